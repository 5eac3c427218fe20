"""The example of a whole decode step runs and finds its own results sound."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]


@pytest.mark.parametrize("options", [[], ["--requests", "1", "--drafts", "1", "--heads", "16",
                                          "--hidden", "2048", "--context", "0"]])
def test_decode_step(cuda, options):
    res = subprocess.run([sys.executable, str(ROOT / "examples" / "decode_step.py"), "--steps", "5",
                          *options], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert res.returncode == 0, res.stderr[-2000:]
    assert "us a step" in res.stdout
