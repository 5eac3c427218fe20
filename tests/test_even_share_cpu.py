"""The deal of items to a grid's blocks, on the CPU: its header compiles with
g++ alone.  (At N = 2^29 and 8 rows an adapter call has 2^25 items; their
product with 152 blocks is past 32 bits.)"""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]


def test_every_item_is_dealt_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = tmp_path / "even_share_check"
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv",
                    f"-I{ROOT / 'mxfp8_gemm_mailbox_gb300' / 'csrc'}",
                    str(ROOT / "tests" / "native" / "even_share_check.cpp"), "-o", str(exe)],
                   check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout + res.stderr
