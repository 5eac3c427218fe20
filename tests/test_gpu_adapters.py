"""Low-rank adapters beside the publishing projection, against float64.

Tolerance: C is rounded once (2^-8 of itself at most), and both adapter sums
are FP32: 2^-18 of the sum of magnitudes covers 16384 products
summed in any order at their typical growth."""
import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from tests.latent_cases import normal

pytestmark = pytest.mark.gpu


def codes(seed, rows, k, low=-4, high=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, k, generator=gen, device="cuda").to(torch.float8_e4m3fn)
    e = torch.randint(low + 127, high + 128, (rows, k // 32), generator=gen, device="cuda")
    return x.view(torch.uint8), e.to(torch.uint8)


def dense(x, scale):
    return (x.view(torch.float8_e4m3fn).float().double()
            * torch.exp2(scale.double() - 127).repeat_interleave(32, 1))


class Projection:
    def __init__(self, n, k, seed=0, **tactic):
        self.n, self.k = n, k
        self.w, self.ws = codes(seed + 100, n, k)
        self.mailbox = mx.Mailbox(8, n)
        self.gemm = mx.PublishGemm(self.w, self.ws, self.mailbox, **tactic)

    def expected(self, x, xs, a, b, gain, ranks, which, alpha=1.0):
        xd, wd = dense(x, xs), dense(self.w, self.ws)
        want, size = alpha * (xd @ wd.t()), abs(alpha) * (xd.abs() @ wd.abs().t())
        for t, i in enumerate(which):
            if 0 <= i < a.shape[0]:
                r = a.shape[1] if ranks is None else min(max(ranks[i], 0), a.shape[1])
                g = 1.0 if gain is None else float(gain[i])
                want[t] += g * (b[i, :, :r].double() @ (a[i, :r].double() @ xd[t]))
                size[t] += abs(g) * (b[i, :, :r].double().abs()
                                     @ (a[i, :r].double().abs() @ xd[t].abs()))
        return want, size


def close(got, want, size):
    assert torch.isfinite(got).all()
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -18 * size
    worst = (err / tol).max().item()
    assert worst <= 1.0, f"{worst:.2f} x the tolerance"


def check(p, m, count, rank, which, gain=True, ranks=None, alpha=None, seed=1):
    x, xs = codes(seed, m, p.k)
    a, b = normal(seed + 1, count, rank, p.k, std=p.k ** -0.5), normal(seed + 2, count, p.n, rank)
    g = torch.linspace(-0.5, 1.5, count, device="cuda") if gain else None
    r = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
    al = None if alpha is None else torch.tensor([alpha], device="cuda")
    adapters = mx.Adapters(a, b, g, r)
    w = torch.tensor(which, dtype=torch.int32, device="cuda")
    c = torch.full((m, p.n), float("nan"), dtype=torch.bfloat16, device="cuda")
    p.gemm.run_adapted(x, xs, adapters, w, alpha=al, c=c)
    out = p.mailbox.consume(m)
    close(out, *p.expected(x, xs, a, b, g, ranks, which, alpha or 1.0))
    assert torch.equal(out, c + 0.0)  # the mailbox clears negative zero
    st, words = p.mailbox.status()
    assert st == mx.OK and words[3] == 0
    return x, xs, out


@pytest.mark.parametrize("rank", [1, 2, 7, 8, 16, 24, 33, 64, 128, 255, 256])
def test_ranks(cuda, rank):
    check(Projection(256, 512), 3, 2, rank, [0, 1, 0])


@pytest.mark.parametrize("m", range(1, 9))
def test_rows_each_with_its_own_adapter(cuda, m):
    check(Projection(384, 1024), m, m, 16, list(range(m)))


@pytest.mark.parametrize("k", [32, 96, 256, 1056, 4096, 8224])
def test_ragged_k(cuda, k):
    check(Projection(256, k), 5, 3, 20, [2, 0, -1, 1, 2])


@pytest.mark.parametrize("tactic", [dict(split_k=1, fold=1), dict(split_k=2), dict(split_k=4),
                                    dict(split_k=8), dict(split_k=1, fold=2),
                                    dict(split_k=2, fold=4), dict(split_k=4, fold=2),
                                    dict(fold=8, split_k=1), dict(cta_k=256, split_k=2),
                                    dict(tmem_load=2, fold=1)])
def test_every_epilogue(cuda, tactic):
    check(Projection(512, 2048, **tactic), 8, 4, 32, [0, 1, 2, 3, -1, 3, 2, 0], alpha=0.75)


def test_workload_shapes(cuda):
    check(Projection(7168, 16384, split_k=4), 8, 8, 64, list(range(8)))
    check(Projection(4096, 4096, split_k=1), 1, 2, 16, [1])


def test_own_ranks_and_unused_parts(cuda):
    p = Projection(256, 512)
    x, xs = codes(1, 4, 512)
    a, b = normal(2, 3, 20, 512, std=0.05), normal(3, 3, 256, 20)
    ranks = [20, 5, 0]
    for i, r in enumerate(ranks):
        a[i, r:] = float("nan")
        b[i, :, r:] = float("inf")
    r = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    which = [1, 0, 2, 1]
    p.gemm.run_adapted(x, xs, mx.Adapters(a, b, None, r),
                       torch.tensor(which, dtype=torch.int32, device="cuda"))
    out = p.mailbox.consume(4)
    close(out, *p.expected(x, xs, a, b, None, ranks, which))


def test_rows_without_an_adapter_keep_the_projections_bits(cuda):
    p = Projection(512, 4096)
    x, xs, out = check(p, 8, 2, 8, [-1, 0, -1, 1, -1, -1, 0, -1])
    p.gemm.run(x, xs)
    plain = p.mailbox.consume(8)
    for t in (0, 2, 4, 5, 7):
        assert torch.equal(out[t], plain[t])
    assert not torch.equal(out[1], plain[1])


def test_an_index_out_of_range_counts_as_none_and_raises_the_flag(cuda):
    p = Projection(256, 512)
    x, xs = codes(1, 3, 512)
    a, b = normal(2, 2, 8, 512), normal(3, 2, 256, 8)
    p.gemm.run(x, xs)
    plain = p.mailbox.consume(3)
    p.gemm.run_adapted(x, xs, mx.Adapters(a, b),
                       torch.tensor([2, -5, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(p.mailbox.consume(3), plain)
    st, words = p.mailbox.status()
    assert st == mx.ERR_INVALID and words[3] == mx.FLAG_BAD_INDEX


def test_non_finite_adapters_reach_their_rows_alone(cuda):
    p = Projection(256, 512)
    x, xs = codes(1, 3, 512)
    a, b = normal(2, 2, 8, 512).abs(), normal(3, 2, 256, 8)
    b[0, 7, 3] = float("inf")
    b[0, 9, 3] = float("nan")
    p.gemm.run_adapted(x, xs, mx.Adapters(a, b),
                       torch.tensor([1, 0, -1], dtype=torch.int32, device="cuda"))
    out = p.mailbox.consume(3)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()
    assert torch.isinf(out[1, 7]) and torch.isnan(out[1, 9])
    keep = torch.ones(256, dtype=torch.bool)
    keep[[7, 9]] = False
    assert torch.isfinite(out[1, keep.cuda()]).all()


def test_same_bits_again_and_from_a_graph(cuda):
    p = Projection(1024, 8192, split_k=2)
    x, xs = codes(1, 8, 8192)
    adapters = mx.Adapters(normal(2, 4, 40, 8192, std=0.01), normal(3, 4, 1024, 40))
    which = torch.tensor([0, 1, 2, 3, 3, 2, -1, 0], dtype=torch.int32, device="cuda")
    p.gemm.run_adapted(x, xs, adapters, which)
    first = p.mailbox.consume(8)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.gemm.run_adapted(x, xs, adapters, which)
        p.mailbox.consume(8, out)
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # the rows' adapters are read on the device
    which.fill_(-1)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    p.gemm.run(x, xs)
    assert torch.equal(out, p.mailbox.consume(8))


def test_a_padded_copy_is_there_for_a_run_on_any_stream(cuda):
    p = Projection(256, 512)
    x, xs = codes(1, 3, 512)
    a, b = normal(2, 2, 12, 512, std=0.05), normal(3, 2, 256, 12)
    which = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    p.gemm.run_adapted(x, xs, mx.Adapters(a, b), which)
    want = p.mailbox.consume(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.full((2, 256, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    del junk  # what the copy's block holds before it
    torch.cuda._sleep(20_000_000)  # the copy waits behind it
    adapters = mx.Adapters(a, b)
    p.gemm.run_adapted(x, xs, adapters, which, stream=side)
    got = p.mailbox.consume(3, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals_of_the_binding(cuda):
    p = Projection(256, 512)
    x, xs = codes(1, 3, 512)
    adapters = mx.Adapters(normal(2, 2, 8, 512), normal(3, 2, 256, 8))
    which = torch.zeros(3, dtype=torch.int32, device="cuda")
    alpha = torch.ones(1, device="cuda")
    c = torch.empty((3, 256), dtype=torch.bfloat16, device="cuda")
    run = p.gemm.run_adapted
    for error, text, args, more in (
            (ValueError, "CUDA", (x.cpu(), xs, adapters, which), {}),
            (ValueError, "CUDA", (x, xs.cpu(), adapters, which), {}),
            (ValueError, "CUDA", (x, xs, adapters, which.cpu()), {}),
            (ValueError, "which", (x, xs, adapters, which.long()), {}),
            (ValueError, "which", (x, xs, adapters, which[:2]), {}),
            (ValueError, "x_scale", (x, xs[:2], adapters, which), {}),
            (ValueError, r"x must be", (x[:, :256].contiguous(), xs, adapters, which), {}),
            (TypeError, "one-byte", (x.float(), xs, adapters, which), {}),
            (TypeError, "alpha", (x, xs, adapters, which), dict(alpha=alpha.cpu())),
            (TypeError, "alpha", (x, xs, adapters, which), dict(alpha=alpha.double())),
            (ValueError, "alpha", (x, xs, adapters, which), dict(alpha=alpha[:0])),
            (ValueError, "alpha", (x, xs, adapters, which), dict(alpha=alpha.repeat(2))),
            (ValueError, "c must be", (x, xs, adapters, which), dict(c=c[:2])),
            (TypeError, "two-byte", (x, xs, adapters, which), dict(c=c.float())),
            (ValueError, "adapters are for",
             (x, xs, mx.Adapters(normal(2, 2, 8, 256), normal(3, 2, 256, 8)), which), {})):
        with pytest.raises(error, match=text):
            run(*args, **more)
    with pytest.raises(ValueError, match="alpha"):
        p.gemm.run_scaled(x, xs, alpha[:0])
    # Nothing was launched: the mailbox still takes a call.
    run(x, xs, adapters, which, alpha=alpha[0])  # a scalar tensor is one number too
    assert torch.isfinite(p.mailbox.consume(3)).all() and p.mailbox.status()[0] == mx.OK


@pytest.mark.parametrize("n,heads,rank,which,tactic", [
    (4096, 32, 16, [0], dict(split_k=1)),
    (1024, 64, 40, [0, 1, 2, 3, -1, 2, 1, 0], dict(split_k=2)),
    (512, 16, 8, [-1, -1, -1], dict(split_k=4)),
    (256, 128, 200, [3, 2, 1, 0], dict(fold=4))])
def test_the_projection_reads_the_activations_made_right_before_it(cuda, n, heads, rank, which,
                                                                   tactic):
    """The projection waits for its adapters in its epilogue alone: nothing it reads before that
    may be of the call before.  Steps in a row with other queries each, through the same x,
    x_scale, which and alpha, that their kernels write right before the call."""
    value, latent, rows, steps = 128, 512, len(which), 8
    p = Projection(n, heads * value, **tactic)
    wv = normal(1, heads, value, latent, std=latent ** -0.5)
    outputs = [normal(20 + i, rows, heads, latent) for i in range(steps)]
    adapters = mx.Adapters(normal(2, 4, rank, p.k, std=p.k ** -0.5), normal(3, 4, n, rank))
    lists = [torch.tensor(which[i % rows:] + which[:i % rows], dtype=torch.int32, device="cuda")
             for i in range(steps)]
    alphas = [torch.full((1,), 0.5 + i, device="cuda") for i in range(steps)]
    x, xs = mx.latent_values(outputs[0], wv)
    index, alpha = torch.empty_like(lists[0]), torch.empty_like(alphas[0])

    def step(i, out, wait):
        index.copy_(lists[i])
        alpha.copy_(alphas[i])
        wait()
        mx.latent_values(outputs[i], wv, x, xs)
        wait()
        p.gemm.run_adapted(x, xs, adapters, index, alpha=alpha)
        wait()
        p.mailbox.consume(rows, out)
        wait()

    want = torch.empty((steps, rows, n), dtype=torch.bfloat16, device="cuda")
    for i in range(steps):
        step(i, want[i], torch.cuda.synchronize)
    assert not any(torch.equal(want[i], want[i - 1]) for i in range(1, steps))
    got = torch.empty_like(want)
    for _ in range(5):
        got.fill_(float("nan"))
        for i in range(steps):
            step(i, got[i], lambda: None)
        assert torch.equal(got, want)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        for i in range(steps):
            step(i, got[i], lambda: None)
    for turn in range(20):
        # Other queries at each replay as well.
        outputs[0].copy_(outputs[1 + turn % (steps - 1)])
        got.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1:], want[1:])
        first = torch.empty_like(want[0])
        step(0, first, torch.cuda.synchronize)
        assert torch.equal(got[0], first)
    assert p.mailbox.status()[0] == mx.OK
