"""A layer of routed experts on the GPU against float64.

Tolerances (tests/experts_cases.py).  product: half a BF16 step of the value (2^-8), and
the FP32 sums: 2^-22 of the sum of magnitudes for every 32 products.  Rounded results:
half a step of the element type (E4M3 2^-4 of the value or 2^-10 of the scale, E2M1 2^-2
of either), the same sums, and a scale that is right for a value that near.  quantize,
route's indexes: equal.  combine: half a BF16 step, and k + 1 roundings of FP32 sums.
route's weights: 2^-20 of the value (an exponential of 2 ulps, a sum, a quotient) and
2^-24 of it for each unit of z_max - z, whose rounding the exponential turns into a
relative error of that size (the sum's own such error is the mean of z_max - z under the
weights, at most the logarithm of their number: 6.3 units, within the 2^-20)."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from tests.experts_cases import (begin_of, close_bf16, close_codes, gate, generator, products,
                                 random_codes, rounded, sum_error, values)

pytestmark = pytest.mark.gpu


def shares(seed, rows, experts):
    """Rows of each expert, some of them none."""
    at = torch.randint(0, experts, (rows,), generator=generator(seed, "cpu"))
    return torch.bincount(at, minlength=experts).tolist()


class Case:
    def __init__(self, counts, n, k, bits=4, x_bits=8, gated=False, seed=1):
        self.counts, self.n, self.k, self.gated = counts, n, k, gated
        self.rows = sum(counts)
        outputs = 2 * n if gated else n
        self.w, self.w_scale = random_codes(seed, (len(counts), outputs), k, bits, -6, -3)
        self.x, self.x_scale = random_codes(seed + 1, (self.rows,), k, x_bits)
        self.begin = begin_of(counts)
        self.product = mx.ExpertProduct(self.w, self.w_scale, gated=gated)

    def expected(self):
        y, size = products(self.w, self.w_scale, self.x, self.x_scale, self.counts)
        error = sum_error(size, self.k)
        return gate(y, error) if self.gated else (y, error)

    def check(self, format=None):
        got = self.product.run(self.x, self.x_scale, self.begin, format=format)
        assert self.product.status() == 0
        if format is None:
            close_bf16(got, *self.expected())
        else:
            close_codes(*got, *self.expected())
        return got


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("format,bits", [("mxfp8", 8), ("mxfp4", 4)])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (7, 7168), (129, 512), (1000, 160)])
def test_quantize(cuda, dtype, format, bits, rows, k):
    gen = generator(rows + k)
    size = torch.exp2(torch.randint(-12, 13, (rows, k // 32, 1), generator=gen,
                                    device="cuda").float())
    x = (torch.randn(rows, k // 32, 32, generator=gen, device="cuda") * size).view(rows, k)
    x = x.to(dtype)
    codes, scale = mx.quantize(x, format)
    want, want_scale = rounded(x, bits)
    assert torch.equal(scale.view(torch.uint8), want_scale)
    assert torch.equal(codes.view(torch.uint8), want)
    assert torch.equal(mx.dequantize(codes, scale, torch.float32).double(), values(codes, scale))


@pytest.mark.parametrize("format,bits", [("mxfp8", 8), ("mxfp4", 4)])
def test_quantize_every_bf16(cuda, format, bits):
    """Every finite BF16 number, each beside a largest element that puts it anywhere in its
    block's range, and the borders of the scale."""
    every = torch.arange(65536, device="cuda").to(torch.uint16).view(torch.bfloat16)
    every = every[torch.isfinite(every)]
    every = every[: every.numel() // 32 * 32]
    for order in (torch.arange(every.numel(), device="cuda"),
                  torch.randperm(every.numel(), generator=generator(3), device="cuda")):
        x = every[order].view(-1, 32)
        codes, scale = mx.quantize(x, format)
        want, want_scale = rounded(x, bits)
        assert torch.equal(scale.view(torch.uint8), want_scale)
        # Zeros keep their sign in both; compared as values too.
        assert torch.equal(codes.view(torch.uint8), want)


@pytest.mark.parametrize("format,bits", [("mxfp8", 8), ("mxfp4", 4)])
def test_quantize_ties(cuda, format, bits):
    """Halfway between two codes, at many scales: to the even one."""
    grid = torch.arange(0, 449, 0.25, device="cuda") if bits == 8 else torch.arange(
        0, 6.25, 0.125, device="cuda")
    rows = []
    for top in ((448.0, 256.0) if bits == 8 else (6.0, 4.0)):
        x = grid[grid <= top]
        x = torch.nn.functional.pad(x, (0, -x.numel() % 31)).view(-1, 31)
        rows.append(torch.cat((x, torch.full_like(x[:, :1], top)), 1))
    x = torch.cat(rows)
    x = torch.cat([x * 2.0 ** e for e in (-100, -20, 0, 3, 90)] + [-x])
    codes, scale = mx.quantize(x, format)
    want, want_scale = rounded(x, bits)
    assert torch.equal(scale.view(torch.uint8), want_scale)
    assert torch.equal(codes.view(torch.uint8), want)


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
def test_quantize_non_finite_and_zero(cuda, format):
    x = torch.randn(4, 96, generator=generator(0), device="cuda")
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    x[3, :32] = 0.0
    codes, scale = mx.quantize(x, format)
    want, want_scale = rounded(x, 8 if format == "mxfp8" else 4)
    assert torch.equal(scale.view(torch.uint8), want_scale)
    v = mx.dequantize(codes, scale, torch.float32)
    if format == "mxfp8":
        assert torch.equal(torch.isnan(v), ~torch.isfinite(x))
    else:
        assert torch.equal(codes, want)
        assert torch.equal(torch.isnan(v).view(4, 3, 32).all(-1), torch.isnan(v).view(4, 3, 32).any(-1))
        assert torch.equal(torch.isnan(v).view(4, 3, 32).all(-1),
                           ~torch.isfinite(x).view(4, 3, 32).all(-1))


def test_quantize_gathers_strided_rows_and_leaves_others(cuda):
    base = torch.randn(40, 256, generator=generator(4), device="cuda").to(torch.bfloat16)
    x = base[:, 64:192]  # rows of 128, 256 apart
    rows = torch.tensor([3, 39, -1, 0, 3, 40, -2, 17], dtype=torch.int32, device="cuda")
    codes = torch.full((8, 128), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.full((8, 4), 0x5A, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.quantize(x, "mxfp8", rows=rows, codes=codes, scale=scale, flags=flags)
    want, want_scale = rounded(x, 8)
    for r, i in enumerate(rows.tolist()):
        if 0 <= i < 40:
            assert torch.equal(codes[r], want[i]) and torch.equal(scale[r], want_scale[i])
        else:
            assert (codes[r] == 0xA5).all() and (scale[r] == 0x5A).all()
    assert int(flags) == mx.FLAG_BAD_INDEX


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bits", [4, 8])
def test_dequantize_every_code_and_scale(cuda, bits, dtype):
    """Every code under every scale: the value rounded once to the type, infinite past its largest,
    NaN under 255.  (FP32 is wider than E2M1 and E4M3 by their own digits, so that rounding its
    value rounds once.)"""
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(256, 1)
    scale = torch.arange(256, device="cuda").to(torch.uint8)[:, None]
    scale = scale.expand(256, 256 * 8 // bits // 32).contiguous()
    got = mx.dequantize(codes, scale, dtype)
    exact = values(codes, scale)
    assert got.dtype == dtype and got.shape == exact.shape
    if bits == 4:
        assert torch.equal(torch.isnan(exact), (scale == 255).repeat_interleave(32, 1))
    want = exact.float().to(dtype)  # 4 digits down to 2^-136: exact in FP32 below its largest
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.double(), nan=0.0, posinf=1e300, neginf=-1e300),
                       torch.nan_to_num(want.double(), nan=0.0, posinf=1e300, neginf=-1e300))
    assert torch.equal(torch.signbit(got)[~torch.isnan(got)], torch.signbit(want)[~torch.isnan(want)])


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_and_back_next_to_the_largest(cuda, bits):
    """Finite numbers that a block rounds up past FP32's largest come back infinite; all others
    within half a step of the element type."""
    top = torch.finfo(torch.bfloat16).max
    x = top * torch.linspace(0.25, 1.0, 64, device="cuda")
    x = torch.stack((x, -x)).bfloat16()
    back = mx.dequantize(*mx.quantize(x, "mxfp%d" % bits), torch.float32).double()
    past = x.double().abs() >= 2.0 ** 128 * (1 - 2.0 ** -5 if bits == 8 else 7 / 8)
    assert past.any() and torch.equal(torch.isinf(back), past)
    near = (back - x.double()).abs() <= x.double().abs() * 2.0 ** -(4 if bits == 8 else 2)
    assert (near | past).all() and torch.equal(torch.signbit(back), torch.signbit(x))


def test_quantize_shapes(cuda):
    x = torch.randn(2, 3, 5, 64, generator=generator(5), device="cuda")
    codes, scale = mx.quantize(x, "mxfp4")
    assert codes.shape == (2, 3, 5, 32) and scale.shape == (2, 3, 5, 2)
    assert mx.dequantize(codes, scale).shape == x.shape
    for rows in (0, None):
        index = None if rows is None else torch.empty(0, dtype=torch.int32, device="cuda")
        c, s = mx.quantize(torch.empty(0 if rows is None else 4, 64, device="cuda"), "mxfp8",
                           rows=index)
        assert c.shape == (0, 64) and s.shape == (0, 2)


# ------------------------------------------------------------------ route, combine
def routed(logits, k, normalize):
    """The definition, token by token, on the host."""
    z = logits.double().cpu()
    weight, expert, entries = [], [], []
    for t, row in enumerate(z.tolist()):
        # NaN before all numbers, infinity among them.
        key = lambda e: (0, 0.0, e) if row[e] != row[e] else (1, -row[e], e)  # noqa: E731
        chosen = sorted(range(len(row)), key=key)[:k]
        chosen = [e for e in chosen if row[e] != -float("inf")]
        first = row[chosen[0]] if chosen else 0.0
        exps = torch.exp(torch.tensor(row, dtype=torch.float64) - first)
        total = exps[chosen].sum() if normalize else exps.sum()
        pad = k - len(chosen)
        weight.append([float(exps[e] / total) for e in chosen] + [0.0] * pad)
        expert.append(chosen + [-1] * pad)
        entries += [(e, t, j) for j, e in enumerate(chosen)]
    entries.sort(key=lambda i: (i[0], i[1]))
    slot = torch.full((len(z), k), -1, dtype=torch.int32)
    row = torch.full((len(z) * k,), -1, dtype=torch.int32)
    for s, (e, t, j) in enumerate(entries):
        slot[t, j], row[s] = s, t
    begin = [sum(i[0] < e for i in entries) for e in range(z.shape[1] + 1)] if len(z) < 600 else (
        torch.tensor([0] + torch.bincount(torch.tensor([i[0] for i in entries]),
                                          minlength=z.shape[1]).tolist()).cumsum(0).tolist())
    return (torch.tensor(weight, dtype=torch.float64).view(len(z), k),
            torch.tensor(expert, dtype=torch.int32).view(len(z), k), slot, row,
            torch.tensor(begin, dtype=torch.int32))


def check_route(logits, k, normalize=True):
    got = mx.route(logits, k, normalize)
    weight, expert, slot, row, begin = routed(logits, k, normalize)
    assert torch.equal(got.expert.cpu(), expert)
    assert torch.equal(got.slot.cpu(), slot)
    assert torch.equal(got.row.cpu(), row)
    assert torch.equal(got.begin.cpu(), begin)
    w = got.weight.double().cpu()
    assert torch.equal(torch.isnan(w), torch.isnan(weight))
    off, weight = torch.nan_to_num((w - weight).abs()), torch.nan_to_num(weight)
    distance = torch.log(weight[:, :1].clamp(min=1e-300) / weight.clamp(min=1e-300)).clamp(min=0)
    assert (off <= (2.0 ** -20 + 2.0 ** -24 * distance) * weight + 1e-37).all()
    return got


@pytest.mark.parametrize("tokens", [0, 1, 2, 31, 32, 33, 128, 300, 1024, 1025])
@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (33, 5), (64, 8), (256, 8)])
def test_route_sizes(cuda, tokens, experts, k):
    check_route(torch.randn(tokens, experts, generator=generator(tokens), device="cuda"), k)


@pytest.mark.parametrize("experts,k", [(65, 1), (257, 32), (512, 16), (32, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_types(cuda, experts, k, dtype, normalize):
    z = torch.randn(77, experts + 8, generator=generator(k), device="cuda") * 3
    check_route(z.to(dtype)[:, 8:], k, normalize)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_route_unaligned_pairs(cuda, dtype):
    z = torch.randn(40, 71, generator=generator(2), device="cuda").to(dtype)
    for part in (z, z[:, 1:], z[:, 1:70], z[:, 2:], torch.cat((z, z), 1)[:, 3:85]):
        check_route(part, 6)
    every = torch.arange(65536, device="cuda").to(torch.uint16).view(dtype).view(-1, 512)
    check_route(every, 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("experts,k", [(7, 7), (71, 8), (128, 8), (129, 9), (250, 7), (257, 8), (512, 8)])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_up_to_eight_and_more(cuda, dtype, experts, k, normalize):
    """Rows on 16-byte boundaries and between them, with ties among them."""
    z = torch.randn(70, experts, generator=generator(k), device="cuda") * 3
    z[10:20] = torch.round(z[10:20])
    z[20, ::3] = -float("inf")
    z = z.to(dtype)
    wide = torch.zeros(70, 528, dtype=dtype, device="cuda")[:, 8:8 + experts]
    odd = torch.zeros(70, 531, dtype=dtype, device="cuda")[:, 1:1 + experts]
    for part in (wide, odd):
        part.copy_(z)
        check_route(part, k, normalize)
    check_route(wide[3:4], k, normalize)


def test_route_ties_infinities_and_nan(cuda):
    inf, nan = float("inf"), float("nan")
    z = torch.zeros(10, 40, device="cuda")  # all equal: the lowest indexes
    z[1] = -inf                             # nothing to choose
    z[2] = torch.finfo(torch.float32).min   # the lowest number is chosen
    z[3, 7:] = -inf                         # fewer than k
    z[4, 20], z[4, 21] = -0.0, 0.0          # equal
    z[5, 11] = nan                          # the largest
    z[6, 30] = inf
    z[7] = torch.arange(40, device="cuda") % 3
    z[8, ::2] = -inf
    z[9] = torch.finfo(torch.float32).max
    check_route(z, 8)
    check_route(z.to(torch.bfloat16), 3, normalize=False)


def check_many(tokens, experts, k):
    """Against the definition in sorts: the lowest index first among equal logits."""
    z = torch.randn(tokens, experts, generator=generator(tokens), device="cuda").to(torch.bfloat16)
    z[::7] = -float("inf")
    got = mx.route(z, k)
    top, expert = torch.sort(z.double(), dim=1, descending=True, stable=True)
    expert = torch.where(top > -float("inf"), expert, -1)[:, :k]
    assert torch.equal(got.expert.long(), expert)
    key = torch.where(expert >= 0, expert, experts).flatten()
    order = torch.sort(key, stable=True)[1]
    begin = torch.tensor([0] + torch.bincount(key, minlength=experts + 1).tolist()).cumsum(0)
    assert got.begin.tolist() == begin[:experts + 1].tolist()
    total = int(got.begin[-1])
    assert torch.equal(got.row[:total].long(), order[:total] // k)
    assert (got.row[total:] == -1).all()
    assert torch.equal(got.slot.flatten()[order[:total]].long(), torch.arange(total, device="cuda"))
    assert (got.slot.flatten()[order[total:]] == -1).all()


@pytest.mark.parametrize("tokens", [2048, 8192, 8193, 32769, 40000])
def test_route_many_tokens(cuda, tokens):
    check_many(tokens, 37, 3)


@pytest.mark.parametrize("tokens,experts,k", [(2049, 100, 8), (9000, 300, 9), (33000, 260, 8),
                                              (33001, 64, 12), (70000, 128, 6)])
def test_route_many_tokens_and_choices(cuda, tokens, experts, k):
    check_many(tokens, experts, k)


@pytest.mark.parametrize("tokens,experts,k", [(8193, 33, 4), (9000, 300, 8), (33000, 260, 8),
                                              (40000, 100, 5), (9000, 64, 9), (33001, 64, 12),
                                              (34000, 500, 10)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_weights_of_many_tokens(cuda, tokens, experts, k, dtype, normalize):
    """Blocks of 64 and 256 tokens, whose logits are loaded while those before are chosen from.
    The tolerance of the file's head, and of all experts' sum a rounding for each of a lane's
    experts (an eighth, or fewer) and of its reduction's steps."""
    z = (torch.randn(tokens, experts, generator=generator(k), device="cuda") * 3).to(dtype)
    z[::7] = -float("inf")
    z[1::7, k - 1:] = -float("inf")  # fewer than k
    got = mx.route(z, k, normalize)
    top, expert = torch.sort(z.double(), dim=1, descending=True, stable=True)
    chosen = top[:, :k] > -float("inf")
    assert torch.equal(got.expert.long(), torch.where(chosen, expert[:, :k], -1))
    exps = torch.exp(torch.where(top > -float("inf"), top - top[:, :1], top))
    total = (exps[:, :k] if normalize else exps).sum(1, keepdim=True)
    weight = torch.where(chosen, exps[:, :k] / total, 0.0)
    distance = torch.where(chosen, top[:, :1] - top[:, :k], 0.0)
    sums = 0.0 if normalize else (experts / 8 + 5) * 2.0 ** -24
    off = (got.weight.double() - weight).abs()
    assert (off <= (2.0 ** -20 + sums + 2.0 ** -24 * distance) * weight + 1e-37).all()


def test_route_one_expert_for_all(cuda):
    z = torch.zeros(700, 16, device="cuda")
    z[:, 5] = 4.0
    got = check_route(z, 1)
    assert got.begin.tolist() == [0] * 6 + [700] * 11


@pytest.mark.parametrize("tokens", [0, 1, 5, 200])
@pytest.mark.parametrize("k,n", [(1, 8), (3, 40), (8, 4096), (9, 1000), (32, 64)])
def test_combine(cuda, tokens, k, n):
    gen = generator(tokens + n)
    slots = tokens * k + 3
    y = torch.randn(slots, n + 16, generator=gen, device="cuda").to(torch.bfloat16)[:, 8:-8]
    weight = torch.rand(tokens, k, generator=gen, device="cuda")
    slot = torch.randperm(slots, generator=gen, device="cuda")[:tokens * k].view(tokens, k).int()
    add = torch.randn(tokens, n, generator=gen, device="cuda").to(torch.bfloat16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    if tokens > 1:
        slot[1] = -1
        slot[-1, 0], weight[-1, 0] = -1, float("nan")
    for extra in (None, add):
        got = mx.combine(y, weight, slot, add=extra, flags=flags)
        live = (slot >= 0)[..., None]
        terms = torch.where(live, y.double()[slot.clamp(min=0).long()] * weight.double()[..., None],
                            0.0)
        want, size = terms.sum(1), terms.abs().sum(1)
        if extra is not None:
            want, size = want + extra.double(), size + extra.double().abs()
        close_bf16(got, want, (k + 1) * 2.0 ** -24 * size)
    assert int(flags) == 0


def test_combine_bad_slots(cuda):
    y = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([[0, 4], [-2, 3], [-1, -1]], dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mx.combine(y, torch.ones(3, 2, device="cuda"), slot, flags=flags)
    assert out[:, 0].tolist() == [1.0, 1.0, 0.0] and int(flags) == mx.FLAG_BAD_INDEX


# ------------------------------------------------------------------ the products
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("x_bits", [4, 8])
def test_product_one_tile(cuda, bits, x_bits):
    Case([8], 128, 128, bits, x_bits).check()


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 31, 32, 33, 64, 100])
def test_product_few_rows(cuda, rows):
    Case([rows, 0, 3], 256, 512, seed=rows).check()


@pytest.mark.parametrize("n", [8, 40, 120, 136, 1000])
@pytest.mark.parametrize("k", [128, 384, 640])
def test_product_odd_sizes(cuda, n, k):
    Case([5, 40, 0, 17], n, k, seed=n + k).check()


@pytest.mark.parametrize("bits,x_bits", [(4, 8), (8, 4), (4, 4), (8, 8)])
@pytest.mark.parametrize("rows", [129, 300, 1000])
def test_product_many_rows(cuda, bits, x_bits, rows):
    Case([rows, 1, rows // 3, 0], 264, 768, bits, x_bits, seed=rows).check()


@pytest.mark.parametrize("experts,rows", [(64, 8), (64, 300), (256, 40), (512, 700), (3, 5000)])
def test_product_experts(cuda, experts, rows):
    Case(shares(experts, rows, experts), 384, 256, seed=rows).check()


def test_product_long_sums(cuda):
    """Few tiles, each cut along k over many CTAs, and whole rounds beside cut tiles."""
    Case([3], 128, 16384).check()
    Case([3, 9], 512, 16384, 8, 8).check()
    Case([20], 160 * 128, 1024).check()
    Case([600], 1280, 7168).check()
    Case([40], 256, 8192).check()
    Case([40], 264, 8192 + 128, 8, 4).check()
    # More tiles than the means suggest: all rows on one expert.
    Case([0] * 30 + [64] + [0] * 33, 64, 8192).check()


@pytest.mark.parametrize("bits,x_bits", [(4, 8), (8, 8), (4, 4)])
@pytest.mark.parametrize("format", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", [[1], [6, 0, 30], [200, 333]])
def test_gated(cuda, bits, x_bits, format, counts):
    Case(counts, 160, 512, bits, x_bits, gated=True).check(format)


@pytest.mark.parametrize("n", [32, 64, 96, 736])
@pytest.mark.parametrize("rows", [5, 150])
def test_gated_widths(cuda, n, rows):
    Case([rows, 4], n, 256, gated=True, seed=n).check("mxfp8")


@pytest.mark.parametrize("power", [-60, 0, 60, 120])
@pytest.mark.parametrize("rows", [3, 40])
def test_gated_far_from_zero(cuda, power, rows):
    """Gates from -240 to 240, ups of 2^power, up to 0.94 of BF16's largest.  y is exact (one product each): what remains is
    the exponential's error, 2 ulps and 1.2 for each unit of its argument, and some roundings."""
    n, k = 64, 128
    w = torch.zeros(2 * n, k, dtype=torch.uint8, device="cuda")
    gates = torch.linspace(-240.0, 240.0, n, device="cuda").to(torch.float8_e4m3fn)
    w[:n, 0], w[n:, 0] = gates.view(torch.uint8), 0x38
    w_scale = torch.full((2 * n, k // 32), 127, dtype=torch.uint8, device="cuda")
    w_scale[n:] = 127 + power
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    x[:, 0] = 0x38
    x_scale = torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")
    product = mx.ExpertProduct(w, w_scale, gated=True)
    g = gates.double()
    h = g * torch.sigmoid(g) * 2.0 ** power
    want = h.expand(rows, n)
    got = product.run(x, x_scale)
    assert product.status() == 0
    close_bf16(got, want, want.abs() * ((4 + 1.2 * g.abs()) * 2.0 ** -23 + 2.0 ** -21))


@pytest.mark.parametrize("format", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,n", [(3, 64), (40, 64), (3000, 512)])
def test_gated_next_to_the_largest(cuda, format, rows, n):
    """Results just below 2^128, of either sign, whose g u is past it for many gates.  The error as
    in test_gated_far_from_zero."""
    k = 128
    gates = torch.cat([torch.arange(1.0, 2.0, 0.125) * p for p in (1, 2, 4, 8)]).double()
    most = 0.99 * 2.0 ** 128 / (gates * torch.sigmoid(gates))  # of the ups, in steps of E4M3's
    power = torch.floor(torch.log2(most)).clamp(max=127)
    ups = torch.floor(most / torch.exp2(power) * 8).clamp(max=15) / 8
    assert (gates * ups * torch.exp2(power) >= 2.0 ** 128).sum() >= 8
    gates, power = gates.repeat(n // 32).cuda(), power.repeat(n // 32).cuda()
    ups = torch.cat((ups, -ups)).repeat(n // 64).cuda()
    w = torch.zeros(2 * n, k, dtype=torch.uint8, device="cuda")
    w[:n, 0] = gates.to(torch.float8_e4m3fn).view(torch.uint8)
    w[n:, 0] = ups.to(torch.float8_e4m3fn).view(torch.uint8)
    w_scale = torch.full((2 * n, k // 32), 127, dtype=torch.uint8, device="cuda")
    w_scale[n:] = (127 + power).to(torch.uint8)[:, None]
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    x[:, 0] = 0x38
    x_scale = torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")
    product = mx.ExpertProduct(w, w_scale, gated=True)
    want = (gates * torch.sigmoid(gates) * ups * torch.exp2(power)).expand(rows, n)
    error = want.abs() * ((4 + 1.2 * gates) * 2.0 ** -23 + 2.0 ** -21)
    got = product.run(x, x_scale, format=format)
    assert product.status() == 0
    if format is None:
        close_bf16(got, want, error)
    else:
        close_codes(*got, want, error)


@pytest.mark.parametrize("format", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows", [3, 40])
def test_gated_far_below_zero(cuda, format, rows):
    """Gates from -160 to -191, a block each, times ups near 2^128: results down to FP32's and the
    scales' smallest, while the exponential's root is subnormal from -175 on.  The error as in
    test_gated_far_from_zero; a step (2^-149) of the root, which stands squared, and of what is
    subnormal after it."""
    gates = -torch.arange(160, 192, dtype=torch.float64)
    n, k = 32 * len(gates), 128
    w = torch.zeros(2 * n, k, dtype=torch.uint8, device="cuda")
    code = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    most = 16 * torch.ceil(gates / 16)  # E4M3 takes -160 and -176, and the rest
    w[:n, 0] = code(most).repeat_interleave(32)
    w[:n, 1] = code(gates - most).repeat_interleave(32)
    ups = (1 + torch.arange(32) % 8 / 8) * torch.where(torch.arange(32) < 16, 1.0, -1.0)
    w[n:, 0] = code(ups).repeat(len(gates))
    w_scale = torch.full((2 * n, k // 32), 127, dtype=torch.uint8, device="cuda")
    w_scale[n:] = 254
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda")
    x[:, :2] = 0x38
    x_scale = torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda")
    product = mx.ExpertProduct(w, w_scale, gated=True)
    g = gates.cuda().repeat_interleave(32)
    want = g * torch.sigmoid(g) * ups.double().cuda().repeat(len(gates)) * 2.0 ** 127
    relative = (4 + 1.2 * g.abs()) * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -148 / torch.exp(g / 2)
    error = want.abs() * relative + 2.0 ** -148
    got = product.run(x, x_scale, format=format)
    assert product.status() == 0
    if format is None:
        close_bf16(got, want.expand(rows, n), error.expand(rows, n))
    else:
        close_codes(*got, want.expand(rows, n), error.expand(rows, n))


def test_gated_cut_tiles(cuda):
    Case([4], 64, 8192, gated=True).check("mxfp8")
    Case([300], 192, 8192, gated=True).check("mxfp4")
    Case([33, 50], 96, 8192, gated=True).check("mxfp8")


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
def test_product_rounded(cuda, format):
    Case([3, 50], 192, 512).check(format)


def test_one_matrix_without_begin(cuda):
    c = Case([77], 136, 384)
    one = mx.ExpertProduct(c.w[0], c.w_scale[0])
    close_bf16(one.run(c.x, c.x_scale), *c.expected())


@pytest.mark.parametrize("rows,n", [(5, 136), (100, 2560), (1000, 2560)])
@pytest.mark.parametrize("words", [1, 2, 3])
def test_scales_between_16_byte_boundaries(cuda, rows, n, words):
    w, w_scale = random_codes(90, (n,), 512, 4)
    x, x_scale = random_codes(91, (rows,), 512, 8)
    product = mx.ExpertProduct(w, w_scale)
    moved = torch.empty(x_scale.numel() + 16, dtype=torch.uint8, device="cuda")
    moved = moved[4 * words:][:x_scale.numel()].view_as(x_scale)
    moved.copy_(x_scale)
    assert moved.data_ptr() % 16 == 4 * words
    assert torch.equal(product.run(x, moved), product.run(x, x_scale))
    assert product.status() == 0


@pytest.mark.parametrize("rows", [5, 50, 1000])
def test_codes_written_in_place_are_read(cuda, rows):
    """By the kernel right before the call, too."""
    c = Case([rows], 2560, 512)
    c.check()
    other, _ = random_codes(92, (1, 2560), 512, 4)
    c.w.copy_(other)
    got = c.product.run(c.x, c.x_scale, c.begin)
    close_bf16(got, *c.expected())


def test_rows_of_no_expert_are_left(cuda):
    for counts, total in (([5, 3], 12), ([100, 90], 260)):
        c = Case(counts, 128, 256)
        rows = sum(counts)
        x, x_scale = random_codes(9, (total,), 256, 8)
        x[:rows], x_scale[:rows] = c.x, c.x_scale
        x[rows:] = 0x7F  # NaN
        out = torch.full((total, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        assert c.product.run(x, x_scale, c.begin, out=out) is out
        close_bf16(out[:rows], *c.expected())
        assert (out[rows:] == 7.0).all()
        # A first expert that does not begin at 0.
        out.fill_(7.0)
        c.product.run(x, x_scale, (c.begin + 2).clamp(max=rows), out=out)
        assert (out[:2] == 7.0).all() and (out[rows:] == 7.0).all()
        assert c.product.status() == 0


def test_same_bits_every_time(cuda):
    for c in (Case([3, 9], 512, 16384), Case([50], 256, 16384, gated=True),
              Case([260, 77], 320, 4096, gated=True)):
        first = c.product.run(c.x, c.x_scale, c.begin)
        for _ in range(5):
            assert torch.equal(c.product.run(c.x, c.x_scale, c.begin), first)
        zeros = c.product.workspace[:1024]  # as a call finds them, so it leaves them
        assert not zeros.any()


def test_non_finite_operands_stay_in_their_rows_and_outputs(cuda):
    c = Case([6, 40], 128, 512, 8, 8)
    y, error = c.expected()
    c.x[2, 17] = 0x7F           # NaN in row 2
    c.x_scale[9, 3] = 255       # a NaN block in row 9
    c.w[1, 5, 100] = 0xFF       # NaN in output 5 of expert 1
    got = c.product.run(c.x, c.x_scale, c.begin)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[2], bad[9], bad[6:, 5] = True, True, True
    assert torch.equal(torch.isnan(got), bad)
    close_bf16(torch.where(bad, torch.zeros_like(got), got),
               torch.where(bad, torch.zeros_like(y), y), error)


def test_bad_begin_is_cut_and_flagged(cuda):
    c = Case([5, 3, 8], 128, 256)
    for begin in ([0, 5, 3, 16], [-1, 5, 8, 16], [0, 5, 8, 17], [0, 2 ** 31 - 1, -2 ** 31, 5]):
        c.product.flags.zero_()
        out = c.product.run(c.x, c.x_scale, torch.tensor(begin, dtype=torch.int32, device="cuda"))
        assert out.shape == (16, 128) and c.product.status() == mx.FLAG_BAD_INDEX
    c.product.flags.zero_()
    c.check()


# ------------------------------------------------------------------ together
def layer(x, logits, gate_up, down, k, form="mxfp8"):
    routing = mx.route(logits, k)
    h, s = mx.quantize(x, form, rows=routing.row)
    h, s = gate_up.run(h, s, routing.begin, format=form)
    y = down.run(h, s, routing.begin)
    return mx.combine(y, routing.weight, routing.slot, add=x)


class Layer:
    def __init__(self, experts, hidden, inner, bits=4):
        self.up = random_codes(11, (experts, 2 * inner), hidden, bits, -6, -4)
        self.down = random_codes(12, (experts, hidden), inner, bits, -6, -4)
        self.gate_up = mx.ExpertProduct(*self.up, gated=True)
        self.second = mx.ExpertProduct(*self.down, workspace=self.gate_up.workspace)
        self.experts, self.hidden = experts, hidden

    def inputs(self, tokens, seed=3):
        gen = generator(seed)
        x = torch.randn(tokens, self.hidden, generator=gen, device="cuda").to(torch.bfloat16)
        logits = torch.randn(tokens, self.experts, generator=gen, device="cuda")
        if tokens > 3:
            logits[3] = -float("inf")  # a padded token
        return x, logits

    def run(self, x, logits, k):
        return layer(x, logits, self.gate_up, self.second, k)


@pytest.mark.parametrize("tokens", [1, 6, 200])
@pytest.mark.parametrize("bits", [4, 8])
def test_layer(cuda, tokens, bits):
    """Step by step against 64 bits, each step on the step before as it came, and the whole
    against the sum over experts in 64 bits."""
    m, k = Layer(16, 512, 256, bits), 4
    x, logits = m.inputs(tokens)
    out = m.run(x, logits, k)
    assert m.gate_up.status() == 0 and m.second.status() == 0
    r = mx.route(logits, k)
    total = int(r.begin[-1])
    counts = (r.begin[1:] - r.begin[:-1]).tolist()
    h, s = mx.quantize(x, "mxfp8", rows=r.row)
    y, size = products(*m.up, h[:total], s[:total], counts)
    h, s = m.gate_up.run(h, s, r.begin, format="mxfp8")
    close_codes(h[:total], s[:total], *gate(y, sum_error(size, m.hidden)))
    want, size = products(*m.down, h[:total], s[:total], counts)
    y = m.second.run(h, s, r.begin)
    close_bf16(y[:total], want, sum_error(size, 256))
    weight = r.weight.double()[..., None]
    here = (r.slot >= 0)[..., None]
    at = r.slot.clamp(min=0).long()
    terms = torch.where(here, want[at] * weight, 0.0) if total else torch.zeros_like(x)[:, None]
    # Each term's BF16 rounding and sums, then one rounding.
    error = torch.where(here, (2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + 2 * sum_error(size, 256)
                               )[at] * weight, 0.0).sum(1) if total else 0.0
    whole = x.double() + terms.sum(1)
    close_bf16(out, whole, error + (k + 1) * 2.0 ** -23 * (x.double().abs() + terms.abs().sum(1)))
    if tokens > 3:
        assert torch.equal(out[3], x[3])


def test_layer_in_a_graph(cuda):
    """Captured once, replayed on other inputs with another routing."""
    m, k, tokens = Layer(16, 512, 256), 4, 12
    x, logits = m.inputs(tokens)
    out = torch.empty_like(x)
    m.run(x, logits, k)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out.copy_(m.run(x, logits, k))
    for seed in range(4, 9):
        a, b = m.inputs(tokens, seed)
        x.copy_(a), logits.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, m.run(a, b, k))
    assert m.gate_up.status() == 0 and m.second.status() == 0


def test_calls_on_another_stream(cuda):
    m, k = Layer(8, 256, 128), 2
    x, logits = m.inputs(9)
    want = m.run(x, logits, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = mx.route(logits, k, stream=side)
    h, s = mx.quantize(x, "mxfp8", rows=r.row, stream=side)
    h, s = m.gate_up.run(h, s, r.begin, format="mxfp8", stream=side)
    y = m.second.run(h, s, r.begin, stream=side.cuda_stream)
    out = mx.combine(y, r.weight, r.slot, add=x, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_quantized_rows_into_the_projection(cuda):
    """The activations of the publishing projection, from BF16 rows."""
    x = torch.randn(5, 512, generator=generator(8), device="cuda").to(torch.bfloat16)
    codes, scale = mx.quantize(x, "mxfp8")
    w, w_scale = random_codes(13, (256,), 512, 8)
    mailbox = mx.Mailbox(8, 256)
    gemm = mx.PublishGemm(w, w_scale, mailbox)
    gemm.run(codes, scale)
    got = mailbox.consume(5)
    want, size = products(w, w_scale, codes, scale, [5])
    close_bf16(got, want, sum_error(size, 512))


FAR = (1 << 30) + 16  # elements between three rows: the last lies past 2^31


def test_rows_past_31_bits(cuda):
    far = torch.empty(2 * FAR + 1024, dtype=torch.bfloat16, device="cuda")
    gen = generator(95)
    for columns in (256, 1024):
        view = far.as_strided((3, columns), (FAR, 1))
        near = torch.randn(3, columns, generator=gen, device="cuda").bfloat16()
        view.copy_(near)
        for got, want in zip(mx.quantize(view, "mxfp8"), mx.quantize(near, "mxfp8")):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
        slot = torch.tensor([[2, 0], [1, 2]], dtype=torch.int32, device="cuda")
        weight = torch.rand(2, 2, generator=gen, device="cuda")
        assert torch.equal(mx.combine(view, weight, slot), mx.combine(near, weight, slot))
        if columns == 256:
            for got, want in zip(mx.route(view, 8), mx.route(near, 8)):
                assert torch.equal(got, want)


def test_codes_past_31_bits(cuda):
    rows, k = (1 << 16) + 33, 1 << 15
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_(generator=generator(96))
    codes, scale = mx.quantize(x, "mxfp8")
    back = mx.dequantize(codes, scale)
    for at in (0, rows - 40):
        want, want_scale = rounded(x[at:at + 40], 8)
        assert torch.equal(codes[at:at + 40].view(torch.uint8), want)
        assert torch.equal(scale[at:at + 40].view(torch.uint8), want_scale)
        assert torch.equal(back[at:at + 40].double(), values(want, want_scale))


@pytest.mark.parametrize("gated", [False, True])
def test_products_past_31_bits(cuda, gated):
    """4 GB of results (codes where gated), their last rows against their own product."""
    rows, n, k = (1 << 18) + 100, 8192, 128
    w, w_scale = random_codes(97, ((2 if gated else 1) * n,), k, 4, -6, -3)
    x, x_scale = random_codes(98, (rows,), k, 8)
    product = mx.ExpertProduct(w, w_scale, gated=gated)
    format = "mxfp8" if gated else None
    got = product.run(x, x_scale, format=format)
    assert product.status() == 0
    for at in (0, rows - 50):
        y, size = products(w, w_scale, x[at:at + 50], x_scale[at:at + 50], [50])
        if gated:
            close_codes(got[0][at:at + 50], got[1][at:at + 50], *gate(y, sum_error(size, k)))
        else:
            close_bf16(got[at:at + 50], y, sum_error(size, k))


def test_the_example_with_experts(cuda):
    root = Path(__file__).resolve().parents[1]
    res = subprocess.run([sys.executable, str(root / "examples" / "decode_step.py"), "--steps", "5",
                          "--context", "100", "--heads", "16", "--hidden", "2048", "--experts", "16",
                          "--inner", "512"], capture_output=True, text=True, timeout=300, cwd=root)
    assert res.returncode == 0, res.stderr[-2000:]
    assert "4 of 16 experts" in res.stdout
