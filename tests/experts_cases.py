"""Inputs of the tests of a layer of routed experts and their results in 64 bits,
from the formulas alone (torch float64, no code of the package)."""
import torch

BLOCK = 32
# (largest value, its exponent's distance from the block's, half a step relative to a value,
# half the smallest step) of the element types.
E4M3 = (448.0, 2.0 ** -4, 2.0 ** -10)
E2M1 = (6.0, 2.0 ** -2, 2.0 ** -2)
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def generator(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def random_codes(seed, shape, k, bits, low=-2, high=2):
    """Random codes (no NaN) and scales 2^low .. 2^high, as uint8."""
    gen = generator(seed)
    scale = torch.randint(127 + low, 128 + high, (*shape, k // BLOCK), generator=gen, device="cuda")
    if bits == 8:
        x = torch.randn(*shape, k, generator=gen, device="cuda").to(torch.float8_e4m3fn)
        return x.view(torch.uint8), scale.to(torch.uint8)
    x = torch.randint(0, 256, (*shape, k // 2), generator=gen, device="cuda")
    return x.to(torch.uint8), scale.to(torch.uint8)


def values(codes, scale):
    """What codes stand for, in 64 bits; NaN for the scale 255."""
    codes, scale = codes.view(torch.uint8), scale.view(torch.uint8)
    if codes.shape[-1] == scale.shape[-1] * BLOCK:
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        table = torch.tensor(E2M1_VALUES + tuple(-x for x in E2M1_VALUES), dtype=torch.float64,
                             device=codes.device)
        v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    power = torch.exp2(scale.double() - 127.0)
    power = torch.where(scale == 255, torch.full_like(power, float("nan")), power)
    return v * power.repeat_interleave(BLOCK, -1)


def rounded(x, bits):
    """(codes, scale) of x [...][K], as the definition says, in 64 bits."""
    x = x.double()
    largest = 448.0 if bits == 8 else 6.0
    y = x.unflatten(-1, (-1, BLOCK))
    finite = torch.isfinite(y)
    top = torch.where(finite, y.abs(), torch.zeros_like(y)).amax(-1, keepdim=True)
    e = torch.zeros_like(top)
    some = top > 0
    e[some] = torch.ceil(torch.log2(top[some] / largest))
    # (A logarithm may be off next to a power of two.)
    e = torch.where(some & (top > largest * torch.exp2(e)), e + 1, e)
    e = torch.where(some & (top <= largest * torch.exp2(e - 1)), e - 1, e)
    e = e.clamp(-127, 127)
    y = y / torch.exp2(e)
    scale = (e.squeeze(-1) + 127).to(torch.uint8)
    sign = torch.signbit(y)
    if bits == 8:
        # Steps of 2^-9 up to 2^-6, then 2^-3 of the value's power of two.
        m = y.abs()
        power = torch.floor(torch.log2(m.clamp(min=2.0 ** -6)))
        power = torch.where(m < torch.exp2(power), power - 1, power)
        power = torch.where(m >= torch.exp2(power + 1), power + 1, power)
        step = torch.exp2(power.clamp(min=-6) - 3)
        m = torch.round(m / step) * step  # half to even
        codes = m.to(torch.float8_e4m3fn).view(torch.uint8) | (sign.to(torch.uint8) << 7)
        codes = torch.where(finite, codes, torch.full_like(codes, 0x7F))
        return codes.flatten(-2), scale
    m = y.abs()
    code = torch.zeros_like(m, dtype=torch.int32)
    for i in range(7):
        border = (E2M1_VALUES[i] + E2M1_VALUES[i + 1]) / 2
        code += ((m >= border) if i % 2 else (m > border)).int()
    code = (code + 8 * sign.int()).flatten(-2)
    whole = finite.all(-1)
    code = torch.where(whole.repeat_interleave(BLOCK, -1), code, torch.zeros_like(code))
    scale = torch.where(whole, scale, torch.full_like(scale, 255))
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale


def begin_of(counts):
    return torch.tensor([0] + list(counts), device="cuda").cumsum(0).int()


def products(w, w_scale, x, x_scale, counts):
    """(y, sum of magnitudes) of every expert's rows, in 64 bits."""
    wv, xv = values(w, w_scale), values(x, x_scale)
    if wv.dim() == 2:
        wv = wv[None]
    y, size, at = [], [], 0
    for e, c in enumerate(counts):
        rows = xv[at:at + c]
        y.append(rows @ wv[e].t())
        size.append(rows.abs() @ wv[e].abs().t())
        at += c
    return torch.cat(y), torch.cat(size)


def sum_error(size, k):
    """What FP32 sums of the tensor core may be off by: 2^-22 of the magnitudes' sum a step of 32
    products (a sum's rounding, and a shift that drops bits below it)."""
    return (k // BLOCK + 1) * 2.0 ** -22 * size


def close_bf16(got, want, error):
    """Within half a BF16 step of a value that is within `error` of `want`."""
    assert got.shape == want.shape and got.dtype == torch.bfloat16
    off = (got.double() - want).abs()
    tol = error + 2.0 ** -8 * (want.abs() + error) + 1e-38
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{worst:.2f} x the tolerance"


def close_codes(codes, scale, want, error):
    """`codes`, `scale`: within half a step of a value that is within `error` of `want`, and the
    scale that of such a block."""
    bits = 8 if codes.shape[-1] == want.shape[-1] else 4
    largest, relative, smallest = E4M3 if bits == 8 else E2M1
    code = scale.view(torch.uint8).double()
    power = torch.exp2(code - 127.0)
    block = lambda t: t.unflatten(-1, (-1, BLOCK))  # noqa: E731
    top, slack = block(want.abs()).amax(-1), block(error).amax(-1)
    # No element above the largest, and half the power would not do; zeros take 2^0.
    zero = (top == 0) & (code == 127)
    assert (zero | (top - slack <= largest * power)).all()
    assert (zero | (top + slack > largest * power / 2) | (code == 0)).all()
    off = (values(codes, scale) - want).abs()
    each = power.repeat_interleave(BLOCK, -1)
    tol = error + torch.maximum(relative * (want.abs() + error), smallest * each)
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{worst:.2f} x the tolerance"


def gate(y, size_error):
    """silu(gate) x up of the halves of y, and what errors in them and in the functions (2^-19
    of the result, the exponential's included) come to."""
    g, u = y.chunk(2, -1)
    dg, du = size_error.chunk(2, -1)
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * dg * (u.abs() + du) + (s.abs() + 1.1 * dg) * du + 2.0 ** -19 * h.abs()
