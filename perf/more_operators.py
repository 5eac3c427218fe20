"""What follows the output projection of a decode step or a prompt, as measurable cases: a layer of
routed experts in microscaled formats.

Five operators, each in a plain form (elementary torch operations in 32 bits) and through the
package's entry points:

- ``route``     the top-k experts of each token, their weights, and the tokens in the experts'
                order;
- ``quantize``  rows in MXFP8 or MXFP4 (elements of 8 or 4 bits, one power of two a block of 32),
                gathered on the way, or a matrix to MXFP4 and back;
- ``product``   every expert's MXFP8 or MXFP4 matrix times its rows, BF16 out; one expert is the
                product of a whole prompt;
- ``gated``     the same with a gate and an up half, silu(gate) x up, rounded to MXFP8;
- ``combine``   the weighted sum of each token's rows.
"""
import math
import random

import torch

own = False

BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One token of a decode step.
        dict(name="route token", op="route", tokens=1, experts=64, k=8, half=False, padded=0),
        # A prompt of 16k tokens, some of them padding, many experts, BF16 logits with their ties.
        dict(name="route prompt", op="route", tokens=16384, experts=256, k=8, half=True,
             padded=100),
        # A decode step's eight tokens, each to the rows of its eight experts.
        dict(name="quantize rows", op="quantize", tokens=8, k=7168, bits=8, gather=8),
        # A weight matrix made into MXFP4, and read back.
        dict(name="quantize matrix", op="quantize", tokens=16384, k=8192, bits=4, gather=0),
        # The second product of one token's eight experts: the stream of their matrices.
        dict(name="product token", op="product", rows=8, experts=64, n=4096, k=2048, bits=4,
             x_bits=8),
        # Few rows on many experts of odd sizes, both operands in 4 bits.
        dict(name="product odd", op="product", rows=333, experts=24, n=1000, k=640, bits=4,
             x_bits=4),
        # The output projection of a prompt of 4096 tokens: one matrix, N and K of the headline.
        dict(name="product prompt", op="product", rows=4096, experts=1, n=7168, k=16384, bits=8,
             x_bits=8),
        # A decode step of eight tokens with eight experts each.
        dict(name="gated step", op="gated", rows=64, experts=64, n=2048, k=4096, bits=4, x_bits=8),
        # Unequal shares on few experts, MXFP8 throughout.
        dict(name="gated odd", op="gated", rows=999, experts=7, n=736, k=896, bits=8, x_bits=8),
        # A prompt of 4096 tokens with eight experts each.
        dict(name="gated prompt", op="gated", rows=32768, experts=64, n=2048, k=4096, bits=4,
             x_bits=8),
        # One token.
        dict(name="combine token", op="combine", tokens=1, k=8, n=4096, padded=0),
        # A prompt.
        dict(name="combine prompt", op="combine", tokens=4096, k=8, n=4096, padded=50),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("route", "quantize", "product", "product", "gated", "gated", "combine"))
    if op == "route":
        experts = _log(rng, 2, 256)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts,
                    k=rng.randint(1, min(8, experts)), half=rng.random() < 0.5,
                    padded=rng.choice((0, 100, 500)))
    if op == "quantize":
        gather = rng.choice((0, rng.randint(1, 8)))
        tokens = _log(rng, 1, 2048 if gather else 16384)
        return dict(op=op, tokens=tokens, k=BLOCK * _log(rng, 1, 256), bits=rng.choice((4, 8)),
                    gather=gather)
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 4096), k=rng.randint(1, 8),
                    n=8 * _log(rng, 1, 512), padded=rng.choice((0, 50, 500)))
    experts = _log(rng, 1, 64)
    k = 128 * _log(rng, 1, 32)
    n = (32 if op == "gated" else 8) * _log(rng, 4, 64 if op == "gated" else 512)
    return dict(op=op, rows=_log(rng, 1, 16384), experts=experts, n=n, k=k,
                bits=rng.choice((4, 8)), x_bits=rng.choice((4, 8)))


# ------------------------------------------------------------------ the cases' derived sizes
def _counts(case):
    """Rows of each expert: unequal shares, the same for every seed up to the experts' order."""
    rows, experts = case["rows"], case["experts"]
    rng = random.Random("%d of %d" % (rows, experts))
    share = [math.exp(rng.gauss(0.0, 0.5)) for _ in range(experts)]
    if rows > 64 * experts:  # a long prompt: everybody's share of it
        counts = [int(rows * s / sum(share)) for s in share]
        counts[0] += rows - sum(counts)
        return counts
    counts = [0] * experts
    for e in rng.choices(range(experts), share, k=rows):
        counts[e] += 1
    return counts


def _out_rows(case):
    return case["tokens"] * (case["gather"] or 1)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": t * e * (2 if case["half"] else 4) + t * k * 16 + (e + 1) * 4,
                "flops": t * e}
    if op == "quantize":
        t, k, r = case["tokens"], case["k"], _out_rows(case)
        back = 0 if case["bits"] == 8 else r * k * 2  # 4 bits: the values, read back
        return {"bytes": t * k * 2 + r * k // BLOCK + (r * k if case["bits"] == 8 else back),
                "flops": 2 * r * k}
    if op == "combine":
        t, k, n = case["tokens"], case["k"], case["n"]
        return {"bytes": t * k * (2 * n + 8) + t * n * 2, "flops": 2 * t * k * n}
    rows, n, k = case["rows"], case["n"], case["k"]
    outputs = 2 * n if op == "gated" else n
    active = sum(c > 0 for c in _counts(case))
    data = active * outputs * (k * case["bits"] // 8 + k // BLOCK)
    data += rows * (k * case["x_bits"] // 8 + k // BLOCK)
    data += rows * (n + n // BLOCK if op == "gated" else 2 * n)
    return {"bytes": data, "flops": 2 * rows * outputs * k}


# ------------------------------------------------------------------ inputs
def _codes(gen, shape, k, bits, low, high):
    """Codes of normal samples and uniform exponents: E4M3 or two E2M1 a byte (the first in the
    low half), and E8M0."""
    scale = torch.randint(low + 127, high + 128, (*shape, k // BLOCK), generator=gen,
                          device="cuda").to(torch.uint8)
    x = torch.empty((*shape, k if bits == 8 else k // 2), dtype=torch.uint8, device="cuda")
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for part in (x if len(shape) > 1 else x[None]):  # one matrix at a time: 32-bit samples
        y = torch.randn(*part.shape[:-1], k, generator=gen, device="cuda")
        if bits == 8:
            part.copy_(y.to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            code = torch.bucketize(y.abs() * 2, borders, out_int32=True) + 8 * (y < 0).int()
            part.copy_(code[..., 0::2] + 16 * code[..., 1::2])
    return x, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "route":
        t, e = case["tokens"], case["experts"]
        z = torch.randn(t, e, generator=gen, device="cuda") * 2
        if case["padded"]:  # every so many tokens one is padding: nothing to choose from
            z[torch.arange(t, device="cuda") % case["padded"] == case["padded"] - 1] = -math.inf
        s["logits"] = z.to(torch.bfloat16) if case["half"] else z
    elif op == "quantize":
        t, k = case["tokens"], case["k"]
        size = torch.exp2(torch.randint(-6, 7, (t, 1), generator=gen, device="cuda").float())
        s["x"] = (torch.randn(t, k, generator=gen, device="cuda") * size).to(torch.bfloat16)
        if case["gather"]:
            rows = torch.arange(t, device="cuda").repeat(case["gather"])
            s["rows"] = rows[torch.randperm(len(rows), generator=gen, device="cuda")].int()
    elif op == "combine":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["y"] = torch.randn(t * k, n, generator=gen, device="cuda").to(torch.bfloat16)
        s["weight"] = torch.softmax(torch.randn(t, k, generator=gen, device="cuda"), -1)
        s["slot"] = torch.randperm(t * k, generator=gen, device="cuda").view(t, k).int()
        if case["padded"]:
            gone = torch.arange(t, device="cuda") % case["padded"] == case["padded"] - 1
            s["slot"][gone] = -1
            s["weight"][gone] = 0
    else:
        outputs = 2 * case["n"] if op == "gated" else case["n"]
        counts = _counts(case)
        random.Random(seed).shuffle(counts)
        s["counts"] = counts  # the plain form's: a program of torch operations knows its sizes
        ends = torch.tensor([0] + counts, device="cuda").cumsum(0)
        s["begin"] = ends.int()
        # Exponents that make outputs of the order of one.
        low = -3 - int(math.log2(case["k"]) / 2)
        s["w"], s["w_scale"] = _codes(gen, (case["experts"], outputs), case["k"], case["bits"],
                                      low, low + 3)
        s["x"], s["x_scale"] = _codes(gen, (case["rows"],), case["k"], case["x_bits"], -1, 1)
        if own:
            import mxfp8_gemm_mailbox_gb300 as mx
            s["product"] = mx.ExpertProduct(s["w"], s["w_scale"], gated=op == "gated")
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_route(s):
    import mxfp8_gemm_mailbox_gb300 as mx
    return mx.route(s["logits"], s["k"])._asdict()


def _own_quantize(s):
    import mxfp8_gemm_mailbox_gb300 as mx
    x, scale = mx.quantize(s["x"], "mxfp%d" % s["bits"], rows=s.get("rows"))
    return (x if s["bits"] == 8 else mx.dequantize(x, scale)), scale


def _own_product(s):
    return s["product"].run(s["x"], s["x_scale"], s["begin"])


def _own_gated(s):
    return s["product"].run(s["x"], s["x_scale"], s["begin"], format="mxfp8")


def _own_combine(s):
    import mxfp8_gemm_mailbox_gb300 as mx
    return mx.combine(s["y"], s["weight"], s["slot"])


_own = {"route": _own_route, "quantize": _own_quantize, "product": _own_product,
        "gated": _own_gated, "combine": _own_combine}


def _plain_route(s):
    z, k = s["logits"].float(), s["k"]
    tokens, experts = z.shape
    top, expert = torch.sort(z, dim=1, descending=True, stable=True)  # the lowest index first
    top, expert = top[:, :k], expert[:, :k]
    routed = top > -math.inf
    e = torch.where(routed, torch.exp(top - top[:, :1]), torch.zeros_like(top))
    total = e.sum(1, keepdim=True)
    weight = torch.where(routed, e / total, torch.zeros_like(e))
    key = torch.where(routed, expert, torch.full_like(expert, experts)).flatten()
    order = torch.sort(key, stable=True)[1]
    begin = torch.searchsorted(key[order], torch.arange(experts + 1, device="cuda"))
    slot = torch.empty_like(order)
    slot[order] = torch.arange(tokens * k, device="cuda")
    none = torch.full_like(expert, -1)
    row = torch.where(torch.arange(tokens * k, device="cuda") < begin[-1], order // k,
                      none.flatten())
    return {"weight": weight, "expert": torch.where(routed, expert, none).int(),
            "slot": torch.where(routed, slot.view(tokens, k), none).int(), "row": row.int(),
            "begin": begin.int()}


def _to_mx(y, bits):
    """(values of the elements, E8M0 scales) of the last axis in blocks of 32: the smallest power
    of two under which no element passes the largest code (448 or 6), then to nearest, ties to
    even."""
    rows = y.shape[0]
    y = y.reshape(rows, -1, BLOCK)
    part, e = torch.frexp(y.abs().amax(-1))
    shift, border = (9, 0.875) if bits == 8 else (3, 0.75)
    e = torch.where(part == 0, torch.zeros_like(e), e - shift + (part > border).int())
    y = torch.ldexp(y, -e[..., None])
    scale = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    if bits == 8:
        return y.to(torch.float8_e4m3fn).view(rows, -1), scale
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return torch.ldexp(torch.round(y / step) * step, e[..., None]).view(rows, -1), scale


def _plain_quantize(s):
    x = s["x"].float()
    if s["gather"]:
        x = x[s["rows"].long()]
    x, scale = _to_mx(x, s["bits"])
    return (x if s["bits"] == 8 else x.to(torch.bfloat16)), scale


def _values(x, scale):
    """What MXFP8 or MXFP4 codes stand for, in 32 bits."""
    if x.shape[-1] == scale.shape[-1] * BLOCK:
        v = x.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        v = torch.stack((table[(x & 15).int()], table[(x >> 4).int()]), -1).flatten(-2)
    v = v.unflatten(-1, (-1, BLOCK)) * torch.exp2(scale.float() - 127.0)[..., None]
    return v.flatten(-2)


def _plain_product(s):
    """Rows of the experts that have any, padded to one length."""
    counts = torch.tensor(s["counts"])
    active = counts.nonzero().flatten()
    longest = int(counts.max())
    count, active = counts[active].cuda(), active.cuda()
    at = s["begin"].long()[active][:, None] + torch.arange(longest, device="cuda")
    live = torch.arange(longest, device="cuda") < count[:, None]
    x = _values(s["x"], s["x_scale"])[torch.where(live, at, torch.zeros_like(at))]
    w = _values(s["w"][active], s["w_scale"][active])
    return torch.matmul(x, w.transpose(1, 2))[live]


def _plain_gated(s):
    gate, up = _plain_product(s).chunk(2, -1)
    return _to_mx(gate / (1.0 + torch.exp(-gate)) * up, 8)


def _plain_combine(s):
    here = s["slot"] >= 0
    y = s["y"].float()[torch.where(here, s["slot"], torch.zeros_like(s["slot"])).long()]
    y = torch.where(here[..., None], y * s["weight"][..., None], torch.zeros_like(y))
    return y.sum(1).to(torch.bfloat16)


_plain = {"route": _plain_route, "quantize": _plain_quantize,
          "product": lambda s: _plain_product(s).to(torch.bfloat16), "gated": _plain_gated,
          "combine": _plain_combine}


# ------------------------------------------------------------------ in 64 bits
def _scaled(y, largest):
    """y over its blocks' powers of two, and those: not rounded to the elements' type."""
    y = y.reshape(y.shape[0], -1, BLOCK)
    top = y.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / largest)), torch.zeros_like(top))
    return (y / torch.exp2(e)).flatten(1), torch.exp2(e).squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        z = s["logits"].double()
        weight = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device="cuda")
        left = z.clone()
        for j in range(case["k"]):
            weight[:, j] = left.amax(1)
            left.scatter_(1, (left == weight[:, j:j + 1]).int().argmax(1, keepdim=True), -math.inf)
        weight = torch.softmax(weight, 1).nan_to_num(0.0)  # a padded token's: nothing
        return {"begin": None, "expert": None, "row": None, "slot": None, "weight": weight}
    if op == "quantize":
        x = s["x"].double()
        if case["gather"]:
            x = x.index_select(0, s["rows"])
        y, scale = _scaled(x, 448.0 if case["bits"] == 8 else 6.0)
        if case["bits"] == 4:  # the nearest of the codes' values, the even code of two
            code = torch.zeros_like(y, dtype=torch.int32)
            for i in range(7):
                border = (E2M1[i] + E2M1[i + 1]) / 2
                code += y.abs() >= border if i % 2 else y.abs() > border
            low = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
            y = torch.sign(y) * low[code] * scale.repeat_interleave(BLOCK, 1)
        return y, scale
    if op == "combine":
        out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (s["slot"][:, j] >= 0).nonzero().flatten()
            rows = s["y"].index_select(0, s["slot"][t, j]).double()
            out.index_add_(0, t, s["weight"][t, j, None].double() * rows)
        return out
    byte = torch.arange(256, dtype=torch.int32, device="cuda")
    low = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    nibble = torch.where(byte % 16 < 8, 1.0, -1.0).double() * low[byte % 8]
    pairs = torch.stack((nibble, nibble[byte // 16]), 1)
    e4m3 = byte.to(torch.uint8).view(torch.float8_e4m3fn).double()

    def dense(x, scale, bits):
        v = e4m3[x.int()] if bits == 8 else pairs[x.int()].flatten(1)
        return v * torch.exp2(scale.double() - 127).repeat_interleave(BLOCK, 1)

    out, at = [], 0
    for e, c in enumerate(s["counts"]):
        if c:
            x = dense(s["x"][at:at + c], s["x_scale"][at:at + c], case["x_bits"])
            out.append(x @ dense(s["w"][e], s["w_scale"][e], case["bits"]).t())
            at += c
    y = torch.cat(out)
    if op == "product":
        return y
    gate, up = y[:, :case["n"]], y[:, case["n"]:]
    return _scaled(gate * torch.sigmoid(gate) * up, 448.0)
