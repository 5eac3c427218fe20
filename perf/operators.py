"""What a decode step around the output projection does, as measurable cases.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and through the package's entry points:

- ``query``   the absorbed query of latent attention: every head's query
              multiplied into the latent space, the rotary part beside it;
- ``attend``  attention of those queries over a paged cache of latents, with
              the drafted tokens of each request under a tree mask;
- ``values``  every head's latent output multiplied by its value matrix and
              rounded to MXFP8, the form in which the projection reads it;
- ``adapted`` the publishing MXFP8 projection with a low-rank adapter of each
              row's own added before the one rounding.
"""
import math

import torch

own = False

ROPE = 64
WIDTHS = (256, 512)           # latent widths
PAGE_SIZES = (8, 16, 32, 64, 128)


def listed():
    return [
        # One request, one token, few heads, a cache that fits two tiles: latency alone.
        dict(name="attend first tokens", op="attend", requests=1, drafts=1, heads=16, latent=512,
             context=100, page=64, ragged=False),
        # A full decode batch of ordinary contexts, every row a request of its own.
        dict(name="attend batch 4k", op="attend", requests=8, drafts=1, heads=128, latent=512,
             context=4096, page=64, ragged=True),
        # One request whose eight rows are a tree of drafts: many query rows on one cache.
        dict(name="attend tree 16k", op="attend", requests=1, drafts=8, heads=128, latent=512,
             context=16384, page=64, ragged=False),
        # The largest: a full batch of long contexts, bound by reading the cache.
        dict(name="attend batch 64k", op="attend", requests=8, drafts=1, heads=128, latent=512,
             context=65536, page=128, ragged=False),
        # Odd sizes: heads that do not fill a tile, small pages that end inside one, the
        # narrow latent, requests with unequal numbers of drafts.
        dict(name="attend odd", op="attend", requests=3, drafts=3, heads=40, latent=256,
             context=2501, page=16, ragged=True),
        # A single token on a small head count: latency.
        dict(name="query single", op="query", rows=1, heads=16, latent=512, nope=128),
        # The full row count at the projection's K = 16384 (128 heads of 128).
        dict(name="query full", op="query", rows=8, heads=128, latent=512, nope=128),
        # K = 4096 (32 heads of 128), one token.
        dict(name="values single", op="values", rows=1, heads=32, latent=512, value=128),
        # K = 16384, eight rows.
        dict(name="values full", op="values", rows=8, heads=128, latent=512, value=128),
        # The chain workload's shape with one row and a small adapter.
        dict(name="adapted one row", op="adapted", n=4096, k=4096, rows=1, split=1, adapters=2,
             rank=16, bare=False),
        # The graph workload's shape; rows that share adapters, rows without one.
        dict(name="adapted shared", op="adapted", n=7168, k=8192, rows=5, split=2, adapters=2,
             rank=24, bare=True),
        # The headline shape, every row with an adapter of its own.
        dict(name="adapted full", op="adapted", n=7168, k=16384, rows=8, split=4, adapters=8,
             rank=64, bare=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend", "query", "values", "adapted"))
    if op == "attend":
        requests = rng.randint(1, 8)
        drafts = rng.randint(1, 8 // requests)
        return dict(op=op, requests=requests, drafts=drafts, heads=_log(rng, 1, 128),
                    latent=rng.choice(WIDTHS), context=_log(rng, 1, 60000) - 1,
                    page=rng.choice(PAGE_SIZES), ragged=rng.random() < 0.5)
    if op == "query":
        return dict(op=op, rows=rng.randint(1, 8), heads=_log(rng, 1, 128),
                    latent=rng.choice(WIDTHS), nope=rng.choice((32, 64, 96, 128, 192)))
    if op == "values":
        return dict(op=op, rows=rng.randint(1, 8), heads=_log(rng, 1, 128),
                    latent=rng.choice(WIDTHS), value=rng.choice((32, 64, 96, 128)))
    return dict(op=op, n=128 * _log(rng, 2, 56), k=32 * _log(rng, 8, 512), rows=rng.randint(1, 8),
                split=rng.choice((1, 2, 4)), adapters=rng.randint(1, 8), rank=_log(rng, 1, 128),
                bare=rng.random() < 0.5)


# ------------------------------------------------------------------ the cases' derived sizes
def _drafts(case):
    """Rows of each request."""
    t = case["drafts"]
    return [t - 1 if case["ragged"] and t > 1 and b % 2 else t for b in range(case["requests"])]


def _contexts(case):
    """Tokens of each request before its drafts."""
    n, c = case["requests"], case["context"]
    return [c - (b * c) // (2 * n) if case["ragged"] else c for b in range(n)]


def _which(case):
    """The adapter of each row, -1 for none."""
    return [-1 if case["bare"] and t % 3 == 2 else t % case["adapters"]
            for t in range(case["rows"])]


def _ranks(case):
    """The rank of each adapter: every other one is smaller than the widest."""
    r = case["rank"]
    return [max(1, r - r // 4) if a % 2 else r for a in range(case["adapters"])]


def work(case):
    op = case["op"]
    if op == "attend":
        t, c = _drafts(case), _contexts(case)
        d, w, h = case["latent"], case["latent"] + ROPE, case["heads"]
        keys = [a + b for a, b in zip(t, c)]
        data = sum(keys) * w * 2 + sum(t) * h * (w + d) * 2
        return {"bytes": data, "flops": 2 * h * sum(a * b for a, b in zip(t, keys)) * (w + d)}
    h, m = case.get("heads"), case["rows"]
    if op == "query":
        i, o = case["nope"], case["latent"]
        return {"bytes": 2 * h * (i * o + m * (i + o + 2 * ROPE)), "flops": 2 * m * h * i * o}
    if op == "values":
        i, o = case["latent"], case["value"]
        return {"bytes": h * (2 * i * o + m * (2 * i + o + o // 32)), "flops": 2 * m * h * i * o}
    n, k = case["n"], case["k"]
    which, ranks = _which(case), _ranks(case)
    low = sum(ranks[a] for a in set(which) if a >= 0) * (n + k) * 2
    return {"bytes": n * k + n * k // 32 + m * (k + k // 32 + 2 * n) + low,
            "flops": 2 * m * n * k + sum(2 * ranks[a] * (n + k) for a in which if a >= 0)}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _codes(gen, rows, k, low, high):
    """MXFP8 rows: E4M3 codes of normal samples, E8M0 codes of uniform exponents."""
    x = torch.randn(rows, k, generator=gen, device="cuda").to(torch.float8_e4m3fn)
    e = torch.randint(low + 127, high + 128, (rows, k // 32), generator=gen, device="cuda")
    return x.view(torch.uint8), e.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "attend":
        t, c = _drafts(case), _contexts(case)
        n, p, w = case["requests"], case["page"], case["latent"] + ROPE
        lengths = [a + b for a, b in zip(t, c)]
        per = (max(lengths) + p - 1) // p
        pool = n * per + 3
        s["cache"] = _normal(gen, pool, p, w)
        s["table"] = torch.randperm(pool, generator=gen, device="cuda")[:n * per].view(n, per).to(torch.int32)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        begin = [0]
        for x in t:
            begin.append(begin[-1] + x)
        s["begin"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
        s["request"] = torch.tensor([b for b, x in enumerate(t) for _ in range(x)], device="cuda")
        # Each draft's parent is any earlier draft of its request, or the context itself.
        host = torch.Generator().manual_seed(seed)
        tree = []
        for x in t:
            sees = []
            for j in range(x):
                up = int(torch.randint(-1, j, (1,), generator=host)) if j else -1
                sees.append((sees[up] if up >= 0 else 0) | 1 << j)
            tree += sees
        s["tree"] = torch.tensor(tree, dtype=torch.int64, device="cuda")
        s["q"] = _normal(gen, begin[-1], case["heads"], w)
        s["scale"] = 1.0 / math.sqrt(128 + ROPE)
        if own:
            import mxfp8_gemm_mailbox_gb300 as mx
            s["attention"] = mx.LatentAttention(case["heads"], case["latent"])
    elif op == "query":
        s["q"] = _normal(gen, case["rows"], case["heads"], case["nope"])
        s["rope"] = _normal(gen, case["rows"], case["heads"], ROPE)
        s["w"] = _normal(gen, case["heads"], case["latent"], case["nope"],
                         std=case["nope"] ** -0.5)
    elif op == "values":
        s["o"] = _normal(gen, case["rows"], case["heads"], case["latent"], std=0.1)
        s["w"] = _normal(gen, case["heads"], case["value"], case["latent"],
                         std=case["latent"] ** -0.5)
    else:
        n, k, m, r = case["n"], case["k"], case["rows"], case["rank"]
        s["w"], s["w_scale"] = _codes(gen, n, k, -4, 2)
        s["x"], s["x_scale"] = _codes(gen, m, k, -4, 2)
        s["a"] = _normal(gen, case["adapters"], r, k, std=k ** -0.5)
        s["b"] = _normal(gen, case["adapters"], n, r)
        s["gain"] = torch.rand(case["adapters"], generator=gen, device="cuda") + 0.5
        s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
        s["which"] = torch.tensor(_which(case), dtype=torch.int32, device="cuda")
        if own:
            import mxfp8_gemm_mailbox_gb300 as mx
            s["mailbox"] = mx.Mailbox(8, n)
            s["gemm"] = mx.PublishGemm(s["w"], s["w_scale"], s["mailbox"], split_k=case["split"])
            s["adapters"] = mx.Adapters(s["a"], s["b"], s["gain"], s["ranks"])
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_attend(s):
    return s["attention"].run(s["q"], s["cache"], s["table"], s["lengths"], s["begin"], s["scale"],
                              tree=s["tree"])


def _own_query(s):
    import mxfp8_gemm_mailbox_gb300 as mx
    return mx.latent_query(s["q"], s["rope"], s["w"])


def _own_values(s):
    import mxfp8_gemm_mailbox_gb300 as mx
    return mx.latent_values(s["o"], s["w"])


def _own_adapted(s):
    s["gemm"].run_adapted(s["x"], s["x_scale"], s["adapters"], s["which"])
    return s["mailbox"].consume(s["rows"])


_own = {"attend": _own_attend, "query": _own_query, "values": _own_values,
        "adapted": _own_adapted}


def _visible(s, keys):
    """Which of the request's first `keys` tokens each row sees: [rows][keys]."""
    begin, lengths = s["begin"].long(), s["lengths"].long()
    at = torch.arange(keys, device="cuda")
    context = (lengths - (begin[1:] - begin[:-1]))[s["request"]][:, None]
    draft = at[None, :] - context
    bit = (s["tree"][:, None] >> draft.clamp(0, 63)) & 1
    return (draft < 0) | ((at < lengths[s["request"]][:, None]) & (bit == 1))


def _plain_attend(s):
    d = s["latent"]
    kv = s["cache"][s["table"].long()].flatten(1, 2)
    live = torch.arange(kv.shape[1], device="cuda") < s["lengths"][:, None]
    kv = torch.where(live[:, :, None], kv, torch.zeros_like(kv)).float()[s["request"]]
    z = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
    sees = _visible(s, kv.shape[1])[:, None, :]
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    top = z.amax(-1, keepdim=True)
    e = torch.where(sees, torch.exp(z - top), torch.zeros_like(z))
    return (torch.matmul(e, kv[:, :, :d]) / e.sum(-1, keepdim=True)).to(torch.bfloat16)


def _plain_query(s):
    y = torch.matmul(s["w"].float(), s["q"].float().unsqueeze(-1)).squeeze(-1)
    return torch.cat((y.to(torch.bfloat16), s["rope"]), -1)


def _to_mx(y):
    """MXFP8 of the last axis in blocks of 32: the smallest power of two under which no
    element passes 448, then E4M3 to nearest, ties to even."""
    rows = y.shape[0]
    y = y.reshape(rows, -1, 32)
    part, e = torch.frexp(y.abs().amax(-1))
    e = torch.where(part == 0, torch.zeros_like(e), e - 9 + (part > 0.875).int())
    x = torch.ldexp(y, -e[..., None]).to(torch.float8_e4m3fn)
    return x.view(rows, -1), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_values(s):
    y = torch.matmul(s["w"].float(), s["o"].float().unsqueeze(-1)).squeeze(-1)
    return _to_mx(y.flatten(1))


def _unpack(x, scale):
    """The values of MXFP8 codes."""
    v = x.view(torch.float8_e4m3fn).float().view(x.shape[0], -1, 32)
    return (v * torch.exp2(scale.float() - 127.0)[..., None]).view(x.shape)


def _plain_adapted(s):
    x, w = _unpack(s["x"], s["x_scale"]), _unpack(s["w"], s["w_scale"])
    a = s["which"].long().clamp(min=0)
    inner = torch.matmul(s["a"].float()[a], x[:, :, None]).squeeze(-1)
    alive = (torch.arange(s["rank"], device="cuda") < s["ranks"][a][:, None]) & (s["which"] >= 0)[:, None]
    inner = torch.where(alive, inner * s["gain"][a][:, None], torch.zeros_like(inner))
    low = torch.matmul(s["b"].float()[a], inner[:, :, None]).squeeze(-1)
    return (torch.matmul(x, w.t()) + low).to(torch.bfloat16) + 0.0  # no negative zero


_plain = {"attend": _plain_attend, "query": _plain_query, "values": _plain_values,
          "adapted": _plain_adapted}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        out = []
        page, d = case["page"], case["latent"]
        for b, (t, c) in enumerate(zip(_drafts(case), _contexts(case))):
            first = sum(_drafts(case)[:b])
            rows = torch.cat([s["cache"][int(i)] for i in s["table"][b, :(c + t + page - 1) // page]])
            rows = rows[:c + t].double()
            for j in range(first, first + t):
                tree = int(s["tree"][j])
                keep = torch.tensor(list(range(c)) + [c + i for i in range(t) if tree >> i & 1],
                                    device="cuda")
                mine = rows[keep]
                p = torch.softmax(s["q"][j].double() @ mine.t() * s["scale"], -1)
                out.append(p @ mine[:, :d])
        return torch.stack(out)
    if op == "query":
        y = torch.einsum("thi,hoi->tho", s["q"].double(), s["w"].double())
        return torch.cat((y, s["rope"].double()), -1)
    if op == "values":
        y = torch.einsum("thi,hoi->tho", s["o"].double(), s["w"].double())
        y = y.reshape(case["rows"], -1, 32)
        top = y.abs().amax(-1, keepdim=True)
        e = torch.where(top > 0, torch.ceil(torch.log2(top / 448.0)), torch.zeros_like(top))
        # Not rounded to E4M3, as the other operators' results are not rounded to BF16.
        return (y / torch.exp2(e)).flatten(1), torch.exp2(e).squeeze(-1)
    value = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()

    def dense(x, scale):
        return value[x.long()] * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)

    x = dense(s["x"], s["x_scale"])
    y = x @ dense(s["w"], s["w_scale"]).t()
    for t, (a, r) in enumerate((a, _ranks(case)[a]) for a in _which(case)):
        if a >= 0:
            inner = s["a"][a, :r].double() @ x[t]
            y[t] += s["gain"][a].double() * (s["b"][a, :, :r].double() @ inner)
    return y
