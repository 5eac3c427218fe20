"""Latent attention on the GPU against float64.

Tolerances.  attend: the softmax weights are rounded to BF16 (2^-8 of each at
most, so 2^-8 of the weights' sum over |c|) and the result once more (2^-8 of
itself): 2^-8 (|y| + sum p |c|), of which the roundings' mixed signs leave
room for the FP32 sums, the exponential and the normaliser (some 2^-20).
query: half a BF16 step at the value, and FP32 sums of up to 512 products,
512 x 2^-24 of the absolute sum.
values: E4M3's half step, 2^-4 of an element or 2^-10 of its block's scale."""
import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from tests.latent_cases import ROPE, Paged, masks_tensor, normal

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def close(got, want, weight):
    assert got.shape == want.shape and got.dtype == torch.bfloat16
    assert torch.isfinite(got).all()
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * (want.abs() + weight) + 1e-30
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{worst:.2f} x the tolerance"


def attend(cuda, paged, heads, masks=None, seed=5, scale=SCALE, q=None, cache=None, at=None):
    at = at or mx.LatentAttention(heads, paged.latent)
    q = normal(seed, paged.rows, heads, paged.latent + ROPE) if q is None else q
    tree = None if masks is None else masks_tensor(masks)
    got = at.run(q, paged.cache if cache is None else cache, paged.table, paged.lengths,
                 paged.begin, scale, tree=tree)
    assert at.status() == 0
    close(got, *paged.expected(q, scale, masks))
    return got


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("context", [0, 1, 62, 63, 64, 65, 127, 128, 700])
def test_context_lengths_around_a_tile(cuda, latent, context):
    attend(cuda, Paged([context], [1], latent, 64), 16)


@pytest.mark.parametrize("heads", [1, 5, 31, 32, 33, 64, 100, 128, 130, 256])
def test_head_counts(cuda, heads):
    attend(cuda, Paged([300, 70], [2, 1], 512, 32), heads)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 96, 128, 1024])
@pytest.mark.parametrize("latent", [256, 512])
def test_page_sizes(cuda, page, latent):
    attend(cuda, Paged([517, 90, 8], [3, 1, 2], latent, page, seed=page), 24)


@pytest.mark.parametrize("drafts", [1, 2, 7, 8, 33, 64])
def test_chains_and_trees(cuda, drafts):
    paged = Paged([201, 0, 64], [drafts, drafts, max(1, drafts - 1)], 512, 32, seed=drafts)
    attend(cuda, paged, 20)
    attend(cuda, paged, 20, masks=paged.random_tree(drafts))


def test_a_long_chain_without_a_tree(cuda):
    attend(cuda, Paged([100], [150], 256, 16), 6)


def test_long_contexts_split_over_the_gpu(cuda):
    attend(cuda, Paged([20011], [1], 512, 64), 128)
    attend(cuda, Paged([9000, 17, 4000], [2, 4, 2], 512, 128, seed=1), 64)


def test_many_requests_some_without_rows(cuda):
    contexts = [(37 * b) % 211 for b in range(256)]
    drafts = [(b * 5) % 3 for b in range(256)]
    attend(cuda, Paged(contexts, drafts, 256, 8), 3)


def test_rows_that_see_nothing_give_zeros(cuda):
    paged = Paged([0, 5], [3, 2], 512, 16)
    masks = [0, 0b010, 0, 0, 0b10]
    got = attend(cuda, paged, 40, masks=masks)
    assert (got[0] == 0).all() and (got[2] == 0).all()
    assert (got[3] != 0).any()
    # a length of zero, with rows: nothing to see either
    at = mx.LatentAttention(40)
    empty = torch.zeros_like(paged.lengths)
    out = at.run(normal(1, 5, 40, 576), paged.cache, paged.table, empty, paged.begin, SCALE)
    assert (out == 0).all() and at.status() == 0


def test_rows_outside_every_request_give_zeros(cuda):
    paged = Paged([30], [2], 256, 16)
    at = mx.LatentAttention(8, 256)
    q = normal(2, 5, 8, 320)
    out = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
    want, weight = paged.expected(q[:2], SCALE)
    close(out[:2], want, weight)
    assert (out[2:] == 0).all()


def test_no_rows_launch_nothing(cuda):
    paged = Paged([30], [0], 256, 16)
    at = mx.LatentAttention(8, 256)
    out = at.run(normal(2, 0, 8, 320), paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
    assert out.shape == (0, 8, 256)
    assert mx.latent_query(normal(1, 0, 4, 64), normal(1, 0, 4, 64), normal(1, 4, 256, 64)).shape \
        == (0, 4, 320)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -3e38])
def test_poison_past_the_length_has_no_effect(cuda, poison):
    for context in (0, 40, 63, 64, 100):
        attend(cuda, Paged([context, 3], [1, 2], 512, 32, poison=poison), 16)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at_column", [0, 200, 300, 511, 512, 575])
def test_poison_in_a_draft_reaches_only_the_rows_that_see_it(cuda, value, at_column):
    paged = Paged([61], [6], 512, 16)
    bad = 2
    masks = [0b1, 0b11, 0b111, 0b1001, 0b11001, 0b100111]
    q = normal(9, 6, 40, 576)
    want, weight = paged.expected(q, SCALE, masks)
    position = 61 + bad
    page = int(paged.table[0, position // 16])
    paged.cache[page, position % 16, at_column] = value
    at = mx.LatentAttention(40)
    got = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE,
                 tree=masks_tensor(masks))
    for row, mask in enumerate(masks):
        if not mask >> bad & 1:
            close(got[row], want[row], weight[row])
        elif at_column < 512:
            assert torch.isnan(got[row]).all()


def test_growing_scores_move_the_running_maximum(cuda):
    # Keys along q with growing length: every tile holds a new maximum, far past the last.
    def keys(b, n, width):
        base = normal(3, 1, width)
        return (base * torch.linspace(0.01, 3.0, n, device="cuda")[:, None]).to(torch.bfloat16)

    paged = Paged([640], [1], 512, 64, keys=keys)
    q = (normal(3, 1, 576) * torch.linspace(0.5, 2, 128, device="cuda")[:, None]).to(torch.bfloat16)
    attend(cuda, paged, 128, q=q[None], scale=1.0)
    attend(cuda, paged, 128, q=-q[None], scale=1.0)  # falling ones: the first tile holds it


def test_scores_of_very_negative_and_equal_values(cuda):
    def keys(b, n, width):
        return torch.full((n, width), -8.0, dtype=torch.bfloat16, device="cuda")

    paged = Paged([130], [2], 256, 32, keys=keys)
    q = torch.full((2, 16, 320), 64.0, dtype=torch.bfloat16, device="cuda")
    got = attend(cuda, paged, 16, q=q, scale=4.0)
    assert (got == -8.0).all()


def test_strided_pool(cuda):
    paged = Paged([300], [2], 512, 16)
    pool = torch.full((paged.cache.shape[0], 3, 16, 584), float("nan"), dtype=torch.bfloat16,
                      device="cuda")
    pool[:, 1, :, :576] = paged.cache
    attend(cuda, paged, 48, cache=pool[:, 1, :, :576])


def test_offsets_past_32_bits(cuda):
    # 2^32 elements before the pages in use.
    paged = Paged([400], [2], 512, 64, spare=0)
    first = (1 << 32) // (64 * 576) + 1
    pool = torch.empty((first + paged.cache.shape[0], 64, 576), dtype=torch.bfloat16, device="cuda")
    pool[first:] = paged.cache
    paged.table += first
    attend(cuda, paged, 16, cache=pool)


def test_same_bits_again_on_another_stream_and_from_a_graph(cuda):
    paged = Paged([5000, 300], [3, 2], 512, 64)
    at = mx.LatentAttention(128)
    q = normal(4, 5, 128, 576)
    args = (q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
    first = at.run(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        second = at.run(*args)
    third = at.run(*args, out=torch.full_like(first, float("nan")), stream=side)
    side.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            at.run(*args, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # lengths are read on the device: the same graph serves a shorter cache
    paged.lengths.copy_(torch.tensor([1003, 17], dtype=torch.int32))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    paged.contexts = [1000, 15]
    paged.tokens = [paged.tokens[0][:1003], paged.tokens[1][:17]]
    close(out, *paged.expected(q, SCALE))
    assert at.status() == 0


def test_indexes_out_of_range_raise_the_flag(cuda):
    paged = Paged([100], [2], 512, 32)
    q = normal(4, 2, 16, 576)

    def run(table=None, lengths=None, begin=None):
        at = mx.LatentAttention(16)
        out = at.run(q, paged.cache, paged.table if table is None else table,
                     paged.lengths if lengths is None else lengths,
                     paged.begin if begin is None else begin, SCALE)
        return out, at.status()

    assert run()[1] == 0
    for page in (-1, paged.cache.shape[0], 1 << 30):
        table = paged.table.clone()
        table[0, 1] = page
        out, flags = run(table=table)
        assert flags == mx.FLAG_BAD_INDEX and torch.isfinite(out).all()
    long = torch.full_like(paged.lengths, 10 ** 9)
    # cut at the table's end: the last slots hold poison there, so only the flag is checked
    assert run(lengths=long)[1] & mx.FLAG_BAD_INDEX
    begin = paged.begin.clone()
    begin[1] = 40
    assert run(begin=begin)[1] & mx.FLAG_BAD_INDEX


@pytest.mark.parametrize("rows,heads,nope,latent", [
    (1, 1, 32, 256), (1, 16, 128, 512), (3, 7, 96, 512), (8, 128, 128, 512), (9, 5, 192, 256),
    (40, 3, 64, 512), (2, 4, 512, 512)])
def test_query(cuda, rows, heads, nope, latent):
    q, rope = normal(1, rows, heads, nope), normal(2, rows, heads, ROPE)
    w = normal(3, heads, latent, nope)
    got = mx.latent_query(q, rope, w)
    want = torch.einsum("thi,hoi->tho", q.double(), w.double())
    size = torch.einsum("thi,hoi->tho", q.double().abs(), w.double().abs())
    assert got.shape == (rows, heads, latent + ROPE)
    err = (got[..., :latent].double() - want).abs()
    half_step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -126))) - 8)
    assert (err <= half_step + 512 * 2.0 ** -24 * size).all()
    assert torch.equal(got[..., latent:], rope)


@pytest.mark.parametrize("rows,heads,value,latent", [
    (1, 1, 32, 256), (1, 32, 128, 512), (3, 7, 96, 512), (8, 128, 128, 512), (9, 5, 64, 256),
    (40, 3, 160, 512), (2, 4, 512, 512)])
def test_values(cuda, rows, heads, value, latent):
    o, w = normal(1, rows, heads, latent), normal(3, heads, value, latent, std=0.1)
    x, scale = mx.latent_values(o, w)
    y = torch.einsum("thi,hoi->tho", o.double(), w.double()).reshape(rows, -1, 32)
    size = torch.einsum("thi,hoi->tho", o.double().abs(), w.double().abs()).reshape(rows, -1, 32)
    top = y.abs().amax(-1)
    s = torch.exp2(scale.view(torch.uint8).double() - 127)
    slack = 512 * 2.0 ** -24 * size.amax(-1)
    assert (top <= 448 * s + slack).all(), "an element passes 448"
    assert (top >= 224 * s - slack).all(), "the scale is not the smallest"
    v = x.float().double().reshape(rows, -1, 32) * s[..., None]
    err = (v - y).abs()
    tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s[..., None]) + 512 * 2.0 ** -24 * size
    assert (err <= tol).all()


def test_values_of_zeros_extremes_and_nan(cuda):
    w = torch.zeros((2, 64, 256), dtype=torch.bfloat16, device="cuda")
    w[:, torch.arange(64), torch.arange(64)] = 1.0  # y = o's first 64 numbers
    o = torch.zeros((5, 2, 256), dtype=torch.bfloat16, device="cuda")
    o[0, 0, 0], o[0, 0, 1] = 448.0, -1.0
    o[0, 1, 40] = 898.0  # 896 in BF16: 448 x 2 exactly
    o[0, 0, 40] = 900.0  # past it: the next power, 225 rounded to 224
    o[1, 0, 3], o[1, 0, 4] = float("nan"), 2.0
    o[2, 0, 0] = 2.0 ** -126
    o[3, 0, 0] = 3.0e38
    x, scale = mx.latent_values(o, w)
    codes = scale.view(torch.uint8)
    v = x.float()
    assert codes[4].eq(127).all() and v[4].eq(0).all()
    assert codes[0, 0] == 127 and v[0, 0] == 448 and v[0, 1] == -1
    assert codes[0, 3] == 128 and v[0, 64 + 40] == 448
    assert codes[0, 1] == 129 and v[0, 40] == 224
    # 0 x NaN is NaN: every output of the head; blocks of NaN alone take 2^0
    assert torch.isnan(v[1, :64]).all() and codes[1, :2].eq(127).all() and v[1, 64:].eq(0).all()
    assert codes[2, 0] == 0 and v[2, 0] > 0
    assert codes[3, 0] == 127 + 127 - 8 + 1 and v[3, 0] == 224
    w[0, 3, 200] = float("nan")  # one output alone: it does not count towards the scale
    o[4, 0, 4] = 2.0
    x, scale = mx.latent_values(o, w)
    v, codes = x.float(), scale.view(torch.uint8)
    assert torch.isnan(v[4, 3]) and v[4, 4] == 256 and codes[4, 0] == 120


def test_the_whole_step_feeds_the_projection(cuda):
    """query, attend, values, projection with adapters, consumer, in one graph,
    against float64 of the rounded intermediates."""
    heads, value, nope, latent, n, rows = 16, 128, 64, 512, 256, 4
    k = heads * value
    paged = Paged([90, 300], [3, 1], latent, 16)
    masks = paged.random_tree(1)
    wq, wv = normal(1, heads, latent, nope, std=0.1), normal(2, heads, value, latent, std=0.05)
    q_nope, q_rope = normal(3, rows, heads, nope), normal(4, rows, heads, ROPE)
    w = torch.randn(n, k, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.randint(120, 130, (n, k // 32), dtype=torch.uint8, device="cuda")
    mailbox = mx.Mailbox(8, n)
    gemm = mx.PublishGemm(w, ws, mailbox)
    a, b = normal(5, 2, 12, k, std=0.02), normal(6, 2, n, 12)
    adapters = mx.Adapters(a, b)
    which = torch.tensor([1, -1, 0, 1], dtype=torch.int32, device="cuda")
    at = mx.LatentAttention(heads, latent)
    out = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    tree = masks_tensor(masks)

    def step():
        q = mx.latent_query(q_nope, q_rope, wq)
        o = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE, tree=tree)
        x, xs = mx.latent_values(o, wv)
        gemm.run_adapted(x, xs, adapters, which)
        mailbox.consume(rows, out)
        return q, o, x, xs

    q, o, x, xs = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    eager = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    close(o, *paged.expected(q, SCALE, masks))
    dense = lambda c, s: (c.view(torch.float8_e4m3fn).float().double()  # noqa: E731
                          * torch.exp2(s.view(torch.uint8).double() - 127).repeat_interleave(32, 1))
    xd = dense(x, xs)
    want = xd @ dense(w, ws).t()
    size = xd.abs() @ dense(w, ws).abs().t()
    for t, i in enumerate([1, -1, 0, 1]):
        if i >= 0:
            want[t] += b[i].double() @ (a[i].double() @ xd[t])
            size[t] += b[i].double().abs() @ (a[i].double().abs() @ xd[t].abs())
    err = (eager.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all()
    assert mailbox.status()[0] == mx.OK


@pytest.mark.parametrize("latent,page", [(256, 8), (512, 64)])
@pytest.mark.parametrize("heads", [3, 100])
@pytest.mark.parametrize("contexts", [(30, 150), (150, 30), (300, 30)])
def test_several_row_tiles_in_a_share(cuda, latent, page, heads, contexts):
    # More row tiles than the GPU takes at once: each share holds parts of several.
    attend(cuda, Paged(contexts * 60, [1] * 120, latent, page), heads)


@pytest.mark.parametrize("latent", [256, 512])
def test_long_shares_of_one_and_of_several_row_tiles(cuda, latent):
    attend(cuda, Paged([30011, 29000], [1, 2], latent, 64), 128)
    attend(cuda, Paged([700 + 13 * b for b in range(90)], [1] * 90, latent, 32), 128)


def test_short_tables_are_never_cut_long_ones_are(cuda):
    # 256 tokens at most: one kernel; the same lengths under a table of more pages: two.
    short = Paged([200, 0, 256], [2, 1, 0], 512, 64)
    attend(cuda, short, 70)
    short.table = torch.cat([short.table, torch.full_like(short.table, -7)], 1)
    attend(cuda, short, 70)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_draft_is_nan_whatever_its_scores(cuda, value):
    # q . c is -inf or +inf by the sign of q there: NaN for the rows that see it either way.
    for column in (0, 255, 256, 511):
        paged = Paged([70], [2], 512, 32)
        paged.cache[int(paged.table[0, 70 // 32]), 70 % 32, column] = value
        q = normal(4, 2, 32, 576)
        q[:, ::2, column], q[:, 1::2, column] = 1.0, -1.0
        at = mx.LatentAttention(32)
        got = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE,
                     tree=masks_tensor([1, 2]))
        assert torch.isnan(got[0]).all() and at.status() == 0
        want, weight = paged.expected(q, SCALE, [1, 2])
        close(got[1], want[1], weight[1])


def test_rows_given_twice_are_refused_on_the_device(cuda):
    # Descending row ranges would be more rows than the call has.
    paged = Paged([30] * 8, [1] * 8, 256, 16)
    begin = torch.tensor([0, 8] * 4 + [0], dtype=torch.int32, device="cuda")
    at = mx.LatentAttention(128, 256)
    out = at.run(normal(1, 8, 128, 320), paged.cache, paged.table, paged.lengths, begin, SCALE)
    assert out.shape == (8, 128, 256)
    assert at.status() & mx.FLAG_BAD_INDEX


def test_streams_outputs_and_refusals_of_the_calls(cuda):
    paged = Paged([100], [2], 256, 16)
    at = mx.LatentAttention(8, 256)
    q = normal(1, 2, 8, 320)
    args = (q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
    first = at.run(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(first)
    assert at.run(*args, out=out, stream=side.cuda_stream) is out  # a handle in place of a Stream
    side.synchronize()
    assert torch.equal(out, first)
    with pytest.raises(TypeError):
        at.run(*args, stream=object())
    with pytest.raises(TypeError, match="int32"):
        at.run(q, paged.cache, paged.table, paged.lengths.long(), paged.begin, SCALE)
    with pytest.raises(ValueError, match="row_begin"):
        at.run(q, paged.cache, paged.table, paged.lengths, paged.begin[:1], SCALE)
    with pytest.raises(ValueError, match="contiguous"):
        at.run(q.transpose(0, 1).contiguous().transpose(0, 1), *args[1:])
    with pytest.raises(ValueError, match="cache"):
        at.run(q, paged.cache.transpose(1, 2).contiguous().transpose(1, 2), *args[2:])
    with pytest.raises(ValueError, match="out"):
        at.run(*args, out=out[:1])
    with pytest.raises(mx.Mxfp8Error, match="scale"):
        at.run(*args[:5], 0.0)
    w = normal(2, 8, 64, 256)
    x, scale = mx.latent_values(first, w)
    x2, scale2 = torch.empty_like(x), torch.empty_like(scale)
    got = mx.latent_values(first, w, x2, scale2)
    assert got[0] is x2 and got[1] is scale2
    assert torch.equal(x.view(torch.uint8), x2.view(torch.uint8))
    assert torch.equal(scale.view(torch.uint8), scale2.view(torch.uint8))
    with pytest.raises(TypeError, match="one-byte"):
        mx.latent_values(first, w, x2.float(), scale2)
    assert at.status() == 0


def test_calls_in_a_row_share_the_sms_with_the_projections_clusters(cuda):
    """The next kernels' CTAs take an SM as soon as one of a pair has left it: nothing of the
    pair may still be on its way to that shared memory."""
    paged = Paged([900, 130], [3, 1], 512, 64)
    at, q = mx.LatentAttention(64), normal(1, 4, 64, 576)
    narrow = Paged([300], [2], 256, 32, seed=3)
    at2, q2 = mx.LatentAttention(16, 256), normal(2, 2, 16, 320)
    n, k = 4096, 1024
    mailbox = mx.Mailbox(8, n)
    gemm = mx.PublishGemm(torch.randint(0, 0x78, (n, k), dtype=torch.uint8, device="cuda"),
                          torch.full((n, k // 32), 120, dtype=torch.uint8, device="cuda"), mailbox,
                          split_k=4)
    x = torch.randint(0, 0x78, (8, k), dtype=torch.uint8, device="cuda")
    xs = torch.full((8, k // 32), 120, dtype=torch.uint8, device="cuda")

    def step():
        a = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
        gemm.run(x, xs)
        b = mailbox.consume(8)
        return a, b, at2.run(q2, narrow.cache, narrow.table, narrow.lengths, narrow.begin, SCALE)

    first = step()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        for got, want in zip(step(), first):
            differ += (got.view(torch.int16) != want.view(torch.int16)).sum()
    assert differ.item() == 0
    close(first[0], *paged.expected(q, SCALE))
    assert at.status() == 0 and at2.status() == 0 and mailbox.status()[0] == mx.OK


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("offset", [8, 16, 24])
def test_outputs_on_any_16_byte_boundary(cuda, latent, offset):
    # Uncut row tiles (a short table), cut ones, and rows of zeros.
    for contexts, heads in (([60, 0, 200], 40), ([9000, 30], 70)):
        drafts = [2, 0, 1][:len(contexts)]
        paged = Paged(contexts, drafts, latent, 16, seed=offset)
        at, q = mx.LatentAttention(heads, latent), normal(5, paged.rows + 1, heads, latent + ROPE)
        args = (paged.cache, paged.table, paged.lengths, paged.begin, SCALE)
        want = at.run(q, *args)
        pool = torch.full((want.numel() + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = pool[offset:offset + want.numel()].view(want.shape)
        assert out.data_ptr() % 32 == offset * 2 % 32
        at.run(q, *args, out=out)
        assert torch.equal(out, want) and (want[-1] == 0).all()
        assert (pool[:offset] == 7).all() and (pool[offset + want.numel():] == 7).all()
        assert at.status() == 0


def test_infinite_values_become_nan(cuda):
    # An infinity has no E4M3 code: it is NaN, and as little part of its block's scale.
    w = torch.zeros((2, 64, 256), dtype=torch.bfloat16, device="cuda")
    w[:, torch.arange(64), torch.arange(64)] = 1.0  # y = o's first 64 numbers
    o = normal(1, 3, 2, 256)

    def values(o, w):
        torch.cuda.synchronize()  # w may not be written by the kernel right before the call
        return mx.latent_values(o, w)

    for value in (float("inf"), float("-inf")):
        w[0, 5, 5], w[1, 40, 7] = value, value  # o[t][0][5] x inf, o[t][1][7] x inf
        x, scale = values(o, w)
        v, codes = x.float(), scale.view(torch.uint8)
        assert torch.isnan(v[:, 5]).all() and torch.isnan(v[:, 64 + 40]).all()
        # The rest of a block as if that number were not there.
        rest = o.clone()
        rest[:, 0, 5] = 0
        clean = torch.zeros_like(w)
        clean[:, torch.arange(64), torch.arange(64)] = 1.0
        clean[1, 40] = 0
        y, y_scale = values(rest, clean)
        y, keep = y.float(), torch.ones(128, dtype=torch.bool, device="cuda")
        keep[[5, 64 + 40]] = False
        assert torch.equal(v[:, keep], y[:, keep])
        assert torch.equal(codes, y_scale.view(torch.uint8))
    # A sum past FP32 is such an infinity too.
    w.zero_()
    w[0, 3, :2] = 3e38
    o[:, 0, :2] = 3.0
    assert torch.isnan(values(o, w)[0].float()[:, 3]).all()


@pytest.mark.parametrize("drafts,length", [(2, 1), (6, 4), (70, 65), (70, 3)])
def test_fewer_tokens_than_drafts(cuda, drafts, length):
    # Token p is draft p - (length - drafts): the first drafts have no token.
    first = drafts - length
    paged = Paged([0], [drafts], 512, 16)
    q, heads = normal(7, drafts, 9, 576), 9
    at = mx.LatentAttention(heads)
    lengths = torch.full_like(paged.lengths, length)
    masks = [(0x9E3779B97F4A7C15 * (t + 1)) & (1 << 64) - 1 for t in range(drafts)]
    for tree in (None, masks):
        got = at.run(q, paged.cache, paged.table, lengths, paged.begin, SCALE,
                     tree=None if tree is None else masks_tensor(tree))
        for t in range(drafts):
            sees = [p for p in range(length)
                    if (p + first <= t if tree is None
                        else p + first < 64 and tree[t] >> (p + first) & 1)]
            if not sees:
                assert (got[t] == 0).all()
                continue
            mine = paged.tokens[0][torch.tensor(sees, device="cuda")].double()
            p = torch.softmax(q[t].double() @ mine.t() * SCALE, -1)
            close(got[t], p @ mine[:, :512], p @ mine[:, :512].abs())


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20, 2.0 ** 40])
@pytest.mark.parametrize("context", [30, 5000])
def test_scores_far_past_the_exponentials_range(cuda, size, context):
    # Spreads of 1e5 and more, so that one token has all of the weight: the errors of an FP32
    # score do not reach the next.
    def keys(b, n, width):
        k = normal(8, n, width) * 2.0 ** -9
        k[:, 0] = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to("cuda") % 256
        k[(k[:, 0] == 255).nonzero()[1:, 0], 0] = 0.0
        return k.to(torch.bfloat16)

    paged = Paged([context], [1], 512, 64, keys=keys)
    q = normal(9, 1, 20, 576) * 2.0 ** -9
    q[:, :, 0] = torch.where(torch.arange(20, device="cuda") % 2 == 0, size, size * 1.5)
    attend(cuda, paged, 20, q=q.to(torch.bfloat16), scale=1.0)


@pytest.mark.parametrize("context", [40, 700, 9000])
def test_scores_of_minus_infinity(cuda, context):
    # Infinite keys under a positive query: those tokens alone drop out.
    paged = Paged([context], [2], 512, 32)
    q = normal(3, 2, 40, 576)
    q[:, :, 570] = 1.0
    page = paged.table[0].long()
    keys = paged.tokens[0].clone()
    keys[:context * 3 // 4, 570] = float("-inf")
    for i in range(len(page)):
        part = keys[i * 32:(i + 1) * 32]
        paged.cache[page[i], :part.shape[0]] = part
    paged.tokens[0] = keys
    attend(cuda, paged, 40, q=q)
    # Every key: the formula is inf - inf, which must not pass for a row that sees nothing.
    keys[:, 570] = float("-inf")
    for i in range(len(page)):
        part = keys[i * 32:(i + 1) * 32]
        paged.cache[page[i], :part.shape[0]] = part
    at = mx.LatentAttention(40)
    masks = masks_tensor([0, 0b11])
    got = at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, SCALE, tree=masks)
    assert torch.isnan(got).all()
    short = Paged([0], [2], 512, 32)
    short.cache[short.table[0, 0], :, 570] = float("-inf")
    got = at.run(q, short.cache, short.table, short.lengths, short.begin, SCALE, tree=masks)
    assert (got[0] == 0).all() and torch.isnan(got[1]).all()
    assert at.status() == 0


@pytest.mark.parametrize("scale", [3e38, 1e38, 1e-38, 1e-44])
def test_the_scale_over_its_whole_range(cuda, scale):
    # Scores of small integers: exact, with ties, which share the weight at a great scale.
    def keys(b, n, width):
        k = torch.zeros((n, width), device="cuda")
        k[:, 0] = torch.arange(n, device="cuda") % 7 - 3
        k[:, 1:100] = normal(8, n, 99)
        return k.to(torch.bfloat16)

    paged = Paged([300, 40], [1, 2], 512, 64, keys=keys)
    q = torch.zeros((3, 12, 576), dtype=torch.bfloat16, device="cuda")
    q[:, ::2, 0], q[:, 1::2, 0] = 1.0, -2.0
    attend(cuda, paged, 12, q=q, scale=scale)
