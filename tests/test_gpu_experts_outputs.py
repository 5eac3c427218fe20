"""Outputs of the calls of a layer of routed experts: they belong to the call's stream; threads
and other streams beside them."""
import threading

import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from tests.experts_cases import begin_of, generator, random_codes
from tests.test_gpu_outputs import (
    test_an_output_is_not_memory_that_the_current_stream_still_reads as check_output,
    test_other_threads_run_while_a_launch_waits_for_its_turn as check_threads)

pytestmark = pytest.mark.gpu


def _rows(n=512):
    return torch.randn(64, n, generator=generator(1), device="cuda").to(torch.bfloat16)


def _quantize():
    x = _rows()
    return lambda stream: mx.quantize(x, "mxfp8", stream=stream)[0]


def _dequantize():
    codes, scale = random_codes(2, (64,), 512, 4)
    return lambda stream: mx.dequantize(codes, scale, stream=stream)


def _product(gated=False):
    w, w_scale = random_codes(3, (4, 512), 256, 4, -6, -4)
    x, x_scale = random_codes(4, (40,), 256, 8)
    begin = begin_of([10, 0, 25, 5])
    product = mx.ExpertProduct(w, w_scale, gated=gated)
    if gated:
        return lambda stream: product.run(x, x_scale, begin, format="mxfp8", stream=stream)[0]
    return lambda stream: product.run(x, x_scale, begin, stream=stream)


def _gated():
    return _product(True)


def _combine():
    y = _rows(2048)
    weight = torch.rand(32, 2, generator=generator(5), device="cuda")
    slot = torch.randperm(64, generator=generator(6), device="cuda").view(32, 2).int()
    return lambda stream: mx.combine(y, weight, slot, stream=stream)


MAKERS = [_quantize, _dequantize, _product, _gated, _combine]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("make", MAKERS)
def test_an_output_is_the_calls_streams_memory(cuda, make, handle):
    check_output(cuda, make, handle)


@pytest.mark.parametrize("make", MAKERS)
def test_other_threads_run_while_a_launch_waits(cuda, make):
    check_threads(cuda, make)


def test_a_routing_is_one_piece_of_the_calls_streams_memory(cuda):
    logits = torch.randn(300, 64, generator=generator(7), device="cuda")
    want = [t.clone() for t in mx.route(logits, 8)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mx.route(logits, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len({t.untyped_storage().data_ptr() for t in got}) == 1
    assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in got)
    begin = got.begin  # any of the five keeps the memory
    del got
    again = mx.route(torch.zeros_like(logits), 8, stream=side)
    side.synchronize()
    assert torch.equal(begin, want[4]) and again.begin.data_ptr() != begin.data_ptr()


def test_two_products_on_two_streams_at_once(cuda):
    """Each with a workspace of its own."""
    makers = [(_product(), torch.cuda.Stream()), (_gated(), torch.cuda.Stream())]
    # Long sums on few tiles too, whose pieces meet in the workspace.
    w, w_scale = random_codes(8, (256,), 16384, 8, -9, -7)
    x, x_scale = random_codes(9, (6,), 16384, 8)
    for _ in range(2):
        product = mx.ExpertProduct(w, w_scale)
        makers.append((lambda stream, p=product: p.run(x, x_scale, stream=stream),
                       torch.cuda.Stream()))
    want = [call(None).clone() for call, _ in makers]
    torch.cuda.synchronize()
    got = [[] for _ in makers]

    def work(i):
        call, stream = makers[i]
        with torch.cuda.stream(stream):
            for _ in range(50):
                got[i].append(call(None))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(makers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert all(torch.equal(t.view(torch.uint8), v.view(torch.uint8)) for t in g)


def test_rows_that_are_left_in_deterministic_mode(cuda):
    """What torch fills new memory with there: NaN, a type's largest where it has none."""
    w, w_scale = random_codes(3, (1, 512), 256, 4, -6, -4)
    x, x_scale = random_codes(4, (40,), 256, 8)
    begin = begin_of([10])
    product = mx.ExpertProduct(w, w_scale)
    rows = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    rows[:10] = torch.arange(10, device="cuda")
    calls = [lambda: [product.run(x, x_scale, begin)]]
    for format in ("mxfp8", "mxfp4"):
        calls.append(lambda f=format: product.run(x, x_scale, begin, format=f))
        calls.append(lambda f=format: mx.quantize(_rows(), f, rows=rows))
    was = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled()
    for call in calls:
        plain = call()
        for t in plain:  # (what the next outputs' memory holds)
            t.view(torch.uint8).fill_(0x11)
        plain = [t.clone() for t in call()]
        torch.use_deterministic_algorithms(True, warn_only=True)
        try:
            got = call()
        finally:
            torch.use_deterministic_algorithms(was[0], warn_only=was[1])
        for a, b in zip(got, plain):
            assert torch.equal(a[:10].view(torch.uint8), b[:10].view(torch.uint8))
            rest = a[10:]
            assert torch.isnan(rest.float()).all() if rest.is_floating_point() else (rest == 255).all()
