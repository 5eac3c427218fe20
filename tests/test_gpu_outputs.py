"""Outputs that the calls make: they belong to the call's stream."""
import threading
import time

import pytest
import torch

import mxfp8_gemm_mailbox_gb300 as mx
from tests.latent_cases import ROPE, Paged, normal

pytestmark = pytest.mark.gpu


def _latent():
    paged = Paged([300, 20], [3, 1], 512, 32)
    at, q = mx.LatentAttention(32), normal(1, 4, 32, 512 + ROPE)
    return lambda stream: at.run(q, paged.cache, paged.table, paged.lengths, paged.begin, 0.07,
                                 stream=stream)


def _query():
    q, rope, w = normal(1, 4, 32, 64), normal(2, 4, 32, ROPE), normal(3, 32, 512, 64)
    torch.cuda.synchronize()  # w may not be written by the kernel right before the call
    return lambda stream: mx.latent_query(q, rope, w, stream=stream)


def _values():
    o, w = normal(1, 4, 32, 512), normal(2, 32, 128, 512)
    torch.cuda.synchronize()  # as above
    return lambda stream: mx.latent_values(o, w, stream=stream)[0]


def _mailbox():
    mailbox, c = mx.Mailbox(8, 4096), normal(1, 4, 4096)

    def call(stream):
        mailbox.publish(c, stream=stream)
        return mailbox.consume(4, stream=stream)
    return call


def _tagged():
    mailbox, c = mx.TaggedMailbox(8, 4096), normal(1, 4, 4096)

    def call(stream):
        mailbox.publish(c, 5, stream=stream)
        return mailbox.consume(4, 5, stream=stream)
    return call


def _gather():
    gather, c = mx.LamportGather(1 << 16), normal(1, 4, 4096)
    return lambda stream: gather(c, stream=stream)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("make", [_latent, _query, _values, _mailbox, _tagged, _gather])
def test_an_output_is_not_memory_that_the_current_stream_still_reads(cuda, make, handle):
    call, side = make(), torch.cuda.Stream()
    want = call(None).clone()
    torch.cuda.synchronize()
    before = torch.full_like(want.view(torch.uint8), 7)
    kept, at = torch.empty_like(before), before.data_ptr()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    kept.copy_(before)  # waits behind it
    del before  # its block is the current stream's next of that size
    got = call(side.cuda_stream if handle else side)
    assert got.data_ptr() != at
    side.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    torch.cuda.synchronize()
    assert (kept == 7).all()
    # And on its release the block is the side stream's, not the current one's.
    at = got.data_ptr()
    del got
    assert torch.empty_like(kept).data_ptr() != at
    with torch.cuda.stream(side):
        assert call(None).data_ptr() == at


def test_the_default_streams_handles(cuda):
    call = _query()
    want = call(None)
    for handle in (0, 1):  # both the legacy default stream, torch's own
        assert torch.equal(call(handle), want)
    call = _tagged()
    want = call(None)
    for handle in (0, 1):
        assert torch.equal(call(handle), want)


def _weights():
    w = torch.randint(0, 0x78, (256, 512), dtype=torch.uint8, device="cuda")
    return w, torch.full((256, 16), 120, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("make,buffer", [
    (lambda stream: mx.Mailbox(8, 4096, stream=stream), "words"),
    (lambda stream: mx.TaggedMailbox(8, 4096, stream=stream), "pairs"),
    (lambda stream: mx.LamportGather(1 << 16, stream=stream), "words"),
    (lambda stream: mx.PublishGemm(*_weights(), mx.Mailbox(8, 256), stream=stream), "workspace")])
def test_an_objects_buffers_are_not_memory_that_the_current_stream_still_reads(cuda, make, buffer):
    side = torch.cuda.Stream()
    size = getattr(make(None), buffer).nbytes
    _weights()
    torch.cuda.synchronize()
    before = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    kept, at = torch.empty_like(before), before.data_ptr()
    torch.cuda._sleep(20_000_000)
    kept.copy_(before)
    del before
    made = make(side)
    assert getattr(made, buffer).data_ptr() != at
    torch.cuda.synchronize()
    assert (kept == 7).all()


@pytest.mark.parametrize("make", [_latent, _query, _values])
def test_other_threads_run_while_a_launch_waits_for_its_turn(cuda, make):
    """A launch blocks its thread where the GPU's queue is full."""
    call, gaps, stop = make(), [], threading.Event()
    call(None)
    torch.cuda.synchronize()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=tick)
    thread.start()
    start = time.perf_counter()
    torch.cuda._sleep(1_000_000_000)  # some 500 ms
    for _ in range(3000):
        call(None)
    issued = time.perf_counter() - start
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert issued > 0.3, "the queue was never full"
    assert max(gaps) < issued / 2


def test_a_consume_without_a_limit(cuda):
    mailbox, c = mx.Mailbox(8, 256), normal(1, 4, 256)
    for limit in (-1, 2 ** 64 - 1, 0):
        mailbox.publish(c)
        assert torch.equal(mailbox.consume(4, timeout_ns=limit), c)
    assert mailbox.status()[0] == mx.OK
