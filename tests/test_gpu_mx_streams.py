"""MXFP4 values given back on another stream than the current one: the memory of the result belongs to that stream."""
import pytest
import torch

from test_gpu_mxfp4 import draw, f8lin  # noqa: F401

pytestmark = pytest.mark.gpu

WAIT = 20_000_000  # clock ticks that a stream is held up for: long beside the calls after it


@pytest.fixture
def q(f8lin):
    q = f8lin.new_mxfp4(512, 520)
    f8lin.mxfp4_quantize(draw((512, 520), torch.bfloat16, 1).cuda(), q)
    return q


def test_a_block_that_the_current_stream_still_reads(q):
    want = q.dequantize()
    other, fives, kept = torch.cuda.Stream(), torch.full_like(want, 5.0), torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    kept.copy_(fives)
    del fives
    got = q.dequantize(stream=other)
    torch.cuda.synchronize()
    assert (kept == 5).all() and torch.equal(got, want)


def test_a_result_dropped_before_it_is_written(q):
    want, other = q.dequantize(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(WAIT)
    got = q.dequantize(stream=other)
    del got
    sevens = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    assert (sevens == 7).all()


def test_a_result_read_on_the_current_stream(q):
    """Dropped while the current stream, which waited for it, still has to read it; its memory is not given out before."""
    want, other = q.dequantize(), torch.cuda.Stream()
    kept = torch.empty_like(want)
    torch.cuda.synchronize()
    got = q.dequantize(stream=other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(WAIT)
    kept.copy_(got)
    del got
    with torch.cuda.stream(other):
        torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_streams_as_objects_and_handles(q):
    want, other = q.dequantize(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (other, other.cuda_stream, torch.cuda.current_stream(), torch.cuda.default_stream().cuda_stream, 0):
        got = q.dequantize(torch.bfloat16, stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(other):
        got = q.dequantize(stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
