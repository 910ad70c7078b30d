"""The allocating forms on a stream that is not the current one: their outputs and workspaces
are memory of that stream, so that work still queued on the current one cannot write into
them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _flat(x):
    return [t for y in x for t in _flat(y)] if isinstance(x, (tuple, list)) else [x]


def test_calls_do_not_take_memory_that_the_current_stream_still_uses():
    import exact_io_aware_13_gb300 as ea
    g = torch.Generator("cuda").manual_seed(90)
    q, k, v, do = (torch.randn(1, 4, 300, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    o, lse = ea.forward(q, k, v, mask_kind=ea.MASK_CAUSAL)

    def calls(stream):
        return _flat([ea.forward(q, k, v, mask_kind=ea.MASK_CAUSAL, stream=stream),
                      ea.backward(q, k, v, o, lse, do, mask_kind=ea.MASK_CAUSAL, stream=stream),
                      ea.quantize_fp8(q, stream=stream),
                      ea.forward_fp8(q, k, v, mask_kind=ea.MASK_CAUSAL, stream=stream),
                      ea.classify_tiles(ea.MASK_CAUSAL, 1000, 1000, stream=stream)])

    want = calls(None)
    sizes = [t.nbytes for t in want] + [max(ea.bwd_workspace_size(q, k), 256)]
    s = torch.cuda.Stream()
    for stream in (s, torch.cuda.ExternalStream(s.cuda_stream)):
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)                  # some 10 ms on the current stream
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        del junk                                       # its fills are still queued
        got = calls(stream)
        s.synchronize()
        torch.cuda.synchronize()
        assert ea.device_status() == 0
        for a, b in zip(got, want):
            if a.dtype == torch.uint8:                 # rows of codes may have bytes that mean nothing
                a, b = a[..., :300], b[..., :300]
            assert torch.equal(a, b)
        del got
