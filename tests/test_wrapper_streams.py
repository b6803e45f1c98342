"""What the allocating functions allocate belongs to the stream that they launch on.

torch's allocator hands a freed block out again at once to the stream that it was allocated for, whose
queue then orders the old use before the new one.  A kernel on another stream is not in that queue: memory
taken from the current stream may still be written by work queued there before.  So with ``stream`` given,
outputs and scratch come from that stream's memory, and the outputs are kept, once freed, until what the
caller's current stream had queued is done.

Without a GPU: the allocations and the streams that are current then, through stand-ins.  With one
(``gpu``): the segments that the outputs lie in, and the results with work held back on either stream.
"""
import contextlib

import numpy as np
import pytest

import fp8_fine_grained_fp8bs_gb300 as fp8bs
from _gpu import require_gpu
from test_wrapper_checks import _codes, claim, launched  # noqa: F401

torch = pytest.importorskip("torch")


def calls(tensor, codes):
    """Every allocating function on small inputs: name -> call taking ``stream``."""
    bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    x, w = tensor((128, 256), bf16), tensor((256, 256), bf16)
    q, s = tensor((128, 256), u8), tensor((2, 128), torch.float32)
    wq, ws = tensor((256, 256), u8), tensor((2, 2), torch.float32)
    off = torch.tensor([0, 128], dtype=i32, device=x.device)
    off = claim(off) if not off.is_cuda else off
    z, idx, dw = tensor((40, 16), torch.float32), tensor((40, 2), i32), tensor((40, 2), torch.float32)
    a, b, e = codes(128, 128, 0), codes(256, 128, 0), codes(256, 128, 0, 1)
    return {
        "quantize_act": lambda st: fp8bs.quantize_act(x, True, stream=st),
        "quantize_weight": lambda st: fp8bs.quantize_weight(w, True, False, st),
        "quantize_act_weight": lambda st: fp8bs.quantize_act_weight(x, w, stream=st),
        "swiglu_quantize": lambda st: fp8bs.swiglu_quantize(x, stream=st),
        "requant_1x128_to_128x1": lambda st: fp8bs.requant_1x128_to_128x1(q, s, stream=st),
        "gemm": lambda st: fp8bs.gemm(q, s, wq, ws, stream=st),
        "grouped_gemm": lambda st: fp8bs.grouped_gemm(q, s, off, wq[None], ws[None], stream=st),
        "diag_gemm_unpromoted": lambda st: fp8bs.diag_gemm_unpromoted(q, wq, st),
        "quantize_fp4": lambda st: fp8bs.quantize_fp4(x, stream=st),
        "quantize_fp4 of experts": lambda st: fp8bs.quantize_fp4(w.view(2, 128, 256), 0, None, st),
        "swiglu_quantize_fp4": lambda st: fp8bs.swiglu_quantize_fp4(x, stream=st),
        "dequantize_fp4": lambda st: fp8bs.dequantize_fp4(*a, stream=st),
        "gemm_fp4": lambda st: fp8bs.gemm_fp4(a, b, stream=st),
        "grouped_gemm_fp4": lambda st: fp8bs.grouped_gemm_fp4(a, off, e, stream=st),
        "moe_route": lambda st: fp8bs.moe_route(z, 2, stream=st),
        "moe_route with the loss": lambda st: fp8bs.moe_route(z, 2, alpha=0.1, stream=st),
        "moe_route_backward": lambda st: fp8bs.moe_route_backward(z, idx, dw, stream=st),
        "moe_layout": lambda st: fp8bs.moe_layout(idx, 16, st),
    }


class Side:
    """A stream by its handle alone, as another library's would be."""
    cuda_stream = 0x1234


@pytest.mark.parametrize("as_handle", [False, True])
def test_allocations_are_made_on_the_given_stream(launched, monkeypatch, as_handle):  # noqa: F811
    main, side = Side(), Side()
    main.cuda_stream = 0x77
    active, allocated, kept = [main], [], []

    @contextlib.contextmanager
    def enter(stream):
        active.append(stream)
        yield
        active.pop()

    def external(handle, device=None):
        assert handle == side.cuda_stream
        return side

    def empty(*a, _make=torch.empty, **k):
        allocated.append(active[-1].cuda_stream)
        return claim(_make(*a, **k))

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: active[-1])
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    table = calls(lambda shape, dtype: claim(torch.zeros(shape, dtype=dtype)), _codes)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: kept.append((t.data_ptr(), st.cuda_stream)))
    for name, call in table.items():
        allocated.clear()
        kept.clear()
        out = call(side.cuda_stream if as_handle else side)
        assert allocated and set(allocated) == {side.cuda_stream}, name
        out = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
        assert {(t.data_ptr(), main.cuda_stream) for t in out} <= set(kept), name
        allocated.clear()
        kept.clear()
        call(main)                                       # the current stream, named
        call(None)
        assert set(allocated) == {main.cuda_stream} and not kept, name
        assert active == [main], name


def _device_calls(fp8bs):
    def codes(M, K, fmt, G=None):
        x = torch.ones((M, K) if G is None else (G, M, K), dtype=torch.bfloat16, device="cuda:0")
        return fp8bs.quantize_fp4(x, fmt)

    return calls(lambda shape, dtype: torch.ones(shape, dtype=dtype, device="cuda:0"), codes)


def _stream_of(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.gpu
def test_outputs_lie_in_the_given_streams_memory():
    _, fp8bs = require_gpu()
    table = _device_calls(fp8bs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert side.cuda_stream != torch.cuda.current_stream().cuda_stream
    for name, call in table.items():
        ref = call(None)
        torch.cuda.synchronize()
        for given in (side, side.cuda_stream):
            out = call(given)
            torch.cuda.synchronize()
            pairs = zip(out, ref) if isinstance(out, tuple) else [(out, ref)]
            for a, b in pairs:
                if a is not None:
                    assert _stream_of(a) == side.cuda_stream and torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def _hold():
    """Some tens of milliseconds of work on the current stream: 20 float32 products of 137 GFLOP."""
    a = torch.ones((4096, 4096), device="cuda:0")
    for _ in range(20):
        a = a @ a * 0.0


def _logits():
    return torch.from_numpy(np.random.default_rng(0).standard_normal((20000, 64)).astype(np.float32)).to("cuda:0")


def _route_and_layout(fp8bs, z, k, stream=None):
    out = fp8bs.moe_route(z, k, alpha=0.1, stream=stream)
    return out + fp8bs.moe_layout(out[0], z.shape[1], stream=stream)


def _same_sizes(fp8bs, T, E, k):
    """Tensors of the sizes that moe_route (with the loss) and moe_layout allocate, scratch included."""
    n = [T * k * 4, T * k * 4, E * 4, 4, 4, fp8bs.moe_route_workspace_bytes(T, E), (E + 1) * 4, fp8bs.moe_layout_rows(T, k, E) * 4,
         fp8bs.moe_layout_workspace_bytes(T, k, E)]
    return [torch.empty(b, dtype=torch.uint8, device="cuda:0") for b in n for _ in range(3)]


@pytest.mark.gpu
def test_memory_with_work_pending_on_the_current_stream_is_not_taken():
    """Freed blocks of the very sizes wanted, with fills of them still queued on the current stream: the
    call on the other stream runs first, and the fills do not touch what it wrote."""
    _, fp8bs = require_gpu()
    z, k = _logits(), 4
    ref = _route_and_layout(fp8bs, z, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _route_and_layout(fp8bs, z, k, side)                  # both streams' memory is there: no cudaMalloc below, which may wait
    _same_sizes(fp8bs, *z.shape, k)
    torch.cuda.synchronize()
    _hold()
    blocks = _same_sizes(fp8bs, *z.shape, k)
    for b in blocks:
        b.fill_(0xFF)
    del blocks, b
    got = _route_and_layout(fp8bs, z, k, side)
    done_first = torch.cuda.Event()
    done_first.record(torch.cuda.current_stream())
    side.synchronize()
    assert not done_first.query()                         # the fills were still to come
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.gpu
def test_scratch_is_kept_until_the_given_stream_has_run():
    """The call waits behind work on its stream; meanwhile the current stream allocates and fills blocks
    of the scratch's own sizes."""
    _, fp8bs = require_gpu()
    z, k = _logits(), 4
    ref = _route_and_layout(fp8bs, z, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _route_and_layout(fp8bs, z, k, side)
    _same_sizes(fp8bs, *z.shape, k)
    with torch.cuda.stream(side):
        _hold()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _hold()
    got = _route_and_layout(fp8bs, z, k, side)
    for b in _same_sizes(fp8bs, *z.shape, k):
        b.fill_(0xFF)
    torch.cuda.current_stream().synchronize()
    assert not side.query()                               # the call was still to come
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.gpu
def test_outputs_freed_early_are_kept_for_the_current_stream():
    """Read on the current stream behind work queued there and freed on the host: calls that follow on
    the other stream are not given the block before it has been read."""
    _, fp8bs = require_gpu()
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((512, 1024)).astype(np.float32)).to("cuda:0").bfloat16()
    ref = fp8bs.quantize_fp4(x)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = fp8bs.quantize_fp4(x, stream=side)[0]
    side.synchronize()
    _hold()
    copy = q.clone()
    del q
    for _ in range(4):
        fp8bs.quantize_fp4(-x, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, ref)
