"""The training step's operators on several streams at once, on streams given by argument, and in graphs that share
nothing: each call gives the bits that it gives alone."""
import pytest

from fp8_fine_grained_fp8bs_gb300 import moe
from _gpu import require_gpu

pytestmark = pytest.mark.gpu


def _calls(torch, fp8bs, seed):
    """name -> call taking a stream, on inputs of the seed."""
    torch.manual_seed(seed)
    M, K, I, T, N, E, k = 700, 1024, 512, 150, 384, 6, 3
    bf16 = lambda *s: torch.randn(s, device="cuda:0").bfloat16()  # noqa: E731
    x, res, dy, dres, gain = bf16(M, K), bf16(M, K), bf16(M, K), bf16(M, K), torch.randn(K, device="cuda:0")
    h, dv = bf16(M, 2 * I), bf16(M, I)
    rstd = torch.rand(M, device="cuda:0") + 0.5
    idx = torch.rand((T, E), device="cuda:0").argsort(1)[:, :k].int().contiguous()
    offsets, row_token, row_of = fp8bs.moe_layout(idx, E)
    rows = row_token.shape[0]
    dout, y, d, w = bf16(T, N), bf16(rows, N), bf16(rows, N), torch.rand((T, k), device="cuda:0")
    a, b = ([*fp8bs.quantize_act(bf16(rows, n), True, True)[2:]] for n in (N, 256))
    return {
        "norm": lambda st: fp8bs.rmsnorm_quantize(x, gain, res, pow2=True, bf16=True, stream=st),
        "norm's gradient": lambda st: fp8bs.rmsnorm_backward(dy, x, gain, rstd, dres, stream=st),
        "swiglu's gradient": lambda st: fp8bs.swiglu_backward_quantize(h, dv, pow2=True, bf16=True, stream=st),
        "combine's gradient": lambda st: fp8bs.moe_combine_backward(dout, y, row_of, row_token, w, True, True, st),
        "dispatch's gradient": lambda st: fp8bs.moe_dispatch_backward(d, row_of, dout, st),
        "weight gradients": lambda st: fp8bs.grouped_wgrad(*a, *b, offsets, stream=st),
    }


def _tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def _same(torch, got, want, name):
    assert len(got) == len(want) and all(torch.equal(p, q) for p, q in zip(got, want)), name


def test_streams_at_once():
    torch, fp8bs = require_gpu()
    sets = [_calls(torch, fp8bs, seed) for seed in (0, 1, 2)]
    want = [{n: _tensors(c(None)) for n, c in calls.items()} for calls in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(4):                      # every operator beside every other, started in another order on each
        for i, (calls, stream) in enumerate(zip(sets, streams)):
            names = list(calls)
            for name in names[2 * i:] + names[:2 * i]:
                got.append((i, name, _tensors(calls[name](stream))))
    torch.cuda.synchronize()
    for i, name, out in got:
        _same(torch, out, want[i][name], name)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_two_graphs_at_once():
    """Graphs captured one after the other, replayed side by side: scratch is a graph's own."""
    torch, fp8bs = require_gpu()
    sets = [_calls(torch, fp8bs, seed) for seed in (3, 4)]
    want = [{n: _tensors(c(None)) for n, c in calls.items()} for calls in sets]
    graphs = []
    for calls in sets:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for c in calls.values():
                c(None)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = {n: _tensors(c(None)) for n, c in calls.items()}
        graphs.append((side, graph, out))
    torch.cuda.synchronize()
    for _ in range(5):
        for side, graph, _ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, out), ref in zip(graphs, want):
        for name in ref:
            _same(torch, out[name], ref[name], name)
    assert fp8bs.fp8bs_get_device_status() == 0


def test_inputs_made_on_the_same_stream_just_before():
    """A launch begins before the kernel in front of it has ended; it reads its inputs only after."""
    torch, fp8bs = require_gpu()
    torch.manual_seed(5)
    H, I, E, T, k = 512, 256, 4, 300, 2
    experts = moe.quantize_experts_fp8(*(torch.randn(s, device="cuda:0").bfloat16() * 0.06 for s in ((E, 2 * I, H), (E, H, I))))
    x, z, gain = torch.randn((T, H), device="cuda:0").bfloat16(), torch.randn((T, E), device="cuda:0"), torch.ones(H, device="cuda:0")

    def step(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        outs = []
        for _ in range(3):
            q, s, _, r, rstd = fp8bs.rmsnorm_quantize(x, gain, x, pow2=True)
            pause()
            out, saved = moe.moe_layer_fp8(q, s, z, experts, k)
            pause()
            grads = moe.moe_layer_fp8_backward(out, saved, experts)
            pause()
            outs += [out, *grads, *fp8bs.rmsnorm_backward(grads[0], r, gain, rstd, out)]
            pause()
        return outs

    want = step(True)
    for _ in range(10):
        _same(torch, step(False), want, "step")
    assert fp8bs.fp8bs_get_device_status() == 0
