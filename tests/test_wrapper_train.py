"""The allocating functions of the training operators: what they refuse, and the stream that they allocate for.

Runs without a GPU, through the stand-ins of test_wrapper_checks and test_wrapper_streams."""
import contextlib

import pytest

import fp8_fine_grained_fp8bs_gb300 as fp8bs
from test_wrapper_checks import claim, launched  # noqa: F401
from test_wrapper_streams import Side

torch = pytest.importorskip("torch")
BF16, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def zeros(shape, dtype):
    return claim(torch.zeros(shape, dtype=dtype))


def arguments():
    """name -> the arguments of a call that is accepted."""
    M, K, T, k, rows, G = 6, 256, 6, 2, 128, 3
    x, gain, rstd = zeros((M, K), BF16), zeros(K, F32), zeros(M, F32)
    row_of, row_token = zeros((T, k), I32), zeros(rows, I32)
    return {
        "rmsnorm_quantize": dict(x=x, gain=gain, residual=x),
        "rmsnorm_backward": dict(dy=x, r=x, gain=gain, rstd=rstd, dres=x),
        "swiglu_backward_quantize": dict(h=x, dv=zeros((M, K // 2), BF16), live=zeros(M, I32)),
        "moe_combine_backward": dict(dout=x, y=zeros((rows, K), BF16), row_of=row_of, row_token=row_token, w=zeros((T, k), F32)),
        "moe_dispatch_backward": dict(d=zeros((rows, K), BF16), row_of=row_of, add=x),
        "grouped_wgrad": dict(a_t=zeros((256, rows), U8), sa_t=zeros((1, 256), F32), b_t=zeros((128, rows), U8),
                              sb_t=zeros((1, 128), F32), offsets=zeros(G + 1, I32)),
    }


@pytest.mark.parametrize("name", sorted(arguments()))
def test_accepted(launched, name):  # noqa: F811
    out = getattr(fp8bs, name)(**arguments()[name])
    assert len(launched) == 1 and launched[0].startswith("fp8bs_")
    assert out is not None


@pytest.mark.parametrize("name,changes", [
    ("rmsnorm_quantize", dict(x=zeros((6, 256), F32))), ("rmsnorm_quantize", dict(x=torch.zeros((6, 256), dtype=BF16))),
    ("rmsnorm_quantize", dict(gain=zeros(255, F32))), ("rmsnorm_quantize", dict(gain=zeros(256, torch.float64))),
    ("rmsnorm_quantize", dict(residual=zeros((5, 256), BF16))), ("rmsnorm_quantize", dict(x=zeros((6, 512), BF16)[:, ::2])),
    ("rmsnorm_backward", dict(r=None)), ("rmsnorm_backward", dict(r=zeros((6, 128), BF16))),
    ("rmsnorm_backward", dict(rstd=zeros(5, F32))), ("rmsnorm_backward", dict(rstd=zeros(6, BF16))),
    ("rmsnorm_backward", dict(dgain=zeros(128, F32))), ("rmsnorm_backward", dict(dgain=zeros(256, BF16))),
    ("rmsnorm_backward", dict(dres=zeros((6, 256), F32))),
    ("swiglu_backward_quantize", dict(h=zeros((6, 255), BF16))), ("swiglu_backward_quantize", dict(dv=None)),
    ("swiglu_backward_quantize", dict(dv=zeros((6, 256), BF16))), ("swiglu_backward_quantize", dict(live=zeros(5, I32))),
    ("swiglu_backward_quantize", dict(live=zeros(6, torch.int64))),
    ("moe_combine_backward", dict(y=None)), ("moe_combine_backward", dict(y=zeros((127, 256), BF16))),
    ("moe_combine_backward", dict(w=zeros((6, 3), F32))), ("moe_combine_backward", dict(row_of=zeros((6, 2), torch.int64))),
    ("moe_combine_backward", dict(row_of=zeros((5, 2), I32), w=zeros((5, 2), F32))),
    ("moe_combine_backward", dict(row_token=zeros(128, torch.int64))),
    ("moe_dispatch_backward", dict(add=zeros((5, 256), BF16))), ("moe_dispatch_backward", dict(d=zeros((128, 512), BF16)[:, ::2])),
    ("moe_dispatch_backward", dict(row_of=zeros((6, 2), torch.int64))),
    ("grouped_wgrad", dict(b_t=zeros((128, 256), U8))), ("grouped_wgrad", dict(sa_t=zeros((256, 1), F32))),
    ("grouped_wgrad", dict(sb_t=zeros((1, 256), F32))), ("grouped_wgrad", dict(offsets=zeros(4, torch.int64))),
    ("grouped_wgrad", dict(out_dtype=torch.float16)), ("grouped_wgrad", dict(out=zeros((3, 256, 256), F32))),
    ("grouped_wgrad", dict(accumulate=True)), ("grouped_wgrad", dict(accumulate=True, out=zeros((3, 256, 128), BF16))),
    ("grouped_wgrad", dict(out=zeros((3, 256, 128), torch.float16)))])
def test_refused(launched, name, changes):  # noqa: F811
    with pytest.raises(ValueError):
        getattr(fp8bs, name)(**{**arguments()[name], **changes})
    assert launched == []


@pytest.mark.parametrize("name", sorted(arguments()))
def test_allocations_are_made_on_the_given_stream(launched, monkeypatch, name):  # noqa: F811
    main, side = Side(), Side()
    main.cuda_stream = 0x77
    active, allocated, kept = [main], [], []

    @contextlib.contextmanager
    def enter(stream):
        active.append(stream)
        yield
        active.pop()

    args = arguments()[name]

    def empty(*a, _make=torch.empty, **k):
        allocated.append(active[-1].cuda_stream)
        return claim(_make(*a, **k))

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: active[-1])
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: side)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: kept.append(st.cuda_stream))
    getattr(fp8bs, name)(**args, stream=side)
    assert allocated and set(allocated) == {side.cuda_stream}
    assert kept and set(kept) == {main.cuda_stream}


def test_layer_refusals(launched):  # noqa: F811
    """The 8-bit layer: rows, widths and experts that do not fit, and a gradient without what it needs."""
    from fp8_fine_grained_fp8bs_gb300 import moe
    T, E, H, I = 6, 4, 256, 128
    one = lambda n, k: (zeros((E, n, k), U8), zeros((E, n // 128, k // 128), F32))  # noqa: E731
    experts = moe.Fp8Experts(one(2 * I, H), one(H, I), None, None)
    xq, sx, z = zeros((T, H), U8), zeros((H // 128, T), F32), zeros((T, E), F32)
    for bad in (dict(xq=zeros((5, H), U8)), dict(logits=zeros((T, E + 1), F32)), dict(sx=zeros((T, H // 128), F32)),
                dict(xq=zeros((T, 128), U8), sx=zeros((1, T), F32))):
        with pytest.raises(ValueError):
            moe.moe_layer_fp8(**{**dict(xq=xq, sx=sx, logits=z, experts=experts, k=2), **bad})
    saved = moe.Fp8Saved(z, (zeros((T, 2), I32), zeros((T, 2), F32)), {}, None, None, None, None, None)
    with pytest.raises(ValueError):       # no transposed copies
        moe.moe_layer_fp8_backward(zeros((T, H), BF16), saved, experts)
    with pytest.raises(ValueError):       # no balance loss in the forward pass
        moe.moe_layer_fp8_backward(zeros((T, H), BF16), saved, experts._replace(gate_up_t=one(H, 2 * I), down_t=one(I, H)),
                                   dloss=zeros(1, F32))
    for w in (zeros((E, 200, H), BF16), zeros((E, 2 * I, H), F32)):
        with pytest.raises(ValueError):
            moe.quantize_experts_fp8(w, zeros((E, H, I), BF16))
    assert launched == []


def test_layer_refuses_what_the_products_could_not_read(launched):  # noqa: F811
    """Codes and scales of another type, layout or size, which the C entry points see as pointers."""
    from fp8_fine_grained_fp8bs_gb300 import moe
    T, E, H, I = 6, 4, 384, 128
    one = lambda n, k: (zeros((E, n, k), U8), zeros((E, n // 128, k // 128), F32))  # noqa: E731
    experts = moe.Fp8Experts(one(2 * I, H), one(H, I), one(H, 2 * I), one(I, H))
    good = dict(xq=zeros((T, H), U8), sx=zeros((H // 128, T), F32), logits=zeros((T, E), F32), experts=experts, k=2)
    up, down = experts.gate_up, experts.down
    for bad in (dict(xq=zeros((T, H), torch.int8)), dict(xq=claim(torch.zeros((H, T), dtype=U8).t())),
                dict(sx=zeros((H // 128, T), torch.float64)), dict(sx=claim(torch.zeros((T, H // 128)).t())), dict(xq=torch.zeros((T, H), dtype=U8)),
                dict(experts=experts._replace(gate_up=(up[0], zeros((E, 3, 2), F32)))),
                dict(experts=experts._replace(gate_up=(up[0], torch.zeros((E, 2, 3))))),
                dict(experts=experts._replace(down=(down[0].to(torch.int32), down[1]))),
                dict(experts=experts._replace(down=(down[0], zeros((E, 1, 3), F32))))):
        with pytest.raises(ValueError):
            moe.moe_layer_fp8(**{**good, **bad})
    saved = moe.Fp8Saved(good["logits"], (zeros((T, 2), I32), zeros((T, 2), F32)), {}, None, None, None, None, None)
    for bad in (dict(gate_up_t=one(2 * I, H)), dict(down_t=one(H, I)), dict(down_t=(experts.down_t[0], zeros((E, 1, 1), F32)))):
        with pytest.raises(ValueError):
            moe.moe_layer_fp8_backward(zeros((T, H), BF16), saved, experts._replace(**bad))
    assert launched == []
