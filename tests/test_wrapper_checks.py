"""The allocating functions refuse what the C entry points could not see, before they launch anything.

Runs without a GPU: CPU tensors that claim to be CUDA ones, and entry points that record their calls
instead of making them.
"""
import pytest

import fp8_fine_grained_fp8bs_gb300 as fp8bs

torch = pytest.importorskip("torch")


class ClaimsCuda(torch.Tensor):
    """A CPU tensor that the wrappers take for a CUDA one."""
    is_cuda = True


def claim(t):
    return t.as_subclass(ClaimsCuda)


@pytest.fixture
def launched(monkeypatch):
    """The entry points called; none of them runs."""
    fp8bs.build()
    fp8bs.load_library()
    calls = []
    for name in fp8bs.__all__:
        if name.startswith("fp8bs_") and not name.endswith(("_bytes", "_string")):
            monkeypatch.setattr(fp8bs, name, lambda *a, _name=name, **k: calls.append(_name))
    return calls


def _codes(M, K, fmt, G=None):
    lead = (M,) if G is None else (G, M)
    n = fp8bs.fp4_scale_bytes(M, K, fmt)
    return (claim(torch.zeros((*lead, K // 2), dtype=torch.uint8)), claim(torch.zeros((*lead[:-1], n), dtype=torch.uint8)),
            claim(torch.ones(lead)) if fmt == 0 else None)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float8_e4m3fn, torch.uint8, torch.float64])
def test_dequantize_writes_float32_or_bfloat16_only(launched, dtype, fmt):
    """The kernel writes two or four bytes an element, whatever the output was allocated as."""
    q, sf, g = _codes(5, 128, fmt)
    with pytest.raises(ValueError):
        fp8bs.dequantize_fp4(q, sf, g, fmt, out_dtype=dtype)
    assert launched == []
    for dtype in (None, torch.bfloat16, torch.float32):
        assert fp8bs.dequantize_fp4(q, sf, g, fmt, out_dtype=dtype).shape == (5, 128)
    assert launched == ["fp8bs_dequantize_fp4"] * 3


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_products_write_float32_or_bfloat16_only(launched, grouped, pow2):
    """An output of another type, of another shape or with gaps between its rows is refused."""
    M, N, K = 128, 256, 128
    a, sa = claim(torch.zeros((M, K), dtype=torch.uint8)), claim(torch.zeros((K // 128, M)))
    b, sb = claim(torch.zeros((N, K), dtype=torch.uint8)), claim(torch.zeros((N // 128, K // 128)))
    offsets = claim(torch.tensor([0, M], dtype=torch.int32))

    def call(**kw):
        if grouped:
            return fp8bs.grouped_gemm(a, sa, offsets, b[None], sb[None], pow2=pow2, **kw)
        return fp8bs.gemm(a, sa, b, sb, pow2=pow2, **kw)

    for dtype in (torch.float16, torch.uint8, torch.float64):
        with pytest.raises(ValueError):
            call(out_dtype=dtype)
        with pytest.raises(ValueError):
            call(out=claim(torch.zeros((M, N), dtype=dtype)))
    for out in (torch.zeros((M, N - 8)), torch.zeros((M - 1, N)), torch.zeros((M, 2 * N))[:, :N]):
        with pytest.raises(ValueError):
            call(out=claim(out))
    with pytest.raises(ValueError):
        call(out=torch.zeros((M, N)))
    assert launched == []
    for kw in ({}, dict(out_dtype=torch.float32), dict(out=claim(torch.zeros((M, N)))),
               dict(out=claim(torch.zeros((M, N), dtype=torch.bfloat16)))):
        assert call(**kw).shape == (M, N)
    assert len(launched) == 4


def test_router_gradient_checks_what_the_loss_reads(launched):
    """counts, tokens and dloss are read as int32 [S, E], int32 [S] and one float32."""
    T, E, k, S = 6, 16, 2, 3
    z, seq = claim(torch.zeros((T, E))), claim(torch.tensor([0, 2, 4, T], dtype=torch.int32))
    idx, dw = claim(torch.zeros((T, k), dtype=torch.int32)), claim(torch.zeros((T, k)))
    good = dict(seq=seq, counts=claim(torch.ones((S, E), dtype=torch.int32)), tokens=claim(torch.ones(S, dtype=torch.int32)),
                dloss=claim(torch.ones(1)))
    for bad in (dict(tokens=good["tokens"].long()), dict(tokens=torch.ones(S, dtype=torch.int32)),
                dict(tokens=claim(torch.ones(2 * S, dtype=torch.int32))[::2]), dict(tokens=good["tokens"][:2]),
                dict(tokens=good["tokens"][:, None]), dict(tokens=None), dict(counts=None),
                dict(counts=good["counts"].float()), dict(counts=good["counts"][:2]), dict(counts=good["counts"][:, :15]),
                dict(dloss=claim(torch.ones(0))), dict(dloss=claim(torch.ones(2))), dict(dloss=claim(torch.ones(1).double())),
                dict(dloss=torch.ones(1))):
        with pytest.raises(ValueError):
            fp8bs.moe_route_backward(z, idx, dw, **{**good, **bad})
    assert launched == []
    for dloss in (good["dloss"], claim(torch.tensor(1.0)), None):
        assert fp8bs.moe_route_backward(z, idx, dw, **{**good, "dloss": dloss}).shape == (T, E)
    assert fp8bs.moe_route_backward(z, idx, dw, seq=seq).shape == (T, E)


@pytest.mark.parametrize("rows", [5, 7])
def test_layer_takes_one_row_of_logits_per_token(launched, rows):
    """Missing tokens became rows of zeros, surplus ones were dropped."""
    from fp8_fine_grained_fp8bs_gb300 import moe
    T, E, H, I, fmt = 6, 4, 64, 64, 0
    experts = _codes(2 * I, H, fmt, E), _codes(H, I, fmt, E)
    x, z = claim(torch.zeros((rows, H), dtype=torch.bfloat16)), claim(torch.zeros((T, E)))
    with pytest.raises(ValueError):
        moe.moe_layer_fp4(x, z, experts, 2, fmt)
    assert launched == []


@pytest.mark.parametrize("N", [128, 72])
def test_quantize_gathers_rows_of_a_matrix_only(launched, N):
    """``rows`` was ignored for expert weights [G, N, K]."""
    w = claim(torch.zeros((2, N, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fp8bs.quantize_fp4(w, rows=claim(torch.zeros(3, dtype=torch.int32)))
    assert launched == []
    assert fp8bs.quantize_fp4(w)[0].shape == (2, N, 32)


def test_swiglu_takes_two_halves(launched):
    """A strided view of odd width lost its last column."""
    wide = claim(torch.zeros((3, 136), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fp8bs.swiglu_quantize_fp4(wide[:, :129])
    assert launched == []
    assert fp8bs.swiglu_quantize_fp4(wide[:, :128])[0].shape == (3, 32)
