"""The routing oracle, pinned independently of itself: worked values, its
gradient against differences, and the layout against the host planner."""
import numpy as np
import pytest

from oracle import route
from fp8_fine_grained_fp8bs_gb300 import moe, synth


def test_choice_worked():
    z = np.array([[0.0, 2.0, 2.0, -np.inf], [np.nan, -np.inf, 1.0, -5.0], [-np.inf] * 4])
    idx, w, counts, tokens, _ = route.route(z, 3, 0, scale=2.0)
    assert idx.tolist() == [[1, 2, 0], [2, 3, -1], [-1, -1, -1]]     # ties to the lower index, none left
    assert np.allclose(w.sum(1), [2, 2, 0]) and w[0, 0] == w[0, 1] and w[1, 2] == 0
    assert counts.tolist() == [[1, 1, 2, 1]] and tokens.tolist() == [2]


def test_bias_moves_the_choice_not_the_weight():
    z = np.array([[1.0, 0.0, -1.0]])
    idx, w, *_ = route.route(z, 1, 1, bias=np.array([0.0, 0.0, 0.9]), normalize=False)
    assert idx.tolist() == [[2]] and np.isclose(w[0, 0], 1 / (1 + np.e))


def test_loss_of_uniform_routing_is_alpha():
    """f_i = 1 and sum P_i = 1 where every expert is chosen equally often."""
    z = np.tile(np.eye(4), (2, 1)) * 1e-9
    _, _, counts, _, loss = route.route(z, 1, 0, alpha=0.3)
    assert counts.tolist() == [[2, 2, 2, 2]] and np.isclose(loss, 0.3)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(score, normalize):
    rng = np.random.default_rng(score)
    T, E, k, seq = 9, 6, 3, [0, 4, 4, 9]
    z = rng.standard_normal((T, E))
    z[2, 1], z[5, :4] = -np.inf, -np.inf
    valid = np.ones(T)
    valid[7] = 0
    dw, dloss = rng.standard_normal((T, k)), 0.7
    kw = dict(score=score, valid=valid, seq=seq, normalize=normalize, scale=1.5, alpha=0.9)
    idx = route.route(z, k, **kw)[0]

    def value(zz):
        _, w, _, _, loss = route.route(zz, k, idx=idx, **kw)
        return (w * np.where(idx >= 0, dw, 0)).sum() + dloss * loss

    dz = route.backward(z, idx, dw, dloss, **kw)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(z[t, e]):
                assert dz[t, e] == 0
                continue
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            # central differences: h^2 / 6 times the third derivative, and rounding of 1e-16 / h
            assert abs((value(up) - value(down)) / (2 * h) - dz[t, e]) < 1e-8


def test_layout_is_the_host_planners():
    E, T, k = 7, 90, 3
    topk = synth.moe_routing(seed=3, tokens=T, experts=E, top_k=k)
    plan = moe.MoePlan(topk, E, 1)
    recv = moe.RecvPlan(plan.expert_counts.reshape(1, E))
    offsets, row_token, row_of = route.layout(topk, E, 128 * 16)
    assert np.array_equal(offsets, recv.offsets)
    assert np.array_equal(row_of, recv.back_idx[plan.send_pos])
    tokens = np.where(recv.unpack_idx >= 0, plan.send_token[np.maximum(recv.unpack_idx, 0)], -1)
    assert np.array_equal(row_token[:recv.padded_rows], tokens) and np.all(row_token[recv.padded_rows:] == -1)
