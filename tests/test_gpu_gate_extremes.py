"""The router gate's weights at the ends of fp32, against 64 bits.

Tolerance: the exponentials are off by 2 ulp and by the rounding of their
argument (2^-24 of the selected logits' span), the sum and the divisions by a few
roundings of 2^-24; what fp32 holds with fewer bits (below 2^-126) by 2^-149 a step.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def sigmoid_ref(l, K, renorm, scale):
    l = l.double().cpu().numpy()
    order = np.argsort(-l, axis=-1, kind="stable")[:, :K]
    v = np.take_along_axis(l, order, -1)
    s = 1.0 / (1.0 + np.exp(-v))
    if renorm:
        s = s / s.sum(-1, keepdims=True)
    return order, s * scale, v[:, :1] - v


@pytest.mark.parametrize("E,K", [(40, 8), (256, 8), (256, 3), (64, 20), (600, 8)])
@pytest.mark.parametrize("T", [6, 5000])                # a token a warp, and four
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_weights_far_below_zero(api, E, K, T, dtype, renorm):
    g = torch.Generator(device=DEV).manual_seed(E + K + T)
    l = torch.randn((T, E), generator=g, device=DEV)
    l[0::6] -= 95.0                                     # scores below 2^-126
    l[1::6] = l[1::6] * 8 - 300.0                       # far below
    l[2::6] = l[2::6] * 40 - 86.0                       # on both sides
    l[3::6] = -104.0                                    # all equal
    l[4::6] -= 700.0                                    # where binary64 still has them
    l[4::6].clamp_(min=-708.0)
    l = l.to(dtype)
    ids, w = api.topk_gate(l, K, api.MOE_SCORE_SIGMOID, renorm, 2.5)
    rids, rw, span = sigmoid_ref(l, K, renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), rids)
    got = w.double().cpu().numpy()
    tol = (32 + 2 * span) * 2.0 ** -24 * rw + 8 * 2.0 ** -149
    assert (np.abs(got - rw) <= tol).all(), float((np.abs(got - rw) / tol).max())
    if renorm:
        assert np.abs(got.sum(-1) / 2.5 - 1.0).max() < 1e-5


@pytest.mark.parametrize("E,K", [(40, 8), (256, 8), (64, 20), (600, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
def test_places_without_an_expert_weigh_nothing_at_any_scale(api, E, K, dtype, scale):
    l = torch.full((5, E), -float("inf"), device=DEV)
    l[1, 3], l[2, :K], l[4, :2] = 0.5, 1.0, float("nan")
    for sigmoid in (api.MOE_SCORE_SOFTMAX, api.MOE_SCORE_SIGMOID):
        for renorm in (True, False):
            ids, w = api.topk_gate(l.to(dtype), K, sigmoid, renorm, scale)
            assert (ids >= 0).sum(-1).tolist() == [0, 1, K, 0, 0]
            assert (w[ids < 0] == 0).all()
            assert not torch.isfinite(w[ids >= 0]).any()
