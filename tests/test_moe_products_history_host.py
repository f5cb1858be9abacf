"""The experts' map on tensors that require gradients (host only): it returns no history,
so it is refused where one is expected."""
import pytest

torch = pytest.importorskip("torch")

from test_moe_device_host import Stand, api, handle  # noqa: E402,F401

BF, I32 = torch.bfloat16, torch.int32


def forward(api, grad_of):
    ragged = handle(api.MoeGemmRagged, 0, groups=2, max_rows=4, N=8, hidden=16)
    t = {"x": Stand((4, 16), BF, 0), "w": Stand((2, 8, 16), BF, 0)}
    for name in t:
        t[name].requires_grad = name == grad_of
    return ragged.forward(t["x"], t["w"], Stand((3,), I32, 0), out=Stand((4, 8), BF, 0))


@pytest.mark.parametrize("grad_of", ["x", "w"])
def test_tensors_that_require_gradients_are_refused(api, grad_of):  # noqa: F811
    with pytest.raises(ValueError, match="no history"):
        forward(api, grad_of)
    assert api._lib.calls == []
    with torch.no_grad():
        forward(api, grad_of)
    with torch.inference_mode():
        forward(api, grad_of)
    assert api._lib.calls == ["moe_gemm_ragged"] * 2


def test_others_are_taken(api):  # noqa: F811
    forward(api, None)
    assert api._lib.calls == ["moe_gemm_ragged"]
