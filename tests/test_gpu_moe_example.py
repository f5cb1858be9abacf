"""The 8-bit layer of examples/int8_moe.py at decode and at prefill.

A row whose largest magnitude is r times its rms is quantised with an error of
r / (127 * sqrt(12)) of the rms: 1.1 % for r = 5 (normal rows of 1024 values),
2.8 % for r = 12 (the products silu(gate) * up, whose tails are longer); the
two together, in quadrature, stay below 3 %, and the bf16 roundings (2^-8
each, three of them) below 1 %.  At decode the activations are not quantised:
the bf16 rounding of the output alone, 2^-8 at most, remains beside fp32 sums.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from conftest import ROOT  # noqa: E402


@pytest.fixture(scope="module")
def example():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    spec = importlib.util.spec_from_file_location(
        "int8_moe", os.path.join(ROOT, "examples", "int8_moe.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_prefill_and_decode_on_the_same_weights(example):
    torch.manual_seed(3)
    errors = example.main()
    assert errors["prefill"] < 0.04
    assert errors["decode"] < 2.0 ** -8


def test_one_rank_and_ragged_sizes(example):
    torch.manual_seed(4)
    errors = example.main(ranks=1, tokens=77, hidden=272, inter=144, experts=6, top_k=2)
    assert errors["prefill"] < 0.04
    assert errors["decode"] < 2.0 ** -8


@pytest.mark.parametrize("expert_layout", [False, True])
def test_dispatch_straight_after_the_gate(example, expert_layout):
    """The one-launch dispatches read ids and weights before they wait for the
    kernel in front of them: they have to be the gate's finished ones."""
    moe = example.moe
    R, T, H, E, K = 8, 64, 128, 1024, 8
    layout = moe.MOE_LAYOUT_EXPERT if expert_layout else moe.MOE_LAYOUT_RANK
    a, b = (moe.MoeA2A(R, T, H, E, K, "cuda", layout=layout) for _ in range(2))
    x = torch.randn((R, T, H), device="cuda").to(torch.bfloat16)
    ids = torch.empty((R, T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((R, T, K), device="cuda")
    for i in range(40):
        logits = torch.randn((R, T, E), device="cuda")
        ids.fill_(-1), w.zero_()
        torch.cuda.synchronize()
        moe.topk_gate(logits, K, out_ids=ids, out_w=w)
        va = a.dispatch(ids, w, x)
        torch.cuda.synchronize()
        vb = b.dispatch(ids, w, x)
        torch.cuda.synchronize()
        assert va.kernels == 1 and int(va.local_expert_counts.sum()) == R * T * K
        for name in ("recv_counts", "local_expert_counts", "send_slot", "dest_weight"):
            assert torch.equal(getattr(va, name), getattr(vb, name)), (i, name)
        a.combine(va.recv_x), b.combine(vb.recv_x)
