"""Host-side refusals of the experts' products and the block quantiser (no GPU):
sizes, pointers and alignments are checked before anything is queued."""
import pytest

A = 1 << 20  # an aligned stand-in pointer (never touched)


@pytest.fixture(scope="module")
def abi():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


QUANT = dict(d_x=A, bf16=1, groups=2, rows=3, hidden=64, row_stride=64, block_rows=1, d_counts=0,
             d_q=A, d_scale=A)


@pytest.mark.parametrize("bad", [
    dict(d_x=0), dict(d_q=0), dict(d_scale=0), dict(d_x=A + 8), dict(d_q=A + 8),
    dict(d_scale=A + 2), dict(d_counts=A + 2), dict(groups=-1), dict(rows=-1), dict(hidden=0),
    dict(hidden=56, row_stride=56), dict(row_stride=56), dict(row_stride=68),
    dict(bf16=0, row_stride=66), dict(block_rows=0), dict(block_rows=64),
    dict(block_rows=128, d_counts=A), dict(hidden=2 ** 31 - 16, row_stride=2 ** 31 - 16)])
def test_quantize_refusals(abi, bad):
    assert abi.moe_quantize_blocks_fp8(**{**QUANT, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_quantize_without_rows_queues_nothing(abi):
    assert abi.moe_quantize_blocks_fp8(**{**QUANT, "rows": 0, "d_x": 0}) == abi.MOE_OK
    assert abi.moe_quantize_blocks_fp8(**{**QUANT, "groups": 0, "d_x": 0}) == abi.MOE_OK


FP8 = dict(d_xq=A, d_x_scale=A, d_wq=A, d_w_scale=A, d_counts=0, d_offsets=0, groups=2, rows=5,
           N=70, hidden=48, d_out=A, d_scratch=A, scratch_bytes=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(d_xq=0), dict(d_x_scale=0), dict(d_wq=0), dict(d_w_scale=0), dict(d_out=0),
    dict(d_scratch=0), dict(d_xq=A + 8), dict(d_wq=A + 8), dict(d_x_scale=A + 2),
    dict(d_w_scale=A + 1), dict(d_counts=A + 2), dict(d_offsets=A + 2), dict(d_out=A + 1),
    dict(d_scratch=A + 128), dict(d_counts=A, d_offsets=A), dict(groups=-1), dict(groups=1025),
    dict(rows=-1), dict(N=0), dict(hidden=0), dict(hidden=40), dict(groups=1024, rows=1 << 22),
    dict(groups=1024, N=1 << 22), dict(groups=1024, hidden=1 << 22),
    dict(groups=1, N=2 ** 31 - 1), dict(groups=1, rows=2 ** 31 - 1, d_offsets=A),
    dict(groups=1, rows=2 ** 30, N=2 ** 30, hidden=16)])
def test_fp8_refusals(abi, bad):
    assert abi.moe_gemm_fp8(**{**FP8, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_fp8_scratch_size(abi):
    assert abi.moe_gemm_fp8_scratch_bytes(0) == 0
    need = abi.moe_gemm_fp8_scratch_bytes(5)
    assert 0 < need <= abi.moe_gemm_fp8_scratch_bytes(300)
    assert abi.moe_gemm_fp8(**{**FP8, "scratch_bytes": need - 1}) == abi.MOE_ERR_CAPACITY
    assert abi.moe_gemm_fp8(**{**FP8, "rows": 0, "d_xq": 0}) == abi.MOE_OK
    assert abi.moe_gemm_fp8(**{**FP8, "groups": 0, "d_xq": 0}) == abi.MOE_OK


SIZES = dict(d_offsets=A, groups=2, rows=5, N=72, hidden=48, d_scratch=A, scratch_bytes=1 << 30)
CALLS = {"moe_gemm_ragged": dict(d_x=A, d_w=A, d_out=A),
         "moe_gemm_ragged_input_grad": dict(d_dy=A, d_w=A, d_dx=A),
         "moe_gemm_ragged_weight_grad": dict(d_dy=A, d_x=A, d_dw=A, fp32=1, accumulate=1)}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_ragged_refusals(abi, name):
    call, good = getattr(abi, name), {**SIZES, **CALLS[name]}
    pointers = [k for k in good if k.startswith("d_")]
    bad = [{k: 0} for k in pointers] + [{k: A + 1} for k in pointers]
    bad += [{k: A + 8} for k in pointers if k in ("d_x", "d_w", "d_dy", "d_dw", "d_scratch")]
    bad += [dict(groups=-1), dict(groups=1025), dict(rows=-1), dict(N=0), dict(hidden=0),
            dict(hidden=44), dict(groups=1024, N=1 << 22), dict(groups=1024, hidden=1 << 22),
            dict(rows=2 ** 31 - 1), dict(hidden=2 ** 31 - 8), dict(groups=1, N=2 ** 31 - 8)]
    if name != "moe_gemm_ragged":
        bad += [dict(N=71), dict(N=68)]
    for b in bad:
        assert call(**{**good, **b}) == abi.MOE_ERR_INVALID_ARG, b
    need = abi.moe_gemm_ragged_scratch_bytes()
    assert call(**{**good, "scratch_bytes": need - 1}) == abi.MOE_ERR_CAPACITY
    assert call(**{**good, "groups": 0}) == abi.MOE_OK
    assert call(**{**good, "rows": 0}) == abi.MOE_OK


def test_weight_grad_adds_to_fp32_only(abi):
    good = {**SIZES, **CALLS["moe_gemm_ragged_weight_grad"]}
    assert abi.moe_gemm_ragged_weight_grad(**{**good, "fp32": 0}) == abi.MOE_ERR_INVALID_ARG


def test_sizes_past_32_bits_are_refused(abi):
    torch = pytest.importorskip("torch")
    for cls in (abi.MoeGemmFp8, abi.MoeGemmRagged):
        for sizes in ((2 ** 32 + 1, 8, 16, 16), (1, 2 ** 32 + 8, 16, 16), (1, 8, 2 ** 32 + 16, 16),
                      (1, 8, 16, 2 ** 32 + 16), (1, 0, 16, 16)):
            with pytest.raises(abi.MoeA2AError):
                cls(*sizes, device="cpu")
    x = torch.empty(0)
    with pytest.raises(ValueError):
        abi.quantize_blocks_fp8(x)
