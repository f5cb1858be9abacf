"""The torch forms of the experts' products on tensors and streams of a device that is
not the current one (host only), and sizes past the limits of their entry points."""
import pytest

torch = pytest.importorskip("torch")

from test_moe_device_host import Stand, StandStream, api, handle  # noqa: E402,F401

BF, F8, F32, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32


def calls(api, index, stream=None):
    S = lambda shape, dtype: Stand(shape, dtype, index)
    eight = handle(api.MoeGemmFp8, index, groups=1, max_rows=4, N=8, hidden=16)
    ragged = handle(api.MoeGemmRagged, index, groups=2, max_rows=4, N=8, hidden=16)
    x, dy, w, off = S((4, 16), BF), S((4, 8), BF), S((2, 8, 16), BF), S((3,), I32)
    return {
        "moe_quantize_blocks_fp8": lambda: api.quantize_blocks_fp8(
            x, out=S((4, 16), F8), scale=S((4, 1), F32), stream=stream),
        "moe_gemm_fp8": lambda: eight.gemm(S((4, 16), F8), S((4, 1), F32), S((8, 16), F8),
                                           S((1, 1), F32), out=S((4, 8), BF), stream=stream),
        "moe_gemm_ragged": lambda: ragged.forward(x, w, off, out=S((4, 8), BF), stream=stream),
        "moe_gemm_ragged_input_grad": lambda: ragged.input_grad(dy, w, off, out=S((4, 16), BF),
                                                                stream=stream),
        "moe_gemm_ragged_weight_grad": lambda: ragged.weight_grad(
            dy, x, off, out=S((2, 8, 16), F32), accumulate=True, stream=stream),
    }


NAMES = ["moe_quantize_blocks_fp8", "moe_gemm_fp8", "moe_gemm_ragged",
         "moe_gemm_ragged_input_grad", "moe_gemm_ragged_weight_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(api, name):  # noqa: F811
    with pytest.raises(ValueError, match="not the current CUDA device"):
        calls(api, 1)[name]()
    with pytest.raises(ValueError):
        calls(api, 1, stream=StandStream(1))[name]()
    assert api._lib.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(api, name):  # noqa: F811
    with pytest.raises(ValueError, match="a stream of cuda:1"):
        calls(api, 0, stream=StandStream(1))[name]()
    assert api._lib.calls == []


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [None, StandStream(0), 0])
def test_tensors_of_the_current_device_are_taken(api, name, stream):  # noqa: F811
    calls(api, 0, stream=stream)[name]()
    assert api._lib.calls == [name]


A = 1 << 20  # an aligned stand-in pointer (never touched)


@pytest.fixture(scope="module")
def abi():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def test_sizes_past_the_limits_are_refused(abi):
    """Blocks of k and tiles whose numbers would pass 32 bits, and rows of the quantiser
    whose number does when it is rounded up."""
    fp8 = dict(d_xq=A, d_x_scale=A, d_wq=A, d_w_scale=A, d_counts=0, d_offsets=A, groups=2,
               rows=5, N=70, hidden=48, d_out=A, d_scratch=A, scratch_bytes=1 << 30)
    ragged = dict(d_offsets=A, groups=2, rows=5, N=72, hidden=48, d_scratch=A,
                  scratch_bytes=1 << 30)
    over = (1 << 28) + 16
    for call in (
            lambda: abi.moe_gemm_fp8(**{**fp8, "hidden": over}),
            # 2^15 x 2^16 tiles of 128 x 128
            lambda: abi.moe_gemm_fp8(**{**fp8, "rows": 1 << 23, "N": 1 << 22}),
            lambda: abi.moe_gemm_ragged(**{**ragged, "hidden": over}, d_x=A, d_w=A, d_out=A),
            lambda: abi.moe_gemm_ragged_input_grad(**{**ragged, "N": over}, d_dy=A, d_w=A, d_dx=A),
            lambda: abi.moe_quantize_blocks_fp8(
                d_x=A, bf16=1, groups=1, rows=2 ** 31 - 8, hidden=16, row_stride=16, block_rows=128,
                d_counts=0, d_q=A, d_scale=A)):
        assert call() == abi.MOE_ERR_INVALID_ARG


def test_a_part_has_room_for_the_widest_tile(abi):
    """Scratch of the 8-bit product: tiles of 256 channels from 33 rows on."""
    size = abi.moe_gemm_fp8_scratch_bytes
    assert size(16) < size(17) == size(32) < size(33) == size(1 << 20)
