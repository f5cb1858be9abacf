"""Thin ctypes binding of the C ABI in include/moe_a2a.h (libmoe_a2a.so).

The module-level functions carry the C names and take raw device pointers
(ints) and sizes; they return the C status codes.  `MoeA2A` wraps them for
torch tensors: it allocates the workspace with torch, checks dtypes, shapes
and devices, passes data pointers and the current CUDA stream, and raises
`MoeA2AError` on any status other than MOE_OK.  Every step of the path runs
in the library's CUDA kernels; there is no fallback: if the library is
missing, importing this module fails.
"""
import ctypes
import os

try:
    import torch as _torch
except ImportError:  # the raw C functions need no torch
    _torch = None

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_a2a.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_PHASE = 2
MOE_ERR_CAPACITY = 3
MOE_ERR_CUDA = 4
MOE_ERR_ROUTING = 5
MOE_ERR_DEVICE_TIMEOUT = 6
MOE_ERR_INTERNAL = 7
MOE_ERR_SETUP_IN_CAPTURE = 8
MOE_DEVICE_FLAG_BAD_EXPERT_ID = 0x1
MOE_DEVICE_FLAG_WAIT_TIMEOUT = 0x2
MOE_DEVICE_FLAG_BAD_SLOT = 0x4

EXPORTS = ("moe_a2a_workspace_bytes", "moe_a2a_create", "moe_dispatch",
           "moe_combine_payload", "moe_combine", "moe_a2a_get_error",
           "moe_a2a_destroy", "moe_a2a_phase", "moe_a2a_status_string",
           "moe_route_static_scratch_bytes", "moe_route_static_scratch",
           "moe_a2a_set_reduction", "moe_dispatch_varlen", "moe_a2a_set_active_ranks",
           "moe_a2a_set_recv_format", "moe_combine_fp8", "moe_quantize_rows_fp8",
           "moe_a2a_workspace_bytes_layout", "moe_a2a_create_layout",
           "moe_expert_gemm", "moe_expert_gemm_fp8", "moe_expert_gemm_rank_scratch_bytes",
           "moe_expert_gemm_rank", "moe_expert_gemm_rank_fp8", "moe_topk_gate",
           "moe_quantize_rows_int8", "moe_gemm_int8_scratch_bytes", "moe_gemm_int8",
           "moe_layer_small_scratch_bytes", "moe_layer_small", "moe_scratch_init",
           "moe_scratch_get_error", "moe_quantize_blocks_fp8", "moe_gemm_fp8_scratch_bytes",
           "moe_gemm_fp8", "moe_gemm_ragged_scratch_bytes", "moe_gemm_ragged",
           "moe_gemm_ragged_input_grad", "moe_gemm_ragged_weight_grad")
MOE_REDUCE_FP32_RANK_ORDER = 0
MOE_REDUCE_BF16_TOPK_TREE = 1
MOE_STATIC_SCRATCH_BYTES = 4 << 20
MOE_FORMAT_BF16 = 0
MOE_FORMAT_FP8_E4M3 = 1
MOE_FORMAT_INT8 = 2
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_LAYER_MAX_TOKENS = 64
MOE_SCALE_BLOCK = 128  # codes, and output channels, that share a scale of moe_gemm_fp8
MOE_LAYOUT_RANK = 0
MOE_LAYOUT_EXPERT = 1


class MoeA2AConfig(ctypes.Structure):
    _fields_ = [("ep_size", ctypes.c_int32), ("max_tokens_per_rank", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32)]


class MoeDispatchView(ctypes.Structure):
    _fields_ = [("recv_x", ctypes.c_void_p), ("recv_topk_ids", ctypes.c_void_p),
                ("recv_topk_w", ctypes.c_void_p), ("src_token", ctypes.c_void_p),
                ("recv_counts", ctypes.c_void_p), ("local_expert_counts", ctypes.c_void_p),
                ("send_slot", ctypes.c_void_p), ("dest_weight", ctypes.c_void_p),
                ("plane_stride", ctypes.c_int32), ("tokens_per_rank", ctypes.c_int32),
                ("send_stride", ctypes.c_int32), ("token_stride", ctypes.c_int32),
                ("recv_scale", ctypes.c_void_p), ("recv_format", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("kernels", ctypes.c_int32)]


class MoeA2AError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, status_string(status), status))


def _load(path: str = LIBRARY):
    if not os.path.exists(path):
        raise ImportError("libmoe_a2a.so is not built (%s); run __graft_entry__.build()" % path)
    # torch first, so that the CUDA runtime it loaded is the one the library binds to
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    p, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(MoeA2AConfig)
    lib.moe_a2a_workspace_bytes.argtypes = [cfgp]
    lib.moe_a2a_workspace_bytes.restype = sz
    lib.moe_a2a_create.argtypes = [cfgp, p, sz, ctypes.POINTER(p)]
    lib.moe_a2a_create.restype = ctypes.c_int
    lib.moe_a2a_workspace_bytes_layout.argtypes = [cfgp, i32]
    lib.moe_a2a_workspace_bytes_layout.restype = sz
    lib.moe_a2a_create_layout.argtypes = [cfgp, i32, p, sz, ctypes.POINTER(p)]
    lib.moe_a2a_create_layout.restype = ctypes.c_int
    lib.moe_dispatch.argtypes = [p, p, p, p, i32, i32, p, ctypes.POINTER(MoeDispatchView)]
    lib.moe_dispatch.restype = ctypes.c_int
    lib.moe_combine_payload.argtypes = [p]
    lib.moe_combine_payload.restype = p
    lib.moe_combine.argtypes = [p, p, i32, p, p, ctypes.c_float, p, p, p]
    lib.moe_combine.restype = ctypes.c_int
    lib.moe_a2a_get_error.argtypes = [p, p, ctypes.POINTER(ctypes.c_uint32)]
    lib.moe_a2a_get_error.restype = ctypes.c_int
    lib.moe_a2a_destroy.argtypes = [p]
    lib.moe_a2a_destroy.restype = ctypes.c_int
    lib.moe_a2a_phase.argtypes = [p]
    lib.moe_a2a_phase.restype = ctypes.c_int
    lib.moe_dispatch_varlen.argtypes = [p, p, p, p, ctypes.POINTER(ctypes.c_int32), i32, p,
                                        ctypes.POINTER(MoeDispatchView)]
    lib.moe_dispatch_varlen.restype = ctypes.c_int
    lib.moe_a2a_set_active_ranks.argtypes = [p, ctypes.c_uint32]
    lib.moe_a2a_set_active_ranks.restype = ctypes.c_int
    lib.moe_combine_fp8.argtypes = [p, p, i32, p, p, ctypes.c_float, p, p, p, p]
    lib.moe_combine_fp8.restype = ctypes.c_int
    lib.moe_quantize_rows_fp8.argtypes = [p, ctypes.c_int64, i32, p, p, p]
    lib.moe_quantize_rows_fp8.restype = ctypes.c_int
    lib.moe_expert_gemm.argtypes = [p, p, i32, p, p]
    lib.moe_expert_gemm.restype = ctypes.c_int
    lib.moe_expert_gemm_fp8.argtypes = [p, p, p, i32, p, p]
    lib.moe_expert_gemm_fp8.restype = ctypes.c_int
    lib.moe_expert_gemm_rank_scratch_bytes.argtypes = [ctypes.POINTER(MoeA2AConfig), i32]
    lib.moe_expert_gemm_rank_scratch_bytes.restype = ctypes.c_size_t
    lib.moe_expert_gemm_rank.argtypes = [p, p, i32, i32, p, p, ctypes.c_size_t, p]
    lib.moe_expert_gemm_rank.restype = ctypes.c_int
    lib.moe_expert_gemm_rank_fp8.argtypes = [p, p, p, i32, i32, p, p, ctypes.c_size_t, p]
    lib.moe_expert_gemm_rank_fp8.restype = ctypes.c_int
    lib.moe_a2a_set_recv_format.argtypes = [p, i32]
    lib.moe_a2a_set_recv_format.restype = ctypes.c_int
    lib.moe_a2a_set_reduction.argtypes = [p, i32]
    lib.moe_a2a_set_reduction.restype = ctypes.c_int
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.moe_topk_gate.argtypes = [p, i32, i64, i64, i32, i32, i32, i32, f32, p, p, p]
    lib.moe_topk_gate.restype = ctypes.c_int
    lib.moe_quantize_rows_int8.argtypes = [p, i32, i32, i32, i32, i64, p, p, p, p]
    lib.moe_quantize_rows_int8.restype = ctypes.c_int
    lib.moe_gemm_int8_scratch_bytes.argtypes = [i32]
    lib.moe_gemm_int8_scratch_bytes.restype = sz
    lib.moe_gemm_int8.argtypes = [p, p, p, p, p, i32, i32, i32, i32, p, p, sz, p]
    lib.moe_gemm_int8.restype = ctypes.c_int
    lib.moe_layer_small_scratch_bytes.argtypes = [i32, i32, i32, i32]
    lib.moe_layer_small_scratch_bytes.restype = sz
    lib.moe_layer_small.argtypes = [p] * 8 + [i32] * 6 + [p, p, sz, p]
    lib.moe_layer_small.restype = ctypes.c_int
    lib.moe_scratch_init.argtypes = [p, sz, p]
    lib.moe_scratch_init.restype = ctypes.c_int
    lib.moe_scratch_get_error.argtypes = [p, p, ctypes.POINTER(ctypes.c_uint32)]
    lib.moe_scratch_get_error.restype = ctypes.c_int
    lib.moe_quantize_blocks_fp8.argtypes = [p, i32, i32, i32, i32, i64, i32, p, p, p, p]
    lib.moe_quantize_blocks_fp8.restype = ctypes.c_int
    lib.moe_gemm_fp8_scratch_bytes.argtypes = [i32]
    lib.moe_gemm_fp8_scratch_bytes.restype = sz
    lib.moe_gemm_fp8.argtypes = [p] * 6 + [i32] * 4 + [p, p, sz, p]
    lib.moe_gemm_fp8.restype = ctypes.c_int
    lib.moe_gemm_ragged_scratch_bytes.argtypes = []
    lib.moe_gemm_ragged_scratch_bytes.restype = sz
    for f in (lib.moe_gemm_ragged, lib.moe_gemm_ragged_input_grad):
        f.argtypes = [p] * 3 + [i32] * 4 + [p, p, sz, p]
        f.restype = ctypes.c_int
    lib.moe_gemm_ragged_weight_grad.argtypes = [p] * 3 + [i32] * 6 + [p, p, sz, p]
    lib.moe_gemm_ragged_weight_grad.restype = ctypes.c_int
    lib.moe_a2a_status_string.argtypes = [ctypes.c_int]
    lib.moe_a2a_status_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


# ---- the C ABI, one function per entry point ---------------------------------

def config(ep_size, max_tokens_per_rank, hidden, num_experts, top_k) -> MoeA2AConfig:
    return MoeA2AConfig(ep_size, max_tokens_per_rank, hidden, num_experts, top_k)


def moe_a2a_workspace_bytes(cfg: MoeA2AConfig) -> int:
    return int(_lib.moe_a2a_workspace_bytes(ctypes.byref(cfg)))


def moe_a2a_create(cfg: MoeA2AConfig, d_workspace: int, workspace_bytes: int):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = _lib.moe_a2a_create(ctypes.byref(cfg), ctypes.c_void_p(d_workspace),
                             workspace_bytes, ctypes.byref(h))
    return st, h


def moe_a2a_workspace_bytes_layout(cfg: MoeA2AConfig, layout: int) -> int:
    return int(_lib.moe_a2a_workspace_bytes_layout(ctypes.byref(cfg), layout))


def moe_a2a_create_layout(cfg: MoeA2AConfig, layout: int, d_workspace: int,
                          workspace_bytes: int):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = _lib.moe_a2a_create_layout(ctypes.byref(cfg), layout, ctypes.c_void_p(d_workspace),
                                    workspace_bytes, ctypes.byref(h))
    return st, h


def moe_dispatch(h, d_topk_ids: int, d_topk_w: int, d_x: int, tokens_per_rank: int,
                 runtime_max_tokens_per_rank: int, stream: int = 0):
    """Returns (status, MoeDispatchView)."""
    view = MoeDispatchView()
    st = _lib.moe_dispatch(h, ctypes.c_void_p(d_topk_ids), ctypes.c_void_p(d_topk_w),
                           ctypes.c_void_p(d_x), tokens_per_rank, runtime_max_tokens_per_rank,
                           ctypes.c_void_p(stream), ctypes.byref(view))
    return st, view


def moe_dispatch_varlen(h, d_topk_ids: int, d_topk_w: int, d_x: int, tokens_per_rank,
                        runtime_max_tokens_per_rank: int, stream: int = 0):
    """Returns (status, MoeDispatchView); tokens_per_rank is a host sequence."""
    view = MoeDispatchView()
    counts = (ctypes.c_int32 * len(tokens_per_rank))(*[int(c) for c in tokens_per_rank])
    st = _lib.moe_dispatch_varlen(h, ctypes.c_void_p(d_topk_ids), ctypes.c_void_p(d_topk_w),
                                  ctypes.c_void_p(d_x), counts, runtime_max_tokens_per_rank,
                                  ctypes.c_void_p(stream), ctypes.byref(view))
    return st, view


def moe_a2a_set_active_ranks(h, active: int) -> int:
    return _lib.moe_a2a_set_active_ranks(h, active)


def moe_combine_payload(h) -> int:
    return _lib.moe_combine_payload(h) or 0


def moe_combine(h, d_expert_out: int, weighted: bool, d_residual: int, d_gamma: int, eps: float,
                d_out: int, d_residual_out: int, stream: int = 0) -> int:
    return _lib.moe_combine(h, ctypes.c_void_p(d_expert_out), int(bool(weighted)),
                            ctypes.c_void_p(d_residual), ctypes.c_void_p(d_gamma),
                            float(eps), ctypes.c_void_p(d_out), ctypes.c_void_p(d_residual_out),
                            ctypes.c_void_p(stream))


def moe_combine_fp8(h, d_expert_out: int, weighted: bool, d_residual: int, d_gamma: int,
                    eps: float, d_out_fp8: int, d_out_scale: int, d_residual_out: int,
                    stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_combine_fp8(h, v(d_expert_out), int(bool(weighted)), v(d_residual),
                                v(d_gamma), float(eps), v(d_out_fp8), v(d_out_scale),
                                v(d_residual_out), v(stream))


def moe_quantize_rows_fp8(d_x: int, rows: int, hidden: int, d_q: int, d_scale: int,
                          stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_quantize_rows_fp8(v(d_x), rows, hidden, v(d_q), v(d_scale), v(stream))


def quantize_rows_fp8(x, out=None, scale=None, stream=None):
    """fp32 [..., H] CUDA tensor -> (float8_e4m3fn [..., H], float32 [...])."""
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    H = x.shape[-1]
    rows = x.numel() // H if H else 0
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    st = moe_quantize_rows_fp8(x.data_ptr(), rows, H, out.data_ptr(), scale.data_ptr(),
                               _raw_stream(stream, x.device))
    if st != MOE_OK:
        raise MoeA2AError(st, "moe_quantize_rows_fp8")
    return out, scale


def moe_expert_gemm(h, d_w: int, N: int, d_out: int, stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_expert_gemm(h, v(d_w), N, v(d_out), v(stream))


def moe_expert_gemm_rank_scratch_bytes(cfg: MoeA2AConfig, N: int) -> int:
    return _lib.moe_expert_gemm_rank_scratch_bytes(ctypes.byref(cfg), N)


def moe_expert_gemm_rank(h, d_w: int, N: int, apply_gates: int, d_out: int, d_scratch: int,
                         scratch_bytes: int, stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_expert_gemm_rank(h, v(d_w), N, apply_gates, v(d_out), v(d_scratch),
                                     scratch_bytes, v(stream))


def moe_expert_gemm_rank_fp8(h, d_w8: int, d_w_scale: int, N: int, apply_gates: int,
                             d_out: int, d_scratch: int, scratch_bytes: int,
                             stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_expert_gemm_rank_fp8(h, v(d_w8), v(d_w_scale), N, apply_gates, v(d_out),
                                         v(d_scratch), scratch_bytes, v(stream))


def moe_expert_gemm_fp8(h, d_w8: int, d_w_scale: int, N: int, d_out: int,
                        stream: int = 0) -> int:
    v = ctypes.c_void_p
    return _lib.moe_expert_gemm_fp8(h, v(d_w8), v(d_w_scale), N, v(d_out), v(stream))


def moe_a2a_set_recv_format(h, fmt: int) -> int:
    return _lib.moe_a2a_set_recv_format(h, fmt)


def moe_a2a_get_error(h, stream: int = 0):
    """Returns (status, device flag bits)."""
    flags = ctypes.c_uint32(0)
    st = _lib.moe_a2a_get_error(h, ctypes.c_void_p(stream), ctypes.byref(flags))
    return st, int(flags.value)


def moe_a2a_destroy(h) -> int:
    return _lib.moe_a2a_destroy(h)


def moe_a2a_phase(h) -> int:
    return _lib.moe_a2a_phase(h)


def moe_a2a_set_reduction(h, reduction: int) -> int:
    return _lib.moe_a2a_set_reduction(h, reduction)


def status_string(status: int) -> str:
    return _lib.moe_a2a_status_string(status).decode()


def moe_route_static_scratch_bytes(ep_size: int, num_experts: int, tokens_per_rank: int) -> int:
    f = _lib.moe_route_static_scratch_bytes
    f.argtypes = [ctypes.c_int32] * 3
    f.restype = ctypes.c_size_t
    return int(f(ep_size, num_experts, tokens_per_rank))


def moe_route_static_scratch(ep_size: int, num_experts: int, top_k: int, tokens_per_rank: int,
                             runtime_max_tokens_per_rank: int, d_topk_ids: int, d_topk_w: int,
                             d_send_slot: int, d_dest_weight: int, d_src_token: int,
                             d_recv_counts: int, d_local_expert_counts: int,
                             d_recv_topk_ids: int, d_recv_topk_w: int, d_flags: int = 0,
                             stream: int = 0) -> int:
    """The routing pass with no device allocation (see include/moe_a2a.h):
    every buffer is the caller's, the temporary memory is the library's
    fixed device array.  Returns the C status code."""
    f = _lib.moe_route_static_scratch
    f.argtypes = [ctypes.c_int32] * 5 + [ctypes.c_void_p] * 11
    f.restype = ctypes.c_int
    v = ctypes.c_void_p
    return f(ep_size, num_experts, top_k, tokens_per_rank, runtime_max_tokens_per_rank,
             v(d_topk_ids), v(d_topk_w), v(d_send_slot), v(d_dest_weight), v(d_src_token),
             v(d_recv_counts), v(d_local_expert_counts), v(d_recv_topk_ids), v(d_recv_topk_w),
             v(d_flags), v(stream))


def moe_topk_gate(d_logits: int, bf16: bool, tokens: int, row_stride: int, num_experts: int,
                  top_k: int, scoring: int, renormalize: bool, scale: float, d_topk_ids: int,
                  d_topk_w: int, stream: int = 0) -> int:
    return _lib.moe_topk_gate(d_logits, int(bf16), tokens, row_stride, num_experts, top_k,
                              scoring, int(renormalize), scale, d_topk_ids, d_topk_w, stream)


def moe_quantize_rows_int8(d_x: int, bf16: bool, groups: int, rows: int, hidden: int,
                           row_stride: int, d_counts: int, d_q: int, d_scale: int,
                           stream: int = 0) -> int:
    return _lib.moe_quantize_rows_int8(d_x, int(bf16), groups, rows, hidden, row_stride,
                                       d_counts, d_q, d_scale, stream)


def moe_gemm_int8_scratch_bytes(rows: int) -> int:
    return int(_lib.moe_gemm_int8_scratch_bytes(rows))


def moe_gemm_int8(d_xq: int, d_x_scale: int, d_wq: int, d_w_scale: int, d_counts: int,
                  groups: int, rows: int, N: int, hidden: int, d_out: int, d_scratch: int,
                  scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_gemm_int8(d_xq, d_x_scale, d_wq, d_w_scale, d_counts, groups, rows, N,
                              hidden, d_out, d_scratch, scratch_bytes, stream)


def moe_layer_small_scratch_bytes(tokens: int, top_k: int, hidden: int, inter: int) -> int:
    return int(_lib.moe_layer_small_scratch_bytes(tokens, top_k, hidden, inter))


def moe_layer_small(d_x: int, d_topk_ids: int, d_topk_w: int, d_w13: int, d_w13_scale: int,
                    d_w2: int, d_w2_scale: int, d_residual: int, tokens: int, top_k: int,
                    num_experts: int, hidden: int, inter: int, fmt: int, d_out: int,
                    d_scratch: int, scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_layer_small(d_x, d_topk_ids, d_topk_w, d_w13, d_w13_scale, d_w2, d_w2_scale,
                                d_residual, tokens, top_k, num_experts, hidden, inter, fmt,
                                d_out, d_scratch, scratch_bytes, stream)


def moe_scratch_init(d_scratch: int, scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_scratch_init(d_scratch, scratch_bytes, stream)


def moe_scratch_get_error(d_scratch: int, stream: int = 0):
    """Returns (status, device flag bits)."""
    flags = ctypes.c_uint32(0)
    st = _lib.moe_scratch_get_error(d_scratch, stream, ctypes.byref(flags))
    return st, int(flags.value)


def moe_quantize_blocks_fp8(d_x: int, bf16: bool, groups: int, rows: int, hidden: int,
                            row_stride: int, block_rows: int, d_counts: int, d_q: int,
                            d_scale: int, stream: int = 0) -> int:
    return _lib.moe_quantize_blocks_fp8(d_x, int(bf16), groups, rows, hidden, row_stride,
                                        block_rows, d_counts, d_q, d_scale, stream)


def moe_gemm_fp8_scratch_bytes(rows: int) -> int:
    return int(_lib.moe_gemm_fp8_scratch_bytes(rows))


def moe_gemm_fp8(d_xq: int, d_x_scale: int, d_wq: int, d_w_scale: int, d_counts: int,
                 d_offsets: int, groups: int, rows: int, N: int, hidden: int, d_out: int,
                 d_scratch: int, scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_gemm_fp8(d_xq, d_x_scale, d_wq, d_w_scale, d_counts, d_offsets, groups, rows,
                             N, hidden, d_out, d_scratch, scratch_bytes, stream)


def moe_gemm_ragged_scratch_bytes() -> int:
    return int(_lib.moe_gemm_ragged_scratch_bytes())


def moe_gemm_ragged(d_x: int, d_w: int, d_offsets: int, groups: int, rows: int, N: int,
                    hidden: int, d_out: int, d_scratch: int, scratch_bytes: int,
                    stream: int = 0) -> int:
    return _lib.moe_gemm_ragged(d_x, d_w, d_offsets, groups, rows, N, hidden, d_out, d_scratch,
                                scratch_bytes, stream)


def moe_gemm_ragged_input_grad(d_dy: int, d_w: int, d_offsets: int, groups: int, rows: int,
                               N: int, hidden: int, d_dx: int, d_scratch: int,
                               scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_gemm_ragged_input_grad(d_dy, d_w, d_offsets, groups, rows, N, hidden, d_dx,
                                           d_scratch, scratch_bytes, stream)


def moe_gemm_ragged_weight_grad(d_dy: int, d_x: int, d_offsets: int, groups: int, rows: int,
                                N: int, hidden: int, fp32: bool, accumulate: bool, d_dw: int,
                                d_scratch: int, scratch_bytes: int, stream: int = 0) -> int:
    return _lib.moe_gemm_ragged_weight_grad(d_dy, d_x, d_offsets, groups, rows, N, hidden,
                                            int(fp32), int(accumulate), d_dw, d_scratch,
                                            scratch_bytes, stream)


# ---- torch forms of the operators around dispatch and combine ------------------

def _on_current(device):
    """The C entries launch on the current device and size their grids for it: refuse
    tensors of another one (its default stream has the same number, 0)."""
    if device.index != _current_device():
        raise ValueError("%s is not the current CUDA device (%s): call under "
                         "torch.cuda.device(%s)" % (device, _current_device(), device.index))


def _raw_stream(stream, device) -> int:
    _on_current(device)
    if stream is None:
        return _current_stream(device.index)
    if getattr(stream, "device", device) != device:
        raise ValueError("a stream of %s for tensors of %s" % (stream.device, device))
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _current_device() -> int:
    return _torch.cuda.current_device()


def _current_stream(index: int) -> int:
    return _torch.cuda.current_stream(index).cuda_stream


if hasattr(getattr(_torch, "_C", None), "_cuda_getCurrentRawStream"):
    # the same number without the Stream object around it (1.9 us less a call)
    _current_stream = _torch._C._cuda_getCurrentRawStream  # noqa: F811
if hasattr(getattr(_torch, "_C", None), "_cuda_getDevice"):
    _current_device = _torch._C._cuda_getDevice  # noqa: F811  (a tensor is there: initialised)


def _empty(shape, dtype, device, stream, raw):
    """A new tensor that belongs to the stream (`raw`) it is going to be used on."""
    if stream is None or raw == _current_stream(device.index):
        return _torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = _torch.cuda.ExternalStream(int(stream), device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


_INT32_MAX = 2 ** 31 - 1  # sizes go to the C entries in 32 bits, and ctypes would wrap them


def _expect(t, dtype, shape, device, name):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s: expected %s %s, got %s %s" % (name, dtype, tuple(shape), t.dtype,
                                                            tuple(t.shape)))
    if t.device != device or not t.is_contiguous():
        raise ValueError("%s must be contiguous on %s" % (name, device))


def topk_gate(logits, top_k: int, scoring: int = MOE_SCORE_SOFTMAX, renormalize: bool = True,
              scale: float = 1.0, out_ids=None, out_w=None, stream=None):
    """Router logits, fp32 or bf16 [..., E] with dense rows (2-D logits may
    have any row stride) -> (ids int32 [..., K], weights float32 [..., K])."""
    dtype, device = logits.dtype, logits.device
    bf16 = dtype is _torch.bfloat16
    if not logits.is_cuda or not (bf16 or dtype is _torch.float32) or logits.dim() < 1:
        raise ValueError("logits must be a float32 or bfloat16 CUDA tensor [..., E]")
    *lead, E = logits.shape
    row_stride = E
    if not logits.is_contiguous():
        if logits.dim() != 2 or logits.stride(1) != 1 or logits.stride(0) < E:
            raise ValueError("logits must be contiguous, or 2-D with dense rows")
        row_stride = logits.stride(0)
    if E > _INT32_MAX or top_k > _INT32_MAX:
        raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_topk_gate")
    shape = (*lead, top_k)
    raw = _raw_stream(stream, device)
    if out_ids is None:
        out_ids = _empty(shape, _torch.int32, device, stream, raw)
    else:
        _expect(out_ids, _torch.int32, shape, device, "out_ids")
    if out_w is None:
        out_w = _empty(shape, _torch.float32, device, stream, raw)
    else:
        _expect(out_w, _torch.float32, shape, device, "out_w")
    st = _lib.moe_topk_gate(logits.data_ptr(), bf16, logits.numel() // E if E else 0, row_stride,
                            E, top_k, scoring, bool(renormalize), scale, out_ids.data_ptr(),
                            out_w.data_ptr(), raw)
    if st != MOE_OK:
        raise MoeA2AError(st, "moe_topk_gate")
    return out_ids, out_w


def quantize_rows_int8(x, counts=None, out=None, scale=None, stream=None):
    """fp32 or bf16 [..., H] CUDA tensor -> (int8 [..., H], float32 [...]).
    With counts (int32 [G] on the device) x is [G, rows, H] and rows past a
    plane's count are left alone.  2-D x may have any row stride that is a
    multiple of 16 bytes."""
    dtype, device = x.dtype, x.device
    bf16 = dtype is _torch.bfloat16
    if not x.is_cuda or not (bf16 or dtype is _torch.float32) or x.dim() < 1:
        raise ValueError("x must be a float32 or bfloat16 CUDA tensor [..., H]")
    shape = x.shape
    *lead, H = shape
    row_stride = H
    if not x.is_contiguous():
        if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < H:
            raise ValueError("x must be contiguous, or 2-D with dense rows")
        row_stride = x.stride(0)
    groups, rows = 1, x.numel() // H if H else 0
    if counts is not None:
        if x.dim() != 3:
            raise ValueError("with counts x must be [groups, rows, hidden]")
        groups, rows = lead
        _expect(counts, _torch.int32, (groups,), device, "counts")
    if rows > _INT32_MAX or groups > _INT32_MAX or H > _INT32_MAX:
        raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_quantize_rows_int8")
    raw = _raw_stream(stream, device)
    if out is None:
        out = _empty(shape, _torch.int8, device, stream, raw)
    else:
        _expect(out, _torch.int8, shape, device, "out")
    if scale is None:
        scale = _empty(lead, _torch.float32, device, stream, raw)
    else:
        _expect(scale, _torch.float32, tuple(lead), device, "scale")
    st = _lib.moe_quantize_rows_int8(x.data_ptr(), bf16, groups, rows, H, row_stride,
                                     0 if counts is None else counts.data_ptr(),
                                     out.data_ptr(), scale.data_ptr(), raw)
    if st != MOE_OK:
        raise MoeA2AError(st, "moe_quantize_rows_int8")
    return out, scale


class _Scratch:
    """Device memory that one operator keeps between its calls.  The allocator is
    told of every torch stream that it is used on, so the handle may be dropped
    while a call runs.  For a stream given as a bare number the caller keeps the
    handle until that call is through."""

    def __init__(self, nbytes: int, device, where: str):
        if nbytes == 0:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, where)
        self.device = _torch.device(device if device is not None else "cuda")
        self.scratch = _torch.empty(nbytes, dtype=_torch.uint8, device=self.device)
        self.device = self.scratch.device
        _on_current(self.device)
        self._scratch_ptr, self._scratch_bytes = self.scratch.data_ptr(), nbytes
        stream = _torch.cuda.current_stream(self.device)
        st = moe_scratch_init(self.scratch.data_ptr(), nbytes, stream.cuda_stream)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_scratch_init")
        stream.synchronize()  # calls may come on any stream
        self._streams = {stream.cuda_stream}

    def _launch_stream(self, stream) -> int:
        """The raw stream of a call that is about to use the scratch memory."""
        raw = _raw_stream(stream, self.device)
        if raw not in self._streams:
            if stream is None:
                stream = _torch.cuda.current_stream(self.device)
            if hasattr(stream, "cuda_stream"):
                self.scratch.record_stream(stream)
                self._streams.add(raw)
        return raw

    def get_error(self, stream=None):
        """Synchronise, read and clear the device flag word: (status, bits)."""
        return moe_scratch_get_error(self.scratch.data_ptr(), _raw_stream(stream, self.device))


class MoeGemmInt8(_Scratch):
    """The 8-bit integer product over `groups` weight matrices, with the
    scratch memory it needs.  One call at a time: calls in stream order."""

    def __init__(self, groups: int, max_rows: int, N: int, hidden: int, device=None):
        self.groups, self.max_rows, self.N, self.hidden = groups, max_rows, N, hidden
        if max(groups, max_rows, N, hidden) > _INT32_MAX:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_gemm_int8")
        super().__init__(moe_gemm_int8_scratch_bytes(max_rows), device,
                         "moe_gemm_int8_scratch_bytes")

    def gemm(self, xq, x_scale, wq, w_scale, counts=None, out=None, stream=None):
        """xq int8 [G, rows, H], x_scale float32 [G, rows], wq int8 [G, N, H],
        w_scale float32 [G, N], counts int32 [G] on the device or None (all
        rows) -> out bf16 [G, rows, N], rows past a count untouched (undefined
        in a new tensor).  With one group the leading extent may be left out."""
        G, N, H, dev = self.groups, self.N, self.hidden, self.device
        lead = (G,) if xq.dim() == 3 or G != 1 else ()
        rows = xq.shape[-2] if xq.dim() >= 2 else 0
        _expect(xq, _torch.int8, (*lead, rows, H), dev, "xq")
        _expect(x_scale, _torch.float32, (*lead, rows), dev, "x_scale")
        _expect(wq, _torch.int8, (*lead, N, H), dev, "wq")
        _expect(w_scale, _torch.float32, (*lead, N), dev, "w_scale")
        if counts is not None:
            _expect(counts, _torch.int32, (G,), dev, "counts")
        if rows > self.max_rows:
            raise MoeA2AError(MOE_ERR_CAPACITY, "moe_gemm_int8")
        raw = self._launch_stream(stream)
        if out is None:
            out = _empty((*lead, rows, N), _torch.bfloat16, dev, stream, raw)
        else:
            _expect(out, _torch.bfloat16, (*lead, rows, N), dev, "out")
        st = _lib.moe_gemm_int8(xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(),
                                w_scale.data_ptr(), _ptr(counts), G, rows, N, H, out.data_ptr(),
                                self._scratch_ptr, self._scratch_bytes, raw)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_gemm_int8")
        return out


def _e4m3(t, name):
    """e4m3 codes as torch has them, or as bytes."""
    if t.dtype is not _torch.float8_e4m3fn and t.dtype is not _torch.uint8:
        raise ValueError("%s: expected e4m3 codes, got %s" % (name, t.dtype))
    return t.dtype


def _blocks(n: int) -> int:
    return (n + MOE_SCALE_BLOCK - 1) // MOE_SCALE_BLOCK


def quantize_blocks_fp8(x, block_rows: int = 1, counts=None, out=None, scale=None, stream=None):
    """fp32 or bf16 [..., H] CUDA tensor -> (float8_e4m3fn [..., H], float32
    scales [..., ceil(H / 128)]): one scale for 128 values of a row, or, with
    block_rows = 128, for 128 values of 128 rows (x [..., rows, H], scales
    [..., ceil(rows / 128), ceil(H / 128)]).  With counts (int32 [G] on the
    device, block_rows = 1) x is [G, rows, H] and rows past a plane's count are
    left alone.  2-D x may have any row stride that is a multiple of 16 bytes."""
    dtype, device, shape = x.dtype, x.device, x.shape
    bf16 = dtype is _torch.bfloat16
    tiles = block_rows != 1
    if not x.is_cuda or not (bf16 or dtype is _torch.float32) or len(shape) < 1 + tiles:
        raise ValueError("x must be a float32 or bfloat16 CUDA tensor [..., H]")
    if tiles and block_rows != MOE_SCALE_BLOCK:
        raise ValueError("block_rows must be 1 or %d" % MOE_SCALE_BLOCK)
    *lead, H = shape
    row_stride = H
    if not x.is_contiguous():
        if len(shape) != 2 or x.stride(1) != 1 or x.stride(0) < H:
            raise ValueError("x must be contiguous, or 2-D with dense rows")
        row_stride = x.stride(0)
    n = x.numel()
    groups, rows = 1, n // H if H else 0
    if tiles:
        rows = lead[-1]
        groups = n // (rows * H) if n else 0
        lead[-1] = _blocks(rows)
    if counts is not None:
        if len(shape) != 3 or tiles:
            raise ValueError("with counts x must be [groups, rows, hidden], block_rows 1")
        groups, rows = lead
        _expect(counts, _torch.int32, (groups,), device, "counts")
    if rows > _INT32_MAX or groups > _INT32_MAX or H > _INT32_MAX:
        raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_quantize_blocks_fp8")
    raw = _raw_stream(stream, device)
    if out is None:
        out = _empty(shape, _torch.float8_e4m3fn, device, stream, raw)
    else:
        _expect(out, _e4m3(out, "out"), shape, device, "out")
    lead.append((H + MOE_SCALE_BLOCK - 1) // MOE_SCALE_BLOCK)
    if scale is None:
        scale = _empty(lead, _torch.float32, device, stream, raw)
    else:
        _expect(scale, _torch.float32, tuple(lead), device, "scale")
    st = _lib.moe_quantize_blocks_fp8(x.data_ptr(), bf16, groups, rows, H, row_stride, block_rows,
                                      0 if counts is None else counts.data_ptr(), out.data_ptr(),
                                      scale.data_ptr(), raw)
    if st != MOE_OK:
        raise MoeA2AError(st, "moe_quantize_blocks_fp8")
    return out, scale


class MoeGemmFp8(_Scratch):
    """The 8-bit floating-point product with block scales over `groups` weight
    matrices, with the scratch memory it needs.  One call at a time: calls in
    stream order."""

    def __init__(self, groups: int, max_rows: int, N: int, hidden: int, device=None):
        self.groups, self.max_rows, self.N, self.hidden = groups, max_rows, N, hidden
        if max(groups, max_rows, N, hidden) > _INT32_MAX:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_gemm_fp8")
        super().__init__(moe_gemm_fp8_scratch_bytes(max_rows), device,
                         "moe_gemm_fp8_scratch_bytes")

    def gemm(self, xq, x_scale, wq, w_scale, counts=None, offsets=None, out=None, stream=None):
        """xq e4m3 [G, rows, H], x_scale float32 [G, rows, ceil(H / 128)], wq
        e4m3 [G, N, H], w_scale float32 [G, ceil(N / 128), ceil(H / 128)],
        counts int32 [G] on the device or None (all rows) -> out bf16 [G, rows,
        N], rows past a count untouched (undefined in a new tensor).  With
        offsets (int32 [G + 1] on the device) the rows stand one group after
        another: xq [rows, H], x_scale [rows, ..], out [rows, N], rows of no
        group untouched.  With one group the leading extent may be left out."""
        G, N, H, dev = self.groups, self.N, self.hidden, self.device
        wide = xq.dim()
        lead = (G,) if wide == 3 or (G != 1 and offsets is None) else ()
        wlead = (G,) if wq.dim() == 3 or G != 1 else ()
        rows = xq.shape[-2] if wide >= 2 else 0
        KB = _blocks(H)
        if offsets is not None:
            if counts is not None:
                raise ValueError("counts or offsets, not both")
            lead = ()
            _expect(offsets, _torch.int32, (G + 1,), dev, "offsets")
        elif counts is not None:
            _expect(counts, _torch.int32, (G,), dev, "counts")
        _expect(xq, _e4m3(xq, "xq"), (*lead, rows, H), dev, "xq")
        _expect(x_scale, _torch.float32, (*lead, rows, KB), dev, "x_scale")
        _expect(wq, _e4m3(wq, "wq"), (*wlead, N, H), dev, "wq")
        _expect(w_scale, _torch.float32, (*wlead, _blocks(N), KB), dev, "w_scale")
        if rows > self.max_rows:
            raise MoeA2AError(MOE_ERR_CAPACITY, "moe_gemm_fp8")
        raw = self._launch_stream(stream)
        if out is None:
            out = _empty((*lead, rows, N), _torch.bfloat16, dev, stream, raw)
        else:
            _expect(out, _torch.bfloat16, (*lead, rows, N), dev, "out")
        st = _lib.moe_gemm_fp8(xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(),
                               w_scale.data_ptr(), _ptr(counts), _ptr(offsets), G, rows, N, H,
                               out.data_ptr(), self._scratch_ptr, self._scratch_bytes, raw)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_gemm_fp8")
        return out


class MoeGemmRagged(_Scratch):
    """One linear map per expert (bf16 [G, N, H]) over rows that stand one
    expert after another, and its gradients, with the scratch memory they need.
    offsets: int32 [G + 1] on the device, expert e has rows offsets[e] to
    offsets[e + 1]; rows of no expert are left alone (undefined in a new
    tensor).  One call at a time: calls in stream order.  Autograd does not
    follow these calls: the gradients are called for, and forward refuses
    tensors that expect a history."""

    def __init__(self, groups: int, max_rows: int, N: int, hidden: int, device=None):
        self.groups, self.max_rows, self.N, self.hidden = groups, max_rows, N, hidden
        if max(groups, max_rows, N, hidden) > _INT32_MAX or max_rows < 1:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_gemm_ragged")
        super().__init__(moe_gemm_ragged_scratch_bytes(), device, "moe_gemm_ragged_scratch_bytes")

    def _rows(self, t, cols, name, offsets, where):
        rows = t.shape[0] if t.dim() == 2 else 0
        _expect(t, _torch.bfloat16, (rows, cols), self.device, name)
        _expect(offsets, _torch.int32, (self.groups + 1,), self.device, "offsets")
        if rows > self.max_rows:
            raise MoeA2AError(MOE_ERR_CAPACITY, where)
        return rows

    def _run(self, call, a, b, offsets, rows, cols, out, where, stream):
        """A product whose output has a row for each row of `a`."""
        raw = self._launch_stream(stream)
        if out is None:
            out = _empty((rows, cols), _torch.bfloat16, self.device, stream, raw)
        else:
            _expect(out, _torch.bfloat16, (rows, cols), self.device, "out")
        st = call(a.data_ptr(), b.data_ptr(), offsets.data_ptr(), self.groups, rows, self.N,
                  self.hidden, out.data_ptr(), self._scratch_ptr, self._scratch_bytes, raw)
        if st != MOE_OK:
            raise MoeA2AError(st, where)
        return out

    def forward(self, x, w, offsets, out=None, stream=None):
        """x bf16 [rows, H], w bf16 [G, N, H] -> out bf16 [rows, N].  Under
        torch.no_grad(), or in a torch.autograd.Function, x and w may require
        gradients; elsewhere that is an error."""
        if (getattr(x, "requires_grad", False) or getattr(w, "requires_grad", False)) and \
                _torch.is_grad_enabled():
            raise ValueError("forward returns no history: call it under torch.no_grad(), and "
                             "input_grad and weight_grad for the gradients")
        G, N, H = self.groups, self.N, self.hidden
        rows = self._rows(x, H, "x", offsets, "moe_gemm_ragged")
        _expect(w, _torch.bfloat16, (G, N, H), self.device, "w")
        return self._run(_lib.moe_gemm_ragged, x, w, offsets, rows, N, out, "moe_gemm_ragged",
                         stream)

    def input_grad(self, dy, w, offsets, out=None, stream=None):
        """dy bf16 [rows, N], w bf16 [G, N, H] -> dx bf16 [rows, H].  N a
        multiple of 8."""
        G, N, H = self.groups, self.N, self.hidden
        rows = self._rows(dy, N, "dy", offsets, "moe_gemm_ragged_input_grad")
        _expect(w, _torch.bfloat16, (G, N, H), self.device, "w")
        return self._run(_lib.moe_gemm_ragged_input_grad, dy, w, offsets, rows, H, out,
                         "moe_gemm_ragged_input_grad", stream)

    def weight_grad(self, dy, x, offsets, out=None, dtype=None, accumulate=False, stream=None):
        """dy bf16 [rows, N], x bf16 [rows, H] -> dw [G, N, H], bf16 (or
        dtype = float32; with `out` its type), zero for an expert without rows.
        accumulate: added to a float32 `out`.  N a multiple of 8."""
        G, N, H, dev = self.groups, self.N, self.hidden, self.device
        where = "moe_gemm_ragged_weight_grad"
        rows = self._rows(dy, N, "dy", offsets, where)
        _expect(x, _torch.bfloat16, (rows, H), dev, "x")
        if dtype is None:
            dtype = _torch.bfloat16 if out is None else out.dtype
        if dtype is not _torch.bfloat16 and dtype is not _torch.float32:
            raise ValueError("the weights' gradient is bfloat16 or float32, not %s" % dtype)
        if accumulate and (out is None or dtype is not _torch.float32):
            raise ValueError("accumulate needs a float32 out")
        raw = self._launch_stream(stream)
        if out is None:
            out = _empty((G, N, H), dtype, dev, stream, raw)
        else:
            _expect(out, dtype, (G, N, H), dev, "out")
        st = _lib.moe_gemm_ragged_weight_grad(
            dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), G, rows, N, H,
            dtype is _torch.float32, bool(accumulate), out.data_ptr(), self._scratch_ptr,
            self._scratch_bytes, raw)
        if st != MOE_OK:
            raise MoeA2AError(st, where)
        return out


class MoeLayerSmall(_Scratch):
    """A whole mixture-of-experts layer for at most `max_tokens` tokens (64 at
    most), with the scratch memory it needs.  One call at a time: calls in
    stream order."""

    def __init__(self, num_experts: int, hidden: int, inter: int, top_k: int,
                 max_tokens: int = MOE_LAYER_MAX_TOKENS, fmt: int = MOE_FORMAT_BF16,
                 device=None):
        self.num_experts, self.hidden, self.inter, self.top_k = num_experts, hidden, inter, top_k
        self.max_tokens, self.fmt = max_tokens, fmt
        self._wtypes = {MOE_FORMAT_BF16: (_torch.bfloat16,), MOE_FORMAT_INT8: (_torch.int8,),
                        MOE_FORMAT_FP8_E4M3: (_torch.float8_e4m3fn, _torch.uint8)}.get(fmt)
        if self._wtypes is None or max(num_experts, hidden, inter, top_k,
                                       max_tokens) > _INT32_MAX:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_layer_small")
        super().__init__(moe_layer_small_scratch_bytes(max_tokens, top_k, hidden, inter), device,
                         "moe_layer_small_scratch_bytes")

    def forward(self, x, topk_ids, topk_w, w13, w2, w13_scale=None, w2_scale=None,
                residual=None, out=None, stream=None):
        """x bf16 [T, H], topk_ids int32 [T, K], topk_w float32 [T, K],
        w13 [E, 2I, H] (gate rows, then up rows), w2 [E, H, I] in the
        handle's format, with channel scales float32 [E, 2I], [E, H] for the
        8-bit formats -> out bf16 [T, H] (+ residual)."""
        E, H, I, K, dev = self.num_experts, self.hidden, self.inter, self.top_k, self.device
        T = x.shape[0]
        _expect(x, _torch.bfloat16, (T, H), dev, "x")
        _expect(topk_ids, _torch.int32, (T, K), dev, "topk_ids")
        _expect(topk_w, _torch.float32, (T, K), dev, "topk_w")
        if T > self.max_tokens:
            raise MoeA2AError(MOE_ERR_CAPACITY, "moe_layer_small")
        if w13.dtype not in self._wtypes or w2.dtype not in self._wtypes:
            raise ValueError("w13, w2: expected %s" % (self._wtypes[0],))
        _expect(w13, w13.dtype, (E, 2 * I, H), dev, "w13")
        _expect(w2, w2.dtype, (E, H, I), dev, "w2")
        if self.fmt != MOE_FORMAT_BF16:
            if w13_scale is None or w2_scale is None:
                raise ValueError("w13_scale and w2_scale are needed for 8-bit weights")
            _expect(w13_scale, _torch.float32, (E, 2 * I), dev, "w13_scale")
            _expect(w2_scale, _torch.float32, (E, H), dev, "w2_scale")
        if residual is not None:
            _expect(residual, _torch.bfloat16, (T, H), dev, "residual")
        raw = self._launch_stream(stream)
        if out is None:
            out = _empty((T, H), _torch.bfloat16, dev, stream, raw)
        else:
            _expect(out, _torch.bfloat16, (T, H), dev, "out")
        st = _lib.moe_layer_small(x.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(),
                                  w13.data_ptr(), _ptr(w13_scale), w2.data_ptr(),
                                  _ptr(w2_scale), _ptr(residual), T, K, E, H, I, self.fmt,
                                  out.data_ptr(), self._scratch_ptr, self._scratch_bytes,
                                  raw)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_layer_small")
        return out


# ---- torch convenience wrapper ------------------------------------------------

def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


class DispatchView:
    """torch views into the workspace produced by one dispatch."""

    def __init__(self, owner, raw: MoeDispatchView):
        import torch
        R, K, E = owner.ep_size, owner.top_k, owner.num_experts
        H, m, RP = owner.hidden, raw.plane_stride, raw.send_stride
        T = raw.token_stride

        def region(ptr, dtype, shape):
            n = 1
            for s in shape:
                n *= s
            off = ptr - owner.workspace.data_ptr()
            nbytes = n * torch.empty((), dtype=dtype).element_size()
            return owner.workspace[off:off + nbytes].view(dtype).view(shape)

        self.plane_stride, self.send_stride = m, RP
        self.tokens_per_rank, self.token_stride = raw.tokens_per_rank, T
        self.recv_format, self.layout = raw.recv_format, raw.layout
        self.kernels = raw.kernels
        # planes: (dst rank, src rank) of m rows, or (expert) of cap = m rows
        planes = (E,) if raw.layout == MOE_LAYOUT_EXPERT else (R, R)
        if raw.recv_format == MOE_FORMAT_FP8_E4M3:
            self.recv_x = region(raw.recv_x, torch.float8_e4m3fn, planes + (m, H))
            self.recv_scale = region(raw.recv_scale, torch.float32, planes + (m,))
        else:
            self.recv_x = region(raw.recv_x, torch.bfloat16, planes + (m, H))
            self.recv_scale = None
        if raw.layout == MOE_LAYOUT_EXPERT:
            self.recv_topk_ids = None
            self.recv_topk_w = region(raw.recv_topk_w, torch.float32, (E, m))
            self.src_token = region(raw.src_token, torch.int32, (E, m))
            self.recv_counts = region(raw.recv_counts, torch.int32, (E,))
            self.local_expert_counts = region(raw.local_expert_counts, torch.int32, (E,))
        else:
            self.recv_topk_ids = region(raw.recv_topk_ids, torch.int32, (R, R, m, K))
            self.recv_topk_w = region(raw.recv_topk_w, torch.float32, (R, R, m, K))
            self.src_token = region(raw.src_token, torch.int32, (R, R, m))
            self.recv_counts = region(raw.recv_counts, torch.int32, (R, R))
            self.local_expert_counts = region(raw.local_expert_counts, torch.int32,
                                              (R, E // R))
        self.send_slot = region(raw.send_slot, torch.int32, (R, T, RP))
        self.dest_weight = region(raw.dest_weight, torch.float32, (R, T, RP))


class MoeA2A:
    """One dispatch/combine handle over a torch-allocated device workspace."""

    def __init__(self, ep_size: int, max_tokens_per_rank: int, hidden: int, num_experts: int,
                 top_k: int, device=None, layout: int = MOE_LAYOUT_RANK):
        import torch
        self.ep_size, self.max_tokens_per_rank, self.hidden = ep_size, max_tokens_per_rank, hidden
        self.num_experts, self.top_k, self.layout = num_experts, top_k, layout
        self.cfg = config(ep_size, max_tokens_per_rank, hidden, num_experts, top_k)
        nbytes = moe_a2a_workspace_bytes_layout(self.cfg, layout)
        if nbytes == 0:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_a2a_workspace_bytes_layout")
        self.device = torch.device(device if device is not None else "cuda")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _on_current(self.workspace.device)  # the handle is prepared for the current device
        st, self.handle = moe_a2a_create_layout(self.cfg, layout, self.workspace.data_ptr(),
                                                nbytes)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_a2a_create")
        self.last_view = None
        self._views = {}
        self._payload = None

    def _stream(self, stream) -> int:
        return _raw_stream(stream, self.workspace.device)

    def _check(self, t, dtype, shape, name):
        if t.dtype != dtype or tuple(t.shape) != tuple(shape):
            raise ValueError("%s: expected %s %s, got %s %s" % (name, dtype, tuple(shape),
                                                               t.dtype, tuple(t.shape)))
        if not t.is_contiguous() or t.device != self.workspace.device:
            raise ValueError("%s must be contiguous on %s" % (name, self.workspace.device))

    def _planes(self):
        return (self.num_experts,) if self.layout == MOE_LAYOUT_EXPERT else (
            self.ep_size, self.ep_size)

    @property
    def phase(self) -> int:
        return moe_a2a_phase(self.handle)

    def dispatch(self, topk_ids, topk_w, x, runtime_max_tokens_per_rank: int = None,
                 stream=None) -> DispatchView:
        import torch
        R, H, K = self.ep_size, self.hidden, self.top_k
        T = topk_ids.shape[1]
        m = T if runtime_max_tokens_per_rank is None else runtime_max_tokens_per_rank
        self._check(topk_ids, torch.int32, (R, T, K), "topk_ids")
        self._check(topk_w, torch.float32, (R, T, K), "topk_w")
        self._check(x, torch.bfloat16, (R, T, H), "x")
        st, raw = moe_dispatch(self.handle, _ptr(topk_ids), _ptr(topk_w), _ptr(x), T, m,
                               self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_dispatch")
        return self._view(raw)

    def _view(self, raw) -> DispatchView:
        # The views depend only on (m, token stride, format) and on which of
        # the two count regions holds this call's local-expert counts: reuse
        # them across calls.
        key = (raw.plane_stride, raw.token_stride, raw.recv_format, raw.local_expert_counts)
        view = self._views.get(key)
        if view is None:
            view = self._views[key] = DispatchView(self, raw)
        else:  # the per-call scalars of this call
            view.kernels, view.tokens_per_rank = raw.kernels, raw.tokens_per_rank
        self.last_view = view
        return view

    def dispatch_varlen(self, topk_ids, topk_w, x, tokens_per_rank, stream=None) -> DispatchView:
        """Per-rank token counts: inputs [R, m, ...], rows t < tokens_per_rank[s]."""
        import torch
        R, H, K = self.ep_size, self.hidden, self.top_k
        m = topk_ids.shape[1]
        self._check(topk_ids, torch.int32, (R, m, K), "topk_ids")
        self._check(topk_w, torch.float32, (R, m, K), "topk_w")
        self._check(x, torch.bfloat16, (R, m, H), "x")
        st, raw = moe_dispatch_varlen(self.handle, _ptr(topk_ids), _ptr(topk_w), _ptr(x),
                                      list(tokens_per_rank), m, self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_dispatch_varlen")
        return self._view(raw)

    def set_active_ranks(self, active: int):
        """Bit d set = logical rank d alive (default: all)."""
        st = moe_a2a_set_active_ranks(self.handle, active)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_a2a_set_active_ranks")

    def combine_payload(self):
        """bf16 [R, R, m, H] view of the in-workspace combine payload region."""
        import torch
        if self.last_view is None:
            raise RuntimeError("no dispatch yet")
        R, H, m = self.ep_size, self.hidden, self.last_view.plane_stride
        planes = (self.num_experts,) if self.layout == MOE_LAYOUT_EXPERT else (R, R)
        if self._payload is None or self._payload.shape[-2] != m:
            off = moe_combine_payload(self.handle) - self.workspace.data_ptr()
            n = planes[0] * (planes[1] if len(planes) > 1 else 1) * m * H * 2
            self._payload = self.workspace[off:off + n].view(torch.bfloat16).view(
                *planes, m, H)
        return self._payload

    def combine(self, expert_out=None, weighted: bool = False, residual=None, gamma=None,
                eps: float = 1e-6, out=None, residual_out=None, stream=None):
        import torch
        if self.last_view is None:
            st = moe_combine(self.handle, 0, weighted, 0, 0, eps, 0, 0, self._stream(stream))
            raise MoeA2AError(st if st != MOE_OK else MOE_ERR_PHASE, "moe_combine")
        R, H = self.ep_size, self.hidden
        T, m = self.last_view.token_stride, self.last_view.plane_stride
        if expert_out is not None:
            self._check(expert_out, torch.bfloat16, self._planes() + (m, H), "expert_out")
        if residual is not None:
            self._check(residual, torch.bfloat16, (R, T, H), "residual")
            self._check(gamma, torch.bfloat16, (H,), "gamma")
            if residual_out is not None:
                self._check(residual_out, torch.bfloat16, (R, T, H), "residual_out")
        if out is None:
            out = torch.empty((R, T, H), dtype=torch.bfloat16, device=self.workspace.device)
        self._check(out, torch.bfloat16, (R, T, H), "out")
        st = moe_combine(self.handle, _ptr(expert_out), weighted, _ptr(residual), _ptr(gamma),
                         eps, _ptr(out), _ptr(residual_out), self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_combine")
        return out

    def combine_fp8(self, expert_out=None, weighted: bool = False, residual=None, gamma=None,
                    eps: float = 1e-6, out=None, out_scale=None, residual_out=None,
                    stream=None):
        """As combine, with an e4m3 output and one fp32 scale per token row:
        returns (out float8_e4m3fn [R, T, H], out_scale float32 [R, T])."""
        import torch
        if self.last_view is None:
            st = moe_combine_fp8(self.handle, 0, weighted, 0, 0, eps, 0, 0, 0,
                                 self._stream(stream))
            raise MoeA2AError(st if st != MOE_OK else MOE_ERR_PHASE, "moe_combine_fp8")
        R, H = self.ep_size, self.hidden
        T, m = self.last_view.token_stride, self.last_view.plane_stride
        if expert_out is not None:
            self._check(expert_out, torch.bfloat16, self._planes() + (m, H), "expert_out")
        if residual is not None:
            self._check(residual, torch.bfloat16, (R, T, H), "residual")
            self._check(gamma, torch.bfloat16, (H,), "gamma")
            if residual_out is not None:
                self._check(residual_out, torch.bfloat16, (R, T, H), "residual_out")
        dev = self.workspace.device
        if out is None:
            out = torch.empty((R, T, H), dtype=torch.float8_e4m3fn, device=dev)
        if out_scale is None:
            out_scale = torch.empty((R, T), dtype=torch.float32, device=dev)
        self._check(out, torch.float8_e4m3fn, (R, T, H), "out")
        self._check(out_scale, torch.float32, (R, T), "out_scale")
        st = moe_combine_fp8(self.handle, _ptr(expert_out), weighted, _ptr(residual),
                             _ptr(gamma), eps, _ptr(out), _ptr(out_scale), _ptr(residual_out),
                             self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_combine_fp8")
        return out, out_scale

    def expert_gemm(self, w, out=None, stream=None):
        """Expert layout: out[e][j] = x[e][j] . w[e]^T for the received rows.
        w: bf16 [E, N, H]; out: bf16 [E, cap, N], or None to write the
        combine payload (N == H).  Returns the output tensor."""
        import torch
        E, H = self.num_experts, self.hidden
        N = w.shape[1]
        self._check(w, torch.bfloat16, (E, N, H), "w")
        if out is not None:
            self._check(out, torch.bfloat16, (E, self.last_view.plane_stride, N), "out")
        st = moe_expert_gemm(self.handle, _ptr(w), N, _ptr(out), self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_expert_gemm")
        return out if out is not None else self.combine_payload()

    def _rank_out_scratch(self, N, out, scratch):
        import torch
        R = self.ep_size
        if out is not None:
            self._check(out, torch.bfloat16, (R, R, self.last_view.plane_stride, N), "out")
        need = moe_expert_gemm_rank_scratch_bytes(self.cfg, N)
        if need == 0:
            raise MoeA2AError(MOE_ERR_INVALID_ARG, "moe_expert_gemm_rank_scratch_bytes")
        if scratch is None:
            if getattr(self, "_rank_scratch", None) is None or self._rank_scratch.numel() < need:
                self._rank_scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
            scratch = self._rank_scratch
        if scratch.dtype != torch.uint8 or scratch.device != self.workspace.device:
            raise ValueError("scratch: expected a uint8 tensor on %s" % self.workspace.device)
        return scratch

    def expert_gemm_rank(self, w, apply_gates=True, out=None, scratch=None, stream=None):
        """Rank layout: each received row's local experts applied to it, their
        bf16 outputs summed with the gates (or plainly) in ascending top-k
        order.  w: bf16 [E, N, H]; out: bf16 [R, R, m, N], or None to write the
        combine payload (N == H); scratch: uint8 device tensor of at least
        moe_expert_gemm_rank_scratch_bytes bytes (allocated and kept here if
        None).  Returns the output tensor."""
        import torch
        E, H = self.num_experts, self.hidden
        N = w.shape[1]
        self._check(w, torch.bfloat16, (E, N, H), "w")
        scratch = self._rank_out_scratch(N, out, scratch)
        st = moe_expert_gemm_rank(self.handle, _ptr(w), N, int(bool(apply_gates)), _ptr(out),
                                  scratch.data_ptr(), scratch.numel(), self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_expert_gemm_rank")
        return out if out is not None else self.combine_payload()

    def expert_gemm_rank_fp8(self, w8, w_scale, apply_gates=True, out=None, scratch=None,
                             stream=None):
        """expert_gemm_rank on FP8 operands, for a rank-layout dispatch in the
        FP8 receive format: each expert output is (qx . qw[e]^T) sx sw[e],
        narrowed to bf16, then gated and summed as expert_gemm_rank does.
        w8: e4m3 [E, N, H] (float8_e4m3fn or uint8); w_scale: float32 [E, N];
        out and scratch as for expert_gemm_rank."""
        import torch
        E, H = self.num_experts, self.hidden
        N = w8.shape[1]
        if w8.dtype not in (torch.float8_e4m3fn, torch.uint8) or tuple(w8.shape) != (E, N, H) \
                or not w8.is_contiguous():
            raise ValueError("w8: expected contiguous e4m3 [%d, N, %d]" % (E, H))
        self._check(w_scale, torch.float32, (E, N), "w_scale")
        scratch = self._rank_out_scratch(N, out, scratch)
        st = moe_expert_gemm_rank_fp8(self.handle, _ptr(w8), _ptr(w_scale), N,
                                      int(bool(apply_gates)), _ptr(out), scratch.data_ptr(),
                                      scratch.numel(), self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_expert_gemm_rank_fp8")
        return out if out is not None else self.combine_payload()

    def expert_gemm_fp8(self, w8, w_scale, out=None, stream=None):
        """FP8 receive format: out[e][j] = (qx[e][j] . qw[e]^T) sx[e][j] sw[e].
        w8: e4m3 [E, N, H] (float8_e4m3fn or uint8); w_scale: float32 [E, N];
        out: bf16 [E, cap, N], or None to write the combine payload (N == H)."""
        import torch
        E, H = self.num_experts, self.hidden
        N = w8.shape[1]
        if w8.dtype not in (torch.float8_e4m3fn, torch.uint8) or tuple(w8.shape) != (E, N, H) \
                or not w8.is_contiguous():
            raise ValueError("w8: expected contiguous e4m3 [%d, N, %d]" % (E, H))
        self._check(w_scale, torch.float32, (E, N), "w_scale")
        if out is not None:
            self._check(out, torch.bfloat16, (E, self.last_view.plane_stride, N), "out")
        st = moe_expert_gemm_fp8(self.handle, _ptr(w8), _ptr(w_scale), N, _ptr(out),
                                 self._stream(stream))
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_expert_gemm_fp8")
        return out if out is not None else self.combine_payload()

    def set_recv_format(self, fmt: int):
        """MOE_FORMAT_BF16 (default) or MOE_FORMAT_FP8_E4M3 rows in recv_x."""
        st = moe_a2a_set_recv_format(self.handle, fmt)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_a2a_set_recv_format")

    def set_reduction(self, reduction: int):
        """MOE_REDUCE_FP32_RANK_ORDER (default) or MOE_REDUCE_BF16_TOPK_TREE."""
        st = moe_a2a_set_reduction(self.handle, reduction)
        if st != MOE_OK:
            raise MoeA2AError(st, "moe_a2a_set_reduction")

    def get_error(self, stream=None):
        """Synchronise, read and clear the device flag word: (status, bits)."""
        return moe_a2a_get_error(self.handle, self._stream(stream))

    def close(self):
        if getattr(self, "handle", None):
            moe_a2a_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
