"""The torch forms of the operators on tensors of a device that is not the current
one (host only: the tensors are stand-ins, and the library must not be called)."""
import math

import pytest

torch = pytest.importorskip("torch")


class Stand:
    """What the torch forms read of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream.cuda_stream]


class StandStream:
    def __init__(self, index, raw=0):
        self.device, self.cuda_stream = torch.device("cuda", index), raw


class Library:
    """Counts calls; every entry succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return b"" if name == "moe_a2a_status_string" else 0
        return entry


@pytest.fixture
def api(monkeypatch):
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    monkeypatch.setattr(moe_a2a, "_lib", Library())
    monkeypatch.setattr(moe_a2a, "_current_device", lambda: 0)
    monkeypatch.setattr(moe_a2a, "_current_stream", lambda index: 0)
    return moe_a2a


def handle(cls, index, **fields):
    h = cls.__new__(cls)
    h.__dict__.update(fields, device=torch.device("cuda", index), _scratch_ptr=1 << 20,
                      _scratch_bytes=1 << 20, scratch=Stand((1 << 20,), torch.uint8, index),
                      _streams={0})
    return h


def calls(api, index, stream=None):
    S = lambda shape, dtype: Stand(shape, dtype, index)
    f32, i32, i8, bf = torch.float32, torch.int32, torch.int8, torch.bfloat16
    gemm = handle(api.MoeGemmInt8, index, groups=1, max_rows=4, N=8, hidden=16)
    layer = handle(api.MoeLayerSmall, index, num_experts=4, hidden=16, inter=16, top_k=2,
                   max_tokens=4, fmt=api.MOE_FORMAT_BF16, _wtypes=(bf,))
    return {
        "moe_topk_gate": lambda: api.topk_gate(S((3, 8), f32), 2, out_ids=S((3, 2), i32),
                                               out_w=S((3, 2), f32), stream=stream),
        "moe_quantize_rows_int8": lambda: api.quantize_rows_int8(
            S((3, 16), bf), out=S((3, 16), i8), scale=S((3,), f32), stream=stream),
        "moe_gemm_int8": lambda: gemm.gemm(S((4, 16), i8), S((4,), f32), S((8, 16), i8),
                                           S((8,), f32), out=S((4, 8), bf), stream=stream),
        "moe_layer_small": lambda: layer.forward(
            S((2, 16), bf), S((2, 2), i32), S((2, 2), f32), S((4, 32, 16), bf),
            S((4, 16, 16), bf), out=S((2, 16), bf), stream=stream),
        "moe_scratch_get_error": lambda: gemm.get_error(stream),
    }


NAMES = ["moe_topk_gate", "moe_quantize_rows_int8", "moe_gemm_int8", "moe_layer_small",
         "moe_scratch_get_error"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_are_refused(api, name):
    with pytest.raises(ValueError, match="not the current CUDA device"):
        calls(api, 1)[name]()
    with pytest.raises(ValueError):
        calls(api, 1, stream=StandStream(1))[name]()
    assert api._lib.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(api, name):
    with pytest.raises(ValueError, match="a stream of cuda:1"):
        calls(api, 0, stream=StandStream(1))[name]()
    assert api._lib.calls == []


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [None, StandStream(0), 0])
def test_tensors_of_the_current_device_are_taken(api, name, stream):
    calls(api, 0, stream=stream)[name]()
    assert api._lib.calls == [name]


def test_scratch_on_another_device_is_refused(api, monkeypatch):
    monkeypatch.setattr(api._torch, "empty",
                        lambda n, dtype, device: Stand((n,), dtype, torch.device(device).index))
    monkeypatch.setattr(api, "moe_gemm_int8_scratch_bytes", lambda rows: 1 << 20)
    with pytest.raises(ValueError, match="not the current CUDA device"):
        api.MoeGemmInt8(1, 4, 8, 16, "cuda:1")
    assert api._lib.calls == []


def a2a(api, index):
    a = api.MoeA2A.__new__(api.MoeA2A)
    a.__dict__.update(ep_size=2, hidden=16, top_k=2, num_experts=4, layout=api.MOE_LAYOUT_RANK,
                      handle=None, last_view=None, workspace=Stand((1 << 20,), torch.uint8, index),
                      device=torch.device("cuda", index))
    return a


def test_dispatch_and_combine_on_another_device_are_refused(api):
    S = lambda shape, dtype: Stand(shape, dtype, 1)
    a = a2a(api, 1)
    ids, w, x = (S((2, 3, 2), torch.int32), S((2, 3, 2), torch.float32),
                 S((2, 3, 16), torch.bfloat16))
    for call in (lambda: a.dispatch(ids, w, x), lambda: a.dispatch_varlen(ids, w, x, [3, 1]),
                 lambda: a.combine(), lambda: a.combine_fp8(), lambda: a.get_error(),
                 lambda: a.get_error(StandStream(1)),
                 lambda: api.quantize_rows_fp8(S((3, 16), torch.float32),
                                               S((3, 16), torch.float8_e4m3fn),
                                               S((3,), torch.float32))):
        with pytest.raises(ValueError, match="not the current CUDA device"):
            call()
    assert api._lib.calls == []
    assert a2a(api, 0).get_error()[0] == api.MOE_OK and api._lib.calls == ["moe_a2a_get_error"]


def test_workspace_on_another_device_is_refused(api, monkeypatch):
    monkeypatch.setattr(torch, "empty",
                        lambda n, dtype, device: Stand((n,), dtype, torch.device(device).index))
    monkeypatch.setattr(api, "moe_a2a_workspace_bytes_layout", lambda cfg, layout: 1 << 20)
    with pytest.raises(ValueError, match="not the current CUDA device"):
        api.MoeA2A(2, 8, 16, 4, 2, "cuda:1")
    assert api._lib.calls == []


def test_scratch_is_tied_to_the_streams_it_is_used_on(api, monkeypatch):
    h = handle(api.MoeGemmInt8, 0, groups=1, max_rows=4, N=8, hidden=16)
    S = lambda shape, dtype: Stand(shape, dtype, 0)
    args = (S((4, 16), torch.int8), S((4,), torch.float32), S((8, 16), torch.int8),
            S((8,), torch.float32), None, S((4, 8), torch.bfloat16))
    recorded = lambda: getattr(h.scratch, "recorded", [])
    h.gemm(*args)                                       # where it was allocated
    h.gemm(*args, stream=StandStream(0, 0))
    assert recorded() == []
    side = StandStream(0, 7)
    h.gemm(*args, stream=side)
    h.gemm(*args, stream=side)
    assert recorded() == [7]                            # once a stream
    h.gemm(*args, stream=9)                             # a bare number: the caller's part
    assert recorded() == [7]
    monkeypatch.setattr(api, "_current_stream", lambda index: 11)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: StandStream(0, 11))
    h.gemm(*args)                                       # another stream made current
    assert recorded() == [7, 11]
    assert api._lib.calls == ["moe_gemm_int8"] * 6


def test_sizes_past_32_bits_are_refused(api, monkeypatch):
    # 2^32 + 5 rows are not 5 rows
    S = lambda shape, dtype: Stand(shape, dtype, 0)
    f32, i32, i8 = torch.float32, torch.int32, torch.int8
    monkeypatch.setattr(api._torch, "empty",
                        lambda shape, dtype, device: Stand(
                            shape if isinstance(shape, (tuple, list, torch.Size)) else (shape,),
                            dtype, 0))
    big = 2 ** 32
    for call in (
            lambda: api.quantize_rows_int8(S((big + 5, 8), f32)),
            lambda: api.quantize_rows_int8(S((2, big + 5, 8), f32), S((2,), i32)),
            lambda: api.quantize_rows_int8(S((big + 5, 2, 8), f32), S((big + 5,), i32)),
            lambda: api.quantize_rows_int8(S((2, big + 64), f32)),
            lambda: api.topk_gate(S((2, big + 64), f32), 2),
            lambda: api.topk_gate(S((2, 64), f32), big + 2),
            lambda: api.MoeGemmInt8(1, big + 4, 8, 16, "cuda:0"),
            lambda: api.MoeGemmInt8(1, 4, big + 8, 16, "cuda:0"),
            lambda: api.MoeGemmInt8(1, 4, 8, big + 16, "cuda:0"),
            lambda: api.MoeLayerSmall(4, big + 16, 16, 2, 4, device="cuda:0"),
            lambda: api.MoeLayerSmall(big + 4, 16, 16, 2, 4, device="cuda:0"),
            lambda: api.MoeLayerSmall(4, 16, 16, 2, big + 4, device="cuda:0")):
        with pytest.raises(api.MoeA2AError):
            call()
    # (only the text of the error was asked for)
    assert set(api._lib.calls) <= {"moe_a2a_status_string"}
