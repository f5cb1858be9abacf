"""The products called first thing in a thread of their own, which has no current context
yet (autograd's threads call a backward pass so): the outputs are the main thread's."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def api():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


def ints(*shape):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(BF)


def ragged(api):
    h = api.MoeGemmRagged(2, 20, 64, 64, DEV)
    return h, torch.tensor([0, 4, 20], dtype=I32, device=DEV)


def forward(api):
    h, off = ragged(api)
    x, w = ints(20, 64), ints(2, 64, 64)
    return lambda: h.forward(x, w, off)


def input_grad(api):
    h, off = ragged(api)
    dy, w = ints(20, 64), ints(2, 64, 64)
    return lambda: h.input_grad(dy, w, off)


def weight_grad(api):
    h, off = ragged(api)
    dy, x = ints(20, 64), ints(20, 64)
    return lambda: h.weight_grad(dy, x, off)


def quantize(api):
    x = ints(20, 128)
    return lambda: api.quantize_blocks_fp8(x)[1]


def eight_bit(api):
    h = api.MoeGemmFp8(1, 20, 128, 256, DEV)
    (xq, sx), (wq, sw) = (api.quantize_blocks_fp8(ints(20, 256)),
                          api.quantize_blocks_fp8(ints(128, 256), 128))
    return lambda: h.gemm(xq, sx, wq, sw)


def integer(api):
    h = api.MoeGemmInt8(1, 20, 128, 256, DEV)
    (xq, sx), (wq, sw) = (api.quantize_rows_int8(ints(20, 256)),
                          api.quantize_rows_int8(ints(128, 256)))
    return lambda: h.gemm(xq, sx, wq, sw)


def layer(api):
    h = api.MoeLayerSmall(4, 128, 64, 2, 3, api.MOE_FORMAT_BF16, DEV)
    ids = torch.tensor([[0, 3], [1, 2], [3, 1]], dtype=I32, device=DEV)
    x, w, w13, w2 = ints(3, 128), torch.full((3, 2), 0.5, device=DEV), ints(4, 128, 128), \
        ints(4, 128, 64)
    return lambda: h.forward(x, ids, w, w13, w2)


def planes(api):
    R, T, H, E, K = 2, 40, 128, 4, 2
    a = api.MoeA2A(R, T, H, E, K, DEV, layout=api.MOE_LAYOUT_EXPERT)
    ids = torch.stack([torch.stack([(torch.arange(T) + r + k) % E for k in range(K)], 1)
                       for r in range(R)]).to(I32).to(DEV)
    x, w = ints(R, T, H), torch.full((R, T, K), 0.5, device=DEV)
    maps = ints(E, H, H)

    def run():
        a.dispatch(ids, w, x)
        a.expert_gemm(maps)
        return a.combine(None, True)
    return run


@pytest.mark.parametrize("make", [forward, input_grad, weight_grad, quantize, eight_bit, integer,
                                  layer, planes])
def test_first_call_of_a_thread(api, make):
    run = make(api)
    want = run().clone()
    torch.cuda.synchronize()
    got = []

    def body():
        try:
            got.append(run().clone())
            torch.cuda.synchronize()
        except Exception as e:
            got.append(e)

    thread = threading.Thread(target=body)
    thread.start()
    thread.join()
    assert isinstance(got[0], torch.Tensor), got[0]
    assert torch.equal(got[0], want)
