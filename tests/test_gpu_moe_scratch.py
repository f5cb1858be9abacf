"""A handle that is dropped while its call still runs on another stream."""
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


@pytest.mark.parametrize("make_current", [False, True])
@pytest.mark.parametrize("op", ["gemm", "layer"])
def test_scratch_of_a_dropped_handle_is_not_given_away(api, op, make_current):
    g = torch.Generator(device=DEV).manual_seed(3)
    side = torch.cuda.Stream()
    if op == "gemm":
        # few tiles, long k: every tile is cut, and its parts go through the scratch
        M, N, H = 300, 520, 4096
        codes = lambda *s: torch.randint(-30, 31, s, generator=g, device=DEV).to(torch.int8)
        args = (codes(1, M, H), torch.rand((1, M), generator=g, device=DEV), codes(1, N, H),
                torch.rand((1, N), generator=g, device=DEV))
        make = lambda: api.MoeGemmInt8(1, M, N, H, DEV)
        call = lambda h, s: h.gemm(*args, out=torch.empty((1, M, N), dtype=torch.bfloat16,
                                                          device=DEV), stream=s)
    else:
        T, E, H, I, K = 8, 8, 1024, 512, 2
        normal = lambda *s: (torch.randn(s, generator=g, device=DEV) / s[-1] ** 0.5).to(
            torch.bfloat16)
        args = (normal(T, H), torch.randint(0, E, (T, K), generator=g, device=DEV).int(),
                torch.rand((T, K), generator=g, device=DEV), normal(E, 2 * I, H), normal(E, H, I))
        make = lambda: api.MoeLayerSmall(E, H, I, K, T, api.MOE_FORMAT_BF16, DEV)
        call = lambda h, s: h.forward(*args, out=torch.empty_like(args[0]), stream=s)
    want = call(make(), None)
    torch.cuda.synchronize()
    h = make()
    at, nbytes = h.scratch.data_ptr(), h.scratch.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                  # about 50 ms in front of the call
    if make_current:
        with torch.cuda.stream(side):
            got = call(h, None)
    else:
        got = call(h, side)
    del h
    other = [torch.empty(nbytes, dtype=torch.uint8, device=DEV) for _ in range(3)]
    assert all(o.data_ptr() != at for o in other)
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
