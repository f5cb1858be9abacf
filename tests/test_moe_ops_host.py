"""Host-side refusals of the operators around dispatch and combine (no GPU):
sizes, pointers and alignments are checked before anything is queued."""
import pytest

A = 1 << 20  # an aligned stand-in pointer (never touched)


@pytest.fixture(scope="module")
def abi():
    from combine_topk_ids_rank_gb300 import build_lib
    build_lib.build()
    from combine_topk_ids_rank_gb300 import moe_a2a
    return moe_a2a


GATE = dict(d_logits=A, bf16=0, tokens=4, row_stride=64, num_experts=64, top_k=8, scoring=0,
            renormalize=1, scale=1.0, d_topk_ids=A, d_topk_w=A)


@pytest.mark.parametrize("bad", [
    dict(d_logits=0), dict(d_topk_ids=0), dict(d_topk_w=0), dict(d_logits=A + 2),
    dict(d_logits=A + 1, bf16=1), dict(d_topk_ids=A + 2), dict(d_topk_w=A + 2),
    dict(tokens=-1), dict(row_stride=63), dict(num_experts=0), dict(num_experts=1025,
                                                                    row_stride=1025),
    dict(top_k=0), dict(top_k=33), dict(top_k=65), dict(num_experts=4, top_k=5),
    dict(scoring=2), dict(scoring=-1)])
def test_gate_refusals(abi, bad):
    assert abi.moe_topk_gate(**{**GATE, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_gate_without_tokens_queues_nothing(abi):
    assert abi.moe_topk_gate(**{**GATE, "tokens": 0, "d_logits": 0}) == abi.MOE_OK


QUANT = dict(d_x=A, bf16=1, groups=2, rows=3, hidden=64, row_stride=64, d_counts=0, d_q=A,
             d_scale=A)


@pytest.mark.parametrize("bad", [
    dict(d_x=0), dict(d_q=0), dict(d_scale=0), dict(d_x=A + 8), dict(d_q=A + 8),
    dict(d_scale=A + 2), dict(d_counts=A + 2), dict(groups=-1), dict(rows=-1), dict(hidden=0),
    dict(hidden=60), dict(hidden=16392, row_stride=16392), dict(row_stride=56),
    dict(row_stride=68), dict(bf16=0, row_stride=66)])
def test_quantize_refusals(abi, bad):
    assert abi.moe_quantize_rows_int8(**{**QUANT, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_quantize_without_rows_queues_nothing(abi):
    assert abi.moe_quantize_rows_int8(**{**QUANT, "rows": 0, "d_x": 0}) == abi.MOE_OK
    assert abi.moe_quantize_rows_int8(**{**QUANT, "groups": 0, "d_x": 0}) == abi.MOE_OK


GEMM = dict(d_xq=A, d_x_scale=A, d_wq=A, d_w_scale=A, d_counts=0, groups=2, rows=5, N=70,
            hidden=48, d_out=A, d_scratch=A, scratch_bytes=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(d_xq=0), dict(d_x_scale=0), dict(d_wq=0), dict(d_w_scale=0), dict(d_out=0),
    dict(d_scratch=0), dict(d_xq=A + 8), dict(d_wq=A + 8), dict(d_x_scale=A + 2),
    dict(d_w_scale=A + 1), dict(d_counts=A + 2), dict(d_out=A + 1), dict(d_scratch=A + 128),
    dict(groups=-1), dict(groups=1025), dict(rows=-1), dict(N=0), dict(hidden=0),
    dict(hidden=40), dict(groups=1024, rows=1 << 22), dict(groups=1024, N=1 << 22)])
def test_gemm_refusals(abi, bad):
    assert abi.moe_gemm_int8(**{**GEMM, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_gemm_scratch_size(abi):
    assert abi.moe_gemm_int8_scratch_bytes(0) == 0
    need = abi.moe_gemm_int8_scratch_bytes(5)
    assert 0 < need <= abi.moe_gemm_int8_scratch_bytes(300)
    assert abi.moe_gemm_int8(**{**GEMM, "scratch_bytes": need - 1}) == abi.MOE_ERR_CAPACITY
    assert abi.moe_gemm_int8(**{**GEMM, "rows": 0, "d_xq": 0}) == abi.MOE_OK
    assert abi.moe_gemm_int8(**{**GEMM, "groups": 0, "d_xq": 0}) == abi.MOE_OK


LAYER = dict(d_x=A, d_topk_ids=A, d_topk_w=A, d_w13=A, d_w13_scale=A, d_w2=A, d_w2_scale=A,
             d_residual=0, tokens=4, top_k=2, num_experts=8, hidden=64, inter=32, fmt=2, d_out=A,
             d_scratch=A, scratch_bytes=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(d_x=0), dict(d_topk_ids=0), dict(d_topk_w=0), dict(d_w13=0), dict(d_w2=0),
    dict(d_w13_scale=0), dict(d_w2_scale=0), dict(d_out=0), dict(d_scratch=0), dict(d_x=A + 8),
    dict(d_topk_ids=A + 2), dict(d_topk_w=A + 2), dict(d_w13=A + 8), dict(d_w2=A + 8),
    dict(d_w13_scale=A + 2), dict(d_w2_scale=A + 2), dict(d_residual=A + 4), dict(d_out=A + 4),
    dict(d_scratch=A + 16), dict(tokens=-1), dict(tokens=65), dict(top_k=0), dict(top_k=33),
    dict(num_experts=0), dict(num_experts=1025), dict(hidden=0), dict(hidden=72),
    dict(hidden=16400), dict(inter=0), dict(inter=24), dict(inter=16400), dict(fmt=3),
    dict(fmt=-1)])
def test_layer_refusals(abi, bad):
    assert abi.moe_layer_small(**{**LAYER, **bad}) == abi.MOE_ERR_INVALID_ARG


def test_layer_scratch_size(abi):
    assert abi.MOE_LAYER_MAX_TOKENS == 64
    for bad in ((0, 2, 64, 32), (65, 2, 64, 32), (4, 0, 64, 32), (4, 2, 72, 32), (4, 2, 64, 24)):
        assert abi.moe_layer_small_scratch_bytes(*bad) == 0
    need = abi.moe_layer_small_scratch_bytes(4, 2, 64, 32)
    assert 0 < need <= abi.moe_layer_small_scratch_bytes(64, 2, 64, 32)
    assert abi.moe_layer_small(**{**LAYER, "scratch_bytes": need - 1}) == abi.MOE_ERR_CAPACITY
    assert abi.moe_layer_small(**{**LAYER, "tokens": 0, "d_x": 0}) == abi.MOE_OK


def test_int8_is_not_a_receive_format(abi):
    c = abi.config(8, 64, 128, 32, 2)
    st, h = abi.moe_a2a_create(c, 1 << 30, abi.moe_a2a_workspace_bytes(c))
    assert st == abi.MOE_OK
    assert abi.moe_a2a_set_recv_format(h, abi.MOE_FORMAT_INT8) == abi.MOE_ERR_INVALID_ARG
    abi.moe_a2a_destroy(h)


def test_scratch_entry_refusals(abi):
    assert abi.moe_scratch_init(0, 1 << 20) == abi.MOE_ERR_INVALID_ARG
    assert abi.moe_scratch_init(A + 8, 1 << 20) == abi.MOE_ERR_INVALID_ARG
    assert abi.moe_scratch_init(A, 64) == abi.MOE_ERR_CAPACITY
    assert abi.moe_scratch_get_error(0)[0] == abi.MOE_ERR_INVALID_ARG


def test_cut_covers_every_unit_once():
    # The even split of tiles x k-blocks over CTAs that the persistent products
    # use (stream.cuh), restated: ranges cover all units once, the owner of a unit
    # is found from the unit alone, and every part of a tile has a slot of its own.
    # grain 1 cuts anywhere, grain = blocks between tiles only.
    for tiles, blocks, ctas, whole in [(1, 1, 152, True), (1, 7, 152, True), (3, 5, 4, False),
                                       (152, 3, 152, False), (153, 56, 152, False),
                                       (700, 17, 152, False), (5, 1000, 152, False),
                                       (160, 9, 152, True), (76, 4, 76, True),
                                       (28, 32, 76, False)]:
        grain = blocks if whole else 1
        grains = tiles * blocks // grain
        parts = min(tiles, ctas) if whole else ctas
        q, more = divmod(grains, parts)
        assert q >= 1
        first = lambda c: (c * q + min(c, more)) * grain

        def owner_of(u):
            g, big = u // grain, more * (q + 1)
            return g // (q + 1) if g < big else more + (g - big) // q

        owner = [c for c in range(parts) for _ in range(first(c), first(c + 1))]
        assert len(owner) == tiles * blocks == first(parts)
        assert all(owner_of(u) == owner[u] for u in range(len(owner)))
        used = set()
        for t in range(tiles):
            own = sorted(set(owner[t * blocks:(t + 1) * blocks]))
            assert own == list(range(own[0], own[-1] + 1))
            if len(own) == 1:
                continue
            assert not whole
            for c in own:
                slot = 0 if c != own[0] or first(c) == t * blocks else 1
                assert (c, slot) not in used
                used.add((c, slot))
