"""Host-side checks of the chunk operators: refusals, workspace plan, argument marshalling (no GPU)."""
import ctypes

import pytest
import torch

from sparse_long_context_indexer_b200 import _lib, api, build

P = 1 << 20
BF, FP8, F32 = _lib.DSA_BF16, _lib.DSA_FP8_E4M3, _lib.DSA_F32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def make_dims(**kw):
    d = dict(B=4, Nq=16, H_I=64, d_I=128, H=128, k=2048, T_max=4096, idx_dtype=FP8, kv_dtype=BF, ld_scores=4096)
    d.update(kw)
    return api.Dims(**d)


def paged(block_size=64, max_blocks=64, num_blocks=100, kv=P, table=P, reserved=0, k_I=P, k_scale=P):
    return _lib.DsaPagedCache(k_I=k_I, k_scale=k_scale, kv=kv, block_table=table, block_size=block_size,
                              num_blocks=num_blocks, max_blocks=max_blocks, reserved=reserved)


def rope(freq=P, latent=1, index=2):
    return _lib.DsaRope(freq, latent, index)


def ref(x):
    return None if x is None else ctypes.byref(x)


INVALID, UNSUPPORTED, WORKSPACE = _lib.DSA_ERR_INVALID_ARG, _lib.DSA_ERR_UNSUPPORTED, _lib.DSA_ERR_WORKSPACE


@pytest.mark.parametrize("case,code", [
    (dict(n=-1), INVALID),
    (dict(n=(1 << 24) + 1), UNSUPPORTED),
    (dict(n=0), _lib.DSA_OK),
    (dict(seq=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(kv_new=None), INVALID),
    (dict(kv_new=P + 8), INVALID),
    (dict(kv_stride=568), INVALID),
    (dict(kv_stride=580), INVALID),
    (dict(k_new=P + 4), INVALID),
    (dict(k_stride=120), INVALID),
    (dict(k_stride=132), INVALID),            # bf16 rows of 264 bytes
    (dict(k_dtype=FP8), INVALID),
    (dict(rope=None), INVALID),
    (dict(rope=rope(freq=None)), INVALID),
    (dict(rope=rope(latent=3)), INVALID),
    (dict(rope=rope(index=-1)), INVALID),
    (dict(k_scale=None), INVALID),
    (dict(kv=None), INVALID),
    (dict(k_I=P + 4), INVALID),
    (dict(paged=paged(block_size=48)), INVALID),
    (dict(paged=paged(block_size=32, max_blocks=128)), INVALID),
    (dict(paged=paged(max_blocks=63)), INVALID),
    (dict(paged=paged(reserved=1)), INVALID),
    (dict(paged=paged(table=None)), INVALID),
    (dict(paged=paged(k_scale=None)), INVALID),
    (dict(dims=dict(kv_dtype=F32)), UNSUPPORTED),
    (dict(dims=dict(d_I=96)), UNSUPPORTED),
    (dict(ws=P, ws_bytes=64), WORKSPACE),
])
def test_append_tokens_rope_refuses(lib, case, code):
    d = make_dims(**case.get("dims", {})).c()
    g = lambda k, v: case.get(k, v)  # noqa: E731
    rc = lib.dsa_append_tokens_rope(ctypes.byref(d), g("n", 4), g("seq", P), g("pos", P), g("kv_new", P),
                                    g("kv_stride", 576), g("k_new", P), g("k_stride", 128), g("k_dtype", BF),
                                    ref(g("rope", rope())), g("kv", P), g("k_I", P), g("k_scale", P),
                                    ref(g("paged", None)), g("ws", None), g("ws_bytes", 0), None)
    assert rc == code


@pytest.mark.parametrize("case,code", [
    (dict(pos=None), INVALID),
    (dict(rope=None), INVALID),
    (dict(q_pe=None, qi_new=None), INVALID),
    (dict(q=None), INVALID),
    (dict(q=P + 8), INVALID),
    (dict(q_nope=P + 2), INVALID),
    (dict(head=56), INVALID),
    (dict(head=68), INVALID),
    (dict(row=127 * 192), INVALID),
    (dict(q_I=None), INVALID),
    (dict(q_scale=None), INVALID),
    (dict(q_scale=P + 4), INVALID),
    (dict(qi_dtype=FP8), INVALID),
    (dict(qi_row=64 * 128 - 8), INVALID),
    (dict(qi_row=64 * 128 + 4), INVALID),
    (dict(dims=dict(H_I=32)), UNSUPPORTED),
    (dict(dims=dict(H=64)), UNSUPPORTED),
    (dict(dims=dict(kv_dtype=F32)), UNSUPPORTED),
    (dict(dims=dict(Nq=(1 << 24) + 1)), UNSUPPORTED),
    (dict(dims=dict(Nq=0)), _lib.DSA_OK),
])
def test_rope_queries_refuses(lib, case, code):
    d = make_dims(**case.get("dims", {})).c()
    g = lambda k, v: case.get(k, v)  # noqa: E731
    rc = lib.dsa_rope_queries(ctypes.byref(d), g("pos", P), ref(g("rope", rope())), g("q_nope", P), g("q_pe", P),
                              g("row", 128 * 192), g("head", 192), g("q", P), g("qi_new", P), g("qi_row", 64 * 128),
                              g("qi_dtype", BF), g("q_I", P), g("q_scale", P), None)
    assert rc == code


@pytest.mark.parametrize("case,code", [
    (dict(cache=None), INVALID),
    (dict(cache=paged(table=None)), INVALID),
    (dict(cache=paged(block_size=96)), INVALID),
    (dict(cache=paged(block_size=32, max_blocks=128)), INVALID),
    (dict(cache=paged(max_blocks=32)), INVALID),
    (dict(cache=paged(num_blocks=0)), INVALID),
    (dict(cache=paged(num_blocks=1 << 24)), UNSUPPORTED),
    (dict(cache=paged(kv=None)), INVALID),
    (dict(cache=paged(kv=P + 8)), INVALID),
    (dict(q=None), INVALID),
    (dict(q=P + 2), INVALID),
    (dict(q_len=None), INVALID),
    (dict(out=P + 4), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=P + 16), INVALID),               # its partials are stored 32 bytes at a time
    (dict(ws_bytes=1024), WORKSPACE),
    (dict(dims=dict(kv_dtype=F32)), UNSUPPORTED),
    (dict(dims=dict(H=64)), UNSUPPORTED),
    (dict(dims=dict(Nq=-1)), INVALID),
    (dict(dims=dict(Nq=0)), _lib.DSA_OK),
])
def test_chunk_attn_paged_refuses(lib, case, code):
    d = make_dims(**case.get("dims", {})).c()
    g = lambda k, v: case.get(k, v)  # noqa: E731
    rc = lib.dsa_chunk_attn_paged(ctypes.byref(d), g("q", P), ref(g("cache", paged(k_I=None, k_scale=None))), P,
                                  g("q_len", P), ctypes.c_float(g("scale", 0.07)), g("out", P), P, g("ws", P),
                                  g("ws_bytes", 1 << 30), None)
    assert rc == code


def test_packed_structures_are_the_interface_s(lib):
    # the byte forms that api.py passes are the C structures'
    d = make_dims(Nq=7, ld_scores=1 << 33)
    assert api._dims_arg(d) == bytes(d.c())
    assert api._pack_cache(1, 2, 3, 4, 5, 6, 7, 0) == bytes(_lib.DsaPagedCache(1, 2, 3, 4, 5, 6, 7, 0))
    assert api._pack_rope(9, 1, 2) == bytes(_lib.DsaRope(9, 1, 2))


def test_no_rows_need_no_pointers(lib):
    # the pointers of tensors without elements are null
    d = make_dims(Nq=0).c()
    assert lib.dsa_rope_queries(ctypes.byref(d), None, ref(rope()), None, None, 128 * 192, 192, None, None, 64 * 128, BF,
                                None, None, None) == _lib.DSA_OK
    assert lib.dsa_chunk_attn_paged(ctypes.byref(d), None, ref(paged()), None, None, 0.07, None, None, P, 1 << 30,
                                    None) == _lib.DSA_OK


def test_row_limits_are_the_documented_ones(lib):
    # 16,777,216 rows pass the size checks (the null or misaligned pointer after them is what is refused), one more does not
    rows = 1 << 24
    for nq, code in ((rows, INVALID), (rows + 1, UNSUPPORTED)):
        d = make_dims(Nq=nq).c()
        assert lib.dsa_rope_queries(ctypes.byref(d), None, ref(rope()), P, P, 128 * 192, 192, P, P, 64 * 128, BF, P, P, None) == code
        assert lib.dsa_chunk_attn_paged(ctypes.byref(d), P + 2, ref(paged()), P, P, 0.07, P, P, P, 1 << 30, None) == code
        # the append's limit is on its tokens: query rows play no part
        assert lib.dsa_append_tokens_rope(ctypes.byref(d), 4, None, P, P, 576, P, 128, BF, ref(rope()), P, P, P, None,
                                          None, 0, None) == INVALID


def test_a_table_wider_than_the_pool_is_bounded_by_the_pool(lib):
    # 1,024 sequences of up to a million positions over a pool of 100 blocks
    d = make_dims(B=1024, T_max=1 << 20, ld_scores=1 << 20)
    cache = paged(max_blocks=1 << 14)
    assert api.workspace_size(d, _lib.DSA_OP_CHUNK_ATTN) == api.workspace_size(make_dims(), _lib.DSA_OP_CHUNK_ATTN)
    c = d.c()
    assert lib.dsa_chunk_attn_paged(ctypes.byref(c), P, ref(cache), P, P, 0.07, P, P, None, 0, None) == WORKSPACE
    args = (P, P, P, 576, P, 128, BF, ref(rope()), P, P, P)
    assert lib.dsa_append_tokens_rope(ctypes.byref(c), 4, *args, ref(cache), P, 64, None) == WORKSPACE
    assert lib.dsa_append_tokens_rope(ctypes.byref(c), 4, *args, None, P, 64, None) == UNSUPPORTED  # contiguous caches of 2^30 rows
    assert lib.dsa_chunk_attn_paged(ctypes.byref(c), P, ref(paged(max_blocks=1 << 14, num_blocks=1 << 24)), P, P, 0.07, P,
                                    P, P, 1 << 30, None) == UNSUPPORTED


def test_chunk_workspace_ignores_the_indexer_and_the_selection(lib):
    base = api.workspace_size(make_dims(), _lib.DSA_OP_CHUNK_ATTN)
    assert base >= 256
    for kw in (dict(k=1), dict(k=0), dict(ld_scores=0), dict(d_I=7), dict(H_I=0), dict(idx_dtype=F32)):
        assert api.workspace_size(make_dims(**kw), _lib.DSA_OP_CHUNK_ATTN) == base


def test_python_entries_check_their_tensors(lib):
    d = make_dims()
    cpu = torch.zeros(16, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_queries(d, cpu, api.Rope(torch.zeros(32)))
    with pytest.raises(ValueError, match="dtype"):
        api.rope_queries(d, cpu.long(), api.Rope(torch.zeros(32)))
    with pytest.raises(ValueError, match="elements"):
        api.rope_queries(d, cpu[:3], api.Rope(torch.zeros(32)))
    with pytest.raises(ValueError, match="q_pe|CUDA"):
        api.chunk_attn_paged(d, torch.zeros(16, 128, 576, dtype=torch.bfloat16), None, cpu, cpu, 0.1, None, None, None)
