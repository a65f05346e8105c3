"""Refusals of the 4-bit cache, its attention and the norm, at the C entries
and in the binding, before anything is enqueued (no GPU)."""
import ctypes

import pytest
import torch

F = ctypes.c_float
P = ctypes.c_void_p(1 << 20)      # compared, never dereferenced: the checks fail first
FAR = [ctypes.c_void_p((1 << 40) + (i << 34)) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    from long_context_03_b200 import build
    build.build()
    import long_context_03_b200 as m
    return m.lib()


@pytest.fixture(scope="module")
def dsa(lib):
    import long_context_03_b200 as m
    return m


def test_norm_arguments(lib):
    # (x, x_stride, residual, weight, dtype, n, d, eps, group, codes, scale, summed, normed, stream)
    a = [FAR[0], 512, FAR[1], FAR[2], 1, 4, 512, F(1e-6), 0, FAR[3], FAR[4], FAR[5], FAR[6], None]

    def call(**kw):
        v = list(a)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return lib.dsa_rms_norm_quantize_e4m3_rows(*v)
    assert call(_4=3) == -2 and call(_4=-1) == -2
    assert call(_5=-1) == -1 and call(_6=0) == -1 and call(_6=16385, _1=20000) == -2
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(_7=F(eps)) == -1
    assert call(_8=64) == -2 and call(_8=-128) == -2
    assert call(_1=511) == -1
    for i in (0, 9, 10):
        assert call(**{f"_{i}": None}) == -1
    for i in (0, 2, 3, 11, 12):
        assert call(**{f"_{i}": ctypes.c_void_p(FAR[7].value + 1)}) == -1  # half an element off
    assert call(_10=ctypes.c_void_p(FAR[7].value + 2)) == -1
    assert call(_5=0, _0=None, _9=None, _10=None) == 0  # nothing to do
    row = 512 * 2
    for out in (9, 10, 11, 12):  # into the middle of an input
        for src in (0, 1, 2):
            assert call(**{f"_{out}": ctypes.c_void_p(FAR[src].value + (row if src < 2 else 16))}) == -1, (out, src)
    assert b"overlap" in lib.dsa_last_error()
    assert call(_9=FAR[2]) == -1 and call(_12=FAR[5]) == -1 and call(_12=FAR[1]) == -1
    # the sum over x only where the rows of x are contiguous
    assert call(_11=FAR[0], _1=513) == -1


def test_append_and_gather_arguments(lib):
    # (x, x_stride, dtype, slots, n, pool, pool_rows, stream)
    a = [FAR[0], 576, 1, FAR[1], 4, FAR[2], 100, None]

    def app(**kw):
        v = list(a)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return lib.dsa_latent_q4_append(*v)
    assert app(_2=7) == -2 and app(_1=575) == -1 and app(_4=-1) == -1 and app(_6=0) == -1
    assert app(_0=None) == -1 and app(_3=None) == -1 and app(_5=None) == -1
    assert app(_5=ctypes.c_void_p(FAR[2].value + 16)) == -1  # pool not 32-byte aligned
    assert app(_0=ctypes.c_void_p(FAR[0].value + 1)) == -1 and app(_3=ctypes.c_void_p(FAR[1].value + 2)) == -1
    assert app(_0=ctypes.c_void_p(FAR[2].value + 4160)) == -1 and app(_3=ctypes.c_void_p(FAR[2].value + 416)) == -1
    assert b"overlap" in lib.dsa_last_error()
    assert app(_4=0, _0=None, _3=None) == 0
    # (pool, pool_rows, rows, n, out, stream)
    g = [FAR[0], 100, FAR[1], 4, FAR[2], None]

    def gat(**kw):
        v = list(g)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return lib.dsa_latent_q4_gather(*v)
    assert gat(_1=0) == -1 and gat(_3=-1) == -1 and gat(_0=None) == -1 and gat(_2=None) == -1 and gat(_4=None) == -1
    assert gat(_0=ctypes.c_void_p(FAR[0].value + 16)) == -1 and gat(_4=ctypes.c_void_p(FAR[2].value + 8)) == -1
    assert gat(_2=ctypes.c_void_p(FAR[1].value + 1)) == -1
    assert gat(_4=ctypes.c_void_p(FAR[0].value + 416 * 32)) == -1 and gat(_4=FAR[1]) == -1
    assert gat(_3=0, _2=None, _4=None) == 0


def test_attention_arguments(lib):
    f = F(0.1)
    # (q, kv, idx, T, L, Hq, topk, scale, out, lse, stream)
    assert lib.dsa_sparse_mla_attn_q4(None, None, None, 1, 1, 1, 1, f, None, None, None) == -1
    assert lib.dsa_sparse_mla_attn_q4(P, P, P, 1, 1, 129, 8, f, P, None, None) == -2
    assert lib.dsa_sparse_mla_attn_q4(P, P, P, 1, 1, 16, 2049, f, P, None, None) == -2
    assert lib.dsa_sparse_mla_attn_q4(P, P, P, 1, 1, 16, 8, F(float("nan")), P, None, None) == -1
    assert lib.dsa_sparse_mla_attn_q4(P, P, P, 1, 0, 16, 8, f, P, None, None) == -1
    assert lib.dsa_sparse_mla_attn_q4(P, ctypes.c_void_p((1 << 20) + 16), P, 1, 1, 16, 8, f, P, None, None) == -1
    assert b"32-byte" in lib.dsa_last_error()
    assert lib.dsa_sparse_mla_attn_q4(None, P, None, 0, 4, 16, 8, f, None, None, None) == 0
    # (q, kv, idx, B, L_max, Hq, topk, scale, out, lse, workspace, ws_bytes, stream)
    assert lib.dsa_sparse_mla_attn_q4_decode(P, P, P, 4, 1000, 16, 256, f, P, None, P, 1024, None) == -5
    assert lib.dsa_sparse_mla_attn_q4_decode(P, P, P, 0, 1000, 16, 256, f, P, None, P, 1024, None) == 0
    # (q, pool, table, idx, T, rows, pool_rows, bt_stride, max_blocks, page, Hq, topk, scale, out, lse, ws, bytes, stream)
    call = lambda *a: lib.dsa_sparse_mla_attn_q4_paged(P, P, *a, 16, 8, f, P, None, None, 0, None)
    assert call(None, P, 2, 1000, 4096, 16, 16, 64) == -1
    assert call(P, P, 2, 1000, 4096, 16, 16, 48) == -2
    assert call(P, P, 2, 1000, 4096, 15, 15, 64) == -1
    assert call(P, P, 2, 1000, 0, 16, 16, 64) == -1
    # (q, kv, idx, cu_q, cu_k, nseq, T, total_k, Hq, topk, scale, out, lse, stream)
    assert lib.dsa_sparse_mla_attn_q4_varlen(P, P, P, P, P, 0, 4, 10, 16, 8, f, P, None, None) == -1
    assert lib.dsa_sparse_mla_attn_q4_varlen(P, P, P, None, P, 1, 4, 10, 16, 8, f, P, None, None) == -1


def test_the_binding_refuses_host_tensors(dsa):
    x = torch.zeros((2, 576), dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros((4, 416), dtype=torch.uint8)
    q = torch.zeros((2, 16, 576), dtype=torch.bfloat16)
    idx = torch.zeros((2, 8), dtype=torch.int32)
    for call in (lambda: dsa.rms_norm_quantize_e4m3_rows(x), lambda: dsa.latent_q4_append(x, slots, pool),
                 lambda: dsa.latent_q4_gather(pool, slots), lambda: dsa.sparse_mla_attn_q4(q, pool, idx, 0.1),
                 lambda: dsa.sparse_mla_attn_q4_decode(q, pool.view(2, 2, 416), idx, 0.1),
                 lambda: dsa.sparse_mla_attn_q4_paged(q, pool, idx, idx, 4, 0.1),
                 lambda: dsa.sparse_mla_attn_q4_varlen(q, pool, idx, [0, 2], [0, 4], 0.1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
