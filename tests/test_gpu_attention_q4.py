"""Attention over the 4-bit latent cache against a float64 softmax over the
rows' exact values.

Tolerances. The rows are exact, so what separates the result from float64 is:
the bf16 rounding of each probability (half a step, 2^-8, of p_s |v_s|), the
bf16 rounding of the output (2^-8 of it), and the scores' fp32 sums. A score's
576 products accumulate in fp32: at most 576 roundings of 2^-24 of the sum of
their magnitudes, taken twice for the tensor core's own order; an error e of a
score changes p by the factor exp(e), and the sum of the p once more: 2 e. The
exponential (2^-21) and the row sum (35 roundings) fit into 2^-18. With
A = sum_s p_s |v_s|:
    |out - ref| <= 2^-8 |ref| + A (2^-8 + 2 e + 2^-18) (1 + 2^-8)
    |lse - ref| <= e + 2^-18 (1 + |ref|)"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

SCALE = 1.0 / 24.0


@pytest.fixture(scope="module")
def dsa():
    import long_context_03_b200 as m
    m.lib()
    return m


def _cache(rows, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, 576), generator=g) * spread * torch.exp(0.3 * torch.randn((576,), generator=g))
    return torch.from_numpy(oracle.q4_quantize(x.to(torch.bfloat16).float().numpy()))


def _queries(T, Hq, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, Hq, 576), generator=g)).to(torch.bfloat16)


def _selection(lens, topk, seed, drop=0.0):
    """Distinct rows below each length, shuffled with the -1 entries among them."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((len(lens), topk), -1, dtype=torch.int32)
    for t, n in enumerate(lens):
        k = min(n, topk)
        pick = torch.randperm(n, generator=g)[:k].to(torch.int32)
        pick[torch.rand(k, generator=g) < drop] = -1
        idx[t, :k] = pick
        if drop:
            idx[t] = idx[t, torch.randperm(topk, generator=g)]
    return idx


def _check(out, lse, q, values, idx, scale=SCALE):
    """values: per token a [rows, 576] float64 CUDA tensor (or one for all)."""
    o, l = out.double(), lse.double()
    for t in range(q.shape[0]):
        v = values[t] if isinstance(values, list) else values
        sel = idx[t][idx[t] >= 0].long().cuda()
        if sel.numel() == 0:
            assert (o[t] == 0).all() and (l[t] == float("-inf")).all(), t
            continue
        c = v[sel]
        qq = q[t].double().cuda()
        z = scale * (qq @ c.T)
        e = 2 * 576 * 2.0 ** -24 * scale * float((qq.abs() @ c.abs().T).max())
        p = torch.softmax(z, dim=1)
        ref, mag = p @ c[:, :512], p @ c[:, :512].abs()
        tol = 2.0 ** -8 * ref.abs() + mag * (2.0 ** -8 + 2 * e + 2.0 ** -18) * (1 + 2.0 ** -8)
        assert ((o[t] - ref).abs() <= tol).all(), (t, float(((o[t] - ref).abs() / tol).max()))
        rl = torch.logsumexp(z, dim=1)
        assert ((l[t] - rl).abs() <= e + 2.0 ** -18 * (1 + rl.abs())).all(), t


def _exact(pool):
    return torch.from_numpy(oracle.q4_values(pool.numpy())).cuda()


@pytest.mark.parametrize("T,L,Hq,topk", [(1, 1, 1, 1), (3, 200, 16, 64), (2, 300, 128, 127), (5, 700, 17, 128),
                                         (4, 700, 128, 129), (90, 3000, 100, 300), (3, 2100, 128, 2048),
                                         (2, 5000, 33, 2047)])
def test_prefill_matches_the_definition(dsa, T, L, Hq, topk):
    pool = _cache(L, L)
    q = _queries(T, Hq, T)
    idx = _selection([max(1, L - t) for t in range(T)], topk, 3, drop=0.1 if T > 2 else 0.0)
    if T > 3:
        idx[1] = -1  # nothing selected
    out, lse = dsa.sparse_mla_attn_q4(q.cuda(), pool.cuda(), idx.cuda(), SCALE, want_lse=True)
    dsa.check_device_error()
    _check(out, lse, q, _exact(pool), idx)


def test_steep_scores(dsa):
    # large queries: one row takes nearly all, and the running maximum moves from chunk to chunk
    pool = _cache(1500, 5)
    q = _queries(6, 128, 6, spread=20.0)
    v = _exact(pool)
    idx = _selection([1500] * 6, 1024, 7)
    z = torch.einsum("hd,sd->hs", q[0].double().cuda(), v[idx[0].long()])[0]
    idx[0] = idx[0][torch.argsort(z).cpu()]  # ascending for head 0: its maximum moves all the time
    out, lse = dsa.sparse_mla_attn_q4(q.cuda(), pool.cuda(), idx.cuda(), SCALE, want_lse=True)
    dsa.check_device_error()
    _check(out, lse, q, v, idx)


@pytest.mark.parametrize("B", [1, 2, 5, 36, 38, 80])
@pytest.mark.parametrize("split", [True, False])
def test_decode_matches_the_definition(dsa, B, split):
    L, Hq, topk = 1100, 128 if B < 40 else 24, 1000
    pool = _cache(B * L, B).view(B, L, 416)
    q = _queries(B, Hq, 2)
    lens = [1100, 1, 999, 128, 129][:B] + [1000 + i for i in range(max(0, B - 5))]
    idx = _selection(lens, topk, 9)
    out, lse = dsa.sparse_mla_attn_q4_decode(q.cuda(), pool.cuda(), idx.cuda(), SCALE, want_lse=True, split=split)
    dsa.check_device_error()
    _check(out, lse, q, [_exact(pool[b]) for b in range(B)], idx)


def test_empty_sequences_in_a_split_batch(dsa):
    B, L, topk = 4, 400, 384
    pool = _cache(B * L, 1).view(B, L, 416)
    q = _queries(B, 40, 3)
    idx = _selection([400, 0, 130, 0], topk, 1)
    idx[2, :128] = -1  # a whole chunk absent
    out, lse = dsa.sparse_mla_attn_q4_decode(q.cuda(), pool.cuda(), idx.cuda(), SCALE, want_lse=True)
    dsa.check_device_error()
    _check(out, lse, q, [_exact(pool[b]) for b in range(B)], idx)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("split", [True, False])
def test_paged_equals_contiguous(dsa, page, split):
    B, L, topk = 6, 1024, 512
    pool = _cache(B * L, 21).view(B, L, 416)
    q = _queries(B, 128, 22).cuda()
    idx = _selection([1024, 1, 700, 513, 17, 64], topk, 23).cuda()
    ref, ref_lse = dsa.sparse_mla_attn_q4_decode(q, pool.cuda(), idx, SCALE, want_lse=True, split=split)
    nb = L // page
    perm = torch.randperm(B * nb + 3, generator=torch.Generator().manual_seed(24))
    paged = torch.full(((B * nb + 3) * page, 416), 0xFF, dtype=torch.uint8)
    paged.view(-1, page, 416)[perm[:B * nb]] = pool.reshape(B * nb, page, 416)
    table = perm[:B * nb].to(torch.int32).view(B, nb)
    out, lse = dsa.sparse_mla_attn_q4_paged(q, paged.cuda(), table.cuda(), idx, L, SCALE, page_size=page,
                                            want_lse=True, split=split)
    dsa.check_device_error()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_one_table_for_all_tokens_and_bad_pages(dsa):
    L, page, T, topk = 640, 64, 7, 256
    pool = _cache(L, 31)
    q = _queries(T, 64, 32)
    idx = _selection([L] * T, topk, 33)
    table = torch.arange(L // page, dtype=torch.int32)[None, :].clone()
    out, lse = dsa.sparse_mla_attn_q4_paged(q.cuda(), pool.cuda(), table.cuda(), idx.cuda(), L, SCALE, page_size=page,
                                            want_lse=True)
    dsa.check_device_error()
    ref, ref_lse = dsa.sparse_mla_attn_q4(q.cuda(), pool.cuda(), idx.cuda(), SCALE, want_lse=True)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    for bad in (-1, 10, 2 ** 31 - 1):
        table[0, 4] = bad
        out, lse = dsa.sparse_mla_attn_q4_paged(q.cuda(), pool.cuda(), table.cuda(), idx.cuda(), L, SCALE,
                                                page_size=page, want_lse=True)
        assert dsa.device_error()[0] == -6
        kept = idx.clone()
        kept[(idx >= 256) & (idx < 320)] = -1
        ref, ref_lse = dsa.sparse_mla_attn_q4(q.cuda(), pool.cuda(), kept.cuda(), SCALE, want_lse=True)
        dsa.check_device_error()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_indices_past_the_cache_are_skipped_and_reported(dsa):
    L, T, topk = 300, 3, 200
    pool = _cache(L, 41)
    q = _queries(T, 128, 42)
    idx = _selection([L] * T, topk, 43)
    bad = idx.clone()
    bad[1, 5], bad[1, 150], bad[2, 0] = L, 2 ** 31 - 1, -2 ** 31
    kept = idx.clone()
    kept[1, 5] = kept[1, 150] = kept[2, 0] = -1
    out, lse = dsa.sparse_mla_attn_q4(q.cuda(), pool.cuda(), bad.cuda(), SCALE, want_lse=True)
    assert dsa.device_error()[0] == -6
    _check(out, lse, q, _exact(pool), kept)


def test_packed_batch_equals_separate_calls(dsa):
    sizes, queries, topk, Hq = [900, 1, 333], [20, 1, 9], 130, 31
    pool = _cache(sum(sizes), 51)
    q = _queries(sum(queries), Hq, 52)
    cu_k, cu_q = np.cumsum([0] + sizes).tolist(), np.cumsum([0] + queries).tolist()
    idx = torch.cat([_selection([n] * m, topk, 53 + i) for i, (n, m) in enumerate(zip(sizes, queries))])
    out, lse = dsa.sparse_mla_attn_q4_varlen(q.cuda(), pool.cuda(), idx.cuda(), cu_q, cu_k, SCALE, want_lse=True)
    dsa.check_device_error()
    for i in range(3):
        a, b = slice(cu_q[i], cu_q[i + 1]), slice(cu_k[i], cu_k[i + 1])
        ref, ref_lse = dsa.sparse_mla_attn_q4(q[a].cuda(), pool[b].contiguous().cuda(), idx[a].cuda(), SCALE,
                                              want_lse=True)
        assert torch.equal(out[a], ref) and torch.equal(lse[a], ref_lse)
    _check(out, lse, q, [_exact(pool[cu_k[i]:cu_k[i + 1]]) for i in range(3) for _ in range(queries[i])], idx)
    bad = idx.clone()
    bad[3, 0] = 900  # the next sequence's first row: outside this one's
    dsa.sparse_mla_attn_q4_varlen(q.cuda(), pool.cuda(), bad.cuda(), cu_q, cu_k, SCALE)
    assert dsa.device_error()[0] == -6


def test_rows_past_four_gigabytes(dsa):
    rows, topk = 10_500_000, 64
    pool = torch.zeros((rows, 416), dtype=torch.uint8, device="cuda")
    small = _cache(topk, 61)
    at = torch.tensor([rows - 1 - 160_000 * i for i in range(topk)])
    pool[at.cuda()] = small.cuda()
    q = _queries(2, 16, 62)
    idx = torch.stack([at, at.flip(0)]).to(torch.int32)
    out, lse = dsa.sparse_mla_attn_q4(q.cuda(), pool, idx.cuda(), SCALE, want_lse=True)
    dsa.check_device_error()
    order = torch.arange(topk)
    _check(out, lse, q, _exact(small), torch.stack([order, order.flip(0)]).to(torch.int32))


def test_the_result_does_not_depend_on_other_tokens_or_runs(dsa):
    pool = _cache(2500, 71).cuda()
    q = _queries(150, 128, 72).cuda()
    idx = _selection([2500] * 150, 2048, 73).cuda()
    out, lse = dsa.sparse_mla_attn_q4(q, pool, idx, SCALE, want_lse=True)
    for _ in range(3):
        again, again_lse = dsa.sparse_mla_attn_q4(q, pool, idx, SCALE, want_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)
    part, part_lse = dsa.sparse_mla_attn_q4(q[100:103].contiguous(), pool, idx[100:103].contiguous(), SCALE,
                                            want_lse=True)
    dsa.check_device_error()
    assert torch.equal(part, out[100:103]) and torch.equal(part_lse, lse[100:103])


def test_a_serving_step_end_to_end(dsa):
    """Norm, append to a paged 4-bit cache, selection over the paged FP8 keys and attention, as a decode step
    runs them, eagerly and replayed from a graph with new inputs."""
    B, page, blocks, topk, Hq = 3, 64, 20, 256, 128
    L = page * blocks
    pool_rows = B * L
    g = torch.Generator().manual_seed(81)
    table = torch.randperm(B * blocks, generator=g).to(torch.int32).view(B, blocks)
    lens = torch.tensor([1280, 700, 130], dtype=torch.int32)
    hist = torch.randn((B, L, 576), generator=g).to(torch.bfloat16)
    pool = torch.zeros((pool_rows, 416), dtype=torch.uint8, device="cuda")
    phys = (table.long().repeat_interleave(page, dim=1) * page + torch.arange(L) % page).to(torch.int32)
    before = phys.clone()
    for b in range(B):
        before[b, lens[b] - 1:] = -1  # the new token's row is not yet there
    dsa.latent_q4_append(hist.view(-1, 576).cuda(), before.view(-1).cuda(), pool)
    keys = torch.randn((pool_rows, 128), generator=g)
    k_codes, k_scale = dsa.quantize_e4m3_rows(keys.cuda())
    qi = torch.randn((B, 64 * 128), generator=g)
    q_codes, q_scale = dsa.quantize_e4m3_rows(qi.cuda())
    w = (torch.rand((B, 64), generator=g) / 64).cuda()
    q = _queries(B, Hq, 82).cuda()
    slots = torch.stack([phys[b, lens[b] - 1] for b in range(B)]).cuda()
    new = hist[torch.arange(B), lens.long() - 1].contiguous().cuda()
    hidden, weight = torch.randn((B, 7168), generator=g).to(torch.bfloat16).cuda(), None
    res = torch.randn((B, 7168), generator=g).to(torch.bfloat16).cuda()
    ws = torch.empty(dsa.split_workspace_size(B, topk), dtype=torch.uint8, device="cuda")
    iws = torch.empty(dsa.index_topk_decode_workspace_size(B, L, topk), dtype=torch.uint8, device="cuda")
    tab, ln = table.cuda(), lens.cuda()

    def step():
        n = dsa.rms_norm_quantize_e4m3_rows(hidden, weight, residual=res)
        dsa.latent_q4_append(new, slots, pool)
        idx = dsa.index_topk_decode_paged(q_codes.view(B, 64, 128), q_scale, w, k_codes, k_scale, tab, ln, topk,
                                          page_size=page, workspace=iws)
        return n, idx, *dsa.sparse_mla_attn_q4_paged(q, pool, tab, idx, L, SCALE, page_size=page, want_lse=True,
                                                     split=True, workspace=ws)

    def check(n, idx, out, lse):
        dsa.check_device_error()
        vals = [torch.from_numpy(oracle.q4_values(oracle.q4_quantize(hist[b].float().numpy()))).cuda()
                for b in range(B)]
        for b in range(B):
            assert idx[b].max() < lens[b]
        _check(out, lse, q.cpu(), vals, idx.cpu())
        h, y = oracle.rms_norm(hidden.double().cpu().numpy(), None, res.double().cpu().numpy(), 1e-6)
        got = n[0].cpu().view(torch.float8_e4m3fn).double().numpy() * n[1].double().cpu().numpy()[:, None]
        assert np.abs(got - y).max() <= 2.0 ** -4 * np.abs(y).max()
    check(*step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    fresh = torch.randn((B, 576), generator=g).to(torch.bfloat16)
    new.copy_(fresh)
    hidden.copy_(torch.randn((B, 7168), generator=g).to(torch.bfloat16))
    q.copy_(_queries(B, Hq, 83))
    for b in range(B):
        hist[b, lens[b] - 1] = fresh[b]
    graph.replay()
    torch.cuda.synchronize()
    check(*outs)


def test_empty_batches(dsa):
    pool = _cache(8, 91).cuda()
    q = torch.empty((0, 16, 576), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    out, lse = dsa.sparse_mla_attn_q4(q, pool, idx, SCALE, want_lse=True)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    dsa.check_device_error()


def test_two_streams_at_once(dsa):
    pool = _cache(3000, 95).cuda()
    work = []
    for s in range(2):
        q = _queries(80, 128, 96 + s).cuda()
        idx = _selection([3000 - 7 * t for t in range(80)], 700, 97 + s).cuda()
        work.append((q, idx, dsa.sparse_mla_attn_q4(q, pool, idx, SCALE, want_lse=True), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for q, idx, _, stream in work:
            with torch.cuda.stream(stream):
                outs.append(dsa.sparse_mla_attn_q4(q, pool, idx, SCALE, want_lse=True))
    torch.cuda.synchronize()
    dsa.check_device_error()
    for i, (out, lse) in enumerate(outs):
        ref, ref_lse = work[i % 2][2]
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
