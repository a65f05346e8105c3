"""Residual addition, root-mean-square norm and E4M3 output against the float64
definition.

Tolerances, in units u = 2^-24 of fp32: the sum of squares of d values goes
through at most 8 + 8 + 5 + 8 additions and multiply-adds of positive terms
(8 in a vector, up to 8 vectors, 5 shuffles, 8 warps), so it is within 29 u;
division and the addition of eps add 2 u, the square root halves that and
rounds once: 17 u. y takes one rounding of h, two products and this: 20 u,
taken as 24 u. The scale adds a division. What goes out in x's type is rounded
once more, by at most half a step. A code is the E4M3 value of some number
within the bounds of y / scale."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dsa():
    import long_context_03_b200 as m
    m.lib()
    return m


def _inputs(n, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, d), generator=g) * torch.logspace(-2, 2, n)[:, None]).to(dtype)
    r = (3 * torch.randn((n, d), generator=g)).to(dtype)
    w = (1 + 0.3 * torch.randn((d,), generator=g)).to(dtype)
    return x, r, w


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double().numpy()


def _check(dsa, x, w, r, group, out, eps):
    codes, scale, summed, normed = out
    n, d = x.shape
    f = lambda t: None if t is None else t.double().cpu().numpy()
    h, y = oracle.rms_norm(f(x), f(w), f(r), eps)
    tiny = float(torch.finfo(x.dtype).smallest_normal) * _half_step(x.dtype) * 2
    if r is not None:
        err = np.abs(f(summed) - h)
        assert (err <= np.abs(h) * (_half_step(x.dtype) + 2 * U) + tiny).all()
    if normed is not None:
        assert (np.abs(f(normed) - y) <= np.abs(y) * (_half_step(x.dtype) + 25 * U) + tiny).all()
    size = group or d
    for i, a in enumerate(range(0, d, size)):
        part = y[:, a:a + size]
        top = np.abs(part).max(axis=1)
        want = np.where(top > 0, top / 448, 1.0)
        got = f(scale)[:, i] if group else f(scale)
        assert (np.abs(got - want) <= want * 26 * U).all()
        q = part / want[:, None]
        c = _values(codes)[:, a:a + size]
        lo, hi = oracle.e4m3_nearest(q * (1 - 52 * U)), oracle.e4m3_nearest(q * (1 + 52 * U))
        assert (np.minimum(lo, hi) <= c).all() and (c <= np.maximum(lo, hi)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 8), (9, 100), (17, 256), (8, 257), (5, 512), (33, 576), (2, 1023),
                                 (7, 1024), (4, 1032), (19, 1536), (3, 2049), (2, 4097), (5, 7168), (2, 8200),
                                 (1, 16383), (2, 16384)])
def test_norm_matches_the_definition(dsa, n, d, group, dtype):
    x, r, w = _inputs(n, d, dtype, n + d)
    out = dsa.rms_norm_quantize_e4m3_rows(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5, group=group,
                                          want_normed=True)
    dsa.check_device_error()
    _check(dsa, x, w, r, group, out, 1e-5)
    # without residual, weight and the optional outputs
    bare = dsa.rms_norm_quantize_e4m3_rows(x.cuda(), eps=1e-5, group=group)
    assert bare[2] is None and bare[3] is None
    _check(dsa, x, None, None, group, bare, 1e-5)


def test_codes_equal_the_plain_quantiser_on_the_norm_written_out(dsa):
    x, r, w = (t.cuda() for t in _inputs(70, 1536, torch.float32, 4))
    codes, scale, _, normed = dsa.rms_norm_quantize_e4m3_rows(x, w, residual=r, want_normed=True)
    ref_codes, ref_scale = dsa.quantize_e4m3_rows(normed)
    dsa.check_device_error()
    assert torch.equal(codes, ref_codes) and torch.equal(scale, ref_scale)


@pytest.mark.parametrize("d", [576, 1536, 1001])
def test_in_place_sum_and_strided_rows(dsa, d):
    x, r, w = (t.cuda() for t in _inputs(21, d, torch.bfloat16, d))
    want = dsa.rms_norm_quantize_e4m3_rows(x, w, residual=r, want_normed=True)
    res = r.clone()
    got = dsa.rms_norm_quantize_e4m3_rows(x, w, residual=res, summed=res, want_normed=True)
    assert got[2] is res
    xx = x.clone()
    got2 = dsa.rms_norm_quantize_e4m3_rows(xx, w, residual=r, summed=xx, want_normed=True)
    assert got2[2] is xx
    wide = torch.full((21, d + 1536), 7.0, dtype=x.dtype, device="cuda")
    wide[:, 1530:1530 + d] = x
    got3 = dsa.rms_norm_quantize_e4m3_rows(wide[:, 1530:1530 + d], w, residual=r, want_normed=True)
    dsa.check_device_error()
    for g in (got, got2):
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    # another map of elements to threads sums in another order: within the definition's bounds
    _check(dsa, x.cpu(), w.cpu(), r.cpu(), 0, got3, 1e-6)
    assert float(wide[:, :1530].min()) == 7.0 and float(wide[:, 1530 + d:].max()) == 7.0


@pytest.mark.parametrize("group", [0, 128])
def test_rows_of_zeros_and_of_nan(dsa, group):
    x = torch.zeros((4, 512), dtype=torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, :] = 2.0
    x[3, 7] = float("inf")
    codes, scale, _, normed = dsa.rms_norm_quantize_e4m3_rows(x.cuda(), want_normed=True, group=group)
    dsa.check_device_error()
    v = codes.cpu().view(torch.float8_e4m3fn).float()
    s = scale.cpu().reshape(4, -1)
    assert (v[0] == 0).all() and (s[0] == 1).all()
    assert v[1].isnan().all()
    assert (v[2] == 448).all() and torch.isfinite(s[2]).all()
    assert v[3, 7].isnan() and torch.isfinite(s).all()


def test_unaligned_and_unusual_pointers(dsa):
    # every array at an offset of one element: the element-wise path
    n, d = 6, 640
    x, r, w = _inputs(n, d, torch.bfloat16, 3)
    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)
    for group in (0, 128):
        out = dsa.rms_norm_quantize_e4m3_rows(off(x), off(w), residual=off(r), group=group, eps=1e-6,
                                              summed=off(r), normed=off(r),
                                              codes=off(torch.zeros((n, d), dtype=torch.uint8)))
        dsa.check_device_error()
        _check(dsa, x, w, r, group, out, 1e-6)


def test_graph_replay_reads_new_inputs(dsa):
    a, r, w = (t.cuda() for t in _inputs(5, 1536, torch.bfloat16, 11))
    b = _inputs(5, 1536, torch.bfloat16, 12)[0].cuda()
    buf = a.clone()
    want = [dsa.rms_norm_quantize_e4m3_rows(t, w, residual=r, group=128) for t in (a, b)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dsa.rms_norm_quantize_e4m3_rows(buf, w, residual=r, group=128)
    for src, ref in ((a, want[0]), (b, want[1])):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in range(3))


def test_an_empty_batch(dsa):
    out = dsa.rms_norm_quantize_e4m3_rows(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), group=128)
    assert out[0].shape == (0, 64) and out[1].shape == (0, 1)
