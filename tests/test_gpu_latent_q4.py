"""The 4-bit latent cache: rows quantised as they are written equal the
definition byte for byte, rows read back equal it value for value."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dsa():
    import long_context_03_b200 as m
    m.lib()
    return m


def _rows(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, 576), generator=g) * torch.logspace(-4, 3, n)[torch.randperm(n, generator=g)][:, None]
    return x.to(dtype)


def _ref(x):
    return oracle.q4_quantize(x.float().numpy())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 333])
def test_append_matches_the_definition(dsa, n, dtype):
    x = _rows(n, dtype, n)
    pool = torch.full((2 * n + 5, 416), 0xA5, dtype=torch.uint8, device="cuda")
    slots = torch.randperm(2 * n + 5, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    assert dsa.latent_q4_append(x.cuda(), slots.cuda(), pool) is pool
    dsa.check_device_error()
    want = np.full((2 * n + 5, 416), 0xA5, dtype=np.uint8)
    want[slots.numpy()] = _ref(x)
    assert np.array_equal(pool.cpu().numpy(), want)  # the rows that no slot names are as they were


@pytest.mark.parametrize("dtype", TYPES)
def test_special_groups(dsa, dtype):
    # borders of the codes (k + 1/2) s and of the scales 7 s, with their neighbours in the type; zeros, NaN,
    # infinities, values above the largest scale and below the smallest
    x = torch.zeros((256, 576), dtype=torch.float64)
    for b in range(256):
        s = float(oracle._Q4_STEPS[b])
        x[b, 0:16] = s * torch.tensor([7, -7, 6.5, 5.5, 4.5, 3.5, 2.5, 1.5, 0.5, -0.5, -1.5, -2.5, -3.5, -4.5, -5.5, -6.5])
        x[b, 16] = 7 * s
        x[b, 32] = -7 * s
        x[b, 48:64] = s * torch.arange(-8, 8) / 1.9
        x[b, 64] = 7 * s
    x = x.to(dtype)
    up = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}[dtype]
    for at in (3, 9, 16, 32):  # away from zero by a step of the type (two, for some mantissas)
        x[:256, at] = (x[:256, at].double() * (1 + up)).to(dtype)
    odd = torch.zeros((8, 576), dtype=dtype)
    odd[1, 0], odd[1, 1] = float("nan"), 3.0
    odd[2, 0], odd[2, 1] = float("inf"), -5.0
    odd[3, 5] = float("-inf")
    odd[4, :] = float("nan")
    odd[5, :512] = torch.finfo(dtype).max
    odd[6, :512] = torch.finfo(dtype).tiny
    odd[7, 512:] = float("inf")
    x = torch.cat([x, odd])
    n = x.shape[0]
    pool = torch.zeros((n, 416), dtype=torch.uint8, device="cuda")
    dsa.latent_q4_append(x.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), pool)
    dsa.check_device_error()
    got, want = pool.cpu().numpy(), _ref(x)
    assert np.array_equal(got[:, :288], want[:, :288])
    ga, wa = (torch.from_numpy(v[:, 288:].copy()).view(torch.bfloat16).float() for v in (got, want))
    assert torch.equal(ga.isnan(), wa.isnan()) and torch.equal(ga.nan_to_num(0), wa.nan_to_num(0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("stride,offset", [(2112, 1536), (577, 0), (600, 3), (584, 8)])
def test_append_reads_strided_rows(dsa, dtype, stride, offset):
    # a slice of a fused projection's output, aligned and not
    n = 45
    wide = torch.full((n, stride + 640), 9.0, dtype=dtype, device="cuda").flatten()[: n * stride + 640]
    view = wide[offset:].as_strided((n, 576), (stride, 1)) if stride >= 576 else None
    x = _rows(n, dtype, stride)
    view.copy_(x)
    pool = torch.zeros((n, 416), dtype=torch.uint8, device="cuda")
    dsa.latent_q4_append(view, torch.arange(n, dtype=torch.int32, device="cuda"), pool)
    dsa.check_device_error()
    assert np.array_equal(pool.cpu().numpy(), _ref(x))


def test_negative_slots_are_skipped_and_far_ones_reported(dsa):
    x = _rows(5, torch.bfloat16, 3)
    pool = torch.full((9, 416), 1, dtype=torch.uint8, device="cuda")
    dsa.latent_q4_append(x.cuda(), torch.tensor([-1, 8, -7, 0, -1], dtype=torch.int32, device="cuda"), pool)
    dsa.check_device_error()
    want = np.full((9, 416), 1, dtype=np.uint8)
    want[[8, 0]] = _ref(x)[[1, 3]]
    assert np.array_equal(pool.cpu().numpy(), want)
    dsa.latent_q4_append(x.cuda(), torch.tensor([9, -1, 2, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), pool)
    assert dsa.device_error()[0] == -6
    want[2] = _ref(x)[2]
    assert np.array_equal(pool.cpu().numpy(), want)
    dsa.check_device_error()  # the report is cleared


@pytest.mark.parametrize("n", [1, 9, 4001])
def test_gather_of_any_bytes_is_exact(dsa, n):
    g = torch.Generator().manual_seed(n)
    pool = torch.randint(0, 256, (777, 416), generator=g, dtype=torch.uint8)
    rows = torch.randint(-2, 777, (n,), generator=g).to(torch.int32)
    out = dsa.latent_q4_gather(pool.cuda(), rows.cuda())
    dsa.check_device_error()
    want = oracle.q4_values(pool.numpy())[rows.clamp(min=0).numpy()]
    want[rows.numpy() < 0] = 0
    got = out.cpu().double().numpy()
    assert np.array_equal(got, want, equal_nan=True)


def test_gather_reports_rows_past_the_pool(dsa):
    pool = torch.full((4, 416), 0x99, dtype=torch.uint8, device="cuda")
    out = dsa.latent_q4_gather(pool, torch.tensor([3, 4, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda"))
    assert dsa.device_error()[0] == -6
    assert (out[1:3] == 0).all() and torch.equal(out[0], out[3]) and (out[0, :512] != 0).all()


def test_rows_past_four_gigabytes(dsa):
    rows = 10_500_000  # 4.4 GB: byte offsets past 32 bits
    pool = torch.zeros((rows, 416), dtype=torch.uint8, device="cuda")
    x = _rows(6, torch.bfloat16, 8)
    slots = torch.tensor([rows - 1, 0, 5_200_000, 10_400_000, 5_162_221, rows - 2], dtype=torch.int32, device="cuda")
    dsa.latent_q4_append(x.cuda(), slots, pool)
    out = dsa.latent_q4_gather(pool, slots)
    dsa.check_device_error()
    assert np.array_equal(pool[slots.long()].cpu().numpy(), _ref(x))
    assert np.array_equal(out.cpu().double().numpy(), oracle.q4_values(_ref(x)))
    assert int(pool.view(-1, 416)[1:1000].max()) == 0


def test_empty_calls(dsa):
    pool = torch.full((4, 416), 7, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dsa.latent_q4_append(torch.empty((0, 576), dtype=torch.bfloat16, device="cuda"), none, pool)
    assert dsa.latent_q4_gather(pool, none).shape == (0, 576)
    dsa.check_device_error()
    assert (pool == 7).all()


def test_on_a_side_stream_and_in_a_graph(dsa):
    n = 64
    x, y = _rows(n, torch.bfloat16, 1).cuda(), _rows(n, torch.bfloat16, 2).cuda()
    slots = torch.randperm(200, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32).cuda()
    pool = torch.zeros((200, 416), dtype=torch.uint8, device="cuda")
    buf = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dsa.latent_q4_append(buf, slots, pool)
        dsa.latent_q4_gather(pool, slots)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            dsa.latent_q4_append(buf, slots, pool)
            out = dsa.latent_q4_gather(pool, slots)
    torch.cuda.current_stream().wait_stream(side)
    for src in (x, y):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().double().numpy(), oracle.q4_values(_ref(src.cpu())))
    dsa.check_device_error()
