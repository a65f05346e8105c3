"""Pins of the 4-bit row format and the norm's oracle (CPU)."""
import numpy as np
import torch

import oracle


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, 576), generator=g).to(torch.bfloat16)


def test_every_scale_byte_and_code_is_exact_in_bf16():
    b = np.zeros((256, 416), dtype=np.uint8)
    b[:, 256:288] = np.arange(256)[:, None]
    word = sum(c << (4 * c) for c in range(8))  # codes 0..7, and 8..15 in the other word
    b[:, :256] = np.tile(np.frombuffer(np.array([word, word ^ 0x88888888], dtype=np.uint32).tobytes(), np.uint8), 32)
    v = oracle.q4_values(b)[:, :512]
    t = torch.from_numpy(v)
    assert torch.equal(t.to(torch.bfloat16).double(), t)
    assert v[0].min() == -8 * 2.0 ** -18 and v[255].max() == 7 * 1.875 * 2.0 ** 13


def test_the_order_of_the_values_in_a_word():
    # one large value at place j of a word, the others zero: nibble j/2 or 4 + j/2 holds 7 + 8
    for j in range(8):
        x = np.zeros((1, 576))
        x[0, 8 + j] = 7.0
        w = oracle.q4_quantize(x)[0, 4:8].view(np.uint32)[0]
        nib = j // 2 + 4 * (j % 2)
        assert w == (0x88888888 & ~(15 << (4 * nib))) | (15 << (4 * nib))


def test_round_trip_is_within_half_a_step():
    x = _rows(200, 1).float().numpy().astype(np.float64)
    b = oracle.q4_quantize(x)
    v = oracle.q4_values(b)
    step = oracle._Q4_STEPS[b[:, 256:288]].repeat(16, axis=1)
    assert (np.abs(v[:, :512] - x[:, :512]) <= step / 2).all()
    assert np.array_equal(v[:, 512:], x[:, 512:])
    # the scale is the smallest that fits: one below would not hold the group's largest magnitude
    amax = np.abs(x[:, :512]).reshape(200, 32, 16).max(axis=2)
    assert (7 * oracle._Q4_STEPS[b[:, 256:288]] >= amax).all()
    assert (7 * oracle._Q4_STEPS[b[:, 256:288] - 1] < amax).all()


def test_special_values():
    x = np.zeros((4, 576))
    x[1, 0], x[1, 1] = np.nan, 3.0
    x[2, 0], x[2, 1] = np.inf, -1e9
    x[3, 0] = 1e-30
    v = oracle.q4_values(oracle.q4_quantize(x))
    assert (v[0] == 0).all() and (v[3] == 0).all()
    assert v[1, 0] == 0 and abs(v[1, 1] - 3.0) < 0.25
    assert v[2, 0] == 107520.0 and v[2, 1] == -107520.0


def test_e4m3_nearest_agrees_with_torch():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(100000, generator=g) * torch.logspace(-4, 3, 100000)
    x = torch.cat([x, torch.arange(-448, 449, 0.5)])
    ref = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_nearest(x.double().numpy()), ref)


def test_rms_norm_closed_forms():
    x = np.array([[3.0, -3.0, 3.0, -3.0], [0.0, 0.0, 0.0, 0.0]])
    h, y = oracle.rms_norm(x, eps=0.0 + 1e-300)
    assert np.array_equal(h, x) and np.allclose(y[0], [1, -1, 1, -1], rtol=1e-15) and (y[1] == 0).all()
    h, y = oracle.rms_norm(x, weight=[1, 2, 3, 4], residual=-x, eps=1e-6)
    assert (h == 0).all() and (y == 0).all()
