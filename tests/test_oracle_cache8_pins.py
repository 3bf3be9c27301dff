"""Pins for the oracle of head norms and the 8-bit cache: worked numbers of the
format, every code against PyTorch's float8_e4m3fn, worked scales, a worked
acceptance."""
import numpy as np
import pytest

import oracle


def test_e4m3_worked():
    assert oracle.e4m3_values([0x00, 0x01, 0x07, 0x08, 0x38, 0x39, 0x7E, 0xB8]).tolist() == [
        0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 1.125, 448.0, -1.0]
    assert np.isnan(oracle.e4m3_values([0x7F, 0xFF])).all()
    # ties to even: 1.0625 lies between 1 and 1.125, 1.1875 between 1.125 and 1.25
    x = [1.0625, 1.1875, 1.0626, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, -500.0, 447.0, 0.0, -0.0, np.nan]
    assert oracle.e4m3_codes(x).tolist() == [0x38, 0x3A, 0x39, 0xB8, 0x00, 0x02, 0x7E, 0xFE, 0x7E, 0x00, 0x80, 0x7F]


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.e4m3_values(codes)
    assert np.array_equal(got, want, equal_nan=True)
    ok = ~np.isnan(got)
    assert np.array_equal(oracle.e4m3_codes(got)[ok], codes[ok])
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * np.float32(40)
    x = np.concatenate([x, x * np.float32(1e-3), (got[:126] + got[1:127]).astype(np.float32) / 2])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_codes(x), want)


def test_scales_worked():
    tops = [0.0, 448 * 2.0 ** -15, 0.0137, 1.75, 1.7501, 448.0, 449.0, 61440.0]
    assert oracle.cache8_scale(tops).tolist() == [2.0 ** -15, 2.0 ** -15, 2.0 ** -14, 2.0 ** -8, 2.0 ** -7, 1.0, 2.0, 256.0]
    assert oracle.cache8_limited([np.inf, -7e4, 5.0]).tolist() == [61440.0, -61440.0, 5.0]
    # every value of the cache is an fp16 number
    for e in range(-15, 9):
        v = oracle.e4m3_values(np.arange(127)) * 2.0 ** e
        v = v[v <= 61440]
        assert np.array_equal(v.astype(np.float16).astype(np.float64), v)


def test_rescale_is_exact_above_the_subnormals():
    codes = np.arange(127, dtype=np.uint8)
    v = oracle.e4m3_values(codes)
    again = oracle.e4m3_values(oracle.cache8_rescale(codes, 1.0, 4.0)) * 4.0
    assert np.array_equal(again[v >= 2.0 ** -4], v[v >= 2.0 ** -4])
    assert np.abs(again - v).max() <= 4 * 2.0 ** -10  # half a step of the new scale's subnormals


def test_head_norm_worked():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    assert np.allclose(oracle.head_norm(x, eps=0.0), [[1.2, 1.6, 0, 0]])
    assert np.allclose(oracle.head_norm(x, [1, 2, 3, 4], eps=2.75), x / 3 * [1, 2, 3, 4])
    assert not oracle.head_norm(np.zeros((1, 4)), eps=0.0).any()


def test_accept_worked():
    # pages of 16 positions, one element a row: 15 cached, rows 0 .. 3 at positions 15 .. 18, path 0, 3
    codes = np.zeros((1, 2, 1, 16, 1), np.uint8)
    codes[0, 0, 0, :, 0] = 0x38            # 1.0, scale 1
    codes[0, 1, 0, :4, 0] = [0x38, 0x40, 0x48, 0x50]  # 1, 2, 4, 8 times 4
    scales = np.array([1.0, 4.0]).reshape(1, 2, 1, 1)
    oracle.cache8_accept(codes, scales, [0, 1], 15, 4, [0, 3])
    assert scales.ravel().tolist() == [1.0, 4.0] and codes[0, 1, 0, 0, 0] == 0x48 and (codes[0, 0] == 0x38).all()
    # 14 cached: row 1's place is the last of the first block, whose scale grows and whose rows keep their values
    codes[0, 1, 0, :4, 0] = [0x38, 0x40, 0x48, 0x50]
    oracle.cache8_accept(codes, scales, [0, 1], 14, 4, [0, 2])
    assert scales.ravel().tolist() == [4.0, 4.0]
    assert codes[0, 0, 0, :15, 0].tolist() == [0x28] * 15 and codes[0, 0, 0, 15, 0] == 0x38  # 0.25, and 1.0
