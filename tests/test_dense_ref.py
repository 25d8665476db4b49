"""The formats and rules that the dense operators' tests compare with, pinned
by closed forms (no GPU)."""
import numpy as np
import pytest
import torch

import dense_ref as R


def test_e4m3_table_is_the_format():
    assert R.E4M3[126] == 448.0 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[8] == 2.0 ** -6
    assert np.isnan(R.E4M3[127]) and np.isnan(R.E4M3[255])
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3, equal_nan=True)


def test_e4m3_rounding_is_to_nearest_ties_to_even():
    codes = np.arange(256)
    ok = ~np.isnan(R.E4M3)
    assert np.array_equal(R.e4m3_rne(R.E4M3[ok]), codes[ok])
    mids = (R.E4M3[:126] + R.E4M3[1:127]) / 2
    want = codes[:126] + (codes[:126] % 2)
    assert np.array_equal(R.e4m3_rne(mids), want)
    v = np.random.default_rng(1).standard_normal(4096).astype(np.float32) * 60
    assert np.array_equal(R.e4m3_rne(v), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("m,byte", [(448.0, 127), (448.5, 128), (449.0, 128), (1.75, 119), (1.7500001, 120),
                                    (0.0, 0), (2.0 ** -140, 0), (1.75 * 2.0 ** -119, 0),
                                    (1.7500001 * 2.0 ** -119, 1), (3.4e38, 247)])
def test_scale_is_the_smallest_that_clips_nothing(m, byte):
    v = np.zeros((1, 40), np.float32)
    v[0, 7], v[0, 39] = -m, m
    q, s = R.mxfp8(v)
    assert s.tolist() == [[byte, byte]]
    back = R.tokens8(q, s)
    assert np.all(np.abs(back - v) <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** (byte - 127.0)))


def test_what_is_not_finite_is_nan_and_sets_no_scale():
    v = np.ones((1, 32), np.float32)
    v[0, 3], v[0, 4], v[0, 5] = np.inf, -np.inf, np.nan
    q, s = R.mxfp8(v)
    assert s[0, 0] == 119 and np.isnan(R.E4M3[q[0, 3:6]]).all() and np.all(R.E4M3[q[0, 6:]] == 256.0)


def test_matrix_decode_and_dropped_group():
    p = np.arange(32, dtype=np.uint8).reshape(1, 32) * 7 % 251
    s = np.array([[129, 255]], np.uint8)
    w = R.dense(p, s)
    assert w[0, 0] == R.E2M1[p[0, 0] & 15] * 4 and w[0, 1] == R.E2M1[p[0, 0] >> 4] * 4
    assert np.all(w[0, 32:] == 0)
