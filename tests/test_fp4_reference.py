"""The 4-bit form's rule, as the tests state it: tables, roundings and what it
keeps of a row."""
import numpy as np

from tests import fp4_reference as R


def test_codes_and_their_middles():
    mids = (R.E2M1[:-1] + R.E2M1[1:]) / 2
    assert R.e2m1_of(R.E2M1.astype(np.float32)).tolist() == list(range(8))
    assert R.e2m1_of(mids.astype(np.float32)).tolist() == [0, 2, 2, 4, 4, 6, 6]       # to the even code
    assert R.e2m1_of(np.nextafter(mids.astype(np.float32), np.float32(9))).tolist() == list(range(1, 8))
    assert R.e2m1_of(np.nextafter(mids.astype(np.float32), np.float32(0))).tolist() == list(range(7))
    assert R.e2m1_of(np.array([-6, 7, 1e30, -1e30, -0.0], dtype=np.float32)).tolist() == [15, 7, 7, 15, 8]


def test_e4m3_bytes():
    assert R.e4m3_of(R.E4M3[:127].astype(np.float32)).tolist() == list(range(127))
    mids = ((R.E4M3[:126] + R.E4M3[1:127]) / 2).astype(np.float32)
    assert all(b % 2 == 0 for b in R.e4m3_of(mids))
    assert R.e4m3_of(np.array([449, 1e9], dtype=np.float32)).tolist() == [126, 126]


def test_what_a_row_keeps():
    rng = np.random.default_rng(1)
    for x in (rng.standard_normal((5, 64)), rng.standard_normal((5, 64)) * 1e-30, np.zeros((2, 32)), rng.standard_normal((3, 96)) * 1e30):
        x = x.astype(np.float32)
        c, b, s = R.quantize(x)
        v = R.values(c, b, s)
        # half a step: of the code, relative 2^-2 at most of the value, or half the smallest code of
        # its block's scale (that rounded down by up to 1/16, which may cut the largest by as much)
        step = np.repeat(R.E4M3[b], 16, -1) * s[:, None].astype(np.float64)
        assert (np.abs(v - x) <= np.maximum(np.abs(x) / 4, step / 4) * 1.01 + s[:, None] * 2.0 ** -9 * 6).all()
    assert s[0] == 1.0 or s[0] > 0
    z = R.quantize(np.zeros((1, 32), np.float32))
    assert not z[0].any() and not z[1].any() and z[2][0] == 1.0
