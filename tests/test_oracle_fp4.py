"""Pins of the 4-bit cache's NumPy oracle: the formats' values, the rounding,
the byte layout, and closed-form rows."""
import numpy as np
import pytest

import oracle
from oracle import fp4, twin


def test_code_values_are_e2m1():
    # sign, two exponent bits of bias 1 (0: subnormal), one mantissa bit
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        want = 0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
        assert fp4.code_value(np.uint8(c)) == (-want if c & 8 else want)


def test_scale_values_are_the_non_negative_e4m3_numbers():
    assert fp4.SCALE_VALUES[-1] == 448 and fp4.SCALE_VALUES[0] == 0
    assert (np.diff(fp4.SCALE_VALUES) > 0).all()


@pytest.mark.parametrize("x,code", [(0.0, 0), (0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2),
                                    (1.2500001, 3), (1.75, 4), (2.5, 4), (3.5, 6), (3.4999, 5),
                                    (5.0, 6), (5.0001, 7), (6.0, 7), (1e30, 7), (np.inf, 7)])
def test_codes_round_to_nearest_even_and_saturate(x, code):
    assert fp4._nearest(np.float64(x), fp4.CODE_VALUES) == code


def test_scale_rounding_matches_the_c_oracle():
    x = np.abs(np.random.default_rng(3).standard_normal(4000) * 10.0 ** np.random.default_rng(
        4).uniform(-4, 4, 4000)).astype(np.float32)
    lib = oracle.default()
    want = [lib.e4m3_encode(v) for v in x]
    assert fp4._nearest(x, fp4.SCALE_VALUES).tolist() == want


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("keys", [True, False])
def test_every_byte_of_a_tile_has_one_owner(D, keys):
    cp, sp = fp4.code_place(D, keys), fp4.scale_place(D, keys)
    assert (cp[:, ::2] == cp[:, 1::2]).all()
    owned = np.concatenate([cp[:, ::2].ravel(), sp.ravel()])
    assert sorted(owned) == list(range(9 * D))


def test_documented_places():
    # keys: panels of 128 dims; values: words of 8 dims, the 16 rows beside one another
    assert fp4.code_place(256, True)[3, 130] == 1024 + 3 * 64 + 1
    assert fp4.scale_place(128, True)[5, 7] == 1024 + 5 * 8 + 7
    assert fp4.code_place(128, False)[9, 13] == 64 + 9 * 4 + 2
    assert fp4.scale_place(64, False)[15, 2] == 512 + 2 * 16 + 15


def test_representable_rows_come_back_exactly():
    rng = np.random.default_rng(5)
    t = np.float32(0.25)
    codes = rng.integers(0, 16, (7, 3, 64)).astype(np.uint8)
    codes[..., ::16] = 7                                    # each block reaches 6
    scales = rng.integers(1, 127, (7, 3, 4)).astype(np.uint8)
    x = fp4.code_value(codes) * np.repeat(fp4.SCALE_VALUES[scales], 16, -1) * t
    got_codes, got_scales = fp4.quantise(x.astype(np.float32), t)
    assert (got_scales == scales).all()
    assert (fp4.code_value(got_codes) == fp4.code_value(codes)).all()


def test_zero_tiny_infinite_and_nan_blocks():
    x = np.zeros((5, 16), np.float32)
    x[1] = 1e-9                                              # the scale rounds to zero
    x[2, 3] = np.inf
    x[3, 4] = np.nan
    x[4] = np.linspace(-1, 1, 16)
    codes, scales = fp4.quantise(x, 1.0)
    assert (codes[0] == 0).all() and scales[0, 0] == 0
    assert (codes[1] == 0).all() and scales[1, 0] == 0
    assert scales[2, 0] == 126 and codes[2, 3] == 7 and (np.delete(codes[2], 3) == 0).all()
    assert scales[3, 0] == 127 and (codes[3] == 0).all()
    assert codes[4, 0] == 15 and codes[4, 15] == 7


def test_quantisation_error_is_within_half_a_step():
    # off the saturated end the code is off by at most half the widest step
    # (1 in [4, 6]) of its scale, and the scale by 2^-4 of the ideal one
    rng = np.random.default_rng(6)
    x = rng.standard_normal((50, 2, 128)).astype(np.float32)
    codes, scales = fp4.quantise(x, 0.01)
    s = np.repeat(fp4.SCALE_VALUES[scales], 16, -1) * np.float32(0.01)
    err = np.abs(fp4.code_value(codes) * s - x)
    over = np.maximum(np.abs(x) - 6 * s, 0)                  # saturated part
    assert (err <= s * (1 + 1e-6) + over).all()
    assert (over <= 6 * s * 2.0 ** -4).all()


def test_append_load_and_pack_agree():
    rng = np.random.default_rng(7)
    rows = rng.standard_normal((3, 2, 16, 128)).astype(np.float32)
    for keys in (True, False):
        packed = fp4.pack(rows, 0.02, keys)
        other = np.zeros_like(packed)
        flat = rows.transpose(0, 2, 1, 3).reshape(48, 2, 128)
        order = rng.permutation(48)
        fp4.write_rows(other, order, *fp4.quantise(flat[order], 0.02), keys)
        assert (packed == other).all()
        back = fp4.load(packed, np.array([5, -1, 47, 48, 5]), 0.02, keys)
        full = fp4.unpack(packed, keys).transpose(0, 2, 1, 3).reshape(48, 2, 128)
        assert (back[0] == full[5].astype(np.float32) * np.float32(0.02)).all()
        assert (back[0] == back[4]).all() and (back[[1, 3]] == 0).all()


def test_attention_over_one_key_returns_its_value():
    rng = np.random.default_rng(8)
    k = fp4.pack(rng.standard_normal((2, 2, 16, 64)).astype(np.float32), 0.01, True)
    vr = rng.standard_normal((2, 2, 16, 64)).astype(np.float32)
    v = fp4.pack(vr, 0.01, False)
    q = rng.standard_normal((1, 1, 4, 64)).astype(np.float32)
    out = fp4.attention(q, k, v, np.array([[1]], np.int32), np.array([1], np.int32), 0.3, 0.01,
                        0.01)
    row = fp4.unpack(v, False)[1, :, 0] * float(np.float32(0.01))
    np.testing.assert_allclose(out[0, 0], np.repeat(row, 2, 0), rtol=1e-6)


def test_attention_matches_the_dense_twin():
    rng = np.random.default_rng(9)
    k = fp4.pack(rng.standard_normal((4, 2, 16, 64)).astype(np.float32), 0.01, True)
    v = fp4.pack(rng.standard_normal((4, 2, 16, 64)).astype(np.float32), 0.02, False)
    q = rng.standard_normal((2, 3, 4, 64)).astype(np.float32)
    table, lens = np.array([[2, 0], [3, 1]], np.int32), np.array([30, 17], np.int32)
    out = fp4.attention(q, k, v, table, lens, 0.125, 0.01, 0.02)
    want = twin.contiguous_attention(q, fp4.unpack(k, True).astype(np.float32),
                                     fp4.unpack(v, False).astype(np.float32), table, lens,
                                     0.125 * float(np.float32(0.01)), "f32")
    np.testing.assert_allclose(out, want * float(np.float32(0.02)), rtol=1e-10, atol=1e-12)
