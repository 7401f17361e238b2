"""Pins of the oracle's MXFP4 and router statements (CPU only)."""
import itertools

import numpy as np
import pytest

from oracle import mxfp4, router


def test_mxfp4_hand_values():
    x = np.zeros((1, 32))
    x[0, :10] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0]   # amax 6: e = 0
    codes, scales = mxfp4.quantize(x)
    assert scales[0, 0] == 127
    got = [int(codes[0, i // 2] >> (4 * (i % 2))) & 15 for i in range(10)]
    assert got == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8]                     # ties to the even code, -0 kept
    assert mxfp4.dequantize(codes, scales, 32)[0, :9].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4]


@pytest.mark.parametrize("amax,byte", [(6.0, 127), (6.0000005, 128), (3.0, 126), (0.0, 0), (12.5, 129),
                                       (3.0e38, 253), (2.0 ** -140, 0), (np.inf, 255), (np.nan, 255)])
def test_mxfp4_scale_byte(amax, byte):
    x = np.full((1, 32), np.float32(amax), dtype=np.float32)
    codes, scales = mxfp4.quantize(x)
    assert scales[0, 0] == byte
    if byte == 255:
        assert not codes.any() and np.isnan(mxfp4.dequantize(codes, scales, 32)).all()


def test_mxfp4_nothing_saturates_and_all_codes_come_back():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float32)
    codes, scales = mxfp4.quantize(x)
    v = mxfp4.dequantize(codes, scales, 96)
    step = np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=1)
    assert (np.abs(v - x) <= step).all() and (np.abs(x) <= 6 * step).all()
    again = mxfp4.quantize(v)                      # representable values stay as they are
    assert np.array_equal(mxfp4.dequantize(*again, 96), v)


def test_mxfp4_padding_and_odd_lengths():
    x = np.arange(1, 36, dtype=np.float64)[None]
    codes, scales = mxfp4.quantize(x)
    assert codes.shape == (1, 32) and scales.shape == (1, 2)
    assert not codes[0, 18:].any()
    assert mxfp4.dequantize(codes, scales, 35).shape == (1, 35)


def test_router_even_load_has_balance_one_and_uniform_lse():
    T, E, k = 12, 6, 2
    l = np.full((T, E), -30.0)
    for t, pair in zip(range(T), itertools.cycle([(0, 1), (2, 3), (4, 5)])):
        l[t, list(pair)] = 3.0
    f = router.forward(l, k)
    assert f["counts"].tolist() == [4] * 6
    assert abs(f["losses"][0] - 1.0) < 1e-9
    assert abs(f["losses"][1] - (3 + np.log(2)) ** 2) < 1e-9


def test_router_nobody_valid():
    l = np.full((3, 4), -np.inf)
    l[0] = [1, 2, 3, 4]
    f = router.forward(l, 2, mask=[False, True, True])
    assert f["tokens"] == 0 and f["losses"].tolist() == [0, 0] and f["w"][1].tolist() == [0, 0]
    assert f["ids"].tolist() == [[3, 2], [0, 1], [0, 1]]
    d, _ = router.backward(l, 2, [False, True, True], f, np.zeros((3, 2)), [1.0, 1.0])
    assert not d.any()


@pytest.mark.parametrize("seed,masked", [(0, False), (1, True)])
def test_router_gradient_against_differences(seed, masked):
    rng = np.random.default_rng(seed)
    T, E, k = 5, 7, 3
    l = rng.standard_normal((T, E))
    l[2, 4] = -np.inf
    mask = np.array([1, 0, 1, 1, 1], dtype=bool) if masked else None
    gw, gl = rng.standard_normal((T, k)), np.array([0.7, 0.3])
    f = router.forward(l, k, mask)
    d, _ = router.backward(l, k, mask, f, gw, gl)
    h = 1e-6
    for t, e in itertools.product(range(T), range(E)):
        if l[t, e] == -np.inf:
            assert d[t, e] == 0
            continue
        up, dn = l.copy(), l.copy()
        up[t, e] += h
        dn[t, e] -= h
        num = (router.loss_of(up, k, mask, gw, gl, f["ids"], f["counts"]) -
               router.loss_of(dn, k, mask, gw, gl, f["ids"], f["counts"])) / (2 * h)
        assert abs(num - d[t, e]) < 1e-8 + 1e-6 * abs(num)
