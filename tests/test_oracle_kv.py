"""Pins of the cache and cross-attention oracle (oracle/kv_ref.py), CPU only: closed forms, torch's own E4M3 rounding,
differences for the gradients, and agreement with the self-attention oracle where the two definitions meet."""
import math

import numpy as np
import pytest
import torch

from oracle import (attend, attention_backward, attention_forward, cross_backward, e8_value, gather, page_row,
                    quantise_row, round_e4m3)


def test_e4m3_rounding_is_torchs():
    r = np.random.RandomState(0)
    x = np.concatenate([r.randn(2000) * 2.0 ** r.randint(-12, 7, 2000), [0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10,
                        1.5 * 2.0 ** -9, 17.0, 19.0, 0.015625]])
    x = np.clip(x, -448, 448)
    got = np.array([round_e4m3(float(np.float32(v))) for v in x])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (1.75, -8), (1.76, -7), (0.0, -120), (2.0 ** -130, -120),
                                    (448.0 * 2.0 ** -120, -120), (450.0 * 2.0 ** -120, -119)])
def test_exponent_is_the_least_that_holds_the_row(amax, e):
    codes, byte = quantise_row([amax, -amax / 3, 0.0])
    assert byte == e + 127 and np.abs(codes).max() <= 448
    back = codes * e8_value(byte)
    assert np.all(np.abs(back - np.array([amax, -amax / 3, 0.0])) <= np.abs([amax, amax / 3, 0.0]) * 2.0 ** -4
                  + 2.0 ** (e - 10))


def test_quantised_values_are_bf16_numbers():
    r = np.random.RandomState(1)
    for k in (-125, -100, 0, 100, 126):
        row = torch.tensor(r.randn(64) * 2.0 ** k).to(torch.bfloat16).double().numpy()
        codes, byte = quantise_row(row)
        back = torch.tensor(codes * e8_value(byte))
        assert torch.equal(back.to(torch.bfloat16).double(), back) and torch.isfinite(back.to(torch.bfloat16)).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_rows_that_are_not_finite_read_as_nan(bad):
    codes, byte = quantise_row([1.0, bad])
    assert byte == 255 and not codes.any() and math.isnan(e8_value(byte))


def test_pages():
    assert page_row([3, 1], 16, 4, 17) == (1, 1) and page_row([3, 1], 16, 4, 32) is None
    assert page_row([3, -1], 16, 4, 16) is None and page_row([4], 16, 4, 0) is None and page_row([0], 16, 4, -1) is None
    cache = np.arange(4 * 1 * 16 * 2, dtype=float).reshape(4, 1, 16, 2)
    rows = gather(cache, None, [2, 9, 0], 40)
    assert np.array_equal(rows[0, :16], cache[2, 0]) and not rows[0, 16:32].any()
    assert np.array_equal(rows[0, 32:], cache[0, 0, :8])


def _draw(*shape, seed):
    return np.random.RandomState(seed).randn(*shape)


@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 2)])
def test_attend_is_self_attention_where_they_meet(hq, hkv):
    q, k, v = _draw(hq, 9, 8, seed=1), _draw(hkv, 9, 8, seed=2), _draw(hkv, 9, 8, seed=3)
    for causal in (False, True):
        o, lse = attention_forward(q[None], k[None], v[None], causal, 0.3)
        lims = np.arange(1, 10) if causal else np.full(9, 9)
        got = attend(q, k, v, lims, 0.3)
        assert np.allclose(got[0], o[0], rtol=0, atol=1e-12) and np.allclose(got[1], lse[0], rtol=0, atol=1e-12)
    do = _draw(hq, 9, 8, seed=4)
    want = attention_backward(q[None], k[None], v[None], do[None], False, 0.3)
    for g, w in zip(cross_backward(q, k, v, do, 9, 0.3), want):
        assert np.allclose(g, w[0], rtol=0, atol=1e-11)


def test_rows_without_keys():
    o, lse, _, _ = attend(_draw(2, 3, 4, seed=1), _draw(1, 5, 4, seed=2), _draw(1, 5, 4, seed=3), [0, -2, 1], 1.0)
    assert not o[:, :2].any() and np.all(np.isneginf(lse[:, :2])) and np.all(np.isfinite(lse[:, 2]))


def test_cross_gradients_against_differences():
    q, k, v, do = _draw(4, 3, 5, seed=1), _draw(2, 7, 5, seed=2), _draw(2, 7, 5, seed=3), _draw(4, 3, 5, seed=4)
    n, scale, h = 4, 0.4, 1e-6
    loss = lambda q, k, v: float((attend(q, k, v, [n] * 3, scale)[0] * do).sum())
    for i, (x, g) in enumerate(zip((q, k, v), cross_backward(q, k, v, do, n, scale))):
        for idx in np.ndindex(x.shape):
            a, b = [y.copy() for y in (q, k, v)], [y.copy() for y in (q, k, v)]
            a[i][idx] += h
            b[i][idx] -= h
            assert abs((loss(*a) - loss(*b)) / (2 * h) - g[idx]) < 1e-8
    assert not cross_backward(q, k, v, do, n, scale)[1][:, n:].any()
    assert not any(g.any() for g in cross_backward(q, k, v, do, 0, scale))
