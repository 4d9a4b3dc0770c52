"""Pins of the float64 oracle of the attention side (CPU): E4M3 against torch's own conversion,
the exponent rule against its closed form, attention against closed forms and library softmax,
the gated residual norm against torch."""
import numpy as np
import pytest
import torch

from oracle import kv_attention as KV


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(KV.e4m3_values(), codes.astype(np.float64))


@pytest.mark.parametrize("seed", range(3))
def test_quantise_rounds_to_nearest_even(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal(512) * 2.0 ** rng.integers(-12, 3)).astype(np.float32)
    x[:8] = [0.0, -0.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 448.0 * 2.0 ** -9, -17.0]   # ties among them
    q, e = KV.quantise(x)
    want = (torch.from_numpy(x) * 2.0 ** -e).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(q, want)


@pytest.mark.parametrize("most,e", [(448.0, 0), (448.0001, 1), (0.875, -9), (1.0, -8), (0.0, -100), (1e-38, -100),
                                    (float("inf"), 119), (3.3e38, 119), (224.0, -1)])
def test_exponent(most, e):
    assert KV.kv_exponent(np.array([0.0, -most, np.nan, most / 3])) == e


def test_quantise_keeps_nan_and_saturates():
    q, e = KV.quantise(np.array([np.nan, np.inf, -np.inf, 1.0]))
    assert e == 119 and np.isnan(q[0]) and list(q[1:3]) == [448.0, -448.0] and q[3] == 0.0


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (False, 3), (True, 3)])
def test_attention_with_zero_queries_is_the_mean_of_what_is_seen(causal, window):
    rng = np.random.default_rng(1)
    v = [rng.standard_normal((L, 2, 4)) for L in (7, 2, 0)]
    k = [rng.standard_normal((L, 2, 4)) for L in (7, 2, 0)]
    out, lse, _, _ = KV.block_attention(np.zeros((9, 4, 4)), k, v, [7, 2, 0], 3, 0.5, causal, window)
    for r, L in enumerate([7, 2, 0]):
        for i in range(3):
            p = L - 3 + i
            seen = [j for j in range(L) if (not causal or j <= p) and (not window or j > p - window)]
            if not seen:
                assert not out[3 * r + i].any() and np.isneginf(lse[3 * r + i]).all()
                continue
            for h in range(4):
                np.testing.assert_allclose(out[3 * r + i, h], v[r][seen, h // 2].mean(0), atol=1e-14)
                assert abs(lse[3 * r + i, h] - np.log(len(seen))) < 1e-13


def test_attention_is_softmax():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((5, 2, 8), (6, 1, 8), (6, 1, 8)))
    out, lse, _, _ = KV.block_attention(q, [k], [v], [6], 5, 0.3, False, 0)
    s = 0.3 * torch.einsum("ihd,jd->ihj", torch.from_numpy(q), torch.from_numpy(k[:, 0]))
    np.testing.assert_allclose(out, (torch.softmax(s, -1) @ torch.from_numpy(v[:, 0])).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-13)


def test_residual_norm():
    rng = np.random.default_rng(3)
    y, h, wp, wq, g = (rng.standard_normal(s) for s in ((5, 16), (5, 16), 16, 16, (3, 16)))
    t = torch.from_numpy
    yn = torch.nn.functional.rms_norm(t(y), (16,), t(wp), 1e-5)
    hh = t(h) + 0.7 * t(np.repeat(g, 2, 0)[:5]) * yn
    x = torch.nn.functional.rms_norm(hh, (16,), t(wq), 1e-5)
    oh, ox = KV.block_residual_norm(y, h, wp, g, wq, 0.7, 1e-5, P=2)
    np.testing.assert_allclose(oh, hh.numpy(), atol=1e-13)
    np.testing.assert_allclose(ox, x.numpy(), atol=1e-13)
    oh, ox = KV.block_residual_norm(y, h)
    np.testing.assert_allclose(oh, y + h, atol=1e-15)
