"""Pins of the state space oracle (oracle/ssm_oracle.py): torch's own conv and
group norm, the closed (attention-like) form of the recurrence, exact rationals,
and splits of a sequence."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import ssm_oracle as orc


def test_conv_matches_torch_conv1d_and_carries_history():
    rng = np.random.default_rng(1)
    cu, C, K = [0, 5, 5, 7], 6, 3
    x, w, b = rng.normal(size=(7, C)), rng.normal(size=(C, K)), rng.normal(size=C)
    h = rng.normal(size=(3, K - 1, C))
    out, err, new = orc.conv(cu, x, w, b, h)
    for n in range(3):
        X = np.concatenate([h[n], x[cu[n]:cu[n + 1]]])
        if cu[n + 1] > cu[n]:
            ref = torch.nn.functional.silu(torch.nn.functional.conv1d(
                torch.from_numpy(X.T)[None], torch.from_numpy(w)[:, None], torch.from_numpy(b), groups=C))[0].T
            np.testing.assert_allclose(out[cu[n]:cu[n + 1]], ref.numpy(), rtol=1e-12, atol=1e-12)
        assert np.array_equal(new[n], X[-(K - 1):])
    assert np.array_equal(new[1], h[1]) and (err >= 0).all()


def test_scan_matches_exact_rationals():
    # decays that are powers of 1/2, one head, two tokens
    H = P = G = 1
    N = 2
    lam = np.log(np.array([[0.5], [0.25]]))
    dt = np.array([[2.0], [0.5]])
    xbc = np.array([[3.0, 1.0, -2.0, 0.5, 1.0], [-1.0, 4.0, 1.0, 2.0, -1.0]])
    S0 = np.array([[[[1.0, 8.0]]]])
    y, _, S, _ = orc.scan([0, 2], xbc, dt, lam, np.array([0.5]), S0, H, P, G, N)
    F = Fraction
    s = [F(1), F(8)]
    for t, (a, d) in enumerate([(F(1, 2), F(2)), (F(1, 4), F(1, 2))]):
        x, B, C = F(int(xbc[t, 0])), [F(v) for v in xbc[t, 1:3]], [F(v) for v in xbc[t, 3:]]
        s = [a * s[i] + d * x * B[i] for i in range(2)]
        want = s[0] * C[0] + s[1] * C[1] + F(1, 2) * x
        assert abs(y[t, 0, 0] - float(want)) < 1e-14 * max(1, abs(float(want)))
    np.testing.assert_allclose(S[0, 0, 0], [float(v) for v in s], rtol=1e-14)


def test_scan_matches_the_closed_form_with_shared_groups():
    rng = np.random.default_rng(2)
    H, P, G, N, T = 4, 3, 2, 5, 11
    xbc = rng.normal(size=(T, H * P + 2 * G * N))
    dt, lam = orc.step_size(rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=H), 0.1, 0.9)
    assert dt.min() >= 0.1 and dt.max() <= 0.9
    D, S0 = rng.normal(size=H), rng.normal(size=(1, H, P, N))
    y, _, S, _ = orc.scan([0, T], xbc, dt, lam, D, S0, H, P, G, N)
    L = np.cumsum(lam, 0)
    for h in range(H):
        x = xbc[:, h * P:(h + 1) * P]
        B = xbc[:, H * P + (h // 2) * N:][:, :N]
        C = xbc[:, H * P + G * N + (h // 2) * N:][:, :N]
        M = np.tril((C @ B.T) * np.exp(np.minimum(L[:, h, None] - L[None, :, h], 0))) * dt[:, h]
        ref = M @ x + np.exp(L[:, h, None]) * (C @ S0[0, h].T) + D[h] * x
        np.testing.assert_allclose(y[:, h], ref, rtol=1e-10, atol=1e-12)
        Sr = np.exp(L[-1, h]) * S0[0, h] + (x * (np.exp(L[-1, h] - L[:, h]) * dt[:, h])[:, None]).T @ B
        np.testing.assert_allclose(S[0, h], Sr, rtol=1e-10, atol=1e-12)


def test_scan_of_a_split_sequence_equals_the_whole():
    rng = np.random.default_rng(3)
    H, P, G, N = 2, 2, 1, 3
    xbc = rng.normal(size=(9, H * P + 2 * G * N))
    dt, lam = orc.step_size(rng.normal(size=(9, H)), 0.0, np.zeros(H))
    D, S0 = np.ones(H), rng.normal(size=(1, H, P, N))
    y, _, S, _ = orc.scan([0, 9], xbc, dt, lam, D, S0, H, P, G, N)
    y1, _, S1, _ = orc.scan([0, 4], xbc[:4], dt[:4], lam[:4], D, S0, H, P, G, N)
    y2, _, S2, _ = orc.scan([0, 5], xbc[4:], dt[4:], lam[4:], D, S1, H, P, G, N)
    assert np.array_equal(y, np.concatenate([y1, y2])) and np.array_equal(S, S2)


@pytest.mark.parametrize("last", [False, True])
def test_group_norm_matches_torch(last):
    rng = np.random.default_rng(4)
    x, z, w, b = rng.normal(size=(5, 24)) + 3, rng.normal(size=(5, 24)), rng.normal(size=24), rng.normal(size=24)
    y, err = orc.group_norm(x, z, w, b, 3, 1e-5, True, last)
    t, g = torch.from_numpy(x), torch.nn.functional.silu(torch.from_numpy(z))
    ref = torch.nn.functional.group_norm(t if last else t * g, 3, torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(y, (ref * g if last else ref).numpy(), rtol=1e-10, atol=1e-10)
    y, _ = orc.group_norm(x, None, None, None, 1, 1e-5, False, last)
    np.testing.assert_allclose(y, torch.nn.functional.rms_norm(t, (24,), eps=1e-5).numpy(), rtol=1e-12)
    assert (err > 0).all()
