"""Pins of the attention oracle (oracle/attn_oracle.py): torch's own attention and
complex rotations, exact small cases, splits of a prompt."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as orc


def cache_of(rng, lens, KV, D, page, spare=3):
    held = [-(-n // page) for n in lens]
    order = rng.permutation(sum(held) + spare)
    table = np.full((len(lens), max(held + [1])), -1)
    at = 0
    for n, c in enumerate(held):
        table[n, :c] = order[at:at + c]
        at += c
    size = (sum(held) + spare, KV, page, D)
    return table, rng.normal(size=size), rng.normal(size=size)


@pytest.mark.parametrize("window", [0, 3])
def test_attention_matches_torch(window):
    rng = np.random.default_rng(1)
    H, KV, D, page = 4, 2, 8, 4
    new, kv = [5, 1, 0, 3], [5, 9, 2, 10]
    cu = np.concatenate([[0], np.cumsum(new)])
    table, kc, vc = cache_of(rng, kv, KV, D, page)
    q, gate = rng.normal(size=(9, H, D)), rng.normal(size=(9, H, D))
    out, err = orc.attention(cu, kv, table, q, kc, vc, page, 0.3, window, gate)
    for n in range(4):
        p = kv[n] - new[n] + np.arange(new[n])
        j = np.arange(kv[n])
        seen = (j <= p[:, None]) & ((j > p[:, None] - window) if window else True)
        for h in range(H):
            K, V = (torch.from_numpy(orc.keys_of(c, table, n, h // 2, kv[n], page)) for c in (kc, vc))
            ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[cu[n]:cu[n + 1], h])[None], K[None], V[None],
                                                                   attn_mask=torch.from_numpy(seen)[None], scale=0.3)[0]
            ref = ref * torch.sigmoid(torch.from_numpy(gate[cu[n]:cu[n + 1], h]))
            np.testing.assert_allclose(out[cu[n]:cu[n + 1], h], ref.numpy(), rtol=1e-12, atol=1e-12)
    assert (err > 0).all() and err.max() < 1e-4


def test_attention_of_equal_scores_is_the_mean_and_rows_without_keys_are_zero():
    table = np.array([[1, 0]])
    kc, vc = np.ones((2, 1, 2, 2)), np.arange(8.0).reshape(2, 1, 2, 2)
    q = np.ones((5, 1, 2))
    out, _ = orc.attention([0, 5], [3], table, q, kc, vc, 2, 1.0)  # positions -2 .. 2
    assert np.array_equal(out[:2], np.zeros((2, 1, 2)))
    np.testing.assert_allclose(out[2:, 0], [[4, 5], [5, 6], [10 / 3, 13 / 3]], rtol=1e-15)


def test_a_split_prompt_equals_the_whole():
    rng = np.random.default_rng(2)
    table, kc, vc = cache_of(rng, [11], 1, 4, 2)
    q = rng.normal(size=(11, 2, 4))
    whole, _ = orc.attention([0, 11], [11], table, q, kc, vc, 2, 0.5)
    parts = [orc.attention([0, b - a], [b], table, q[a:b], kc, vc, 2, 0.5)[0] for a, b in ((0, 4), (4, 5), (5, 11))]
    np.testing.assert_allclose(np.concatenate(parts), whole, rtol=1e-14, atol=1e-15)


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_product_of_complex_numbers(pairs):
    rng = np.random.default_rng(3)
    x, P = rng.normal(size=(6, 2, 10)), np.array([0, 1, 2, 1000, 100000, 3])
    f = 10.0 ** -np.arange(3)
    y, err = orc.rotated(x, P, f, pairs, scale=1.5)
    z = x[..., 0:6:2] + 1j * x[..., 1:6:2] if pairs else x[..., :3] + 1j * x[..., 3:6]
    z = 1.5 * z * np.exp(1j * P[:, None] * f)[:, None]
    got = y[..., 0:6:2] + 1j * y[..., 1:6:2] if pairs else y[..., :3] + 1j * y[..., 3:6]
    np.testing.assert_allclose(got, z, rtol=1e-12)
    assert np.array_equal(y[..., 6:], x[..., 6:]) and not err[..., 6:].any() and (err[..., :6] > 0).all()
    n, e = orc.rotated(x, P * 0, f, pairs, weight=np.full(10, 2.0), eps=0.0)
    np.testing.assert_allclose((n * n).mean(-1), 4, rtol=1e-12)
    assert (e > 0).all()


def test_positions():
    seq, p = orc.positions([0, 2, 2, 5], [7, 3, 2])
    assert seq.tolist() == [0, 0, 2, 2, 2] and p.tolist() == [5, 6, -1, 0, 1]
