"""Pins of the float64 oracle of the position and serving operators (oracle/ra_serving.py)."""
import numpy as np
import pytest

import oracle
from oracle import ra_serving as S


def _inputs(rng, B, N, Hq, Hkv, D, norm, bias):
    qkv = rng.standard_normal((B, N, (Hq + 2 * Hkv) * D))
    params = [None] * 4
    if norm != "none":
        params[0], params[2] = rng.uniform(0.5, 1.5, D), rng.uniform(0.5, 1.5, D)
    if bias:
        params[1], params[3] = rng.standard_normal(D), rng.standard_normal(D)
    return qkv, params


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_rotation_keeps_lengths_and_depends_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(1)
    qkv = np.repeat(rng.standard_normal((1, 1, 3 * 16)), 6, axis=1)      # one token at six positions
    how = dict(frequencies=rng.uniform(0.01, 1, 6), sections=(4, 2), interleaved=interleaved)
    pos = np.stack([np.arange(6), 3 * np.arange(6)])[:, None]
    q, k, v = S.qk_norm_rope(qkv, 1, 1, positions=pos, **how)
    q0, k0, v0 = S.qk_norm_rope(qkv, 1, 1)
    assert np.allclose((q ** 2).sum(-1), (q0 ** 2).sum(-1)) and np.array_equal(v, v0)
    assert np.array_equal(q[0, 0, 0], q0[0, 0, 0]) and np.array_equal(q[..., 12:], q0[..., 12:])
    s = q[0, 0] @ k[0, 0].T
    for d in range(1, 6):                                                # equal along the diagonals
        assert np.allclose(np.diagonal(s, d), s[0, d])


@pytest.mark.parametrize("norm,bias", [("none", False), ("rms", False), ("layer", False), ("layer", True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_against_differences(norm, bias, interleaved):
    rng = np.random.default_rng(2)
    B, N, Hq, Hkv, D = 2, 3, 4, 2, 8
    qkv, params = _inputs(rng, B, N, Hq, Hkv, D, norm, bias)
    how = dict(norm=norm, eps=1e-5, frequencies=rng.uniform(0.1, 1, 3), sections=(1, 2),
               positions=rng.integers(-5, 50, (2, B, N)), interleaved=interleaved)
    d = [rng.standard_normal((B, h, N, D)) for h in (Hq, Hkv, Hkv)]

    def loss(x, p):
        return sum((g * y).sum() for g, y in zip(d, S.qk_norm_rope(x, Hq, Hkv, params=p, **how)))
    dqkv, dparams = S.qk_norm_rope_bwd(qkv, *d, Hq, Hkv, params=params, **how)
    e = 1e-6
    for at in [tuple(rng.integers(0, n) for n in qkv.shape) for _ in range(24)]:
        hi, lo = qkv.copy(), qkv.copy()
        hi[at] += e
        lo[at] -= e
        assert abs((loss(hi, params) - loss(lo, params)) / (2 * e) - dqkv[at]) < 1e-6 * max(1, abs(dqkv[at]))
    for i, p in enumerate(params):
        if p is not None:
            for j in range(D):
                hi, lo = [[None if x is None else x.copy() for x in params] for _ in range(2)]
                hi[i][j] += e
                lo[i][j] -= e
                assert abs((loss(qkv, hi) - loss(qkv, lo)) / (2 * e) - dparams[i][j]) < 1e-5


def test_layer_norm_is_the_module_oracles():
    rng = np.random.default_rng(3)
    qkv, params = _inputs(rng, 1, 4, 2, 2, 16, "layer", True)
    q, k, _ = S.qk_norm_rope(qkv, 2, 2, norm="layer", params=params)
    x = qkv.reshape(1, 4, 6, 16).transpose(0, 2, 1, 3)
    assert np.allclose(q, oracle.layer_norm(x[:, :2], params[0], params[1]))
    assert np.allclose(k, oracle.layer_norm(x[:, 2:4], params[2], params[3]))


def test_decode_is_the_attention_oracle_on_the_joined_keys():
    rng = np.random.default_rng(4)
    B, Hq, Hkv, C, P, D = 3, 4, 2, 9, 5, 8
    q, k, v = rng.standard_normal((B, Hq, D)) * 3, rng.standard_normal((B, Hkv, C, D)), rng.standard_normal((B, Hkv, C, D))
    pk, pv = rng.standard_normal((Hkv, P, D)), rng.standard_normal((Hkv, P, D))
    length = [4, 0, 9]
    o, w, spread, sums = S.attention_decode(q, k, v, length, pk, pv)
    for b, n in enumerate(length):
        for h in range(Hq):
            keys = np.concatenate([k[b, h // 2, :n], pk[h // 2]])
            vals = np.concatenate([v[b, h // 2, :n], pv[h // 2]])
            O, m, s, _ = oracle.ra_attention_head_fwd(q[b, h][None], keys, vals, D ** -0.5, False)
            assert np.allclose(o[b, h], O[0]) and np.isclose(sums[b, h], s[0])
        assert np.all(w[b, :, n:] == 0)
    # weights of own and shared keys add up to one per query head
    assert np.all(w.sum(-1) < 2) and np.allclose(S.attention_decode(q, k, v, [9] * 3)[1].sum(-1), 2.0)
    o, w, _, _ = S.attention_decode(q, k, v, [0, 1, 0])
    assert np.all(o[0] == 0) and np.all(w[0] == 0) and np.allclose(o[1, :2], v[1, 0, 0])


def test_evict_by_hand():
    w = np.array([[[5, 1, 5, 2, 9, 0.5, 0.1, 0.2]]], dtype=np.float32)
    assert S.cache_evict(w, [8], 4, 1)[0].tolist() == [[[0, 2, 4, 7]]]
    assert S.cache_evict(w, [8], 3, 1)[0].tolist() == [[[0, 4, 7]]]            # of the two fives, the first
    assert S.cache_evict(w, [3], 4, 1)[0].tolist() == [[[0, 1, 2, -1]]]
    assert S.cache_evict(w, [6], 2, 2)[0].tolist() == [[[4, 5]]]
    index, n = S.cache_evict(w, [0], 2, 2)
    assert index.tolist() == [[[-1, -1]]] and n.tolist() == [0]
    w[0, 0, 6] = np.nan
    assert S.cache_evict(w, [8], 2, 0)[0].tolist() == [[[4, 6]]]
