"""The bounds of the KV attention tests, without a GPU: they hold the oracle's own outputs, and they are
narrow enough to tell planted mistakes."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.kv_bounds import attention_bounds, batch_bounds, outside, telling


def data(n, t, H, n_kv, D, seed=0):
    g = np.random.default_rng(seed)
    bf = lambda *s: KV.bf16_round(g.standard_normal(s).astype(np.float32))  # noqa: E731
    return bf(n, H, D) * 1.25, KV.quantise(bf(t, n_kv, D)), KV.quantise(bf(t, n_kv, D))


@pytest.mark.parametrize("n,t,H,n_kv", [(1, 40, 4, 2), (5, 3, 2, 1), (70, 90, 2, 2)])
def test_the_centre_is_the_oracles(n, t, H, n_kv):
    q, k, v = data(n, t, H, n_kv, 64)
    want, bound, drop = attention_bounds(q, k, v, n_kv, 0.125, hidden=[1])
    assert np.allclose(want, KV.attention(q, KV.value(*k), KV.value(*v), n_kv, 0.125, hidden=[1]), rtol=1e-12, atol=1e-13)
    assert not outside(KV.bf16_round(want), want, bound).any()
    assert np.array_equal(bound.any(-1), want.any(-1))           # rows that see nothing are zero exactly


@pytest.mark.parametrize("few", [True, False])
def test_planted_mistakes_are_outside(few):
    n, t, H, n_kv, D = 4, 300, 4, 2, 128
    q, k, v = data(n, t, H, n_kv, D, 1)
    scale = D ** -0.5
    want, bound, drop = attention_bounds(q, k, v, n_kv, scale, few)
    assert telling(want, bound, drop) == (1.0, 1.0)
    for wrong in (attention_bounds(q, k, v, n_kv, scale * 1.05)[0],                                  # another scale
                  attention_bounds(q, k, (np.minimum(v[0] + 1, 15),) + v[1:], n_kv, scale)[0],       # codes one up
                  attention_bounds(q, k, (v[0], v[1] * (1 + 2.0 ** -4), v[2]), n_kv, scale)[0],      # a step too long
                  np.concatenate([want[1:], want[:1]])):                                             # rows changed over
        assert outside(wrong, want, bound).all()


def test_a_lost_half_of_the_weights_is_outside():
    """Of weights in two bf16 halves against 16 + code the low one lost; one half against code - 8 is within
    its own, wider bound."""
    n, t, H, n_kv, D = 4, 16, 2, 1, 64
    q, k, v = data(n, t, H, n_kv, D, 2)
    want, two, _ = attention_bounds(q, k, v, n_kv, 0.125, True)
    one = attention_bounds(q, k, v, n_kv, 0.125, False)[1]
    kk = KV.value(*k)[:, 0]

    def rounded(centre):
        out = np.zeros_like(want)
        for j in range(n):
            for h in range(H):
                m = t - n + j + 1
                s = kk[:m] @ q[j, h] * 0.125
                p = np.exp(s - s.max())[:, None]
                w = KV.bf16_round((p * v[1][:m]).astype(np.float32))
                out[j, h] = (w * (v[0][:m, 0] + centre) + p * (v[2] - centre * v[1])[:m]).sum(0) / p.sum()
        return out

    assert outside(rounded(16), want, two).all()
    assert not outside(rounded(-8), want, one).any()


def test_batches_take_their_own_tokens():
    q, k, v = data(6, 50, 2, 2, 64, 3)
    want, bound, _ = batch_bounds(q, k, v, [2, 4], [20, 30], 2, 0.125, hidden={1: [0]})
    cut = lambda c, a, z: tuple(x[a:z] for x in c)  # noqa: E731
    assert np.array_equal(want[2:], attention_bounds(q[2:], cut(k, 20, 50), cut(v, 20, 50), 2, 0.125, hidden=[0])[0])
    assert bound.shape == want.shape
