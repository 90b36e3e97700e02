"""Pins of the fp64 oracle of the hybrid decoder's operators: closed forms, central differences, and the
distribution that speculative sampling has to leave unchanged."""
import numpy as np
import pytest

from oracle import hybrid as ho

D = 4


def _case(lens, Hq, Hkv, seed=0):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    return r.normal(size=(T, Hq * D)), r.normal(size=(T, Hkv * D)), r.normal(size=(T, Hkv * D)), cu


def test_attention_against_a_loop_over_rows():
    q, k, v, cu = _case([3, 0, 5], 4, 2)
    out, lse, _ = ho.attention(q, k, v, cu, D, 0.5)
    for a, b in zip(cu, cu[1:]):
        for t in range(a, b):
            for h in range(4):
                g = h // 2
                s = np.array([0.5 * q[t, h * D:(h + 1) * D] @ k[j, g * D:(g + 1) * D] for j in range(a, t + 1)])
                w = np.exp(s) / np.exp(s).sum()
                want = sum(w[j - a] * v[j, g * D:(g + 1) * D] for j in range(a, t + 1))
                np.testing.assert_allclose(out[t, h * D:(h + 1) * D], want, rtol=1e-12)
                np.testing.assert_allclose(lse[h, t], np.log(np.exp(s).sum()), rtol=1e-12)


def test_first_token_is_its_value_and_equal_keys_give_the_mean():
    q, k, v, cu = _case([6], 1, 1)
    out, lse, _ = ho.attention(q, np.zeros_like(k), v, cu, D, 1.0)
    np.testing.assert_allclose(out, np.cumsum(v, 0) / np.arange(1, 7)[:, None], rtol=1e-12)
    np.testing.assert_allclose(lse[0], np.log(np.arange(1, 7)), rtol=1e-12, atol=1e-15)


def test_gradients_against_central_differences():
    q, k, v, cu = _case([4, 1, 3], 4, 2, seed=3)
    do = np.random.default_rng(4).normal(size=q.shape)
    grads, _ = ho.attention_backward(q, k, v, cu, D, 0.7, do)

    def loss():
        return (ho.attention(q, k, v, cu, D, 0.7)[0] * do).sum()

    eps = 1e-5
    for x, g in zip((q, k, v), grads):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + eps
            up = loss()
            x[i] = keep - eps
            down = loss()
            x[i] = keep
            assert abs((up - down) / (2 * eps) - g[i]) < 1e-7


@pytest.mark.parametrize("prefix,lens", [(5, [4, 6]), (0, [3, 5]), (7, [2, 2])])
def test_cached_equals_the_last_rows_of_a_prompt(prefix, lens):
    L, S, Hq, Hkv = 2, 4, 4, 2
    r = np.random.default_rng(1)
    pool_k, pool_v = r.normal(size=(12, S, Hkv, D)), r.normal(size=(12, S, Hkv, D))
    order = r.permutation(12)
    pp, table = order[:2], order[2:6].reshape(2, 2)
    q = r.normal(size=(2 * L, Hq * D))
    out, _ = ho.cached(q, pool_k, pool_v, pp, prefix, table, lens, L, 0.5)
    for i, n in enumerate(lens):
        k, v = (np.concatenate([x[pp].reshape(-1, Hkv * D)[:prefix], x[table[i]].reshape(-1, Hkv * D)[:n]])
                for x in (pool_k, pool_v))
        full = np.zeros((prefix + n, Hq * D))
        full[-L:] = q[i * L:(i + 1) * L]
        want, _, _ = ho.attention(full, k, v, [0, prefix + n], D, 0.5)
        np.testing.assert_allclose(out[i * L:(i + 1) * L], want[-L:], rtol=1e-12)


def test_cached_row_without_a_key_is_zero():
    r = np.random.default_rng(2)
    pool = r.normal(size=(2, 2, 1, D))
    out, _ = ho.cached(r.normal(size=(3, D)), pool, pool, [], 0, [[0]], [2], 3, 1.0)
    assert (out[0] == 0).all() and (out[1:] != 0).any()


@pytest.mark.parametrize("with_draft", [True, False])
def test_first_token_follows_the_target(with_draft):
    """Whatever the drafts, the first emitted token is distributed as the target's first row."""
    r = np.random.default_rng(5)
    V, n = 5, 40000
    p, q = r.dirichlet(np.ones(V), 2), r.dirichlet(np.ones(V), 1)
    tokens = r.choice(V, size=(n, 1), p=q[0]) if with_draft else np.full((n, 1), 2)
    a, nxt = ho.accept_drafts(np.tile(p, (n, 1)), tokens, r.random((n, 1)), r.random(n), np.tile(q, (n, 1)) if with_draft else None)
    first = np.where(a > 0, tokens[:, 0], nxt)
    freq = np.bincount(first, minlength=V) / n
    # six standard deviations of a binomial share
    assert (np.abs(freq - p[0]) < 6 * np.sqrt(p[0] * (1 - p[0]) / n)).all()


def test_drafts_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1], [0.2, 0.3, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [0.5, 0.25, 0.25]])
    # draft 0: token 1, q = .5, p = .25: kept for u < .5; draft 1: token 0, q = .5, p = .1: kept for u < .2
    a, nxt = ho.accept_drafts(p, [[1, 0]], np.array([[0.49, 0.1]]), [0.6], q)
    assert (a[0], nxt[0]) == (2, 2)
    a, nxt = ho.accept_drafts(p, [[1, 0]], np.array([[0.49, 0.2]]), [0.0], q)
    assert (a[0], nxt[0]) == (1, 1)               # residual (0, .55, 0)
    a, nxt = ho.accept_drafts(p, [[1, 0]], np.array([[0.5, 0.0]]), [0.9], q)
    assert (a[0], nxt[0]) == (0, 0)               # residual (.25, 0, 0)
    a, nxt = ho.accept_drafts(p, [[1, 0]], np.array([[0.3, 0.0]]), [0.5])
    assert (a[0], nxt[0]) == (0, 0)               # greedy draft: row 0 without token 1 = (.5, 0, .25), half of .75
    a, nxt = ho.accept_drafts(p, [[1, 0]], np.array([[0.49, 0.1]]), [0.1], q, num_drafts=[0])
    assert (a[0], nxt[0]) == (0, 0)
