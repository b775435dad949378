"""Pins of the few-token layer's oracle: scalar loops, the layer built from the
other oracles' pieces, and masked logits."""

import math

import numpy as np

from oracle import router, tokens


def test_layer_against_scalar_loops():
    g = np.random.default_rng(0)
    T, H, F, E, k = 3, 4, 5, 6, 2
    x, w1, w2 = g.standard_normal((T, H)), g.standard_normal((E, 2 * F, H)), g.standard_normal((E, H, F))
    lg = g.standard_normal((T, E)).astype(np.float32)
    res = g.standard_normal((T, H))
    out, bound = tokens.layer(x, lg, w1, w2, k, res)
    for t in range(T):
        ids = sorted(range(E), key=lambda e: -lg[t, e])[:k]
        z = [math.exp(float(lg[t, e])) for e in ids]
        for n in range(H):
            want = res[t, n]
            for e, ze in zip(ids, z):
                for f in range(F):
                    gate = sum(w1[e, f, i] * x[t, i] for i in range(H))
                    up = sum(w1[e, F + f, i] * x[t, i] for i in range(H))
                    want += ze / sum(z) * w2[e, n, f] * gate / (1 + math.exp(-gate)) * up
            assert abs(out[t, n] - want) < 1e-12
    assert (bound > 0).all() and (bound < 0.2 * (1 + np.abs(out))).all()


def test_choice_is_the_routers_without_masked_experts():
    g = np.random.default_rng(1)
    lg = g.standard_normal((20, 9)).astype(np.float32)
    lg[:5, 3] = lg[:5, 7]
    ids, w = router.route_topk(lg, 4)
    for t, (i, wt) in enumerate(tokens.choose(lg, 4)):
        assert i == ids[t].tolist() and np.allclose(wt, w[t], rtol=1e-14)
    lg[2, :] = -np.inf
    lg[3, 2:] = -np.inf
    got = tokens.choose(lg, 4)
    assert got[2][0] == [] and sorted(got[3][0]) == [0, 1] and abs(got[3][1].sum() - 1) < 1e-15
    out, bound = tokens.layer(np.ones((20, 2)), lg, np.ones((9, 4, 2)), np.ones((9, 2, 2)), 4)
    assert (out[2] == 0).all() and (bound[2] <= 2.0 ** -126).all()
