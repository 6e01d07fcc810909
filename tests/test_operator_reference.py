"""The 64-bit references of the decode and backward tests against the oracle's
token recurrence and against central differences (CPU)."""
import numpy as np
import pytest
import torch

import operator_reference as R
import oracle
from helpers import f64


def _case(lens, Hk=1, Hv=2, d=8, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    q, k, v, g, beta = R.rows(gen, T, Hk, Hv, d)
    return (q, k, v, g, beta, torch.randn(T, Hv, d, generator=gen),
            torch.randn(N, Hv, d, d, generator=gen) * 0.3,
            torch.randn(N, Hv, d, d, generator=gen) * 0.3)


@pytest.mark.parametrize("lens", [[5], [3, 0, 1, 7]])
def test_forward_is_the_oracle(lens):
    q, k, v, g, beta, _, h0, _ = _case(lens)
    o, hT = R.forward(q, k, v, g, beta, lens, h0, scale=0.7)
    o_ref, h_ref = oracle.gdn_token(f64(q), f64(k), f64(v), f64(g), f64(beta),
                                    np.array(R.offsets(lens)), f64(h0), scale=0.7)
    np.testing.assert_allclose(o.numpy(), o_ref, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(hT.numpy(), h_ref, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("lens", [[6], [3, 0, 1, 4]])
def test_backward_against_differences_of_the_oracle(lens):
    q, k, v, g, beta, do, h0, dhT = _case(lens, seed=1)
    grads = R.backward(q, k, v, g, beta, lens, do, h0, dhT, scale=0.7)
    base = [f64(x) for x in (q, k, v, g, beta, h0)]
    cu = np.array(R.offsets(lens))

    def loss(x):
        o, hT = oracle.gdn_token(*x[:5], cu, x[5], scale=0.7)
        return float((o * f64(do)).sum() + (hT * f64(dhT)).sum())

    rng = np.random.default_rng(2)
    for i, gr in enumerate(grads):
        for _ in range(3):
            step = rng.standard_normal(base[i].shape)
            eps = 1e-5
            up, down = list(base), list(base)
            up[i], down[i] = base[i] + eps * step, base[i] - eps * step
            diff = (loss(up) - loss(down)) / (2 * eps)
            want = float((gr.numpy() * step).sum())
            # the differences' own error: eps^2 times third derivatives, and 1e-16 / eps
            assert abs(diff - want) <= 1e-7 * (1.0 + np.linalg.norm(gr.numpy()) *
                                               np.linalg.norm(step)), i
