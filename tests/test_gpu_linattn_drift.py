"""Slow decays over thousands of tokens: what one token's decay is off by must not add up.

Bounds are norms for each head.  A token rounds the state a few times by at most U32 of its value;
the roundings of different tokens are independent, so after n tokens a state whose norm does not
fall is off by at most about sqrt(m n) U32 of it, m being the roundings of a token.  A decay that is
itself rounded to fp32 is off the same way every time, by up to n U32."""
import numpy as np
import pytest
import torch

import plain_operators as plain
import ternary_weight_lm_b200 as mmf
from gpu_helpers import DEV, to_dev

pytestmark = pytest.mark.gpu

LG = np.array([-1e-3, -1e-4, -1e-5, -1e-7, -2e-8, 0.0, -0.02, -3.0], dtype=np.float32)


def _states(q, k, v, lg, h0):
    """The state after the last token (64 bits), a token at a time."""
    g = plain.gammas(lg)[:, None, None]
    S = h0.astype(np.float64)
    for t in range(k.shape[0]):
        S = g * S + k[t].astype(np.float64)[:, :, None] * v[t].astype(np.float64)[:, None, :]
    return S


def _check(got, ref, bound):
    for h in range(len(ref)):
        plain.assert_norm(got[h], ref[h], bound, ("head", h))


# three roundings: k v, its sum with the decay's part, the state
@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_thousands_of_steps(dt):
    n, H, d = 4096, len(LG), 64
    rng = np.random.default_rng(41)
    q, k, v = (rng.normal(size=(n, H, d)).astype(dt) for _ in range(3))
    h0 = (rng.normal(size=(H, d, d)) * 60).astype(np.float32)
    dq, dk, dv, lg, state = (to_dev(x) for x in (q, k, v, LG, h0[None]))
    for t in range(n):
        mmf.linattn_step(dq[t:t + 1], dk[t:t + 1], dv[t:t + 1], lg, state)
    torch.cuda.synchronize()
    _check(state[0].cpu().numpy(), _states(q, k, v, LG, h0), np.sqrt(3 * n) * plain.U32)
