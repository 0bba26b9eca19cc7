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


def _backward_states(q, do, lg, scale, dhT):
    """The gradient of the state before the first token (64 bits)."""
    g = plain.gammas(lg)[:, None, None]
    U = dhT.astype(np.float64)
    for t in range(q.shape[0] - 1, -1, -1):
        U = g * (U + scale * q[t].astype(np.float64)[:, :, None] * do[t].astype(np.float64)[:, None, :])
    return U


# Every form of the sweep, in one segment (heads enough to fill the GPU; they share their rows) and
# in many.  The chunked forms round a state twice for each chunk of at least 64 tokens, and what a
# chunk adds has an error of its own, less than 2e-6 of it (as in the tests of prompts); the
# token-by-token form rounds it twice for each token, and what is added once.
@pytest.mark.parametrize("dt,d,T,H,split", [
    (np.float16, 128, 16384, 148, False), (np.float16, 128, 16384, 8, True),
    (np.float16, 64, 16384, 444, False), (np.float16, 64, 16384, 8, True),
    (np.float32, 64, 8192, 444, False), (np.float32, 64, 8192, 8, True)])
def test_long_prompts(dt, d, T, H, split):
    n = len(LG)
    rng = np.random.default_rng(T + d + H)
    x = [rng.normal(size=(T, d)).astype(dt) for _ in range(4)]
    h0, dhT = ((rng.normal(size=(n, d, d)) * 100).astype(np.float32) for _ in range(2))
    q, k, v, do = (to_dev(a)[:, None].expand(T, H, d) for a in x)
    do = do.contiguous()
    lg = to_dev(np.resize(LG, H))
    s0, sT = (torch.zeros(1, H, d, d, device=DEV) for _ in range(2))
    s0[0, :n], sT[0, :n] = to_dev(h0), to_dev(dhT)
    need = mmf.mmf_linattn_workspace_bytes(mmf._linattn(q, k, v, lg, None, None, None, None))
    assert (need > 0) == split
    hT = torch.empty_like(s0)
    mmf.linattn_forward(q, k, v, lg, h0=s0, hT=hT)
    dh0 = mmf.linattn_backward(q, k, v, lg, do, scale=0.1, dhT=sT, want_dh0=True)[3]
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    bound = 2e-6 + np.sqrt(2 * T / 64) * plain.U32 if dt == np.float16 else np.sqrt(3 * T) * plain.U32
    a = [np.broadcast_to(y[:, None], (T, n, d)) for y in x]
    _check(hT[0, :n].cpu().numpy(), _states(*a[:3], LG, h0), bound)
    _check(dh0[0, :n].cpu().numpy(), _backward_states(a[0], a[3], LG, 0.1, dhT), bound)
