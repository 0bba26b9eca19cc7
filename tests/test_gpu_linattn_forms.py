"""GPU tests of which kernel a linear attention call takes, whole and in segments, and of bounds that
it cannot follow.  Tolerances as in test_gpu_linattn."""
import numpy as np
import pytest
import torch

import plain_operators as plain
import ternary_weight_lm_b200 as mmf
from gpu_helpers import DEV, to_dev
from test_gpu_linattn import _check_backward, _decays, _make

pytestmark = pytest.mark.gpu


def _need(q, k, v, lg, cu=None, dout=None):
    d = mmf._linattn(q, k, v, lg, dout, None, cu, None)
    return (mmf.mmf_linattn_workspace_bytes if dout is None else
            mmf.mmf_linattn_backward_workspace_bytes)(d)


# sizes and strides that rule out a tensor-core form, in prompts long enough for segments: one value
# row for all tokens, and heads that only the forward's order of sizes has on the tensor cores
@pytest.mark.parametrize("dk,dv,shared", [(128, 128, True), (64, 192, False), (64, 64, True)])
def test_long_prompts_of_other_forms(dk, dv, shared):
    T, H = 3000, 2
    q, k, v, h0 = _make(T, H, dk, dv, np.float16, seed=50, h0=True)
    do, dhT = np.roll(v, 3, axis=0), np.roll(h0, 1, axis=3)
    if shared:
        v[:] = v[:1]
    dq, dk_, dd, lg = (to_dev(x) for x in (q, k, do, _decays(H)))
    dvv = to_dev(v[:1]).expand(T, H, dv) if shared else to_dev(v)
    assert _need(dq, dk_, dvv, lg) > 0 and _need(dq, dk_, dvv, lg, dout=dd) > 0
    hT = torch.empty(1, H, dk, dv, device=DEV)
    o = mmf.linattn_forward(dq, dk_, dvv, lg, scale=0.1, h0=to_dev(h0), hT=hT)
    got = mmf.linattn_backward(dq, dk_, dvv, lg, dd, scale=0.1, h0=to_dev(h0), dhT=to_dev(dhT),
                               want_dh0=True)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    a = (q, k, v, _decays(H), [0, T], 0.1)
    ref, refT = plain.linattn(*a, h0)
    mag, magT = plain.absolute(plain.linattn, *a, h0=h0)
    plain.assert_close(o.cpu().numpy(), ref, plain.tolerance(ref, mag, True, T, dk), "o")
    plain.assert_close(hT.cpu().numpy(), refT, plain.sum_bound(T, dk) * magT, "hT")
    _check_backward(got, *a, do, h0, dhT, norms=False)


# whole and in segments; almost every token outside, and none
@pytest.mark.parametrize("T,cu", [(300, [3, 40, 170]), (5000, [4000, 4000, 4010]),
                                  (3000, [0, 2900, 2900]), (300, [7, 7]), (200, [0, 200])])
@pytest.mark.parametrize("dt,dk,dv", [(np.float16, 128, 128), (np.float16, 64, 64),
                                      (np.float16, 64, 128), (np.float16, 8, 24),
                                      (np.float32, 200, 40)])
def test_rows_outside_the_sequences_are_zero(T, cu, dt, dk, dv):
    H = 2
    q, k, v, _ = _make(T, H, dk, dv, dt, seed=T)
    do = np.roll(v, 1, axis=0)
    for x in (q, k, v, do):
        x[:cu[0]] = np.nan
        x[cu[-1]:] = np.nan
    dq, dk_, dvv, dd, lg = (to_dev(x) for x in (q, k, v, do, _decays(H)))
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    # memory that the outputs will lie in, full of what must not stay
    rest = [torch.full((T, H, max(dk, dv)), float("nan"), dtype=dq.dtype, device=DEV)
            for _ in range(4)]
    del rest
    o = mmf.linattn_forward(dq, dk_, dvv, lg, cu_seqlens=cud)
    grads = mmf.linattn_backward(dq, dk_, dvv, lg, dd, cu_seqlens=cud)[:3]
    given = torch.full_like(o, 9.0)
    mmf.linattn_forward(dq, dk_, dvv, lg, cu_seqlens=cud, out=given)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    for x in (o, *grads):
        assert bool((x[:cu[0]] == 0).all()) and bool((x[cu[-1]:] == 0).all())
    assert bool((given[:cu[0]] == 9).all()) and bool((given[cu[-1]:] == 9).all())
    assert torch.equal(given[cu[0]:cu[-1]], o[cu[0]:cu[-1]])
    assert bool(torch.isfinite(o).all())
