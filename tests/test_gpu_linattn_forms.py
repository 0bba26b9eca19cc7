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


def _floor(q, k, v, decay, scale, h0=None):
    """What fp16's smallest step can add to an output of the chunked forms, for one sequence.

    A score's power of two brings its row's largest, or a bound on it, to 2^14 .. 2^15.  The bound is
    at most 2^6 times 128 max|q_i| max_j gamma^(i-j) |k_j| (max|k| of keys within 2^6 of one another;
    else the decayed maximum, of keys rounded up to powers of two); half a step of 2^-24 among the
    subnormals is then at most 2^-25 / 2^14 2^6 = 2^-33 of that, times |v_j|.  A state likewise
    brings its largest value, at most the decayed sum of max|k_j| max|v_j| and the start's, there: at
    most 2^-39 of it, times |q_i|."""
    q, k, v = (np.abs(x.astype(np.float64)) for x in (q, k, v))
    g = plain.gammas(decay)
    reach = np.zeros(len(g))
    state = reach if h0 is None else np.abs(h0[0].astype(np.float64)).max(axis=(1, 2))
    out, vs = np.empty(v.shape), np.zeros(v.shape[1:])
    for t in range(len(q)):
        reach = np.maximum(reach * g, k[t].max(axis=-1))
        state = state * g + k[t].max(axis=-1) * v[t].max(axis=-1)
        vs = vs + v[t]
        out[t] = ((2.0 ** -33 * 128 * q[t].max(axis=-1) * reach)[:, None] * vs +
                  (2.0 ** -39 * q[t].sum(axis=-1) * state)[:, None])
    return scale * out


def _backward_floors(q, k, v, decay, scale, do, h0=None):
    """Of dq, dk and dv, each a sweep of its own."""
    flip = None if h0 is None else np.swapaxes(h0, 2, 3)
    return (_floor(do, v, k, decay, scale, flip),
            _floor(v[::-1], do[::-1], q[::-1], decay, scale)[::-1],
            _floor(k[::-1], q[::-1], do[::-1], decay, scale)[::-1])


# A key far larger than the rest, of a later token or of one that has decayed away, must not cost the
# others their bits: all values within their own bounds.  Backwards the keys are dout (for dk) and q
# (for dv), and later tokens come first.
@pytest.mark.parametrize("d", [128, 64, 40])
@pytest.mark.parametrize("lg", [0.0, -0.7])
def test_a_large_key_does_not_cost_others_their_bits(d, lg):
    T, H, at, scale = 200, 2, 100, 2.0 ** -8    # the largest results stay below fp16's 65504
    q, k, v, _ = _make(T, H, d, d, np.float16, seed=60)
    do = np.roll(v, 5, axis=0)
    small = np.float16(1e-4)
    decay = np.full(H, lg, dtype=np.float32)
    kk, qq, dd = k * small, q * small, do * small
    for x in (kk, qq, dd):
        x[at, :, 7] = 60000.0
    o = mmf.linattn_forward(to_dev(q), to_dev(kk), to_dev(v), to_dev(decay), scale=scale)
    ref, _ = plain.linattn(q, kk, v, decay, [0, T], scale)
    mag, _ = plain.absolute(plain.linattn, q, kk, v, decay, [0, T], scale)
    plain.assert_close(o.cpu().numpy(), ref, plain.tolerance(ref, mag, True, T, d) +
                       _floor(q, kk, v, decay, scale), "o")
    for q, k, v, do in ((q, k, v, dd), (qq, k, v, do)):
        got = mmf.linattn_backward(*(to_dev(x) for x in (q, k, v, decay, do)), scale=scale)
        a = (q, k, v, decay, [0, T], scale, do)
        mags = plain.absolute(plain.linattn_backward, *a)
        floors = _backward_floors(q, k, v, decay, scale, do)
        for name, x, ref, mag, low in zip(("dq", "dk", "dv"), got, plain.linattn_backward(*a), mags, floors):
            plain.assert_close(x.cpu().numpy(), ref, plain.tolerance(ref, mag, True, T, d) + low, name)


# Rows of zeros where the rest of a chunk has decayed away, as padding with zeros has them; and
# gradients far below 1 of a length that no chunk divides.  (Where only v is zero, the scores of those
# tokens are what the others' step is set by: _floor.)
@pytest.mark.parametrize("d", [128, 64, 40])
@pytest.mark.parametrize("lg", [-0.1, -0.7, -3.0])
@pytest.mark.parametrize("zero", ["k", "v", "kv", "qkv", ""])
def test_rows_of_zeros_and_small_gradients(d, lg, zero):
    T, H, scale = 210, 2, 0.1
    q, k, v, h0 = _make(T, H, d, d, np.float16, seed=70, h0=True)
    do = np.roll(v, 5, axis=0) * np.float16(1e-3)
    for name, x in (("q", q), ("k", k), ("v", v)):
        if name in zero:
            x[30:64] = 0
            x[90:200] = 0
    decay = np.full(H, lg, dtype=np.float32)
    a = (q, k, v, decay, [0, T], scale)
    hT = torch.empty(1, H, d, d, device=DEV)
    o = mmf.linattn_forward(*(to_dev(x) for x in a[:4]), scale=scale, h0=to_dev(h0), hT=hT)
    ref, refT = plain.linattn(*a, h0)
    mag, magT = plain.absolute(plain.linattn, *a, h0=h0)
    plain.assert_close(o.cpu().numpy(), ref, plain.tolerance(ref, mag, True, T, d) +
                       _floor(q, k, v, decay, scale, h0), "o")
    plain.assert_close(hT.cpu().numpy(), refT, plain.sum_bound(T, d) * magT, "hT")
    for grad in (do, np.where(np.arange(T)[:, None, None] % 70 < 30, do, do * 0)):
        got = mmf.linattn_backward(*(to_dev(x) for x in (*a[:4], grad)), scale=scale,
                                   h0=to_dev(h0), want_dh0=True)
        refs = plain.linattn_backward(*a, grad, h0)
        mags = plain.absolute(plain.linattn_backward, *a, grad, h0=h0)
        floors = _backward_floors(q, k, v, decay, scale, grad, h0)
        for name, x, r, m, low in zip(("dq", "dk", "dv", "dh0"), got, refs, mags, (*floors, 0.0)):
            plain.assert_close(x.cpu().numpy(), r, plain.tolerance(r, m, name != "dh0", T, d) + low, name)


# bounds that descend, overlap or leave the tokens, for every kernel, whole and in segments (heads of
# 128 take their rows by tensor map): nothing outside the outputs is touched, and it is reported
@pytest.mark.parametrize("cu", [[0, 500, 200, 600], [-50, 100, 700, 9000], [600, 0, 600, 0],
                                [2147483647, -2147483648, 5, 9], [0, 4000, 0, 4000, 0, 4000]])
@pytest.mark.parametrize("T", [600, 4000])
@pytest.mark.parametrize("dt,d", [(np.float16, 128), (np.float16, 64), (np.float16, 24),
                                  (np.float32, 128)])
def test_bad_bounds_forwards_and_backwards(cu, T, dt, d):
    H, B, pad = 2, len(cu) - 1, 300
    q, k, v, h0 = _make(T, H, d, d, dt, seed=2, B=B, h0=True)
    dq, dk, dv, lg = (to_dev(x) for x in (q, k, v, _decays(H)))
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if T == 4000:
        assert _need(dq, dk, dv, lg, cu=cud) > 0
        assert _need(dq, dk, dv, lg, cu=cud, dout=dv) > 0
    rows = [torch.full((T + 2 * pad, H, d), 7.0, dtype=dq.dtype, device=DEV) for _ in range(4)]
    o, gq, gk, gv = (x[pad:-pad] for x in rows)
    states = [torch.full((B + 2, H, d, d), 7.0, device=DEV) for _ in range(3)]
    s0, sT, ds = (x[1:-1] for x in states)
    s0.copy_(to_dev(h0))
    mmf.linattn_forward(dq, dk, dv, lg, cu_seqlens=cud, h0=s0, hT=sT, out=o)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 8
    # into buffers with guards, which the convenience does not take
    d_ = mmf._linattn(dq, dk, dv, lg, dv, None, cud, None)
    need = mmf.mmf_linattn_backward_workspace_bytes(d_)
    ws = mmf.workspace(need) if need else None
    mmf.mmf_linattn_backward(d_, dq, dk, dv, dv, s0, sT, gq, gk, gv, ds, ws)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 8
    for x in rows:
        assert bool((x[:pad] == 7).all()) and bool((x[-pad:] == 7).all())
    for x in states:
        assert bool((x[0] == 7).all()) and bool((x[-1] == 7).all())
    assert torch.equal(s0, to_dev(h0))


# Which calls are cut into segments: few heads of a long prompt, not many of them nor a short one
@pytest.mark.parametrize("T,H,d,split", [
    (2700, 40, 128, True), (1300, 300, 128, False), (300, 4, 128, False),
    (2700, 40, 64, True), (4000, 8, 64, True), (1300, 444, 64, False), (100, 4, 64, False)])
def test_which_calls_are_split(T, H, d, split):
    g = torch.Generator(device=DEV).manual_seed(T)
    q, k, v = (torch.randn(T, H, d, generator=g, device=DEV).half() for _ in range(3))
    lg, heads = to_dev(_decays(H)), [0, 1, H - 1]
    assert (_need(q, k, v, lg) > 0) == split
    o = mmf.linattn_forward(q, k, v, lg)
    a = [x[:, heads].cpu().numpy() for x in (q, k, v)]
    ref, _ = plain.linattn(*a, _decays(H)[heads], [0, T], d ** -0.5)
    mag, _ = plain.absolute(plain.linattn, *a, _decays(H)[heads], [0, T], d ** -0.5)
    got = o[:, heads].cpu().numpy()
    plain.assert_close(got, ref, plain.tolerance(ref, mag, True, T, d), "o")
