"""GPU parity of the linear attention with a decay for each head (whole prompts, single tokens,
gradients) against its plain 64-bit form.

Tolerances are element-wise and come from the arithmetic (plain_operators.tolerance): relative to
the sum of the magnitudes of a value's terms for what is rounded before the sum, to the value for
the output's own rounding.  Beside them, where the terms are many and their signs random, the
2-norm of the errors: fp16 outputs have one rounding of up to 2^-11 of the value and two operands
rounded alike, so less than 2 * 2^-11 of the result's norm; fp32 results less than 2e-6 (their
roundings of 2^-24 each, over at most a few hundred tokens, add up in quadrature)."""
import numpy as np
import pytest
import torch

import plain_operators as plain
import ternary_weight_lm_b200 as mmf
from gpu_helpers import DEV, to_dev

pytestmark = pytest.mark.gpu

LG = np.array([-0.25, -0.02, -2.0 ** -9, 0.0, -3.0, -1e-4, -0.7, -0.1], dtype=np.float32)


def _decays(H):
    return np.resize(LG, H)


def _make(T, H, dk, dv, dt, seed, B=1, h0=False):
    rng = np.random.default_rng(seed)
    q, k = (rng.normal(size=(T, H, dk)).astype(dt) for _ in range(2))
    v = rng.normal(size=(T, H, dv)).astype(dt)
    s = (rng.normal(size=(B, H, dk, dv)) * 2).astype(np.float32) if h0 else None
    return q, k, v, s


def _dev(x):
    return None if x is None else to_dev(x)


def _forward(q, k, v, lg, scale, cu=None, batch=None, h0=None, **kw):
    B = len(cu) - 1 if cu is not None else (batch or 1)
    T, H, dk = q.shape
    hT = torch.full((B, H, dk, v.shape[2]), 99.0, device=DEV)
    out = torch.full((T, H, v.shape[2]), 55.0, device=DEV,
                     dtype=torch.from_numpy(v[:1]).dtype)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    mmf.linattn_forward(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), scale=scale, cu_seqlens=cud,
                        batch=batch, h0=_dev(h0), hT=hT, out=out, **kw)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    return out.cpu().numpy(), hT.cpu().numpy()


def _check_forward(o, hT, q, k, v, lg, cu, scale, h0, norms=True):
    f16 = q.dtype == np.float16
    far, d = max(b - a for a, b in zip(cu, cu[1:])), q.shape[2]
    ref, refT = plain.linattn(q, k, v, lg, cu, scale, h0)
    mag, magT = plain.absolute(plain.linattn, q, k, v, lg, cu, scale, h0=h0)
    plain.assert_close(o, ref, plain.tolerance(ref, mag, f16, far, d), "o")
    plain.assert_close(hT, refT, plain.sum_bound(far, d) * magT, "hT")
    untouched = np.isnan(ref)
    assert (o[untouched] == 55.0).all()
    if norms:
        plain.assert_norm(o, ref, 2 * plain.U16 if f16 else 2e-6, "o")
        plain.assert_norm(hT, refT, 2e-6, "hT")


# one token, two, around a tile of 16, 64 and 128 tokens, odd lengths; equal and unequal head
# sizes, the ones with their own tile and the others, up to 256
@pytest.mark.parametrize("T,H,dk,dv", [
    (1, 2, 128, 128), (2, 3, 64, 64), (15, 2, 64, 128), (16, 1, 128, 64), (17, 2, 8, 8),
    (63, 2, 128, 128), (64, 2, 64, 64), (65, 2, 128, 128), (127, 1, 64, 64), (128, 2, 128, 128),
    (129, 3, 64, 64), (200, 5, 96, 40), (300, 8, 128, 128), (300, 8, 64, 64), (70, 2, 256, 256),
    (90, 2, 200, 136), (130, 2, 64, 256), (130, 2, 128, 192), (257, 2, 16, 128)])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_forward_matches_plain_form(T, H, dk, dv, dt):
    q, k, v, h0 = _make(T, H, dk, dv, dt, seed=T + dk, h0=T % 2 == 1)
    lg, scale = _decays(H), dk ** -0.5
    o, hT = _forward(q, k, v, lg, scale, h0=h0)
    _check_forward(o, hT, q, k, v, lg, [0, T], scale, h0)


# lengths of none and of one, bounds inside a tile, tokens before the first and behind the last
# sequence; with and without a start state
@pytest.mark.parametrize("cu", [
    [0, 40], [3, 3, 4, 70, 70, 199, 199], [0, 1, 2, 3, 130, 259], [0, 0, 0], [5, 300],
    [0, 128, 256, 300], [0, 64, 65, 192]])
@pytest.mark.parametrize("dk,dv,dt", [(64, 64, np.float16), (128, 128, np.float16),
                                      (24, 40, np.float16), (128, 96, np.float32)])
@pytest.mark.parametrize("h0", [False, True])
def test_ragged_batches(cu, dk, dv, dt, h0):
    T, H, B = 300, 4, len(cu) - 1
    q, k, v, s = _make(T, H, dk, dv, dt, seed=len(cu), B=B, h0=h0)
    # what lies outside the sequences must not be looked at
    for x in (q, k, v):
        x[:cu[0]] = np.nan
        x[cu[-1]:] = np.inf
    lg = _decays(H)
    o, hT = _forward(q, k, v, lg, 0.3, cu=cu, h0=s)
    _check_forward(o, hT, q, k, v, lg, cu, 0.3, s, norms=False)


def _finite(x):
    return np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)


@pytest.mark.parametrize("d", [64, 128, 40])
def test_infinities_and_nan_stay_in_their_sequence(d):
    T, H, cu, lg = 400, 2, [0, 70, 270, 400], _decays(2)
    q, k, v, _ = _make(T, H, d, d, np.float16, seed=1)
    ref, refT = plain.linattn(q, k, v, lg, cu, 0.125)
    mag, magT = plain.absolute(plain.linattn, q, k, v, lg, cu, 0.125)
    tol = plain.tolerance(ref, mag, True, 200, d)
    q[100:110], k[90], v[95] = np.inf, np.nan, -np.inf
    o, hT = _forward(q, k, v, lg, 0.125, cu=cu)
    # other sequences, and the tokens before the first bad one
    keep = np.r_[0:90, 270:400]
    plain.assert_close(o[keep], ref[keep], tol[keep], "o")
    plain.assert_close(hT[[0, 2]], refT[[0, 2]], plain.sum_bound(130, d) * magT[[0, 2]], "hT")
    # a key that is not a number reaches every output from its token on
    assert not np.isfinite(o[90:270]).any()


# in one segment, and in the first of several; or in the state that the prompt starts from
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("d", [64, 128, 40])
@pytest.mark.parametrize("T,where", [(300, "v"), (3000, "v"), (300, "h0"), (3000, "h0")])
def test_a_bad_value_stays_in_its_column(T, where, d, bad):
    H, lg, col = 2, _decays(2), 5
    q, k, v, h0 = _make(T, H, d, d, np.float16, seed=2, h0=True)
    at = 141 if where == "v" else 0
    if where == "v":
        v[at, 1, col] = bad
    else:
        h0[0, 1, 3, col] = bad
    o, hT = _forward(q, k, v, lg, 0.125, h0=h0)
    a = (q, k, _finite(v), lg, [0, T], 0.125)
    ref, refT = plain.linattn(*a, _finite(h0))
    mag, magT = plain.absolute(plain.linattn, *a, h0=_finite(h0))
    tol, tolT = plain.tolerance(ref, mag, True, T, d), plain.sum_bound(T, d) * magT
    assert not np.isfinite(o[at:at + 20, 1, col]).any()
    assert not np.isfinite(hT[0, 1, :, col]).all()
    ref[at:, 1, col], refT[0, 1, :, col] = np.nan, np.nan      # not compared
    o[at:, 1, col] = 0.0
    plain.assert_close(o, ref, tol, "o")
    plain.assert_close(hT, refT, tolT, "hT")


@pytest.mark.parametrize("dt,d", [(np.float16, 64), (np.float16, 128), (np.float32, 64)])
def test_every_decay(dt, d):
    # none, total, invalid (counted as none), and one whose powers underflow within a tile
    lg = np.array([0.0, -np.inf, 0.5, np.nan, -20.0, -1e-7, -88.0, -300.0], dtype=np.float32)
    T, H = 150, len(lg)
    q, k, v, h0 = _make(T, H, d, d, dt, seed=4, h0=True)
    o, hT = _forward(q, k, v, lg, 1.0, h0=h0)
    _check_forward(o, hT, q, k, v, lg, [0, T], 1.0, h0)


@pytest.mark.parametrize("d", [64, 128])
def test_large_and_small_values(d):
    # scores beyond fp16's largest value, states beyond it, and values among its subnormals
    T, H = 140, 3
    rng = np.random.default_rng(8)
    q, k, v, h0 = _make(T, H, d, d, np.float16, seed=8, h0=True)
    for big_q, big_k, big_v in ((300.0, 300.0, 0.01), (0.01, 900.0, 900.0), (1e-4, 1.0, 1.0),
                                (1.0, 2e-4, 3e-5), (1.0, 1.0, 1e-6)):
        qq, kk, vv = ((x.astype(np.float32) * m).astype(np.float16)
                      for x, m in ((q, big_q), (k, big_k), (v, big_v)))
        ref, _ = plain.linattn(qq, kk, vv, _decays(H), [0, T], 1.0, h0)
        scale = float(2.0 ** -np.ceil(np.log2(max(np.abs(ref).max(), 1e-30) / 2.0 ** 12)))
        o, hT = _forward(qq, kk, vv, _decays(H), scale, h0=h0)
        _check_forward(o, hT, qq, kk, vv, _decays(H), [0, T], scale, h0, norms=False)


@pytest.mark.parametrize("dt,d", [(np.float16, 128), (np.float16, 64), (np.float32, 64)])
@pytest.mark.parametrize("cu", [None, [0, 1500, 1500, 1501, 4000]])
def test_split_sequences(dt, d, cu):
    # long enough for every sequence to be cut into segments, and for a chunked form to be needed
    # for the reference: states at the segment bounds come from the plain form
    T, H = 4000, 2
    q, k, v, h0 = _make(T, H, d, d, dt, seed=6, B=1 if cu is None else 4, h0=True)
    o, hT = _forward(q, k, v, _decays(H), 0.1, cu=cu, h0=h0)
    _check_forward(o, hT, q, k, v, _decays(H), cu or [0, T], 0.1, h0)


# segments of many chunks: unsplit sequences (enough heads to fill the GPU), with and without a
# state as an output, and split ones; a few heads against the plain form
@pytest.mark.parametrize("T,H,split", [(1300, 300, False), (2700, 40, True)])
@pytest.mark.parametrize("d,state", [(128, True), (128, False), (64, True)])
def test_long_segments(T, H, split, d, state):
    heads = [0, 5, H - 1]
    g = torch.Generator(device=DEV).manual_seed(H)
    q, k, v = (torch.randn(T, H, d, generator=g, device=DEV).half() for _ in range(3))
    do = torch.randn(T, H, d, generator=g, device=DEV).half()
    lg, hT = _decays(H), torch.empty(1, H, d, d, device=DEV) if state else None
    assert (mmf.mmf_linattn_workspace_bytes(mmf._linattn(q, k, v, to_dev(lg), None, None, None,
                                                         None)) > 0) == split or d == 64
    o = mmf.linattn_forward(q, k, v, to_dev(lg), hT=hT)
    grads = mmf.linattn_backward(q, k, v, to_dev(lg), do, want_dh0=state)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    a = [x[:, heads].cpu().numpy() for x in (q, k, v, do)]
    ref, refT = plain.linattn(*a[:3], lg[heads], [0, T], d ** -0.5)
    mag, magT = plain.absolute(plain.linattn, *a[:3], lg[heads], [0, T], d ** -0.5)
    got = o[:, heads].cpu().numpy()
    plain.assert_close(got, ref, plain.tolerance(ref, mag, True, T, d), "o")
    plain.assert_norm(got, ref, 2 * plain.U16, "o")
    if state:
        got = hT[:, heads].cpu().numpy()
        plain.assert_close(got, refT, plain.sum_bound(T, d) * magT, "hT")
        plain.assert_norm(got, refT, 2e-6, "hT")
    grads = [x if x is None else x[:, heads] for x in grads]
    ref = plain.linattn_backward(*a[:3], lg[heads], [0, T], d ** -0.5, a[3])
    for name, x, r in zip(("dq", "dk", "dv", "dh0"), grads, ref):
        if x is not None:
            plain.assert_norm(x.cpu().numpy(), r, 2e-6 if name == "dh0" else 2 * plain.U16, name)


@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_equal_batches_and_in_place_states(dt):
    T, H, d, B = 1800, 2, 64, 3
    q, k, v, h0 = _make(T, H, d, d, dt, seed=7, B=B, h0=True)
    lg = _decays(H)
    state = to_dev(h0)
    o = mmf.linattn_forward(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), batch=B, h0=state,
                            hT=state)
    torch.cuda.synchronize()
    _check_forward(o.cpu().numpy(), state.cpu().numpy(), q, k, v, lg, [0, 600, 1200, 1800],
                   d ** -0.5, h0)


def _views(dt, T, H, d):
    """q, k, v as views: of one packed projection, of head-major tensors, of shared heads."""
    g = torch.Generator(device=DEV).manual_seed(3)
    packed = torch.randn(T, 3, H, d, generator=g, device=DEV).to(dt)
    heads = torch.randn(3, H, T, d, generator=g, device=DEV).to(dt)
    wide = torch.randn(T, H * d * 3 + 40, generator=g, device=DEV).to(dt)
    one = torch.randn(T, 1, d, generator=g, device=DEV).to(dt)
    return [tuple(packed[:, i] for i in range(3)),
            tuple(heads[i].transpose(0, 1) for i in range(3)),
            tuple(wide[:, 8 + i * H * d:8 + (i + 1) * H * d].view(T, H, d) for i in range(3)),
            (packed[:, 0], one.expand(T, H, d), one.expand(T, H, d)),
            # one row for every token
            (packed[:, 0], heads[0, :, :1].transpose(0, 1).expand(T, H, d), packed[:, 2])]


@pytest.mark.parametrize("dt,d", [(torch.float16, 64), (torch.float16, 128),
                                  (torch.float32, 64)])
@pytest.mark.parametrize("i", range(5))
def test_layouts(dt, d, i):
    T, H = 150, 4
    q, k, v = _views(dt, T, H, d)[i]
    lg = to_dev(_decays(H))
    want = mmf.linattn_forward(*(x.contiguous() for x in (q, k, v)), lg)
    out = torch.empty(H, T, d, dtype=dt, device=DEV).transpose(0, 1)
    mmf.linattn_forward(q, k, v, lg, out=out)
    do = torch.randn(T, H, d, device=DEV).to(dt)
    grads = mmf.linattn_backward(*(x.contiguous() for x in (q, k, v)), lg, do, want_dh0=True)
    got = mmf.linattn_backward(q, k, v, lg, do.transpose(0, 1).contiguous().transpose(0, 1),
                               want_dh0=True)
    if i == 4 and d == 128:
        # A row that every token shares has no tensor map, so heads of 128 take the kernel of the
        # other sizes for it.  Its roundings are in other places: each result is within its bound of
        # the plain form, which is what both are held to.
        a = [x.contiguous().cpu().numpy() for x in (q, k, v, do)]
        for o in (out, want):
            ref, _ = plain.linattn(*a[:3], _decays(H), [0, T], d ** -0.5)
            mag, _ = plain.absolute(plain.linattn, *a[:3], _decays(H), [0, T], d ** -0.5)
            plain.assert_close(o.contiguous().cpu().numpy(), ref,
                               plain.tolerance(ref, mag, True, T, d), "o")
        for x in (grads, got):
            _check_backward(x, *a[:3], _decays(H), [0, T], d ** -0.5, a[3], None, None, norms=False)
        return
    assert torch.equal(out.contiguous(), want)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 24])
def test_strides_of_single_tokens_and_heads_do_not_matter(d):
    lg = to_dev(_decays(1))
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(3, 1, 1, d, generator=g, device=DEV).half()
    q, k, v = (a.as_strided((1, 1, d), (1, 3, 1)) for a in x)
    out = torch.empty(d, dtype=torch.float16, device=DEV).as_strided((1, 1, d), (5, 7, 1))
    want = mmf.linattn_forward(*x, lg)
    mmf.linattn_forward(q, k, v, lg, out=out)
    assert torch.equal(out.reshape(-1), want.reshape(-1))


def test_strides_of_part_vectors_are_refused():
    T, H, d = 20, 2, 64
    wide = torch.zeros(T, 3 * H * d + 4, dtype=torch.float16, device=DEV)
    q = wide[:, :H * d].view(T, H, d)
    lg = to_dev(_decays(H))
    with pytest.raises(mmf.MMFError, match="ALIGNMENT"):
        mmf.linattn_forward(q, q, q, lg)
    q = torch.zeros(T * H * d + 8, dtype=torch.float16, device=DEV)[4:-4].view(T, H, d)
    with pytest.raises(mmf.MMFError, match="ALIGNMENT"):
        mmf.linattn_forward(q, q, q, lg)


@pytest.mark.parametrize("cu", [[0, 500, 200, 600], [-50, 100, 700, 3000], [600, 0, 600, 0],
                                [2147483647, -2147483648, 5, 9], [0, 600, 0, 600]])
@pytest.mark.parametrize("d", [64, 24])
def test_bad_bounds_are_reported_and_touch_nothing_else(cu, d):
    T, H = 600, 2
    q, k, v, _ = _make(T, H, d, d, np.float16, seed=2)
    guard = torch.full((T + 400, H, d), 7.0, dtype=torch.float16, device=DEV)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    mmf.linattn_forward(to_dev(q), to_dev(k), to_dev(v), to_dev(_decays(H)), cu_seqlens=cud,
                        out=guard[200:-200])
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 8
    assert bool((guard[:200] == 7.0).all()) and bool((guard[-200:] == 7.0).all())


# ------------------------------------------------------------------------------------ steps
@pytest.mark.parametrize("B,H,dk,dv", [(1, 2, 128, 128), (3, 4, 64, 64), (5, 3, 96, 40),
                                       (2, 2, 256, 256), (7, 1, 8, 8), (4, 2, 64, 200),
                                       (33, 8, 128, 128)])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
def test_step_matches_plain_form(B, H, dk, dv, dt):
    q, k, v, h0 = _make(B, H, dk, dv, dt, seed=B + dk, B=B, h0=True)
    state = to_dev(h0)
    o = mmf.linattn_step(to_dev(q), to_dev(k), to_dev(v), to_dev(_decays(H)), state, scale=0.3)
    torch.cuda.synchronize()
    cu = list(range(B + 1))
    ref, refT = plain.linattn(q, k, v, _decays(H), cu, 0.3, h0)
    mag, magT = plain.absolute(plain.linattn, q, k, v, _decays(H), cu, 0.3, h0=h0)
    tol = plain.tolerance(ref, mag, dt == np.float16, 1, dk, tensor_cores=False)
    plain.assert_close(o.cpu().numpy(), ref, tol, "o")
    plain.assert_close(state.cpu().numpy(), refT, plain.sum_bound(1, dk) * magT, "state")


def test_step_slots():
    B, H, d, n = 6, 2, 64, 9
    q, k, v, pool = _make(B, H, d, d, np.float16, seed=5, B=n, h0=True)
    lg, slots = _decays(H), [4, -1, 0, 8, -7, 2]
    state = to_dev(pool)
    sl = torch.tensor(slots, dtype=torch.int32, device=DEV)
    o = mmf.linattn_step(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), state, slots=sl).cpu().numpy()
    assert mmf.mmf_get_device_status() == 0
    alone = to_dev(pool[[max(s, 0) for s in slots]])
    want = mmf.linattn_step(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), alone).cpu().numpy()
    live = [i for i, s in enumerate(slots) if s >= 0]
    assert np.array_equal(o[live], want[live])
    assert (o[[1, 4]] == 0).all()
    got, alone = state.cpu().numpy(), alone.cpu().numpy()
    for i in live:
        assert np.array_equal(got[slots[i]], alone[i])
    for s in set(range(n)) - set(slots):
        assert np.array_equal(got[s], pool[s])


def test_step_slots_named_twice_or_outside():
    B, H, d, n = 5, 1, 64, 4
    q, k, v, pool = _make(B, H, d, d, np.float16, seed=6, B=n, h0=True)
    slots = [2, 2, 4, 1, 2]
    state = to_dev(pool)
    o = mmf.linattn_step(to_dev(q), to_dev(k), to_dev(v), to_dev(_decays(H)), state,
                         slots=torch.tensor(slots, dtype=torch.int32, device=DEV)).cpu().numpy()
    assert mmf.mmf_get_device_status() == 8
    assert (o[[1, 2, 4]] == 0).all() and (o[[0, 3]] != 0).any()
    one = to_dev(pool[[2, 1]])
    mmf.linattn_step(to_dev(q[[0, 3]]), to_dev(k[[0, 3]]), to_dev(v[[0, 3]]), to_dev(_decays(H)),
                     one)
    got, one = state.cpu().numpy(), one.cpu().numpy()
    assert np.array_equal(got[2], one[0]) and np.array_equal(got[1], one[1])
    assert np.array_equal(got[[0, 3]], pool[[0, 3]])


@pytest.mark.parametrize("dt,d", [(np.float16, 128), (np.float32, 48)])
def test_steps_continue_a_prompt(dt, d):
    T, n, H = 90, 77, 2
    q, k, v, _ = _make(T, H, d, d, dt, seed=9)
    lg, scale = _decays(H), d ** -0.5
    dq, dk, dv, dl = (to_dev(x) for x in (q, k, v, lg))
    state = torch.empty(1, H, d, d, device=DEV)
    o = [mmf.linattn_forward(dq[:n], dk[:n], dv[:n], dl, hT=state)]
    for t in range(n, T):
        o.append(mmf.linattn_step(dq[t:t + 1], dk[t:t + 1], dv[t:t + 1], dl, state))
    torch.cuda.synchronize()
    ref, refT = plain.linattn(q, k, v, lg, [0, T], scale)
    mag, magT = plain.absolute(plain.linattn, q, k, v, lg, [0, T], scale)
    plain.assert_close(torch.cat(o).cpu().numpy(), ref,
                       plain.tolerance(ref, mag, dt == np.float16, T, d), "o")
    plain.assert_close(state.cpu().numpy(), refT, plain.sum_bound(T, d) * magT, "state")


# --------------------------------------------------------------------------------- gradients
def _check_backward(got, q, k, v, lg, cu, scale, do, h0, dhT, norms=True):
    f16 = q.dtype == np.float16
    far, d = max(b - a for a, b in zip(cu, cu[1:])), max(q.shape[2], v.shape[2])
    ref = plain.linattn_backward(q, k, v, lg, cu, scale, do, h0, dhT)
    mag = plain.absolute(plain.linattn_backward, q, k, v, lg, cu, scale, do, h0=h0, dhT=dhT)
    for name, g, r, m in zip(("dq", "dk", "dv", "dh0"), got, ref, mag):
        g = g.cpu().numpy()
        half = f16 and name != "dh0"
        plain.assert_close(g, r, plain.tolerance(r, m, half, far, d), name)
        if norms:
            plain.assert_norm(g, r, 2 * plain.U16 if half else 2e-6, name)


@pytest.mark.parametrize("T,H,dk,dv", [(1, 2, 128, 128), (2, 2, 64, 64), (64, 2, 64, 128),
                                       (65, 2, 128, 128), (130, 3, 64, 64), (257, 4, 128, 64),
                                       (150, 2, 96, 40), (80, 1, 256, 256), (1100, 2, 128, 128)])
@pytest.mark.parametrize("dt", [np.float16, np.float32])
@pytest.mark.parametrize("states", [False, True])
def test_backward_matches_plain_form(T, H, dk, dv, dt, states):
    q, k, v, h0 = _make(T, H, dk, dv, dt, seed=T, h0=states)
    rng = np.random.default_rng(T + 1)
    do = rng.normal(size=v.shape).astype(dt)
    dhT = rng.normal(size=(1, H, dk, dv)).astype(np.float32) if states else None
    lg, scale = _decays(H), dk ** -0.5
    got = mmf.linattn_backward(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), to_dev(do),
                               scale=scale, h0=_dev(h0), dhT=_dev(dhT), want_dh0=True)
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    _check_backward(got, q, k, v, lg, [0, T], scale, do, h0, dhT)


@pytest.mark.parametrize("scale", [0.0, -0.7])
@pytest.mark.parametrize("d,dt", [(64, np.float16), (128, np.float16), (40, np.float32)])
def test_scales_of_zero_and_below(scale, d, dt):
    T, H = 140, 2
    q, k, v, h0 = _make(T, H, d, d, dt, seed=3, h0=True)
    do, dhT = np.roll(v, 2, axis=0), np.roll(h0, 1, axis=2)
    lg = _decays(H)
    o, hT = _forward(q, k, v, lg, scale, h0=h0)
    _check_forward(o, hT, q, k, v, lg, [0, T], scale, h0, norms=False)
    got = mmf.linattn_backward(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), to_dev(do),
                               scale=scale, h0=to_dev(h0), dhT=to_dev(dhT), want_dh0=True)
    torch.cuda.synchronize()
    _check_backward(got, q, k, v, lg, [0, T], scale, do, h0, dhT, norms=False)


@pytest.mark.parametrize("cu", [[3, 3, 4, 70, 70, 199, 199], [0, 1, 2, 3, 130, 259], [0, 0, 0]])
@pytest.mark.parametrize("dk,dv,dt", [(64, 64, np.float16), (128, 128, np.float16),
                                      (24, 40, np.float32)])
def test_backward_of_ragged_batches(cu, dk, dv, dt):
    T, H, B = 300, 4, len(cu) - 1
    q, k, v, h0 = _make(T, H, dk, dv, dt, seed=len(cu), B=B, h0=True)
    rng = np.random.default_rng(2)
    do = rng.normal(size=v.shape).astype(dt)
    dhT = rng.normal(size=h0.shape).astype(np.float32)
    for x in (q, k, v, do):
        x[:cu[0]] = np.nan
        x[cu[-1]:] = np.inf
    lg = _decays(H)
    got = mmf.linattn_backward(to_dev(q), to_dev(k), to_dev(v), to_dev(lg), to_dev(do), scale=0.3,
                               cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                               h0=to_dev(h0), dhT=to_dev(dhT), want_dh0=True)
    torch.cuda.synchronize()
    _check_backward(got, q, k, v, lg, cu, 0.3, do, h0, dhT, norms=False)


def test_backward_matches_differences_of_the_forward():
    # in fp32: central differences of a loss that is linear in q, k, v and the state alone, so
    # their only error is rounding, about sum_bound / step of the loss's magnitude
    T, H, d, step = 37, 2, 16, 2.0 ** -3
    q, k, v, h0 = _make(T, H, d, d, np.float32, seed=11, h0=True)
    rng = np.random.default_rng(12)
    do = rng.normal(size=v.shape).astype(np.float32)
    dhT = rng.normal(size=h0.shape).astype(np.float32)
    lg = to_dev(_decays(H))

    def loss(q, k, v, h0):
        hT = torch.empty(1, H, d, d, device=DEV)
        o = mmf.linattn_forward(q, k, v, lg, h0=h0, hT=hT)
        return float((o.double() * to_dev(do)).sum() + (hT.double() * to_dev(dhT)).sum())

    x = [to_dev(a) for a in (q, k, v, h0)]
    grads = mmf.linattn_backward(x[0], x[1], x[2], lg, to_dev(do), h0=x[3], dhT=to_dev(dhT),
                                 want_dh0=True)
    mags = plain.absolute(plain.linattn, q, k, v, _decays(H), [0, T], d ** -0.5, h0=h0)
    size = float((mags[0] * np.abs(do)).sum() + (mags[1] * np.abs(dhT)).sum())
    for i in range(4):
        u = torch.from_numpy(rng.choice([-1.0, 1.0], size=x[i].shape).astype(np.float32)).to(DEV)
        up = loss(*(a + step * u if j == i else a for j, a in enumerate(x)))
        down = loss(*(a - step * u if j == i else a for j, a in enumerate(x)))
        want = float((grads[i].double() * u).sum())
        tol = 2 * plain.sum_bound(T, d) * size * (1 + step) / step
        assert abs((up - down) / (2 * step) - want) <= tol


# ------------------------------------------------------------------------------ how it is run
def test_streams_graphs_and_repeats():
    T, H, d = 700, 4, 128
    q, k, v, _ = _make(T, H, d, d, np.float16, seed=13)
    do = np.roll(v, 1, axis=0)
    dq, dk, dv, dd, lg = (to_dev(x) for x in (q, k, v, do, _decays(H)))
    out, hT = torch.empty_like(dv), torch.empty(1, H, d, d, device=DEV)
    want = mmf.linattn_forward(dq, dk, dv, lg, hT=hT)
    wantT = hT.clone()
    grads = mmf.linattn_backward(dq, dk, dv, lg, dd, want_dh0=True)
    # the same bits every time, and on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = mmf.linattn_forward(dq, dk, dv, lg, hT=hT, stream=side)
    g = mmf.linattn_backward(dq, dk, dv, lg, dd, want_dh0=True, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(hT, wantT)
    assert all(torch.equal(a, b) for a, b in zip(g, grads))
    # captured, with inputs that change between replays, two graphs in turn
    state = torch.zeros(T, H, d, d, device=DEV)[:2].contiguous()
    tok = [x[:2].contiguous() for x in (dq, dk, dv)]
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    mmf.linattn_forward(dq, dk, dv, lg, hT=hT, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mmf.linattn_forward(dq, dk, dv, lg, hT=hT, out=out)
    with torch.cuda.graph(second):
        g2 = mmf.linattn_backward(dq, dk, dv, lg, dd, want_dh0=True)
        so = mmf.linattn_step(*tok, lg, state)
    dv.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((hT == 0).all())
    dv.copy_(to_dev(v))
    graph.replay()
    second.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(hT, wantT)
    assert all(torch.equal(a, b) for a, b in zip(g2, grads))
    alone = torch.zeros_like(state)
    assert torch.equal(mmf.linattn_step(*tok, lg, alone), so) and torch.equal(alone, state)


# each of the three kernels, on rows so far apart that their offsets pass 31 and 32 bits
@pytest.mark.parametrize("d", [128, 64, 24])
def test_offsets_beyond_32_bits(d):
    T, H, far = 80, 2, 1 << 26            # 80 * 2^26 elements: 10 GB of fp16
    wide = torch.empty(T * far, dtype=torch.float16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(4, T, H, d, generator=g, device=DEV).half()
    # q, k, v, do and o side by side in every row
    rows = [wide.as_strided((T, H, d), (far, d, 1), i * H * d) for i in range(5)]
    for r, a in zip(rows, x):
        r.copy_(a)
    lg = to_dev(_decays(H))
    want = mmf.linattn_forward(*x[:3], lg)
    mmf.linattn_forward(*rows[:3], lg, out=rows[4])
    assert torch.equal(rows[4].contiguous(), want)
    got = mmf.linattn_backward(*rows[:3], lg, rows[3])
    for a, b in zip(got[:3], mmf.linattn_backward(*x[:3], lg, x[3])):
        assert torch.equal(a, b)


def test_a_pool_beyond_32_bits():
    n, H, d = 8300, 16, 128               # 2.2e9 values, 8.7 GB
    pool = torch.empty(n, H, d, d, device=DEV)
    q, k, v, h0 = _make(2, H, d, d, np.float16, seed=1, B=2, h0=True)
    slots = [n - 1, 0]
    pool[slots] = to_dev(h0)
    alone = to_dev(h0)
    a = [to_dev(x) for x in (q, k, v, _decays(H))]
    want = mmf.linattn_step(*a, alone)
    got = mmf.linattn_step(*a, pool, slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    assert torch.equal(got, want) and torch.equal(pool[slots], alone)


def test_two_calls_at_once_with_a_workspace_each():
    T, H, d = 3000, 2, 64
    lg = to_dev(_decays(H))
    sides = [torch.cuda.Stream() for _ in range(2)]
    x = [[to_dev(a) for a in _make(T, H, d, d, np.float16, seed=20 + i)[:3]] for i in range(2)]
    want = [mmf.linattn_forward(*a, lg) for a in x]
    torch.cuda.synchronize()
    got = [mmf.linattn_forward(*a, lg, stream=s) for _ in range(5) for a, s in zip(x, sides)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


def test_a_block_of_8_bit_projections_around_the_mixer():
    """norm -> 8-bit q, k, v -> linear attention over a ragged prompt, then single tokens -> 8-bit
    output projection: each stage fed by the one before it, against the plain forms fed alike."""
    K, H, d, cu = 256, 2, 64, [0, 5, 133]
    T, rng = cu[-1], np.random.default_rng(30)
    x = rng.normal(size=(T, K)).astype(np.float16)
    W = [(rng.normal(size=(n, K)) * 0.06).astype(np.float16) for n in (3 * H * d,)][0]
    Wo = (rng.normal(size=(K, H * d)) * 0.06).astype(np.float16)
    (W8, s), (O8, so) = mmf.quantize_weights_int8(to_dev(W)), mmf.quantize_weights_int8(to_dev(Wo))
    lg = _decays(H)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    state = torch.empty(2, H, d, d, device=DEV)

    def block(x, mix):
        qkv = mmf.int8_linear_forward(x, W8, s).view(-1, 3, H, d)
        o = mix(qkv[:, 0], qkv[:, 1], qkv[:, 2])
        return qkv, o, mmf.int8_linear_forward(o.view(-1, H * d), O8, so)

    qkv, o, y = block(to_dev(x), lambda q, k, v: mmf.linattn_forward(
        q, k, v, to_dev(lg), cu_seqlens=cud, hT=state))
    h = state.clone().cpu().numpy()
    new = rng.normal(size=(2, K)).astype(np.float16)
    qkv1, o1, y1 = block(to_dev(new), lambda q, k, v: mmf.linattn_step(q, k, v, to_dev(lg), state))
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    a = [qkv[:, i].cpu().numpy() for i in range(3)]
    _check_forward(o.cpu().numpy(), h, *a, lg, cu, d ** -0.5, None, norms=False)
    a = [qkv1[:, i].cpu().numpy() for i in range(3)]
    ref, refT = plain.linattn(*a, lg, [0, 1, 2], d ** -0.5, h)
    mag, magT = plain.absolute(plain.linattn, *a, lg, [0, 1, 2], d ** -0.5, h0=h)
    plain.assert_close(o1.cpu().numpy(), ref, plain.tolerance(ref, mag, True, 1, d), "step")
    plain.assert_close(state.cpu().numpy(), refT, plain.sum_bound(1, d) * magT, "state")
    for got, inp in ((y, o), (y1, o1)):
        A = torch.empty((inp.shape[0], H * d), dtype=torch.int8, device=DEV)
        gam = torch.empty(inp.shape[0], device=DEV)
        mmf.mmf_quantize_activations(inp.view(-1, H * d), None, 1e-8, A, gam)
        r = plain.int8_product(A.cpu().numpy(), gam.cpu().numpy(), O8.cpu().numpy(),
                               so.cpu().numpy())
        plain.assert_close(got.cpu().numpy(), r,
                           (plain.U16 * 1.001 + 4.01 * plain.U32) * np.abs(r) + plain.TINY16, "y")
