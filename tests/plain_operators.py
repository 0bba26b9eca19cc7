"""Plain 64-bit implementations of the 8-bit projection and of the linear attention with a decay
for each head (numpy, straight from the formulas), and rounding bounds for their tests."""
import numpy as np

U32 = 2.0 ** -24          # half a step of fp32, relative
U16 = 2.0 ** -11          # half a step of fp16, relative
TINY16 = 2.0 ** -25       # half a step among fp16's subnormals


def quantize_rows(W):
    """Codes and scales of a weight matrix in fp32 arithmetic: exact values, no tolerance."""
    W = W.astype(np.float32)
    s = np.abs(W).max(axis=1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.clip(np.rint(W / s[:, None]), -127, 127)
    return np.where(s[:, None] > 0, c, 0).astype(np.int8), s


def int8_product(A, gamma, W8, wscale):
    acc = A.astype(np.int64) @ W8.astype(np.int64).T
    return acc * (gamma.astype(np.float64) / 127)[:, None] * wscale.astype(np.float64)[None, :]


def gammas(log_decay):
    lg = np.asarray(log_decay, dtype=np.float64)
    lg = np.where(np.isnan(lg), 0.0, np.minimum(lg, 0.0))
    return np.exp(lg)


def linattn(q, k, v, log_decay, cu, scale, h0=None):
    """(o, hT); rows of tokens outside the sequences are NaN in o."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    T, H, dk = q.shape
    dv, B = v.shape[2], len(cu) - 1
    g = gammas(log_decay)[:, None, None]
    o = np.full((T, H, dv), np.nan)
    hT = np.zeros((B, H, dk, dv)) if h0 is None else h0.astype(np.float64).copy()
    for b in range(B):
        S = hT[b]
        for t in range(cu[b], cu[b + 1]):
            S = g * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hd,hde->he", q[t], S)
        hT[b] = S
    return o, hT


def linattn_backward(q, k, v, log_decay, cu, scale, do, h0=None, dhT=None):
    q, k, v, do = (x.astype(np.float64) for x in (q, k, v, do))
    T, H, dk = q.shape
    dv, B = v.shape[2], len(cu) - 1
    g = gammas(log_decay)[:, None, None]
    dq, dkk, dvv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    dh0 = np.zeros((B, H, dk, dv)) if dhT is None else dhT.astype(np.float64).copy()
    for b in range(B):
        S = np.zeros((H, dk, dv)) if h0 is None else h0[b].astype(np.float64)
        for t in range(cu[b], cu[b + 1]):
            S = g * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hde,he->hd", S, do[t])
        U = dh0[b]
        for t in range(cu[b + 1] - 1, cu[b] - 1, -1):
            R = U + scale * q[t][:, :, None] * do[t][:, None, :]
            dkk[t] = np.einsum("hde,he->hd", R, v[t])
            dvv[t] = np.einsum("hde,hd->he", R, k[t])
            U = g * R
        dh0[b] = U
    return dq, dkk, dvv, dh0


def absolute(f, *args, **kw):
    """The same with every value's magnitude (the scale's too, the logarithms of decays as they
    are): a bound on the sum of the magnitudes of a result's terms, which its rounding errors are
    relative to."""
    def mag(i, a):
        if isinstance(a, float):
            return abs(a)
        return np.abs(a) if isinstance(a, np.ndarray) and a.dtype.kind == "f" and i != 3 else a
    return f(*(mag(i, a) for i, a in enumerate(args)),
             **{n: None if a is None else np.abs(a) for n, a in kw.items()})


def sum_bound(longest, d):
    """Relative to the sum of magnitudes, of a value held in fp32 throughout: a term is rounded as a
    product, by at most two operations (decay, addition) for each of `longest` tokens, by the sum
    over d, the scale and the decay's own rounding (a relative error of at most 2 U32 for each
    token it is applied to)."""
    return (4 * longest + d + 8) * U32


def tolerance(ref, mag, f16, longest, d, tensor_cores=True):
    """fp32: the sum's bound alone.  fp16: the output's rounding, and with tensor cores two
    operands (the chunk's scores and the state) rounded once to eleven bits."""
    tol = sum_bound(longest, d) * mag
    if f16:
        tol = tol + U16 * np.abs(ref) + TINY16 + (U16 * (1 + U16) * mag if tensor_cores else 0.0)
    return tol


def assert_close(got, ref, tol, what):
    got = got.astype(np.float64)
    real = ~np.isnan(ref)
    bad = ~(np.abs(got - ref) <= tol) & real
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def assert_norm(got, ref, bound, what):
    """Errors of many independent roundings: their 2-norm relative to the result's."""
    real = ~np.isnan(ref)
    if not real.any():
        return
    n = np.linalg.norm(ref[real])
    err = np.linalg.norm(got.astype(np.float64)[real] - ref[real])
    assert err <= bound * n, (what, err / max(n, 1e-300))
