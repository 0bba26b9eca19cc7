"""Cases of the 8-bit product and of the linear attention with a decay for each head.

Each case is one call that a user's program makes of the library: `prepare` makes what the
program has in hand, `run` makes the call (or, with `own` false, computes the same in elementary
torch operations), `exact` gives the operator's values in 64 bits.

The operators:
  int8_weights   a weight matrix to 8-bit codes with one scale for each output channel
  int8_product   activation codes (one scale for each token) times such weights
  linattn        S_t = gamma S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over whole prompts
  linattn_step   the same for one new token of each sequence, states updated in place
  linattn_bwd    gradients of linattn: dq, dk, dv and the initial state's
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "f32": torch.float32}
CHUNK = 128


def listed():
    return [
        # the output head of a 2048-wide model with 32000 tokens of vocabulary, one new token
        dict(name="head, 1 token", op="int8_product", T=1, K=2048, N=32000, out="f32"),
        # an odd layer of odd sizes over a small batch of new tokens
        dict(name="odd layer, 77 tokens", op="int8_product", T=77, K=1040, N=1000, out="f16"),
        # the gate projection of the same model over a long prompt
        dict(name="gate, 8192 tokens", op="int8_product", T=8192, K=2048, N=11264, out="f16"),
        # the output head's weights, once when a model is loaded
        dict(name="head's weights", op="int8_weights", N=32000, K=2048, dt="f32"),
        # a small odd layer's weights
        dict(name="odd layer's weights", op="int8_weights", N=1000, K=1040, dt="f16"),
        # one long prompt: 16 heads of 128 (hidden 2048)
        dict(name="one prompt of 32768", op="linattn", B=1, T=32768, H=16, dk=128, dv=128, dt="f16",
             ragged=False, h0=False),
        # prompts of unlike lengths packed into one call, continuing earlier states; heads of 64
        dict(name="13 unlike prompts", op="linattn", B=13, T=9001, H=16, dk=64, dv=64, dt="f16",
             ragged=True, h0=True),
        # single precision with unequal head sizes
        dict(name="3 prompts in f32", op="linattn", B=3, T=1500, H=8, dk=96, dv=128, dt="f32",
             ragged=False, h0=False),
        # generation: one sequence, then a full batch
        dict(name="step of 1", op="linattn_step", B=1, H=16, dk=128, dv=128, dt="f16"),
        dict(name="step of 256", op="linattn_step", B=256, H=16, dk=128, dv=128, dt="f16"),
        # training: a batch of equal sequences, and a small ragged one with a state's gradient
        dict(name="backward, 4 x 2048", op="linattn_bwd", B=4, T=8192, H=16, dk=128, dv=128,
             dt="f16", ragged=False, h0=False),
        dict(name="backward, 5 unlike", op="linattn_bwd", B=5, T=1111, H=8, dk=64, dv=64, dt="f16",
             ragged=True, h0=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["int8_product", "int8_product", "int8_weights", "linattn", "linattn",
                     "linattn_step", "linattn_bwd"])
    if op == "int8_product":
        while True:
            T, K, N = _log(rng, 1, 8192), _log(rng, 256, 8192, 16), _log(rng, 256, 32000, 8)
            if T * K * N <= 8192 * 2048 * 11264 and T * N <= 8192 * 11264:
                return dict(op=op, T=T, K=K, N=N, out=rng.choice(["f16", "f16", "f32"]))
    if op == "int8_weights":
        while True:
            N, K = _log(rng, 256, 32000, 8), _log(rng, 256, 8192, 16)
            if N * K <= 32000 * 2048:
                return dict(op=op, N=N, K=K, dt=rng.choice(["f16", "f32"]))
    if op == "linattn_step":
        while True:
            B, H, d = _log(rng, 1, 256), rng.choice([4, 8, 16, 20, 32]), rng.choice([64, 128])
            if B * H * d * d <= 256 * 16 * 128 * 128:
                return dict(op=op, B=B, H=H, dk=d, dv=d, dt=rng.choice(["f16", "f16", "f32"]))
    H, d = rng.choice([4, 8, 16]), rng.choice([64, 128])
    dt = rng.choice(["f16", "f16", "f16", "f32"])
    dk, dv = (d, d) if dt == "f16" else (rng.choice([64, 96, 128]), d)
    top = (32768 if op == "linattn" else 8192) * 16 * 128 // (H * d) // (1 if dt == "f16" else 8)
    T = _log(rng, 16, min(top, 32768))
    B = max(1, min(_log(rng, 1, 16), T // 4))
    ragged = rng.random() < 0.5
    if not ragged:
        T = T // B * B
    return dict(op=op, B=B, T=T, H=H, dk=dk, dv=dv, dt=dt, ragged=ragged, h0=rng.random() < 0.5)


# ------------------------------------------------------------------------------------ inputs
def _log_decay(H):
    """Decays from exp(-1/4) to exp(-1/512) for a token, evenly spread over the heads' logarithms."""
    e = torch.linspace(2.0, 9.0, H, dtype=torch.float64) if H > 1 else torch.tensor([5.0]).double()
    return (-(2.0 ** -e)).float()


def _lengths(case, seed):
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T // B] * B
    g = torch.Generator().manual_seed(seed + 77)
    cuts = torch.randint(0, T + 1, (B - 1,), generator=g).sort().values.tolist()
    cuts = [0] + cuts + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    op = case["op"]
    s = dict(op=op)
    if op == "int8_weights":
        s["W"] = normal(case["N"], case["K"], std=0.02, dtype=DT[case["dt"]])
        return s
    if op == "int8_product":
        T, K, N = case["T"], case["K"], case["N"]
        s["A"] = (normal(T, K) * 32.0).round_().clamp_(-128, 127).to(torch.int8)
        s["gamma"] = normal(T).abs_() + 3.0
        s["W8"] = (normal(N, K) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["wscale"] = (normal(N).abs_() + 1.0) * 5e-4
        s["out"] = DT[case["out"]]
        return s
    H, dk, dv, dt = case["H"], case["dk"], case["dv"], DT[case["dt"]]
    s["log_decay"] = _log_decay(H).to(DEV)
    s["scale"] = dk ** -0.5
    if op == "linattn_step":
        B = case["B"]
        s["q"], s["k"] = normal(B, H, dk, dtype=dt), normal(B, H, dk, dtype=dt)
        s["v"] = normal(B, H, dv, dtype=dt)
        s["state"] = normal(B, H, dk, dv, std=3.0)
        return s
    B, T = case["B"], case["T"]
    lens = _lengths(case, seed)
    s["batch"], s["longest"] = B, max(lens)
    cu = torch.tensor([0] + lens).cumsum(0)
    s["cu"] = cu.to(torch.int32).to(DEV)
    s["cu_arg"] = s["cu"] if case["ragged"] else None
    s["q"], s["k"] = normal(T, H, dk, dtype=dt), normal(T, H, dk, dtype=dt)
    s["v"] = normal(T, H, dv, dtype=dt)
    s["h0"] = normal(B, H, dk, dv, std=3.0) if case["h0"] else None
    if op == "linattn":
        s["hT"] = torch.empty(B, H, dk, dv, device=DEV)
    else:
        s["do"] = normal(T, H, dv, dtype=dt)
        s["dhT"] = normal(B, H, dk, dv) if case["h0"] else None
    return s


# -------------------------------------------------------------------------------- plain forms
def _powers(lg, n):
    """exp(n lg) for each head, [H, *n.shape], 0 where n is negative."""
    e = torch.exp(lg.double().view(-1, *([1] * n.dim())) * n.clamp(min=0).double())
    return (e * (n >= 0)).float()


def _rows(cu, longest, T, backwards):
    """Token of each place of a padded [B, L] batch, sequences aligned at its end (so that the
    padding comes first), whether it is one, and each token's place."""
    L = -(-longest // CHUNK) * CHUNK
    cu = cu.long()
    lo, hi = cu[:-1, None], cu[1:, None]
    at = torch.arange(L, device=cu.device)[None, :]
    idx = lo + (L - 1 - at) if backwards else hi - L + at
    real = (idx >= lo) & (idx < hi)
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu, t, right=True).clamp(max=cu.numel() - 1) - 1
    off = t - cu[b]
    place = b * L + (L - 1 - off if backwards else L - (cu[b + 1] - cu[b]) + off)
    return idx.clamp(0, T - 1), real, place


def _sweep(q, k, v, lg, cu, longest, s0, mult=1.0, backwards=False):
    """o_t = S_t^T q_t and the last state, with S_t = gamma S_{t-1} + mult k_t v_t^T, chunk by
    chunk, in 32 bits.  Backwards the tokens come last one first and the decay acts after a token:
    o_t = R_t^T q_t with R_t = U + mult k_t v_t^T, U = gamma R_t."""
    lag = 1 if backwards else 0
    T, H = q.shape[0], q.shape[1]
    B = cu.numel() - 1
    idx, real, place = _rows(cu, longest, T, backwards)
    L, C = idx.shape[1], CHUNK
    n = L // C

    def padded(x):
        x = x.float()[idx] * real[..., None, None]
        return x.view(B, n, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4)  # [B, H, n, C, d]

    qp, kp, vp = padded(q), padded(k), padded(v) * mult
    i = torch.arange(C, device=q.device)
    p = (qp @ kp.transpose(-1, -2)) * _powers(lg, i[:, None] - i[None, :])[:, None]
    o = p @ vp
    del p
    ds = (kp * _powers(lg, C - 1 + lag - i)[:, None, :, None]).transpose(-1, -2) @ vp
    c = torch.arange(n + 1, device=q.device)
    before = _powers(lg, C * (c[:, None] - 1 - c[None, :n]))  # [H, n + 1, n]
    st = (before @ ds.flatten(-2)).view(B, H, n + 1, *ds.shape[-2:])
    del ds
    if s0 is not None:
        pad = L - (cu[1:] - cu[:-1]).long()
        e = (c[None, :] * C - pad[:, None]).clamp(min=0)
        st = st + _powers(lg, e).transpose(0, 1)[..., None, None] * s0.float()[:, :, None]
        first = (i[None, :] + 1 - lag + c[:n, None] * C)[None] - pad[:, None, None]
        reach = first - e[:, :n, None]
    else:
        reach = (i + 1 - lag)[None, None, :].expand(B, n, C)
    o = o + (qp @ st[:, :, :n]) * _powers(lg, reach).transpose(0, 1)[..., None]
    return o.permute(0, 2, 3, 1, 4).reshape(B * L, H, -1)[place], st[:, :, n]


def _plain(s):
    op = s["op"]
    if op == "int8_weights":
        w = s["W"].float()
        top = w.abs().amax(dim=1)
        scale = top / torch.full_like(top, 127.0)
        code = (w / scale[:, None]).round().clamp(-127, 127)
        return torch.where(scale[:, None] > 0, code, torch.zeros_like(code)).to(torch.int8), scale
    if op == "int8_product":
        acc = s["A"].float() @ s["W8"].float().t()
        return (acc * (s["gamma"] / 127.0)[:, None] * s["wscale"][None, :]).to(s["out"])
    lg, scale, dt = s["log_decay"], s["scale"], s["q"].dtype
    if op == "linattn_step":
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
        s["state"].mul_(_powers(lg, torch.ones((), device=DEV))[None, :, None, None])
        s["state"].add_(k[..., :, None] * v[..., None, :])
        o = (q[..., None, :] @ s["state"])[..., 0, :] * scale
        return o.to(dt), s["state"]
    cu, far = s["cu"], s["longest"]
    q, k, v = s["q"], s["k"], s["v"]
    if op == "linattn":
        o, hT = _sweep(q, k, v, lg, cu, far, s["h0"])
        return (o * scale).to(dt), hT
    do, dhT = s["do"], s["dhT"]
    flip = lambda h: None if h is None else h.transpose(-1, -2)  # noqa: E731
    dq, _ = _sweep(do, v, k, lg, cu, far, flip(s["h0"]))
    dk, _ = _sweep(v, do, q, lg, cu, far, flip(dhT), mult=scale, backwards=True)
    dv, dh0 = _sweep(k, q, do, lg, cu, far, dhT, mult=scale, backwards=True)
    return (dq * scale).to(dt), dk.to(dt), dv.to(dt), dh0


# ------------------------------------------------------------------------------ own operators
def _own(s):
    import ternary_weight_lm_b200 as mmf

    op = s["op"]
    if op == "int8_weights":
        return mmf.quantize_weights_int8(s["W"])
    if op == "int8_product":
        return mmf.int8_matmul(s["A"], s["gamma"], s["W8"], s["wscale"], out_dtype=s["out"])
    if op == "linattn_step":
        o = mmf.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
        return o, s["state"]
    if op == "linattn":
        o = mmf.linattn_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                cu_seqlens=s["cu_arg"], batch=s["batch"], h0=s["h0"], hT=s["hT"])
        return o, s["hT"]
    return mmf.linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                cu_seqlens=s["cu_arg"], batch=s["batch"], h0=s["h0"],
                                dhT=s["dhT"], want_dh0=True)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------- work and values
def work(case):
    """Inputs read once, outputs written once; for the recurrence the operations of the
    token-by-token form (decay and update of the state, product with q), which no form needs
    fewer of than half."""
    op = case["op"]
    if op == "int8_weights":
        n, e = case["N"] * case["K"], 2 if case["dt"] == "f16" else 4
        return {"bytes": n * (e + 1) + 4 * case["N"], "flops": 2 * n}
    if op == "int8_product":
        T, K, N, e = case["T"], case["K"], case["N"], 2 if case["out"] == "f16" else 4
        return {"bytes": T * K + N * K + 4 * T + 4 * N + e * T * N, "flops": 2 * T * K * N}
    B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
    e, state = 2 if case["dt"] == "f16" else 4, 4 * B * H * dk * dv
    if op == "linattn_step":
        return {"bytes": 2 * state + e * B * H * 2 * (dk + dv), "flops": 5 * B * H * dk * dv}
    T = case["T"]
    if op == "linattn":
        return {"bytes": e * T * H * 2 * (dk + dv) + state * (2 if case["h0"] else 1),
                "flops": 4 * T * H * dk * dv}
    # q, k, v, do in; dq, dk, dv out; the states' gradients
    return {"bytes": e * T * H * (4 * dk + 3 * dv) + state * (3 if case["h0"] else 1),
            "flops": 10 * T * H * dk * dv}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "int8_weights":
        return None, s["W"].double().abs().max(dim=1).values / 127.0  # codes are held to equality
    if op == "int8_product":
        y = torch.einsum("tk,nk->tn", s["A"].double(), s["W8"].double())
        y = torch.einsum("tn,t,n->tn", y, s["gamma"].double() / 127.0, s["wscale"].double())
        return y
    g = s["log_decay"].double().exp()
    q, k, v, scale = s["q"].double(), s["k"].double(), s["v"].double(), s["scale"]
    if op == "linattn_step":
        S = torch.einsum("h,bhde->bhde", g, s["state"].double())
        S = S + torch.einsum("bhd,bhe->bhde", k, v)
        return torch.einsum("bhd,bhde->bhe", q, S) * scale, S
    cu = s["cu"].tolist()
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=DEV)
    far = int(lens.max())
    start = s["cu"][:-1].long()
    B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
    G = g.view(1, H, 1, 1)

    def token(S, n, x, y, c):
        """S for sequences that have a token n: decayed, with c x y^T added."""
        live = n < lens
        at = (start + n).clamp(max=q.shape[0] - 1)
        new = S * G + (c * x[at])[..., :, None] * y[at][..., None, :]
        return torch.where(live.view(B, 1, 1, 1), new, S), at, live

    def put(out, at, live, val):
        # sequences without this token write to a row behind the last one
        out[torch.where(live, at, torch.full_like(at, out.shape[0] - 1))] = val

    def rows(d):
        return torch.zeros(q.shape[0] + 1, H, d, dtype=torch.float64, device=DEV)

    zero = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV)
    S = zero if s["h0"] is None else s["h0"].double()
    if op == "linattn":
        o = rows(dv)
        for n in range(far):
            S, at, live = token(S, n, k, v, 1.0)
            put(o, at, live, (q[at][..., None, :] @ S)[..., 0, :] * scale)
        return o[:-1], S
    do = s["do"].double()
    dq, dkk, dvv = rows(dk), rows(dk), rows(dv)
    for n in range(far):
        S, at, live = token(S, n, k, v, 1.0)
        put(dq, at, live, (S @ do[at][..., :, None])[..., 0] * scale)
    # R holds the gradient of the state after a token; it decays on its way to the token before
    R = zero if s["dhT"] is None else s["dhT"].double()
    for n in range(far - 1, -1, -1):
        live = n < lens
        at = (start + n).clamp(max=q.shape[0] - 1)
        add = (scale * q[at])[..., :, None] * do[at][..., None, :]
        here = R + add
        put(dkk, at, live, (here @ v[at][..., :, None])[..., 0])
        put(dvv, at, live, (k[at][..., None, :] @ here)[..., 0, :])
        R = torch.where(live.view(B, 1, 1, 1), here * G, R)
    return dq[:-1], dkk[:-1], dvv[:-1], R
