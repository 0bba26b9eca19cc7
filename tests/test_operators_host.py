"""Host-side checks of the 8-bit projection and of the linear attention: every refusal happens
before any launch, the binding refuses tensors that a call would misread, and the plain 64-bit
forms agree with finite differences."""
import ctypes

import numpy as np
import pytest
import torch

import plain_operators as plain
import ternary_weight_lm_b200 as mmf

OK, INVALID, SHAPE, ALIGN, CUDA, TIMEOUT, WS = 0, 1, 2, 3, 4, 5, 6
A16 = 0x10000   # fake, aligned "device" addresses: never dereferenced by rejected calls


# ------------------------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("kw,code", [
    (dict(W=None), INVALID), (dict(W8=None), INVALID), (dict(s=None), INVALID),
    (dict(dt=2), INVALID), (dict(N=0), SHAPE), (dict(N=4), SHAPE), (dict(N=1001), SHAPE),
    (dict(K=8), SHAPE), (dict(K=1000), SHAPE), (dict(K=32784), SHAPE),
    (dict(W=A16 + 8), ALIGN), (dict(W8=A16 + 8), ALIGN), (dict(s=A16 + 2), ALIGN),
])
def test_int8_quantize_weights_rejects_on_host(kw, code):
    a = dict(W=A16, dt=0, N=1000, K=1040, W8=A16, s=A16)
    a.update(kw)
    assert mmf.lib().mmf_int8_quantize_weights(a["W"], a["dt"], a["N"], a["K"], a["W8"], a["s"],
                                               None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), INVALID), (dict(g=None), INVALID), (dict(W8=None), INVALID),
    (dict(s=None), INVALID), (dict(y=None), INVALID), (dict(ydt=2), INVALID),
    (dict(T=0), SHAPE), (dict(T=-1), SHAPE), (dict(K=120), SHAPE), (dict(N=12), SHAPE),
    (dict(N=(1 << 20) + 8), SHAPE), (dict(A=A16 + 8), ALIGN), (dict(g=A16 + 1), ALIGN),
    (dict(W8=A16 + 4), ALIGN), (dict(s=A16 + 3), ALIGN), (dict(y=A16 + 8), ALIGN),
])
def test_int8_forward_quantized_rejects_on_host(kw, code):
    a = dict(A=A16, g=A16, T=7, K=1040, W8=A16, s=A16, N=1000, y=A16, ydt=1)
    a.update(kw)
    assert mmf.lib().mmf_int8_forward_quantized(a["A"], a["g"], a["T"], a["K"], a["W8"], a["s"],
                                                a["N"], a["y"], a["ydt"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INVALID), (dict(W8=None), INVALID), (dict(y=None), INVALID),
    (dict(xdt=3), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(K=1040), SHAPE), (dict(K=8320), SHAPE), (dict(N=4), SHAPE), (dict(T=0), SHAPE),
    (dict(x=A16 + 8), ALIGN), (dict(g=A16 + 4), ALIGN), (dict(ws=A16 + 16), ALIGN),
    (dict(ws=None), WS), (dict(wsb=100), WS),
])
def test_int8_forward_rejects_on_host(kw, code):
    a = dict(x=A16, xdt=1, T=7, K=1024, g=None, eps=1e-8, W8=A16, s=A16, N=1000, y=A16, ydt=1,
             ws=A16, wsb=1 << 20)
    a.update(kw)
    assert mmf.lib().mmf_int8_forward(a["x"], a["xdt"], a["T"], a["K"], a["g"], a["eps"], a["W8"],
                                      a["s"], a["N"], a["y"], a["ydt"], a["ws"], a["wsb"],
                                      None) == code


def test_int8_workspace_sizes():
    assert mmf.mmf_int8_workspace_bytes(3, 128) == 512 + 256
    assert mmf.mmf_int8_workspace_bytes(300, 256) == 300 * 256 + 1280
    assert mmf.mmf_int8_workspace_bytes(0, 128) == 0
    assert mmf.mmf_int8_workspace_bytes(3, 1040) == 0


# -------------------------------------------------------------------------- linear attention
def desc(**kw):
    d = mmf.LinattnDesc()
    a = dict(T=600, B=3, cu_seqlens=None, H=4, dk=64, dv=128, dt=1, scale=0.125, log_decay=A16)
    a.update(kw)
    e = a["H"]
    st = dict(q_t=e * a["dk"], q_h=a["dk"], k_t=e * a["dk"], k_h=a["dk"], v_t=e * a["dv"],
              v_h=a["dv"], o_t=e * a["dv"], o_h=a["dv"])
    for n, v in {**st, **a}.items():
        setattr(d, n, v)
    return d


DESC_FAULTS = [
    (dict(log_decay=None), INVALID), (dict(dt=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(T=0), SHAPE), (dict(B=0), SHAPE),
    (dict(T=601), SHAPE), (dict(H=0, q_t=0, k_t=0, v_t=0, o_t=512), SHAPE), (dict(dk=60), SHAPE),
    (dict(dk=264), SHAPE), (dict(dv=0), SHAPE), (dict(dv=4), SHAPE), (dict(B=(1 << 20) + 1), SHAPE),
    (dict(q_t=-256), INVALID), (dict(k_h=-8), INVALID), (dict(v_t=516), ALIGN),
    (dict(q_h=68), ALIGN), (dict(o_t=0), INVALID), (dict(o_h=64), INVALID),
    (dict(log_decay=A16 + 2), ALIGN), (dict(cu_seqlens=A16 + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", DESC_FAULTS)
def test_linattn_descriptors_are_refused(kw, code):
    L, d = mmf.lib(), desc(**kw)
    r = ctypes.byref(d)
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, A16, 1 << 40, None) == code
    assert L.mmf_linattn_backward(r, A16, A16, A16, A16, None, None, A16, A16, A16, None, A16,
                                  1 << 40, None) == code


@pytest.mark.parametrize("i", range(9))
def test_linattn_pointers_are_refused(i):
    L, r = mmf.lib(), ctypes.byref(desc())
    for bad, code in ((None, INVALID), (A16 + 8, ALIGN)):
        p = [A16] * 9
        p[i] = bad
        # the states may be missing
        if i in (0, 1, 2, 4) or (bad is not None and i in (3, 5)):
            assert L.mmf_linattn_forward(r, *p[:6], A16, 1 << 40, None) == code
        if i in (0, 1, 2, 3, 6, 7, 8) or bad is not None:
            assert L.mmf_linattn_backward(r, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8],
                                          A16 + 256, A16, 1 << 40, None) == code


def test_linattn_workspaces_and_aliases_are_refused():
    L = mmf.lib()
    d = desc(T=6000, B=1, H=16)
    r = ctypes.byref(d)
    need = mmf.mmf_linattn_workspace_bytes(d)
    assert need > 0 and need % 256 == 0
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, A16, need - 1, None) == WS
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, None, 0, None) == WS
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, A16 + 16, need, None) == ALIGN
    need = mmf.mmf_linattn_backward_workspace_bytes(d)
    args = (r, A16, A16, A16, A16, None, A16, A16, A16, A16)
    assert L.mmf_linattn_backward(*args, A16 + 256, A16, need - 1, None) == WS
    # the gradients of the first and of the last state are read and written at unlike times
    assert L.mmf_linattn_backward(*args, A16, A16, need, None) == INVALID
    args = (r, A16, A16, A16, A16, A16, None, A16, A16, A16)
    assert L.mmf_linattn_backward(*args, A16, A16, need, None) == INVALID
    # one short sequence needs none, and a size without a workspace is refused
    d = desc(T=100, B=1)
    assert mmf.mmf_linattn_workspace_bytes(d) == 0
    assert L.mmf_linattn_forward(ctypes.byref(d), A16, A16, A16, None, A16, None, None, 8,
                                 None) == WS
    for kw in (dict(T=0), dict(T=601), dict(dk=60), dict(B=0)):
        assert mmf.mmf_linattn_workspace_bytes(desc(**kw)) == 0
    assert L.mmf_linattn_workspace_bytes(None) == 0
    assert L.mmf_linattn_forward(None, A16, A16, A16, None, A16, None, None, 0, None) == INVALID


@pytest.mark.parametrize("kw,args,code", [
    (dict(), dict(o=None), INVALID), (dict(), dict(state=None), INVALID),
    (dict(T=8), dict(), INVALID), (dict(cu_seqlens=A16), dict(), INVALID),
    (dict(), dict(n=3), INVALID), (dict(), dict(slots=A16), INVALID),
    (dict(), dict(slots=A16, n=(1 << 20) + 1), INVALID), (dict(), dict(slots=A16 + 2, n=9), ALIGN),
    (dict(), dict(state=A16 + 8), ALIGN), (dict(), dict(o=A16 + 8), ALIGN),
    (dict(dk=12), dict(), SHAPE), (dict(o_t=64), dict(), INVALID),
])
def test_linattn_step_rejects_on_host(kw, args, code):
    d = desc(**{**dict(T=4, B=4), **kw})
    a = dict(q=A16, k=A16, v=A16, o=A16, state=A16, slots=None, n=0)
    a.update(args)
    assert mmf.lib().mmf_linattn_step(ctypes.byref(d), a["q"], a["k"], a["v"], a["o"], a["state"],
                                      a["slots"], a["n"], None) == code


def test_valid_calls_without_gpu_report_a_cuda_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L = mmf.lib()
    assert L.mmf_int8_quantize_weights(A16, 0, 8, 16, A16, A16, None) == CUDA
    assert L.mmf_int8_forward_quantized(A16, A16, 1, 16, A16, A16, 8, A16, 1, None) == CUDA
    r = ctypes.byref(desc(T=4, B=4))
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, None, 0, None) == CUDA
    assert L.mmf_linattn_step(r, A16, A16, A16, A16, A16, None, 0, None) == CUDA


def test_binding_refuses_tensors_it_would_misread():
    f = torch.float16
    q, v = torch.zeros(6, 2, 16, dtype=f), torch.zeros(6, 2, 32, dtype=f)
    lg = torch.zeros(2)
    fwd = mmf.linattn_forward
    with pytest.raises(ValueError, match="GPU"):
        fwd(q, q, v, lg)
    with pytest.raises(TypeError, match="k"):
        fwd(q, q.float(), v, lg)
    with pytest.raises(ValueError, match="v"):
        fwd(q, q, v[:5], lg)
    with pytest.raises(ValueError, match="log_decay"):
        fwd(q, q, v, torch.zeros(3))
    with pytest.raises(ValueError, match="last dimension"):
        fwd(q, q, torch.zeros(6, 32, 2, dtype=f).transpose(1, 2), lg)
    with pytest.raises(TypeError, match="cu_seqlens"):
        fwd(q, q, v, lg, cu_seqlens=torch.tensor([0, 6]))
    with pytest.raises(ValueError, match="batch"):
        fwd(q, q, v, lg, cu_seqlens=torch.tensor([0, 6], dtype=torch.int32), batch=2)
    with pytest.raises(ValueError, match="h0"):
        fwd(q, q, v, lg, h0=torch.zeros(1, 2, 32, 16))
    with pytest.raises(ValueError, match="out"):
        fwd(q, q, v, lg, out=torch.zeros(6, 2, 16, dtype=f))
    with pytest.raises(ValueError, match="state"):
        mmf.linattn_step(q, q, v, lg, torch.zeros(5, 2, 16, 32))
    with pytest.raises(TypeError, match="slots"):
        mmf.linattn_step(q, q, v, lg, torch.zeros(9, 2, 16, 32), slots=torch.arange(6))
    with pytest.raises(ValueError, match="dhT"):
        mmf.linattn_backward(q, q, v, lg, v, dhT=torch.zeros(2, 2, 16, 32))
    A, W = torch.zeros(3, 32, dtype=torch.int8), torch.zeros(8, 32, dtype=torch.int8)
    g, s = torch.zeros(3), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        mmf.int8_matmul(A, g, W, s)
    with pytest.raises(TypeError, match="A"):
        mmf.int8_matmul(A.float(), g, W, s)
    with pytest.raises(ValueError, match="W8"):
        mmf.int8_matmul(A, g, W[:, :16], s)
    with pytest.raises(ValueError, match="contiguous"):
        mmf.int8_matmul(A, g, torch.zeros(32, 8, dtype=torch.int8).t(), s)
    with pytest.raises(ValueError, match="out"):
        mmf.int8_matmul(A, g, W, s, out=torch.zeros(3, 9))
    with pytest.raises(TypeError, match="W"):
        mmf.quantize_weights_int8(torch.zeros(8, 32, dtype=torch.float64))
    with pytest.raises(ValueError, match="norm_w"):
        mmf.int8_linear_forward(torch.zeros(3, 32), W, s, norm_w=torch.zeros(31))


# ---------------------------------------------------------------------------- plain forms
def test_plain_gradients_match_differences():
    rng = np.random.default_rng(5)
    H, dk, dv, cu, scale = 2, 3, 2, [0, 3, 3, 7], 0.7
    T, B = cu[-1], len(cu) - 1
    q, k = rng.normal(size=(T, H, dk)), rng.normal(size=(T, H, dk))
    v, do = rng.normal(size=(T, H, dv)), rng.normal(size=(T, H, dv))
    h0, dhT = rng.normal(size=(B, H, dk, dv)), rng.normal(size=(B, H, dk, dv))
    lg = np.array([-0.3, -0.01])
    grads = plain.linattn_backward(q, k, v, lg, cu, scale, do, h0, dhT)

    def loss():
        o, hT = plain.linattn(q, k, v, lg, cu, scale, h0)
        return (o * do).sum() + (hT * dhT).sum()

    # the loss is at most quadratic in any one value of q, k, v or h0: central differences are
    # exact up to rounding, about 2^-52 |loss| / step
    step = 2.0 ** -10
    for x, g in zip((q, k, v, h0), grads):
        it = np.nditer(x, flags=["multi_index"])
        for _ in it:
            i = it.multi_index
            was = x[i]
            x[i] = was + step
            up = loss()
            x[i] = was - step
            down = loss()
            x[i] = was
            assert abs((up - down) / (2 * step) - g[i]) <= 1e-9 * (1 + abs(g[i]))


def test_plain_codes_of_a_row_of_zeros_and_of_ties():
    W = np.zeros((3, 16), dtype=np.float32)
    W[1, :4] = [127.0, 0.5, 1.5, -2.5]
    W[2, 0] = 1e-44          # the scale underflows to zero
    c, s = plain.quantize_rows(W)
    assert c[0].tolist() == [0] * 16 and s[0] == 0
    assert c[1, :4].tolist() == [127, 0, 2, -2] and s[1] == 1
    assert c[2].tolist() == [0] * 16 and s[2] == 0
