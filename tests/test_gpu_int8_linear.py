"""GPU parity of the 8-bit projection against its plain 64-bit form.

Tolerances: codes and scales are equal (one correctly rounded division each).  The product is
exact in int32; y takes at most four fp32 roundings (the sum's conversion, gamma / 127, times the
channel's scale, times the sum), and fp16's own."""
import numpy as np
import pytest
import torch

import plain_operators as plain
import ternary_weight_lm_b200 as mmf
from gpu_helpers import DEV, gpu_act_quant, to_dev

pytestmark = pytest.mark.gpu


def _inputs(T, K, N, seed=0):
    rng = np.random.default_rng(seed)
    A = rng.integers(-128, 128, size=(T, K)).astype(np.int8)
    W8 = rng.integers(-127, 128, size=(N, K)).astype(np.int8)
    gamma = rng.uniform(1e-5, 9.0, size=T).astype(np.float32)
    s = rng.uniform(1e-5, 1e-3, size=N).astype(np.float32)
    return A, gamma, W8, s


def _check(y, ref):
    tol = 4.01 * plain.U32 * np.abs(ref)
    if y.dtype == np.float16:
        tol = tol + plain.U16 * np.abs(ref) * 1.001 + plain.TINY16
    plain.assert_close(y, ref, tol, "y")


def _product(A, gamma, W8, s, dt=torch.float16):
    """Into a buffer with rows behind the last one, which have to stay as they were."""
    T, N = A.shape[0], W8.shape[0]
    buf = torch.full((T + 3, N), 77.0, dtype=dt, device=DEV)
    mmf.int8_matmul(to_dev(A), to_dev(gamma), to_dev(W8), to_dev(s), out=buf[:T])
    torch.cuda.synchronize()
    assert mmf.mmf_get_device_status() == 0
    assert bool((buf[T:] == 77.0).all())
    return buf[:T].cpu().numpy()


# tokens around every tile width, odd channel counts (a tile of 128 cut short, one of 8 rows),
# K of one 16-byte vector, around the 128-byte k-block, and of many blocks
@pytest.mark.parametrize("T,K,N", [
    (1, 16, 8), (1, 2048, 1000), (15, 112, 136), (16, 128, 128), (17, 144, 248), (32, 1040, 1000),
    (33, 256, 2048), (64, 8192, 128), (65, 1040, 264), (77, 1040, 1000), (128, 384, 512),
    (129, 2048, 2048), (200, 1008, 1000), (256, 256, 256), (257, 640, 4104), (513, 2048, 776),
    (1000, 272, 2056), (1025, 2048, 2048), (4, 32768, 24)])
@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_product_matches_plain_form(T, K, N, dt):
    A, gamma, W8, s = _inputs(T, K, N, seed=T + K + N)
    # keep fp16 finite: |sum| <= 128 * 127 * K
    gamma *= np.float32(min(1.0, 3e4 / (128 * 127 * K * 9.0 / 127 * 1e-3)))
    _check(_product(A, gamma, W8, s, dt), plain.int8_product(A, gamma, W8, s))


def test_product_extremes_do_not_wrap():
    # the largest sums of the largest K: 128 * 127 * 32768 = 2^31 - 2^24 does not wrap
    T, K, N = 3, 32768, 16
    A = np.full((T, K), -128, dtype=np.int8)
    W8 = np.full((N, K), 127, dtype=np.int8)
    W8[1] = -127
    gamma, s = np.ones(T, np.float32), np.ones(N, np.float32)
    _check(_product(A, gamma, W8, s, torch.float32), plain.int8_product(A, gamma, W8, s))


def test_product_is_the_same_every_time():
    A, gamma, W8, s = _inputs(40, 4096, 520, seed=3)   # split over a cluster
    a = _product(A, gamma, W8, s)
    b = _product(A, gamma, W8, s)
    assert np.array_equal(a, b)


@pytest.mark.parametrize("N,K", [(8, 16), (24, 1040), (1000, 1040), (64, 4096), (40, 4112),
                                 (16, 32768)])
@pytest.mark.parametrize("dt", [np.float32, np.float16])
def test_weights_match_plain_form(N, K, dt):
    rng = np.random.default_rng(N + K)
    W = (rng.normal(size=(N, K)) * 0.02).astype(dt)
    W[0] = 0
    W[1, 0] = 127.0                       # scale 1: halves round to even
    W[1, 1:9] = [0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5, 0.49]
    W[2, :] = 0
    W[2, K - 1] = np.finfo(dt).max        # the maximum in the last place
    if dt == np.float32:
        W[3, :] = 1e-44                   # the scale underflows
    W8, s = mmf.quantize_weights_int8(to_dev(W))
    ref8, refs = plain.quantize_rows(W)
    assert np.array_equal(s.cpu().numpy(), refs)
    assert np.array_equal(W8.cpu().numpy(), ref8)


@pytest.mark.parametrize("T", [5, 300])
def test_forward_is_the_pre_pass_and_the_product(T):
    K, N = 1024, 1000
    rng = np.random.default_rng(T)
    x = rng.normal(size=(T, K)).astype(np.float16)
    g = rng.uniform(0.5, 1.5, size=K).astype(np.float32)
    W = (rng.normal(size=(N, K)) * 0.02).astype(np.float16)
    W8, s = mmf.quantize_weights_int8(to_dev(W))
    y = mmf.int8_linear_forward(to_dev(x), W8, s, norm_w=to_dev(g), eps=1e-6)
    A, gamma, _ = gpu_act_quant(x, g=g, eps=1e-6)
    z = mmf.int8_matmul(to_dev(A), to_dev(gamma), W8, s)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    _check(z.cpu().numpy(), plain.int8_product(A, gamma, W8.cpu().numpy(), s.cpu().numpy()))
    # two roundings to 8 bits (at most half a step of 1/127 of the largest value) stay small
    # beside the layer itself: independent errors, so far below their worst case
    xh = x.astype(np.float64)
    xh = xh / np.sqrt((xh ** 2).mean(axis=1, keepdims=True) + 1e-6) * g
    full = xh @ W.astype(np.float64).T
    step = np.abs(xh).max(axis=1, keepdims=True) / 127 / np.sqrt(12)
    wstep = (np.abs(W.astype(np.float64)).max(axis=1) / 127 / np.sqrt(12))[None, :]
    std = np.sqrt(step ** 2 * (W.astype(np.float64) ** 2).sum(axis=1)[None, :] +
                  wstep ** 2 * (xh ** 2).sum(axis=1, keepdims=True))
    off = (z.cpu().numpy().astype(np.float64) - full) / std
    assert 0.5 < np.sqrt((off ** 2).mean()) < 1.5


@pytest.mark.parametrize("T", [8, 400])
def test_another_stream_and_a_replayed_graph(T):
    K, N = 512, 520
    A, gamma, W8, s = _inputs(T, K, N, seed=9)
    want = _product(A, gamma, W8, s)
    dA, dg, dW, ds = to_dev(A), to_dev(gamma), to_dev(W8), to_dev(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mmf.int8_matmul(dA, dg, dW, ds, stream=side)
    side.synchronize()
    assert np.array_equal(y.cpu().numpy(), want)
    out = torch.empty((T, N), dtype=torch.float16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmf.int8_matmul(dA, dg, dW, ds, out=out)
    dA.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    dA.copy_(torch.from_numpy(A))
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)


def test_outputs_beyond_32_bits():
    T, K, N = 70000, 16, 32000            # 2.2e9 outputs, 4.5 GB
    A, gamma, W8, s = _inputs(T, K, N, seed=21)
    dA, dg, dW, ds = (to_dev(x) for x in (A, gamma, W8, s))
    y = mmf.int8_matmul(dA, dg, dW, ds)
    for lo in (0, 67000, T - 200):
        want = mmf.int8_matmul(dA[lo:lo + 200], dg[lo:lo + 200], dW, ds)
        assert torch.equal(y[lo:lo + 200], want)
