"""Host-side checks of the linear attention's descriptor and of what the binding passes on."""
import ctypes

import pytest
import torch

import ternary_weight_lm_b200 as mmf
from test_operators_host import A16, CUDA, INVALID, desc


# rows of o in one place: strides that are each at least a row, and are not enough together
@pytest.mark.parametrize("kw", [
    dict(o_t=128, o_h=128), dict(o_t=128, o_h=192), dict(o_t=384, o_h=128), dict(o_t=504, o_h=128),
    dict(o_t=128, o_h=128 * 598), dict(o_t=136, o_h=136),
    # the products pass 64 bits
    dict(o_t=1 << 61, o_h=1 << 61), dict(T=16777215, B=3, o_t=1 << 60, o_h=(1 << 60) + 8),
])
def test_rows_of_an_output_in_one_place_are_refused(kw):
    L, r = mmf.lib(), ctypes.byref(desc(**kw))
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, A16, 1 << 40, None) == INVALID
    T = kw.get("T", 600)
    r = ctypes.byref(desc(**{**kw, "T": min(T, 600), "B": min(T, 600)}))
    assert L.mmf_linattn_step(r, A16, A16, A16, A16, A16, None, 0, None) == INVALID
    if torch.cuda.is_available():
        return                   # what follows is not refused, and the addresses are not real
    # dout is only read
    assert L.mmf_linattn_backward(r, A16, A16, A16, A16, None, None, A16, A16, A16, None, A16,
                                  1 << 40, None) == CUDA


@pytest.mark.parametrize("kw", [
    dict(), dict(o_t=128, o_h=128 * 600), dict(o_t=136, o_h=136 * 600), dict(o_t=552, o_h=136),
    dict(T=1, B=1, o_t=8, o_h=128), dict(H=1, o_t=128, o_h=8), dict(o_t=512, o_h=128),
])
def test_rows_of_an_output_apart_are_taken(kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    L, r = mmf.lib(), ctypes.byref(desc(**kw))
    assert L.mmf_linattn_forward(r, A16, A16, A16, None, A16, None, A16, 1 << 40, None) == CUDA



# Segments are chosen for the kernel that runs.  The workspace has a state for each of them.
def test_segments_are_those_of_the_kernel_that_runs():
    need, grad = mmf.mmf_linattn_workspace_bytes, mmf.mmf_linattn_backward_workspace_bytes
    one = dict(T=16384, B=1, H=4)
    # backward, the tensor cores take heads of 64 and 128 only: other sizes run as in fp32
    for dk, dv in ((64, 192), (64, 256), (128, 192), (96, 128)):
        kw = dict(one, dk=dk, dv=dv)
        assert grad(desc(**kw)) == grad(desc(**kw, dt=0)) > 0
    assert need(desc(**one, dk=64, dv=192)) != need(desc(**one, dk=64, dv=192, dt=0)) > 0
    # heads of 128: a row that all tokens share has no tensor map, whichever tensor has it
    kw = dict(one, dk=128, dv=128)
    shared = {need(desc(**kw, **{n: 0})) for n in ("q_t", "k_t", "v_t")}
    assert len(shared) == 1 and need(desc(**kw)) not in shared and 0 not in shared
    shared = {grad(desc(**kw, **{n: 0})) for n in ("q_t", "k_t", "v_t")}
    assert len(shared) == 1 and grad(desc(**kw)) not in shared and 0 not in shared
    # heads further apart than a tensor map's columns go
    assert need(desc(**kw, k_h=1 << 30)) == need(desc(**kw, q_h=1 << 62)) == need(desc(**kw, q_t=0))


def test_the_descriptor_keeps_its_layout():
    # clear_outside stands where there was padding
    d = mmf.LinattnDesc
    assert (d.scale.offset, d.clear_outside.offset, d.log_decay.offset) == (40, 44, 48)
    assert ctypes.sizeof(d) == 120


class _OnGpu:
    """Stands for a tensor on the second GPU."""
    is_cuda, device = True, torch.device("cuda:1")

    def get_device(self):
        return 1


class _Stream:
    device, cuda_stream = torch.device("cuda:0"), 0


def test_a_stream_of_another_device_is_refused():
    def call(handle):
        raise AssertionError("launched")

    with pytest.raises(ValueError, match="stream is on cuda:0"):
        mmf._on(_OnGpu(), _Stream(), call)


def test_a_workspace_elsewhere_is_refused():
    dev = torch.device("meta")
    with pytest.raises(ValueError, match="ws is on cpu"):
        mmf._scratch(torch.zeros(512, dtype=torch.uint8), 512, dev)
    with pytest.raises(ValueError, match="contiguous"):
        mmf._scratch(torch.zeros(1024, dtype=torch.uint8, device=dev)[::2], 512, dev)
    ws = torch.zeros(512, dtype=torch.uint8, device=dev)
    assert mmf._scratch(ws, 512, dev) is ws and mmf._scratch(None, 0, dev) is None
    assert mmf._scratch(None, 300, dev).numel() == 300


@pytest.mark.parametrize("name", ["linattn_forward", "linattn_backward", "int8_linear_forward"])
def test_every_call_with_a_workspace_checks_it(name, monkeypatch):
    # as far as the workspace on the host: the launches are taken away
    monkeypatch.setattr(mmf, "_on", lambda t, stream, call: call(0))
    for f in ("mmf_linattn_forward", "mmf_linattn_backward", "mmf_int8_forward"):
        monkeypatch.setattr(mmf, f, lambda *a: None)
    x = torch.zeros(4, 2, 16)
    args = {"linattn_forward": (x, x, x, torch.zeros(2)),
            "linattn_backward": (x, x, x, torch.zeros(2), x),
            "int8_linear_forward": (torch.zeros(4, 128), torch.zeros(8, 128, dtype=torch.int8),
                                    torch.zeros(8))}[name]
    getattr(mmf, name)(*args, ws=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws is on meta"):
        getattr(mmf, name)(*args, ws=torch.zeros(1 << 16, dtype=torch.uint8, device="meta"))


def test_the_current_stream_without_torchs_private_calls(monkeypatch):
    for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, n, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda at: type("S", (), {"cuda_stream": 100 + at}))
    monkeypatch.setattr(mmf, "_current", None)
    assert mmf._on(_OnGpu(), None, lambda handle: handle) == 101
