"""The device and the stream that the binding's calls launch on (CPU: tensors without storage on
devices that need not exist, a library that only notes where it was called)."""
import contextlib
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import hadamard_rotated_precision_halo_amd as H


class Machine:
    """Two GPUs, of which 0 is current, and the launches made on them."""

    def __init__(self, monkeypatch):
        self.device, self.streams, self.launches, self.switches = 0, {0: 100, 1: 101}, [], 0
        monkeypatch.setattr(H, "lib", lambda: self)
        monkeypatch.setattr(H, "_current_device", lambda: self.device)
        monkeypatch.setattr(H, "_current_stream", lambda index: self.streams[index])
        monkeypatch.setattr(H, "_ptr", lambda t: None if t is None else 1)
        monkeypatch.setattr(H, "_p", lambda t: None if t is None else 1)
        monkeypatch.setattr(torch.cuda, "current_stream", self.current_stream)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)

    def current_stream(self, device=None):
        index = self.device if device is None else torch.device(device).index
        s = object.__new__(Stream)
        s.device, s.cuda_stream = torch.device("cuda", index), self.streams[index]
        return s

    @contextlib.contextmanager
    def stream(self, s):
        self.switches += 1
        was = self.device, dict(self.streams)
        self.device = s.device.index
        self.streams[self.device] = s.cuda_stream
        yield
        self.device, self.streams = was

    def __getattr__(self, name):
        if name.endswith("_bytes") or name.endswith("_bytes_ex"):
            return lambda *a: 256

        def launch(*a):
            self.launches.append((name, self.device, getattr(a[-1], "value", a[-1])))
            return 0
        return launch


class Stream:
    """What a torch.cuda.Stream shows of itself."""


def calls(dev):
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    x, w, dy = (torch.empty(s, dtype=bf, device=dev) for s in ((64, 128), (32, 128), (64, 32)))
    v, b = torch.empty(128, dtype=bf, device=dev), torch.empty(32, dtype=bf, device=dev)
    one, sw = torch.empty(64, device=dev), torch.empty(32, device=dev)
    q, qw, e = (torch.empty(s, dtype=t, device=dev) for s, t in (((64, 128), i8), ((32, 128), i8),
                                                                 ((64, 128), torch.float8_e4m3fn)))
    idx, tl = torch.empty((64, 4), dtype=torch.int32, device=dev), torch.empty((64, 4), device=dev)
    return {
        "fwht_quant": lambda **k: H.fwht_quant(x, H.COLS, 64, **k),
        "fwht_quant_dual": lambda **k: H.fwht_quant_dual(x, 64, **k),
        "fwht_quant_noalloc": lambda **k: H.fwht_quant_noalloc(x, q, one, H.ROWS, 64, **k),
        "gemm_i8": lambda **k: H.gemm_i8(q, one, q, one, **k),
        "gemm_fp8": lambda **k: H.gemm_fp8(e, one, e, one, **k),
        "linear_fwd": lambda **k: H.linear_fwd(x, w, 64, **k),
        "linear_bwd": lambda **k: H.linear_bwd(dy, x, w, 32, **k),
        "block_norm_fwd": lambda **k: H.block_norm_fwd(x, x, v, v, v, **k),
        "block_norm_bwd": lambda **k: H.block_norm_bwd(x, x, x, x, v, v, v, one, one, **k),
        "distill_fwd": lambda **k: H.distill_fwd(x, idx, tl, **k),
        "distill_bwd": lambda **k: H.distill_bwd(one, x, one, idx, tl, **k),
        "distill_fwd_bwd": lambda **k: H.distill_fwd_bwd(x, idx, tl, one, **k),
        "linear_act_fwd": lambda **k: H.linear_act_fwd(x, w, 64, bias=b, want_z=True, **k),
        "linear_act_q": lambda **k: H.linear_act_q(x, qw, sw, 64, **k),
        "linear_act_bwd": lambda **k: H.linear_act_bwd(dy, dy, x, w, 32, activation="silu", **k),
    }


NAMES = sorted(["fwht_quant", "fwht_quant_dual", "fwht_quant_noalloc", "gemm_i8", "gemm_fp8", "linear_fwd",
                "linear_bwd", "block_norm_fwd", "block_norm_bwd", "distill_fwd", "distill_bwd",
                "distill_fwd_bwd", "linear_act_fwd", "linear_act_q", "linear_act_bwd"])


@pytest.fixture
def machine(monkeypatch):
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")
        yield Machine(monkeypatch)


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_launches_on_its_tensors_device(machine, name, index):
    out = calls(f"cuda:{index}")[name]()
    assert [l[1:] for l in machine.launches] == [(index, 100 + index)]
    assert machine.switches == (0 if index == 0 else 1)      # nothing to switch on the current device
    assert machine.device == 0                               # and the current device is the caller's again
    for t in out if isinstance(out, tuple) else (out,):
        assert t is None or t.device == torch.device("cuda", index)


def test_the_rate_probe_launches_on_its_streams_device(machine, monkeypatch):
    other = machine.current_stream("cuda:1")
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    H.mfma_rate_probe(0, 4, stream=other)
    H.mfma_rate_probe(0, 4)
    assert [l[1:] for l in machine.launches] == [(1, 101), (0, 100)] and machine.device == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_call_given_a_stream_allocates_on_it(machine, monkeypatch, name):
    """The allocator may hand on memory as soon as its stream's work reaches the point where it was
    freed: outputs and workspaces of another stream than the kernels' could be handed on early."""
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    call, at = calls("cuda:0")[name], []
    side = machine.current_stream("cuda:0")
    side.cuda_stream = 777
    for n in ("empty", "empty_like"):
        def spy(*a, real=getattr(torch, n), **k):
            at.append(machine.streams[machine.device])
            return real(*a, **k)
        monkeypatch.setattr(torch, n, spy)
    call(stream=side)
    assert machine.launches[-1][1:] == (0, 777) and machine.streams[0] == 100
    assert set(at) <= {777} and (at or name == "fwht_quant_noalloc"), at
    other = machine.current_stream("cuda:1")
    with pytest.raises(ValueError, match="stream"):
        call(stream=other)
