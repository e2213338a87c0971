"""The device and the stream of the gated layer's calls and of those on kept activations (CPU, on the
machine of test_binding_devices)."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import hadamard_rotated_precision_halo_amd as H
import test_binding_devices as D


def calls(dev):
    bf, i8, u8 = torch.bfloat16, torch.int8, torch.uint8
    x, w, dy = (torch.empty(s, dtype=bf, device=dev) for s in ((64, 128), (64, 128), (64, 32)))
    z, sw = torch.empty((64, 64), dtype=bf, device=dev), torch.empty(64, device=dev)
    qw = torch.empty((64, 128), dtype=i8, device=dev)
    kx = H.Checkpoint(torch.empty((64, 128), dtype=i8, device=dev), torch.empty((64, 4), dtype=u8, device=dev))
    kz = H.Checkpoint(torch.empty((128, 32), dtype=i8, device=dev), torch.empty((128, 1), dtype=u8, device=dev))
    ka = H.Checkpoint(torch.empty((64, 64), dtype=i8, device=dev), torch.empty((64, 2), dtype=u8, device=dev))
    return {
        "checkpoint_pack": lambda **k: H.checkpoint_pack(x, **k),
        "checkpoint_unpack": lambda **k: H.checkpoint_unpack(kx, **k),
        "linear_glu_fwd": lambda **k: H.linear_glu_fwd(x, w, 64, want_z=True, **k),
        "linear_glu_fwd_kept": lambda **k: H.linear_glu_fwd(x, w, 64, want_z=i8, **k)[1],
        "linear_act_fwd_kept": lambda **k: H.linear_act_fwd(x, w, 64, want_z=i8, **k)[1],
        "linear_glu_q": lambda **k: H.linear_glu_q(x, qw, sw, 64, **k),
        "linear_glu_bwd": lambda **k: H.linear_glu_bwd(dy, z, x, w, 32, **k),
        "linear_glu_bwd_kept": lambda **k: H.linear_glu_bwd(dy, kz, kx, w, 32, **k),
        "linear_act_bwd_kept": lambda **k: H.linear_act_bwd(z, ka, kx, w, 32, activation="silu", **k),
    }


NAMES = sorted(["checkpoint_pack", "checkpoint_unpack", "linear_glu_fwd", "linear_glu_fwd_kept",
                "linear_act_fwd_kept", "linear_glu_q", "linear_glu_bwd", "linear_glu_bwd_kept",
                "linear_act_bwd_kept"])


@pytest.fixture
def machine(monkeypatch):
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")
        yield D.Machine(monkeypatch)


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_launches_on_its_tensors_device(machine, name, index):
    out = calls(f"cuda:{index}")[name]()
    assert [l[1:] for l in machine.launches] == [(index, 100 + index)]
    assert machine.switches == (0 if index == 0 else 1) and machine.device == 0
    for t in out if isinstance(out, tuple) else (out,):
        assert t is None or t.device == torch.device("cuda", index)


@pytest.mark.parametrize("name", NAMES)
def test_a_call_given_a_stream_allocates_on_it(machine, monkeypatch, name):
    monkeypatch.setattr(torch.cuda, "Stream", D.Stream)
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
    assert set(at) == {777}, at
    with pytest.raises(ValueError, match="stream"):
        call(stream=machine.current_stream("cuda:1"))


def test_operands_of_another_device_are_refused(machine):
    here, there = calls("cuda:0"), torch.empty((128, 32), dtype=torch.int8, device="cuda:1")
    assert here["linear_glu_bwd_kept"]()
    powers = torch.empty((128, 1), dtype=torch.uint8, device="cuda:0")
    bf = torch.bfloat16
    x, w, dy = (torch.empty(s, dtype=bf, device="cuda:0") for s in ((64, 128), (64, 128), (64, 32)))
    with pytest.raises(ValueError, match="z's codes"):
        H.linear_glu_bwd(dy, H.Checkpoint(there, powers), x, w, 32)
    with pytest.raises(ValueError, match="powers"):
        H.checkpoint_unpack(H.Checkpoint(there, powers))
