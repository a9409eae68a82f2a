"""CPU check that every entry point of the binding runs with the device of its tensors current.
Tensors on a second GPU are stood in for by a tensor that says it lies there; the check ends
where the device would be switched."""
import pytest
import torch

from selective_state_space_naju_amd import binding as nb

ENTRY_POINTS = ("scan_fwd", "block_fwd", "scan_bwd", "block_bwd", "scan_step", "block_step",
                "mixer_fwd", "mixer_bwd", "embed_fwd", "embed_bwd", "distill_fwd", "distill_bwd",
                "distill_fwd_bwd", "logits_process", "w4_quantize", "w4_linear")


class OnDeviceOne(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 1


class Switched(Exception):
    pass


@pytest.fixture
def second_device(monkeypatch):
    def switch(device):
        assert device == 1
        raise Switched
    monkeypatch.setattr(torch.cuda, "device", switch)
    monkeypatch.setattr(nb, "_current_device", lambda: 0, raising=False)
    return torch.zeros(2, 2).as_subclass(OnDeviceOne)


@pytest.mark.parametrize("name", ENTRY_POINTS)
def test_the_tensors_device_is_made_current(name, second_device):
    import inspect
    fn = getattr(nb, name)
    required = [p.name for p in inspect.signature(fn).parameters.values()
                if p.default is p.empty]
    with pytest.raises(Switched):
        fn(*[second_device] * len(required))
    with pytest.raises(Switched):
        fn(**{k: second_device for k in required})


def test_reading_a_workspaces_errors_switches_too(second_device):
    ws = nb.Workspace.__new__(nb.Workspace)
    ws.tensor, ws.nbytes = second_device, 256
    with pytest.raises(Switched):
        ws.error_flags()


def test_the_current_device_is_not_switched(monkeypatch, second_device):
    monkeypatch.setattr(nb, "_current_device", lambda: 1)
    with pytest.raises(Exception) as e:
        nb.w4_linear(second_device, second_device, second_device, 32)
    assert e.type is not Switched
