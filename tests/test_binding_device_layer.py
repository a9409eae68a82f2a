"""CPU check that the entry points of the rest of a layer run with the device of their tensors
current, also where the first argument is not given; and that the update names a tensor that is
missing from its lists."""
import pytest
import torch

from selective_state_space_naju_amd import binding as nb
from test_binding_device import Switched, second_device  # noqa: F401  (a fixture)

CALLS = {
    "res_norm_fwd": lambda t: nb.res_norm_fwd(t, w_pre=t),
    "res_norm_bwd": lambda t: nb.res_norm_bwd(t, None, t, w_pre=t),
    "res_norm_bwd without dxn": lambda t: nb.res_norm_bwd(None, t, t, t),
    "res_norm_bwd by names": lambda t: nb.res_norm_bwd(dxn=None, dx_new=t, x_new=t, y=t),
    "linattn_fwd": lambda t: nb.linattn_fwd(t, t, t, t),
    "linattn_bwd": lambda t: nb.linattn_bwd(t, t, t, t, t),
    "linattn_step": lambda t: nb.linattn_step(t, t, t, t, t),
    "adamw_step": lambda t: nb.adamw_step([t], [t], [t], [t], 1, 1e-3),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device_is_made_current(name, second_device):  # noqa: F811
    with pytest.raises(Switched):
        CALLS[name](second_device)


@pytest.mark.parametrize("which", [1, 2, 3])
def test_a_missing_tensor_is_named(which, monkeypatch):
    monkeypatch.setattr(nb, "_stream", lambda dev: 0)
    lists = [[torch.zeros(4), torch.zeros(4)] for _ in range(4)]
    lists[which][1] = None
    with pytest.raises(ValueError, match=r"%s\[1\] is required" % "pgmv"[which]):
        nb.adamw_step(*lists, 1, 1e-3)
