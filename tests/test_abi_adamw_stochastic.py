"""CPU checks of how the AdamW step's 8-bit states may be rounded (no call here touches a GPU)."""
import pytest
import torch

from selective_state_space_naju_amd import binding as nb


def test_state_bits():
    def call(bits, step=1):
        return nb.lib().naju_adamw_step(0, None, nb.F32, bits, 1e-3, 0.9, 0.999, 1e-8, 0.0, step,
                                        None, None, None, None)
    for bits in (32, 8, 8 + nb.STOCHASTIC):
        assert call(bits) == nb.OK
        assert call(bits, 0) == nb.EINVAL
    for bits in (0, nb.STOCHASTIC, 32 + nb.STOCHASTIC, 8 + 2 * nb.STOCHASTIC, -8):
        assert call(bits) == nb.EUNSUPPORTED
        assert "state_bits" in nb.last_error()


def test_binding_refuses_it_with_32_bits(monkeypatch):
    monkeypatch.setattr(nb, "_stream", lambda dev: 0)
    p = [torch.zeros(5)]
    with pytest.raises(ValueError, match="stochastic goes with 8-bit states"):
        nb.adamw_step(p, p, p, p, 1, 1e-3, stochastic=True)
