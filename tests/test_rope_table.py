"""The rotation table: its values and its arguments, without a GPU."""
import math

import pytest
import torch

import newton_schulz_08_amd as nsa


def test_values():
    t = nsa.rope_table(5, 6, 100.0, device="cpu")
    assert t.shape == (5, 6) and t.dtype == torch.float32
    for p in range(5):
        for i in range(3):
            angle = p * 100.0 ** (-2 * i / 6)
            assert abs(float(t[p, i]) - math.cos(angle)) <= 2.0 ** -24 and abs(float(t[p, 3 + i]) - math.sin(angle)) <= 2.0 ** -24
    assert nsa.rope_table(3, 0, device="cpu").shape == (3, 0)


@pytest.mark.parametrize("rot", [1, 7, -2])
def test_odd_widths_are_refused(rot):
    with pytest.raises(ValueError, match="even"):
        nsa.rope_table(4, rot, device="cpu")


def test_devices_given_by_number(monkeypatch):
    """Device 0 is that device, whichever is current."""
    seen = []
    monkeypatch.setattr(torch.Tensor, "to", lambda self, device: seen.append(device) or self)
    nsa.rope_table(2, 2, device=0)
    nsa.rope_table(2, 2, device=1)
    nsa.rope_table(2, 2)
    assert seen == [0, 1, "cuda"]
    monkeypatch.undo()
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device, **kw: seen.append(device) or empty(*a, **kw))
    for device in (0, 1, None):
        try:
            nsa.alloc_workspace(512, device)
        except RuntimeError:
            pass    # host memory need not be aligned
    assert seen[3:] == [0, 1, "cuda"]
