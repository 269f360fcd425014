"""Sizes of workspaces are the current device's: they grow with its multiprocessors, so a size that was asked for on one
device is not handed out on another. No GPU needed."""
import pytest
import torch

import linear_attention_ssm_gdp_gb300 as gdp


class Fake:
    """A library whose sizes are the current device's number."""

    def __init__(self):
        self.device = 0

    def gdp_attention_paged_workspace_size(self, *a):
        return 1000 + self.device

    def gdp_group_norm_workspace_size(self, *a):
        return 2000 + self.device


@pytest.fixture
def fake(monkeypatch):
    f = Fake()
    monkeypatch.setattr(gdp, "load", lambda: f)
    monkeypatch.setattr(gdp, "_current_device", lambda: f.device)
    return f


def test_attention(fake):
    args = (7, 1, 7, 4, 2, 72, 72, torch.bfloat16)
    for device in (0, 1, 0, 3):
        fake.device = device
        assert gdp.gdp_attention_paged_workspace_size(*args) == 1000 + device


def test_group_norm(fake):
    for device in (0, 1, 0, 3):
        fake.device = device
        assert gdp.gdp_group_norm_workspace_size(3, 77, 96, 2, torch.float32) == 2000 + device


def test_without_a_device(monkeypatch):
    """Where there is none, sizes can be asked for all the same."""
    def none():
        raise RuntimeError("no device")
    monkeypatch.setattr(gdp, "load", lambda: Fake())
    monkeypatch.setattr(gdp, "_current_device", none)
    assert gdp.gdp_attention_paged_workspace_size(5, 1, 5, 4, 2, 72, 72, torch.bfloat16) == 1000
    assert gdp.gdp_group_norm_workspace_size(3, 78, 96, 2, torch.float32) == 2000
