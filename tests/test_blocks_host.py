"""Workspaces of blocks.py, without a GPU: one set for each device, and none made inside a capture."""

import pytest
import torch

from w4a8_codebook_quantized_rotate_b200 import blocks


class Layer:
    """What AttentionBlock asks of a layer, on a device without memory."""

    def __init__(self, n, k, device):
        self.n, self.k, self.device = n, k, torch.device(device)

    def prepare(self, m):
        return torch.zeros(m, device=self.device)


def test_workspaces_are_their_devices():
    held = blocks._Workspaces(lambda m: 64 * m)
    one, two = held.get(4, "cpu"), held.get(4, torch.device("meta"))
    assert one.device.type == "cpu" and two.device.type == "meta" and one.numel() == two.numel() == 256
    assert held.get(4, "cpu") is one and held.get(4, "meta") is two
    assert held.get(2, "cpu") is one and held.get(3, "meta") is two          # the last one of the device serves
    assert held.get(5, "cpu").numel() == 512 and held.get(5, "meta").numel() == 512
    assert held.get(4, "cpu") is one and held.get(8, "meta").numel() == 512


def test_block_prepares_where_its_layers_are():
    block = blocks.AttentionBlock(Layer(4 * 64, 128, "meta"), Layer(128, 2 * 64, "meta"), 2, 1, 64)
    block._workspaces = blocks._Workspaces(lambda m: 64 * m)
    assert block.prepare(3).device.type == "meta"
    assert block.prepare(3, "cpu").device.type == "cpu"


def test_no_workspace_is_made_inside_a_capture(monkeypatch):
    held = blocks._Workspaces(lambda m: 64 * m)
    monkeypatch.setattr(blocks, "_capturing", lambda device: True)
    with pytest.raises(RuntimeError, match="prepare\\(4\\)"):
        held.get(4, "cpu")
    monkeypatch.setattr(blocks, "_capturing", lambda device: False)
    ws = held.get(4, "cpu")
    monkeypatch.setattr(blocks, "_capturing", lambda device: True)
    assert held.get(4, "cpu") is ws and held.get(2, "cpu") is ws             # what is there may be used
    with pytest.raises(RuntimeError):
        held.get(5, "cpu")
    with pytest.raises(RuntimeError):
        held.get(4, "meta")
