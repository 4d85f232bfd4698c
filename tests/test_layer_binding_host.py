"""Refusals of the layer's binding that need no GPU: what would reach past a buffer, or read what the
same call writes."""
import types

import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import kda as binding, layer


def space(workspace, need=4096):
    return layer._space(types.SimpleNamespace(nbytes=need, device=torch.device("cpu")), workspace)


@pytest.mark.parametrize("workspace", [torch.empty(1, dtype=torch.uint8).expand(8192),
                                       torch.empty((2, 4096), dtype=torch.uint8).t(),
                                       torch.empty(16384, dtype=torch.uint8)[::2]])
def test_workspace_has_to_be_one_stretch(workspace):
    """Its bytes are counted from its element count, which only a contiguous tensor has behind its
    address."""
    with pytest.raises(ValueError, match="contiguous"):
        space(workspace)
    with pytest.raises(ValueError, match="contiguous"):
        binding._workspace(4096, workspace, torch.device("cpu"))


def test_workspace_has_to_be_on_the_device():
    ws = torch.empty(8192, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        binding._workspace(4096, ws, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="device"):
        layer._space(types.SimpleNamespace(nbytes=4096, device=torch.device("cuda", 0)), ws)


def test_workspace_of_any_type_and_its_size():
    ws = torch.empty(1024, dtype=torch.float32)
    assert space(ws) == (ws, ws.data_ptr(), 4096)
    with pytest.raises(ValueError, match="4096 bytes"):
        space(ws[1:])


def test_outputs_do_not_overwrite_what_a_call_still_reads():
    x, w, v = torch.zeros(8, 8), torch.zeros(8, 8), torch.zeros(8)
    for out in (x, w, x.view(8, 8)):
        with pytest.raises(ValueError, match="memory of its own"):
            kda.linear(x, w, out=out)
    with pytest.raises(ValueError, match="memory of its own"):
        kda.residual_norm(x, v, out=w, h_out=w)
    e = torch.zeros(0, 8)
    with pytest.raises(ValueError, match="CUDA"):              # no rows: nothing to share
        kda.linear(e, w, out=torch.zeros(0, 8))
