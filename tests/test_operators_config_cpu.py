"""What is given as the configuration is a MoeConfig: other structures are
refused, not read as one."""
import ctypes as C

import pytest
import torch


class Other(C.Structure):
    _fields_ = [("a", C.c_int32)]


@pytest.mark.parametrize("cfg", [Other(1), C.c_int64(3), None, {"H": 128}, (C.c_int32 * 9)(128, 128, 16, 4, 1, 0, 0, 0, 0)],
                         ids=lambda c: type(c).__name__)
def test_other_structures_are_refused(cfg):
    import sparse_moe_layer_expert_b200 as m
    z, idx, off = torch.zeros((1, 2, 16)), torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(m.MoeError, match="MoeConfig"):
        m.moe_balance_loss(cfg, z, idx, off)
    with pytest.raises(m.MoeError, match="MoeConfig"):
        m.moe_router_backward(cfg, z, idx, dlogits=True)
