"""Edges of the router's operators: affinities below FP32's normal range, and
an allocation that fails."""
import numpy as np
import pytest
import torch

from oracle import block as O
from test_gpu_operators import U, f64, z_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


@pytest.mark.parametrize("Nr,scale", [(16, 1.0), (16, 65536.0), (1, 1.0), (33, 2.0 ** -10)])
def test_affinities_below_the_normal_range(m, Nr, scale):
    """Logits in (-88.7, -87.4): s = 1 / (1 + e^-z) is subnormal there (as the router's own affinities are), its shares
    are ordinary numbers, and so are the loss and its gradient, a scaled loss's too."""
    Kr, T = min(4, Nr), 6
    g = torch.Generator().manual_seed(Nr)
    z = -87.4 - 1.3 * torch.rand((1, T, Nr), generator=g)
    z[0, 0] = -88.0
    z[0, 1] = -88.722
    idx = torch.arange(Kr, dtype=torch.int32).repeat(T, 1)
    cfg = m.config(128, 128, Nr, Kr)
    off = [0, 2, T]
    offd = torch.tensor(off, dtype=torch.int32).cuda()
    loss, counts = m.moe_balance_loss(cfg, z.cuda(), idx.cuda(), offd, alpha=0.3)
    zn, idn = z.double().sum(0).numpy(), idx.numpy().astype(np.int64)
    lr, cr = O.balance_loss(zn, idn, off, 0.3)
    # subnormal s: quantum 2^-149, half of one beside at least 2^-128
    sub = 2.0 ** -22
    assert (np.abs(f64(loss) - lr) <= (2 * z_tol(z) + 2 * sub + 60 * U) * lr).all()
    dloss = torch.full((2,), scale)
    dl, _, _ = m.moe_router_backward(cfg, z.cuda(), idx.cuda(), dlogits=True,
                                     balance=dict(seq_offsets=offd, counts=counts, dloss=dloss.cuda(), alpha=0.3))
    ref, mag = O.router_dlogits(zn, idn, off=off, counts=cr, dloss=dloss.numpy(), alpha=0.3)
    assert (np.abs(f64(dl) - ref) <= (4 * z_tol(z) + 4 * sub + 40 * U) * mag + 1e-40).all()


def test_allocation_failure_is_torchs_own(m):
    """An output that does not fit raises torch.OutOfMemoryError (before anything is launched)."""
    T, H, Nr, Kr = 1 << 16, 7168, 4, 1
    cfg = m.config(H, 128, Nr, Kr)
    z = torch.zeros((1, T, Nr), device="cuda")
    idx = torch.zeros((T, Kr), dtype=torch.int32, device="cuda")
    wr = torch.zeros((Nr, H), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.mem_get_info()[1]
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
        with pytest.raises(torch.OutOfMemoryError):
            m.moe_router_backward(cfg, z, idx, wr=wr, dx=True)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
