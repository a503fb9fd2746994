"""The norm's E4M3 codes, bit for bit: the FP32 y is reproduced on the host
from the call's own rstd (two IEEE products), and its codes are those of the
correctly rounded quotient y / S, S the correctly rounded amax / 448 -- as
fp8_quant_1x128 takes them.  Most values are put within a few FP32 steps of the
middle between two codes, where any other rounding of the quotient shows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def host_y(h, rstd, w):
    return (h.cpu().float() * rstd.cpu()[:, None]) * w.cpu()


def near_ties(h, rstd, S, amax, g):
    """Weights that put y next to code midpoints of its tile's scale; channel 0 of each tile keeps the amax."""
    n = (h.cpu().float() * rstd.cpu()[:, None])[0]
    H = n.numel()
    e = torch.randint(-5, 8, (H,), generator=g).double()
    k = torch.randint(0, 8, (H,), generator=g).double()
    tie = (torch.exp2(e) * (1 + (2 * k + 1) / 16)).clamp(max=432.0)
    sign = torch.where(torch.rand((H,), generator=g) < 0.5, -1.0, 1.0).double()
    off = 1 + torch.randint(-3, 4, (H,), generator=g).double() * 2.0 ** -24
    y = sign * tie * S.double().repeat_interleave(128) * off
    w = (y / n.double()).float()
    w[::128] = amax
    return w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 7168), (700, 7168), (2, 32768), (1300, 2048)])
def test_codes_next_to_ties(m, T, H, dtype):
    g = torch.Generator().manual_seed(T + H)
    row = (torch.rand((H,), generator=g) + 0.5).to(dtype)
    x = row.expand(T, H).contiguous().cuda()
    # first only the channel that sets each tile's scale
    amax = torch.rand((H // 128,), generator=g) * 2000 + 300
    w = torch.zeros(H)
    w[::128] = amax
    _, _, _, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, None, w.cuda())
    w = near_ties(x[:1], rstd[:1], s[0].cpu(), amax, g)
    _, y, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x, None, w.cuda())
    y32 = host_y(x, rstd, w)
    assert torch.equal(y.cpu(), y32.to(torch.bfloat16))
    tiles = y32.view(T, H // 128, 128)
    want_s = tiles.abs().amax(2) / 448.0
    assert torch.equal(s.cpu(), want_s)
    codes = (tiles / want_s[:, :, None]).view(T, H).to(torch.float8_e4m3fn).view(torch.uint8)
    diff = (q.cpu() != codes).sum().item()
    assert diff == 0, f"{diff} of {codes.numel()} codes differ"


@pytest.mark.parametrize("pow2", [False, True])
def test_codes_of_small_and_signed_zero_values(m, pow2):
    """Zeros keep their sign, tiny tiles their codes."""
    T, H = 5, 512
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H), generator=g)
    x[0, 5], x[0, 6] = 0.0, -0.0
    w = torch.randn((H,), generator=g)
    w[128:256] *= 2.0 ** -110  # scales below 2^-100
    w[256:384] *= 2.0 ** 90
    _, _, q, s, rstd = m.fp8_add_rmsnorm_quant_1x128(x.cuda(), None, w.cuda(), pow2=pow2)
    tiles = host_y(x, rstd, w).view(T, H // 128, 128)
    if not pow2:
        assert torch.equal(s.cpu(), tiles.abs().amax(2) / 448.0)
    codes = (tiles / s.cpu()[:, :, None]).view(T, H).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(q.cpu(), codes)
