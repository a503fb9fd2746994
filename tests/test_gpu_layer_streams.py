"""The layer's calls on streams of the caller's own."""
import pytest
import torch

from test_gpu_block import EPS, problem
from test_gpu_block_weights import run, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def owner(t):
    """The stream that the allocator keeps t's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


def test_memory_belongs_to_the_stream_it_is_used_on(m):
    T = 64
    cfg, layer, x, resid, w, dout = problem(m, T, 35)
    off = torch.tensor([0, 20, T], dtype=torch.int32).cuda()
    fresh = problem(m, T, 35)[1]
    _, fs = fresh.block_forward(x, resid, w, EPS)
    floss, fbal = fresh.balance_loss(T, off)
    want = fresh.block_backward(fs, dout, balance=fbal)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, saved = layer.block_forward(x, resid, w, EPS, stream=st)
    loss, bal = layer.balance_loss(T, off, stream=st)
    got = layer.block_backward(saved, dout, balance=bal, stream=st)
    torch.cuda.synchronize()
    mine = [out, saved["h"], saved["y"], saved["rstd"], loss, bal["counts"], *got.values(), layer.workspace(T),
            layer.block_backward_workspace(T), *layer._wt.values()]
    assert [owner(t) == st.cuda_stream for t in mine] == [True] * len(mine)
    assert torch.equal(loss, floss)
    same(got, want)


def test_transposed_weights_made_on_another_stream(m):
    """The first backward, held up on one stream, fills the transposed copies; a second one on another stream waits for
    them."""
    T1, T2 = 64, 80
    cfg, layer, x1, r1, w, d1 = problem(m, T1, 37)
    fresh = problem(m, T1, 37)[1]
    g = torch.Generator().manual_seed(1)
    x2, r2, d2 = (torch.randn((T2, cfg["H"]), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    want1, want2 = run(fresh, x1, r1, w, d1), run(fresh, x2, r2, w, d2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(a):
        _, s1 = layer.block_forward(x1, r1, w, EPS)
    with torch.cuda.stream(b):
        _, s2 = layer.block_forward(x2, r2, w, EPS)
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        torch.cuda._sleep(1_000_000_000)
        g1 = layer.block_backward(s1, d1)
    with torch.cuda.stream(b):
        g2 = layer.block_backward(s2, d2)
    torch.cuda.synchronize()
    for got, want in ((g1, want1), (g2, want2)):
        same(got, {k: want[k] for k in got})


def test_layer_freed_while_another_stream_works(m):
    """A workspace made on one stream and used on another is not handed out again before that one is done."""
    T = 64
    cfg, layer, x, resid, w, dout = problem(m, T, 39)
    layer.block_forward(x, resid, w, EPS)
    want = layer.block_forward(x, resid, w, EPS)[0]
    nbytes, ptr = layer.workspace(T).numel(), layer.workspace(T).data_ptr()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(1)
    with torch.cuda.stream(st):
        torch.cuda._sleep(1_000_000_000)
        got = layer.block_forward(x, resid, w, EPS)[0]
    layer._ws.clear()
    layer._guarded = []
    taken = [torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(not (t.data_ptr() <= ptr < t.data_ptr() + nbytes) for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
