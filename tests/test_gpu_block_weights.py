"""The block's backward after its weights have changed, and on streams of the
caller's own."""
import pytest
import torch

import moe_synth as S
from test_gpu_block import EPS, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import sparse_moe_layer_expert_b200 as pkg
    return pkg


def run(layer, x, resid, w, dout):
    out, saved = layer.block_forward(x, resid, w, EPS)
    g = layer.block_backward(saved, dout)
    return dict(g, out=out, layer_dx=layer.backward(saved["y"], dout)[0])


def same(a, b):
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def new_experts(cfg):
    """Other weights of two routed experts and the shared one."""
    return {e: tuple(t.cuda() for t in S.gen_expert(e, cfg["H"], cfg["I"], 900 + e)) for e in (0, 3, cfg["Nr"])}


def test_block_backward_after_new_expert_weights(m):
    """Every gradient is that of the weights the layer has now, in the layer, in a sibling that shares them, and in a
    graph captured before."""
    T = 96
    cfg, layer, x, resid, w, dout = problem(m, T, 31)
    args = (x, resid, w, dout)
    sib = layer.sibling()
    run(layer, *args), run(sib, *args)
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        captured = run(layer, *args)
    fresh = problem(m, T, 31)[1]
    for e, (w13, w2) in new_experts(cfg).items():
        fresh.set_expert(e, w13, w2)
        layer.set_expert(e, w13, w2)
    want = run(fresh, *args)
    same(run(layer, *args), want)
    same(run(sib, *args), want)
    graph.replay()
    torch.cuda.synchronize()
    same(captured, want)
    layer.check(), sib.check()


def test_weights_written_in_place(m):
    """Codes and scales written past set_expert: weights_changed() says so."""
    T = 40
    cfg, layer, x, resid, w, dout = problem(m, T, 33)
    args = (x, resid, w, dout)
    before = run(layer, *args)
    fresh = problem(m, T, 33)[1]
    for e, (w13, w2) in new_experts(cfg).items():
        fresh.set_expert(e, w13, w2)
    for k in ("w13", "s13", "w2", "s2"):
        getattr(layer, k).copy_(getattr(fresh, k))
    layer.weights_changed()
    want = run(fresh, *args)
    assert not torch.equal(before["dx"], want["dx"])
    same(run(layer, *args), want)


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
        torch.cuda._sleep(200_000_000)
        g1 = layer.block_backward(s1, d1)
    with torch.cuda.stream(b):
        g2 = layer.block_backward(s2, d2)
    torch.cuda.synchronize()
    for got, want in ((g1, want1), (g2, want2)):
        same(got, {k: want[k] for k in got})
