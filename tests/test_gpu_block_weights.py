"""The block's backward after its weights have changed."""
import copy

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


def test_other_tensors_in_the_weights_places(m):
    """A layer given another layer's tensors reads those, and the first layer's copies stay its own."""
    T = 40
    cfg, layer, x, resid, w, dout = problem(m, T, 34)
    other = problem(m, T, 35)[1]
    args = (x, resid, w, dout)
    want, mine = run(other, *args), run(layer, *args)
    sib = layer.sibling()
    for k in ("w13", "s13", "w2", "s2", "wr", "bias"):
        setattr(layer, k, getattr(other, k))
    same(run(layer, *args), want)
    same(run(sib, *args), mine)


def test_expert_counted_from_the_end_and_a_copied_layer(m):
    T = 40
    cfg, layer, x, resid, w, dout = problem(m, T, 36)
    args = (x, resid, w, dout)
    run(layer, *args)
    twin = copy.deepcopy(layer)
    before = run(layer, *args)
    w13, w2 = (t.cuda() for t in S.gen_expert(3, cfg["H"], cfg["I"], 950))
    fresh = problem(m, T, 36)[1]
    fresh.set_expert(cfg["Nr"], w13, w2)
    layer.set_expert(-1, w13, w2)  # the shared expert
    same(run(layer, *args), run(fresh, *args))
    same(run(twin, *args), before)
    with pytest.raises(IndexError):
        layer.set_expert(layer.E, w13, w2)
