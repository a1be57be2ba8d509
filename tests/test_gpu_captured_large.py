"""Graphs of the launches that large decoding steps make: the selection in two launches
(beyond one cluster per item), the product on CTA pairs, and a whole captured step of
such sizes, replayed with other inputs.  Replays equal the calls bit for bit."""
import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("b,k,v,m", [(2, 4, 50001, 4), (3, 9, 5000, 18), (20, 4, 3001, 64), (1, 64, 9000, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_selection(dev, b, k, v, m, dtype):
    g = torch.Generator(device=dev).manual_seed(v)
    z = torch.randn(b, k, v, generator=g, device=dev).to(dtype)
    s = -torch.rand(b, k, generator=g, device=dev)
    done = torch.rand(b, k, generator=g, device=dev) < 0.3
    graph = torch.cuda.CUDAGraph()
    flce.beam_select(z, s, num_select=m, finished=done, eos_token=5)
    with torch.cuda.graph(graph):
        out = flce.beam_select(z, s, num_select=m, finished=done, eos_token=5)
    for _ in range(3):
        z.copy_(torch.randn(b, k, v, generator=g, device=dev))
        s.copy_(-torch.rand(b, k, generator=g, device=dev))
        done.copy_(torch.rand(b, k, generator=g, device=dev) < 0.3)
        graph.replay()
        assert _same(out, flce.beam_select(z, s, num_select=m, finished=done, eos_token=5))


@pytest.mark.parametrize("n,v", [(193, 1000), (500, 3001), (77, 5001)])
def test_product(dev, n, v):
    g = torch.Generator(device=dev).manual_seed(n)
    x = torch.randn(n, 320, generator=g, device=dev)
    head = flce.mxfp4_quantize(torch.randn(v, 320, generator=g, device=dev))
    graph = torch.cuda.CUDAGraph()
    flce.mxfp4_logits(x, head, softcap=20.0)
    with torch.cuda.graph(graph):
        z = flce.mxfp4_logits(x, head, softcap=20.0)
    for _ in range(3):
        x.copy_(torch.randn(n, 320, generator=g, device=dev))
        flce.mxfp4_quantize(torch.randn(v, 320, generator=g, device=dev), out=head)  # another head in its place
        graph.replay()
        assert torch.equal(z, flce.mxfp4_logits(x, head, softcap=20.0))
    assert flce.get_error(dev) == flce.FLCE_OK


def test_two_graphs_with_one_workspace(dev):
    """Replayed one after the other on one stream they may share it."""
    lib = flce.load_library()
    g = torch.Generator(device=dev).manual_seed(3)
    head = flce.mxfp4_quantize(torch.randn(2000, 256, generator=g, device=dev))
    xs = [torch.randn(n, 256, generator=g, device=dev) for n in (300, 40)]
    ws = torch.empty(lib.flce_mxfp4_logits_workspace_size(300, 256), dtype=torch.uint8, device=dev)
    want = [flce.mxfp4_logits(x, head) for x in xs]
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            z = flce.mxfp4_logits(x, head, workspace=ws)
        graphs.append((graph, z))
    for order in ((0, 1), (1, 0), (0, 1, 0)):
        for i in order:
            graphs[i][0].replay()
    assert _same([z for _, z in graphs], want)


@pytest.mark.parametrize("b,k,v,h", [(6, 9, 20001, 64), (50, 4, 1500, 130)])
def test_step(dev, b, k, v, h):
    """More than 8 beams; more than 192 rows."""
    g = torch.Generator(device=dev).manual_seed(b)
    head = flce.mxfp4_quantize(torch.randn(v, h, generator=g, device=dev))
    w, bias = torch.rand(h, generator=g, device=dev), torch.randn(h, generator=g, device=dev)
    draw = lambda: (torch.randn(b, k, h, generator=g, device=dev),  # noqa: E731
                    -torch.rand(b, k, generator=g, device=dev), torch.rand(b, k, generator=g, device=dev) < 0.2)
    first = draw()
    states = [torch.randn(b, k, 3, 7, 16, generator=g, device=dev) for _ in range(2)]
    keep = [t.clone() for t in states]
    step = flce.CapturedBeamStep(first[0], head, first[1], norm_weight=w, norm_bias=bias, softcap=30.0,
                                 finished=first[2], eos_token=3, states=states)
    assert _same(states, keep)
    for _ in range(3):
        hidden, scores, done = draw()
        z = flce.mxfp4_logits(flce.layer_norm(hidden, w, bias), head, softcap=30.0)
        want = flce.beam_select(z, scores, finished=done, eos_token=3)
        flce.beam_reorder(keep, want[1])
        step.set_inputs(hidden, scores, done)
        got = step.replay()
        assert _same(got, want) and torch.equal(step.logits, z) and _same(states, keep)
    assert flce.get_error(dev) == flce.FLCE_OK
