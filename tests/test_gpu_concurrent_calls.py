"""Calls from several host threads at once.  The binding releases the interpreter's lock
inside the library, so one thread's call may run between any two steps of another's:
calls of the same kernel that want different amounts of shared memory used to refuse
one another's launch, about once in 3000 products and once in 20000 norms."""
import threading

import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _together(dev, calls, rounds):
    """Each call `rounds` times in a thread and on a stream of its own."""
    gate, failed = threading.Barrier(len(calls)), []

    def work(i, call):
        stream = torch.cuda.Stream(dev)
        stream.wait_stream(torch.cuda.default_stream(dev))
        gate.wait(60)
        for k in range(rounds):
            status = call(stream.cuda_stream)
            if status != flce.FLCE_OK:
                failed.append((i, status))
            if k % 100 == 99:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=work, args=a) for a in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, (len(failed), failed[:4])
    assert flce.get_error(dev) == flce.FLCE_OK


def test_products_of_different_token_counts(dev):
    """Token counts whose stages take different amounts of shared memory."""
    lib = flce.load_library()
    g = torch.Generator().manual_seed(1)
    head = flce.mxfp4_quantize(torch.randn(128, 512, generator=g).to(dev))
    calls, results = [], []
    for n in (8, 77, 40, 120):
        x = torch.randn(n, 512, generator=g).to(torch.bfloat16).to(dev)
        ws = torch.empty(lib.flce_mxfp4_logits_workspace_size(n, 512), dtype=torch.uint8, device=dev)
        z = torch.empty(n, 128, dtype=torch.bfloat16, device=dev)
        results.append((z, flce.mxfp4_logits(x, head)))
        calls.append(lambda s, n=n, x=x, ws=ws, z=z: lib.flce_mxfp4_logits(
            x.data_ptr(), 0, n, 512, 512, head.codes.data_ptr(), head.scales.data_ptr(), 128, 128, 0.0,
            z.data_ptr(), 0, 128, ws.data_ptr(), ws.numel(), s))
    _together(dev, calls, 20000)
    assert all(torch.equal(a, b) for a, b in results)


def test_layer_norms_of_different_widths(dev):
    """Streamed rows of widths whose rings take different amounts of shared memory."""
    lib = flce.load_library()
    g = torch.Generator().manual_seed(2)
    calls, results = [], []
    for n, h in ((300, 8192), (600, 4096), (300, 8192), (600, 4096)):
        x = torch.randn(n, h, generator=g).to(torch.bfloat16).to(dev)
        y = torch.empty_like(x)
        results.append((y, flce.layer_norm_forward(x)[0]))
        calls.append(lambda s, n=n, h=h, x=x, y=y: lib.flce_layer_norm_forward(
            x.data_ptr(), 0, n, h, h, None, None, 1, 1e-5, y.data_ptr(), h, None, None, s))
    _together(dev, calls, 60000)
    assert all(torch.equal(a, b) for a, b in results)


def test_selections_of_different_sizes(dev):
    lib = flce.load_library()
    g = torch.Generator().manual_seed(3)
    calls, results = [], []
    for b, k, v, m in ((1, 4, 30000, 4), (2, 64, 1024, 64), (4, 8, 50001, 16), (1, 1, 131072, 64)):
        z, s = torch.randn(b, k, v, generator=g).to(dev), -torch.rand(b, k, generator=g).to(dev)
        out = [torch.empty(b, m, dtype=t, device=dev) for t in (torch.float32, torch.int64, torch.int64)]
        ws = torch.empty(lib.flce_beam_select_workspace_size(b, k, v, m), dtype=torch.uint8, device=dev)
        results.append((out, flce.beam_select(z, s, num_select=m)))
        calls.append(lambda st, z=z, s=s, out=out, ws=ws, b=b, k=k, v=v, m=m: lib.flce_beam_select(
            z.data_ptr(), 1, b, k, v, v, s.data_ptr(), None, 0, m, *(t.data_ptr() for t in out),
            ws.data_ptr(), ws.numel(), st))
    _together(dev, calls, 2000)
    assert all(torch.equal(a, c) for got, want in results for a, c in zip(got, want))
