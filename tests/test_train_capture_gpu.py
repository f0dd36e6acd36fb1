"""The training-step operators in CUDA graphs: calls that share the context's workspace on parallel branches of one
graph, next to calls outside of it, and what a capture refuses."""
import ctypes

import pytest
import torch

from cross_vendor_gradient_gb300 import Context, GbError
from cross_vendor_gradient_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture()
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with Context([1]) as c:
        yield c


def norm_sets(seed, sizes):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, device="cuda", generator=g) for n in sizes]


class Rows:
    """A gradient of rms_norm, and where it goes."""

    def __init__(self, seed, rows, cols):
        g = torch.Generator("cuda").manual_seed(seed)
        self.dy, self.h = (torch.randn(rows, cols, device="cuda", generator=g) for _ in range(2))
        self.w, self.rstd = torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda")
        self.dx, self.dw = torch.zeros_like(self.h), torch.zeros_like(self.w)

    def run(self, ctx, stream=None):
        ctx.rms_norm_backward(self.dy, self.h, self.w, self.rstd, self.dx, self.dw, stream=stream)


def test_parallel_branches_of_one_graph_do_not_share_partial_sums(ctx):
    """Norms and gradients of one context, captured on two streams that fork and join: every replay has the bits of
    calls one after another."""
    sets = norm_sets(1, [3_000_000, 40_000, 2_000_000, 700])
    rows = [Rows(2, 4000, 512), Rows(3, 3000, 768)]
    want = [torch.zeros(2, device="cuda") for _ in sets]
    for g, o in zip(sets, want):
        ctx.grad_norm([g], o, max_norm=1.0)
    for r in rows:
        r.run(ctx)
    want_rows = [(r.dx.clone(), r.dw.clone()) for r in rows]
    outs = [torch.zeros(2, device="cuda") for _ in sets]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        ctx.grad_norm([sets[0]], outs[0], max_norm=1.0)
        ctx.grad_norm([sets[1]], outs[1], max_norm=1.0, stream=side)
        rows[0].run(ctx)
        ctx.grad_norm([sets[2]], outs[2], max_norm=1.0, stream=side)
        rows[1].run(ctx, stream=side)
        ctx.grad_norm([sets[3]], outs[3], max_norm=1.0)
        main.wait_stream(side)
    for _ in range(20):
        for t in outs + [r.dx for r in rows] + [r.dw for r in rows]:
            t.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
        for r, (dx, dw) in zip(rows, want_rows):
            assert torch.equal(r.dx, dx) and torch.equal(r.dw, dw)


def test_a_graph_runs_next_to_calls_outside_of_it(ctx):
    """A graph's norm and gradient on one stream, others called at the same time on another stream."""
    sets = norm_sets(4, [3_000_000, 1_500_000])
    rows = [Rows(5, 4000, 512), Rows(6, 2000, 1024)]
    want = [torch.zeros(2, device="cuda") for _ in sets]
    for g, o, r in zip(sets, want, rows):
        ctx.grad_norm([g], o, max_norm=1.0)
        r.run(ctx)
    want_rows = [(r.dx.clone(), r.dw.clone()) for r in rows]
    outs = [torch.zeros(2, device="cuda") for _ in sets]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ctx.grad_norm([sets[0]], outs[0], max_norm=1.0)
        rows[0].run(ctx)
    for _ in range(20):
        for t in outs + [r.dw for r in rows]:
            t.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        for _ in range(3):
            ctx.grad_norm([sets[1]], outs[1], max_norm=1.0, stream=side)
            rows[1].run(ctx, stream=side)
        torch.cuda.synchronize()
        for o, w, r, (dx, dw) in zip(outs, want, rows, want_rows):
            assert torch.equal(o, w) and torch.equal(r.dx, dx) and torch.equal(r.dw, dw)


def test_one_capture_after_another(ctx):
    """Calls of a second capture do not wait on what the first one recorded."""
    sets = norm_sets(7, [100_000, 50_000])
    outs, graphs = [torch.zeros(2, device="cuda") for _ in sets], []
    ctx.grad_norm([sets[0]], outs[0])
    torch.cuda.synchronize()
    for g, o in zip(sets, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            ctx.grad_norm([g], o)
        graphs.append(graph)
    for graph in reversed(graphs):
        graph.replay()
    torch.cuda.synchronize()
    for g, o in zip(sets, outs):
        want = float(g.double().norm())
        assert abs(o[0].item() - want) < 1e-6 * want


class Address:
    """What a call needs of a stream."""

    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


def test_a_captured_step_without_a_number_is_refused(ctx):
    """The host's count cannot go on in a replay.  With a number, the capture goes on and each replay is that step."""
    p, g = torch.ones(1000, device="cuda"), torch.full((1000,), 0.5, device="cuda")
    opt, side, graph = ctx.adamw([p], [g], lr=0.1), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    opt.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for stream in (None, side, torch.cuda.ExternalStream(side.cuda_stream), Address(side.cuda_stream)):
            with pytest.raises(GbError) as e:
                opt.step(stream=stream)
            assert e.value.status == B.GB_ERR_INVALID_ARG and opt.steps == 1
        opt.step(step=7, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    q = [t.clone() for t in (p, g)]
    eager = ctx.adamw([q[0]], [q[1]], [opt.exp_avg[0].clone()], [opt.exp_avg_sq[0].clone()], lr=0.1)
    for _ in range(3):
        graph.replay()
        eager.step(step=7)
    torch.cuda.synchronize()
    assert torch.equal(p, q[0]) and torch.equal(opt.exp_avg_sq[0], eager.exp_avg_sq[0])
    opt.step()  # outside of a capture, on from the last number
    assert opt.steps == 8


class DriverStream:
    """A stream that synchronizes with the legacy stream, which torch's streams do not, and its capture."""

    def __init__(self):
        self.cu, self.handle, self.graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(), ctypes.c_void_p()
        assert self.cu.cuStreamCreate(ctypes.byref(self.handle), 0) == 0

    @property
    def cuda_stream(self):
        return self.handle.value

    def begin(self):
        assert self.cu.cuStreamBeginCapture_v2(self.handle, 1) == 0  # thread local

    def end(self):
        status = self.cu.cuStreamEndCapture(self.handle, ctypes.byref(self.graph))
        if self.graph:
            self.cu.cuGraphDestroy(self.graph)
        return status

    def destroy(self):
        self.cu.cuStreamDestroy_v2(self.handle)


def test_the_legacy_stream_during_a_capture_is_refused(ctx):
    """The call is refused, the capture goes on, and the context stays usable."""
    x, out = torch.full((1000,), 2.0, device="cuda"), torch.zeros(2, device="cuda")
    rows = Rows(1, 10, 64)
    ctx.grad_norm([x], out)
    torch.cuda.synchronize()
    other = DriverStream()
    legacy = torch.cuda.default_stream()
    assert legacy.cuda_stream == 0
    other.begin()
    for call in (lambda: ctx.grad_norm([x], out, stream=legacy), lambda: rows.run(ctx, stream=legacy)):
        with pytest.raises(GbError) as e:
            call()
        assert e.value.status == B.GB_ERR_INVALID_ARG
    ctx.grad_norm([x], out, stream=other)
    assert other.end() == 0
    assert ctx.status() == B.GB_OK
    out.zero_()
    ctx.grad_norm([x], out, stream=legacy)
    torch.cuda.synchronize()
    assert abs(out[0].item() - 4000 ** 0.5) < 1e-5
    other.destroy()


def test_a_capture_that_has_been_invalidated_is_refused(ctx):
    x, out = torch.ones(1000, device="cuda"), torch.zeros(2, device="cuda")
    ctx.grad_norm([x], out)
    torch.cuda.synchronize()
    other = DriverStream()
    other.begin()
    assert other.cu.cuStreamSynchronize(other.handle) != 0  # not allowed in a capture: an error, and no capture any more
    with pytest.raises(GbError) as e:
        ctx.grad_norm([x], out, stream=other)
    assert e.value.status == B.GB_ERR_INVALID_ARG and ctx.status() == B.GB_OK
    assert other.end() != 0
    ctx.grad_norm([x], out)
    torch.cuda.synchronize()
    assert abs(out[0].item() - 1000 ** 0.5) < 1e-5
    other.destroy()
