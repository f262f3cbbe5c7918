"""Calls that name a stream other than the current one: what the binding allocates for them (outputs, workspaces) shares
no memory with work that is still queued on either stream."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
B, T, D = 2, 2000, 256


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    x, r, i, dh = (torch.randn(B, T, D, generator=g).to(BF16).cuda() for _ in range(4))
    q, k, v = (torch.randn(B, h, T, 64, generator=g).to(BF16).cuda() for h in (4, 2, 2))
    a, b = torch.rand(B, T, D, generator=g).cuda(), torch.randn(B, T, D, generator=g).cuda()
    return x, r, i, torch.full((D,), -5.0, device="cuda"), dh, q, k, v, a, b


def work(cla, t, stream):
    x, r, i, lam, dh, q, k, v, a, b = t
    o, lse = cla.window_attn_fwd(q, k, v, window=300, sinks=4, stream=stream)
    return (o, lse, *cla.window_attn_bwd(q, k, v, o, lse, q, window=300, sinks=4, stream=stream),
            *cla.gated_scan_bwd(x, r, i, lam, None, dh, stream=stream), *cla.scan_diag_fwd(a, b, stream=stream))


def named(kind, s):
    return s if kind == "object" else s.cuda_stream


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_blocks_that_the_current_stream_still_reads(cla, kind):
    """Tensors freed while a queued kernel of the current stream has yet to read them are not the call's to write."""
    t = inputs(1)
    want = work(cla, t, None)
    sizes = [x.numel() * x.element_size() for x in want] + [
        cla.gated_scan_workspace_size(B, T, D), cla.scan_diag_workspace_size(B, T, D),
        cla.window_attn_bwd_workspace_size(B, 4, 2, T, 64, 300, 4), 256]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    copies = [torch.empty_like(x) for x in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for c, x in zip(copies, freed):
        c.copy_(x)
    del freed, x
    got = work(cla, t, named(kind, s))
    torch.cuda.synchronize()
    for c in copies:
        assert bool((c == 7).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_outputs_that_the_current_stream_still_reads(cla, kind):
    """Outputs dropped while the current stream has yet to read them are not the next call's to write."""
    t, t2 = inputs(1), inputs(2)
    want, want2 = work(cla, t, None), work(cla, t2, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = work(cla, t, named(kind, s))
    copies = [torch.empty_like(x) for x in got]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    for c, x in zip(copies, got):
        c.copy_(x)
    del got, x
    got2 = work(cla, t2, named(kind, s))
    torch.cuda.synchronize()
    for a, b in zip(copies + list(got2), want + want2):
        assert torch.equal(a, b)


def test_default_stream_by_its_handles(cla):
    """0 and 1 (the legacy stream's constant) are the default stream."""
    t = inputs(3)
    want = work(cla, t, None)
    for handle in (0, 1):
        torch.cuda.synchronize()
        got = work(cla, t, handle)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_on_a_stream_that_a_capture_forks_to(cla):
    """Named streams inside a capture: outputs and workspaces come from the graph's own memory, and replays on new inputs
    give what calls outside give."""
    t, t2 = inputs(4), inputs(5)
    static = tuple(x.clone() for x in t)
    work(cla, static, None)
    s, fork = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fork.wait_stream(s)
        got = work(cla, static, fork)
        s.wait_stream(fork)
    for now in (t2, t):
        want = work(cla, now, None)
        for a, b in zip(static, now):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


FIRST_CALLS = """
import torch
import chunkwise_linear_attention_gb300 as cla
g = torch.Generator().manual_seed(0)
rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
x, r, i, dh = (rnd(2, 300, 64) for _ in range(4))
lam, state = torch.full((64,), -5.0, device="cuda"), torch.zeros(2, 64, device="cuda")
q, k, v, dO = rnd(2, 4, 300, 128), rnd(2, 2, 300, 128), rnd(2, 2, 300, 128), rnd(2, 4, 300, 128)
kc, vc = (torch.zeros(2, 2, 104, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
pos = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
kw = dict(window=100, sinks=4)

def work():
    o, lse = cla.window_attn_fwd(q, k, v, **kw)
    cla.window_cache_write(k, v, kc, vc, **kw)
    state.zero_()
    return (cla.gated_scan_fwd(x, r, i, lam) + cla.gated_scan_bwd(x, r, i, lam, None, dh) + (o, lse)
            + cla.window_attn_bwd(q, k, v, o, lse, dO, **kw)
            + (cla.window_attn_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], kc, vc, pos, **kw),
               cla.gated_scan_step(x[:, 0].contiguous(), r[:, 0].contiguous(), i[:, 0].contiguous(), lam, state)))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = work()
graph.replay()
torch.cuda.synchronize()
got = [y.clone() for y in got]
for a, b in zip(got, work()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_of_a_process_are_captured(cla):
    """No entry point needs a call outside a capture before one inside."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
