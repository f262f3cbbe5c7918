"""The norm and rotation, the 8-bit window cache and the delta rule's steps as a hybrid stack uses them together: a layer of
the delta rule and a layer of local attention, trained, prefilled and stepped; calls on several streams and in graphs."""
import os
import subprocess
import sys

import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
B, T, H, K, d, W, N = 2, 200, 4, 2, 64, 70, 3
D = H * d


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)

    def w(*s):
        return (torch.randn(*s, generator=g) * s[0] ** -0.5).cuda()

    return dict(delta=w(D, 3 * D), gates=w(D, 2 * H), qkv=w(D, (H + 2 * K) * d), wq=1 + 0.2 * torch.randn(d, generator=g).cuda(),
                wk=1 + 0.2 * torch.randn(d, generator=g).cuda(), freq=(1000.0 ** (-torch.arange(0, d, 2).float() / d)).cuda(),
                l2=torch.full((d,), d ** -0.5).cuda())


def heads(x, *n):  # [B, T, sum(n) d] -> views [B, heads, T, d]
    return [y.transpose(1, 2) for y in x.view(*x.shape[:2], sum(n), d).split(n, 2)]


# ------------------------------------------------------------------ training
class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cla, q, k, wq, wk, freq, lens):
        ctx.cla, ctx.lens = cla, lens
        ctx.save_for_backward(q, k, wq, wk, freq)
        return cla.qk_norm_rope_fwd(q, k, wq, wk, freq, lens=lens)

    @staticmethod
    def backward(ctx, dq, dk):
        dq, dk, dwq, dwk = ctx.cla.qk_norm_rope_bwd(*ctx.saved_tensors, dq, dk, lens=ctx.lens)
        return None, dq, dk, dwq, dwk, None, None


class Window(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cla, q, k, v, lens):
        o, lse = cla.window_attn_fwd(q, k, v, window=W, sinks=N, lens=lens)
        ctx.cla, ctx.lens = cla, lens
        ctx.save_for_backward(q, k, v, o, lse)
        return o

    @staticmethod
    def backward(ctx, dO):
        return (None, *ctx.cla.window_attn_bwd(*ctx.saved_tensors, dO, window=W, sinks=N, lens=ctx.lens), None)


def plain_norm(x, w, freq):
    y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
    angle = torch.arange(x.shape[2])[:, None].double() * freq.double()
    a, b = y.chunk(2, -1)
    return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)


def test_training_step(cla):
    """Norm, rotation and attention of a padded batch: outputs and every gradient against the 64-bit form.  bf16 rounds each of
    about six tensors on the way by 2^-9 of its size in the root mean square, and the gradients pass through two operators:
    2^-9 sqrt(6) 2, about 1%; 3% is allowed, in the 2-norm."""
    g = torch.Generator().manual_seed(1)
    x0, up = (torch.randn(B, T, D, generator=g).to(BF16) for _ in range(2))
    lens = torch.tensor([T, 90], dtype=torch.int32)
    live = (torch.arange(T) < lens[:, None])[..., None]
    p = weights()
    names = ("qkv", "wq", "wk")
    x = x0.cuda().requires_grad_()
    w = {n: p[n].clone().requires_grad_() for n in names}
    q, k, v = heads(x @ w["qkv"].to(BF16), H, K, K)
    o = Window.apply(cla, *Norm.apply(cla, q, k, w["wq"], w["wk"], p["freq"], lens.cuda()), v, lens.cuda())
    y = o.transpose(1, 2).reshape(B, T, D)
    got = torch.autograd.grad((y.float() * (up * live).cuda().float()).sum(), [x] + [w[n] for n in names])

    x64 = x0.double().requires_grad_()
    w64 = {n: p[n].cpu().double().requires_grad_() for n in names}
    q, k, v = heads(x64 @ w64["qkv"], H, K, K)
    q, k = plain_norm(q, w64["wq"], p["freq"].cpu()), plain_norm(k, w64["wk"], p["freq"].cpu())
    k, v = (z.repeat_interleave(H // K, 1) for z in (k, v))
    s = (q @ k.transpose(2, 3) * d ** -0.5).masked_fill(~M.visible(T, W, N), -float("inf"))
    y64 = (torch.softmax(s, 3) @ v).transpose(1, 2).reshape(B, T, D)
    want = torch.autograd.grad((y64 * (up * live).double()).sum(), [x64] + [w64[n] for n in names])

    def near(name, a, b):
        a, b = a.detach().double().cpu(), b.detach()
        assert float((a - b).norm()) <= 0.03 * float(b.norm()), (name, float((a - b).norm() / b.norm()))

    near("y", y * live.cuda(), y64 * live)
    for n, a, b in zip(("x",) + names, got, want):
        near(n, a, b)


# ------------------------------------------------------------------ serving
def test_prefill_and_steps(cla):
    """A prompt through both layers, then tokens one by one over the state and the 8-bit cache.  Each operator's outputs are
    held to its 64-bit form on the inputs that it was given, with the state and the cache carried along in 64 bits."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, T, D, generator=g).to(BF16).cuda()
    p = weights(3)
    n = 150

    def project(x):
        ld, beta = (x.float() @ p["gates"]).view(*x.shape[:2], 2, H).permute(2, 0, 3, 1)
        return heads(x @ p["delta"].to(BF16), H, H, H), -torch.nn.functional.softplus(ld), torch.sigmoid(beta)

    def attention_in(x):
        return heads(x @ p["qkv"].to(BF16), H, K, K)

    # the prompt
    (q, k, v), ld, beta = project(x[:, :n])
    q, k = cla.qk_norm_rope_fwd(q, k, p["l2"], p["l2"])
    M.assert_within("k", k, *R.norm_rope(heads(x[:, :n] @ p["delta"].to(BF16), H, H, H)[1], p["l2"])["o"])
    o, S = cla.delta_fwd(q, k, v.contiguous(), ld.contiguous(), beta.contiguous())
    y = x[:, :n] + o.transpose(1, 2).reshape(B, n, D).to(BF16)
    q, k, v = attention_in(y)
    q, k = cla.qk_norm_rope_fwd(q, k, p["wq"], p["wk"], p["freq"])
    cla.window_attn_fwd(q, k, v, window=W, sinks=N)
    cache = cla.window_cache8(B, K, d, window=W, sinks=N)
    kept = [R.cache8_write(t, c, f, None, W, N) for t, c, f in ((k, cache[0], cache[2]), (v, cache[1], cache[3]))]
    cla.window_cache8_write(k, v, *cache, window=W, sinks=N)

    pos = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for t in range(n, T):
        xt = x[:, t:t + 1]
        (q, k, v), ld, beta = project(xt)
        q, k = cla.qk_norm_rope_fwd(q, k, p["l2"], p["l2"])
        before = S.clone()
        o = cla.delta_step(q, k, v, ld, beta, S)
        (ro, eo), (rS, eS) = R.delta(q, k, v, ld, beta, before)
        M.assert_within("o", o, ro, eo)
        M.assert_within("S", S, rS, eS)
        y = xt + o.transpose(1, 2).reshape(B, 1, D).to(BF16)
        q, k, v = (z[:, :, 0] for z in attention_in(y))
        raw = k.clone()
        q, k = cla.qk_norm_rope_step(q, k, p["wq"], p["wk"], p["freq"], pos)
        M.assert_within("k", k[:, :, None], *R.norm_rope(raw[:, :, None], p["wk"], p["freq"], pos[:, None])["o"])
        kept = [R.cache8_put(z, *c, pos, W, N) for z, c in ((k, kept[0]), (v, kept[1]))]
        o = cla.window_attn_step8(q, k, v, *cache, pos, window=W, sinks=N)
        M.assert_within("o", o, *R.step8(q, *kept[0], *kept[1], pos))
        pos += 1
    for got, want in zip(cache, (kept[0][0], kept[1][0], kept[0][1], kept[1][1])):
        assert torch.equal(got.double().cpu(), want)


# ------------------------------------------------------------------ streams, graphs, devices
def inputs(seed):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g)

    q, k, dq, dk = (rnd(3, h, 700, 64).to(BF16).cuda() for h in (4, 2, 4, 2))
    wq, wk, freq = rnd(64).cuda(), rnd(64).cuda(), torch.rand(32, generator=g).cuda()
    v = rnd(3, 2, 700, 64).to(BF16).cuda()
    ld, beta, S = -torch.rand(3, 4, 2, generator=g).cuda(), torch.rand(3, 4, 2, generator=g).cuda(), rnd(3, 4, 64, 64).cuda()
    return q, k, dq, dk, wq, wk, freq, v, ld, beta, S


def work(cla, t, stream):
    q, k, dq, dk, wq, wk, freq, v, ld, beta, S = t
    pos = torch.tensor([600, 40, 5000], dtype=torch.int32).cuda()
    cache, S = cla.window_cache8(3, 2, 64, window=500), S.clone()
    s = torch.cuda.current_stream() if stream is None else stream
    if not isinstance(s, torch.cuda.Stream):
        s = torch.cuda.ExternalStream(s) if s > 1 else torch.cuda.default_stream()
    s.wait_stream(torch.cuda.current_stream())
    out = cla.qk_norm_rope_fwd(q, k, wq, wk, freq, stream=stream) + cla.qk_norm_rope_bwd(q, k, wq, wk, freq, dq, dk, stream=stream)
    cla.window_cache8_write(k, v, *cache, window=500, stream=stream)
    out += (cla.window_attn_step8(q[:, :, 0], k[:, :, 0], v[:, :, 0], *cache, pos, window=500, stream=stream),)
    out += cla.qk_norm_rope_step(q[:, :, 1], k[:, :, 1], wq, wk, freq, pos, stream=stream)
    out += (cla.delta_step(q[:, :, :2], q[:, :, 2:4], q[:, :, 4:6], ld, beta, S, stream=stream), S)
    torch.cuda.current_stream().wait_stream(s)
    return out + tuple(x.view(torch.uint8) for x in cache)


def equal(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_calls_on_streams_at_once(cla):
    t = inputs(1)
    want = work(cla, t, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [work(cla, t, streams[i % 3]) for i in range(9)] + [work(cla, t, s) for s in (streams[0].cuda_stream, 0, 1)]
    torch.cuda.synchronize()
    for out in got:
        equal(out, want)


def test_outputs_that_the_current_stream_still_reads(cla):
    """Outputs dropped while the current stream has yet to read them are not the next call's to write."""
    t, t2 = inputs(1), inputs(2)
    want, want2 = work(cla, t, None), work(cla, t2, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = work(cla, t, s)
    copies = [torch.empty_like(x) for x in got]
    torch.cuda._sleep(100_000_000)
    for c, x in zip(copies, got):
        c.copy_(x)
    del got, x
    got2 = work(cla, t2, s)
    torch.cuda.synchronize()
    equal(copies + list(got2), want + want2)


def test_two_graphs_and_eager_calls(cla):
    """Two captured runs, with memory of their own, replayed in turn and beside eager calls."""
    t = [tuple(x.clone() for x in inputs(i)) for i in (1, 2)]
    s = torch.cuda.Stream()
    graphs, got = [], []
    for x in t:
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            q, k, dq, dk, wq, wk, freq, v, ld, beta, S = x
            cache = cla.window_cache8(3, 2, 64, window=500)
            out = cla.qk_norm_rope_fwd(q, k, wq, wk, freq) + cla.qk_norm_rope_bwd(q, k, wq, wk, freq, dq, dk)
            cla.window_cache8_write(k, v, *cache, window=500)
            pos = torch.full((3,), 650, dtype=torch.int32, device="cuda")
            out += (cla.window_attn_step8(q[:, :, 0], k[:, :, 0], v[:, :, 0], *cache, pos, window=500),)
            S = S.clone()
            out += (cla.delta_step(q[:, :, :2], q[:, :, 2:4], q[:, :, 4:6], ld, beta, S), S) + cache
            got.append(out)

    def eager(x):
        q, k, dq, dk, wq, wk, freq, v, ld, beta, S = x
        cache = cla.window_cache8(3, 2, 64, window=500)
        out = cla.qk_norm_rope_fwd(q, k, wq, wk, freq) + cla.qk_norm_rope_bwd(q, k, wq, wk, freq, dq, dk)
        cla.window_cache8_write(k, v, *cache, window=500)
        pos = torch.full((3,), 650, dtype=torch.int32, device="cuda")
        out += (cla.window_attn_step8(q[:, :, 0], k[:, :, 0], v[:, :, 0], *cache, pos, window=500),)
        S = S.clone()
        return out + (cla.delta_step(q[:, :, :2], q[:, :, 2:4], q[:, :, 4:6], ld, beta, S), S) + cache

    want = [eager(x) for x in t]
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        beside = eager(t[1 - i])
        torch.cuda.synchronize()
        for a, b in ((got[i], want[i]), (beside, want[1 - i])):
            equal([x.view(torch.uint8) for x in a], [x.view(torch.uint8) for x in b])


FIRST_CALLS = """
import torch
import chunkwise_linear_attention_gb300 as cla
g = torch.Generator().manual_seed(0)
rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
q, k, v = rnd(2, 20, 300, 128), rnd(2, 2, 300, 128), rnd(2, 2, 300, 128)
w, f = torch.ones(128, device="cuda"), torch.rand(64, generator=g).cuda()
pos = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
gate = torch.rand(2, 20, 300, generator=g).cuda()
S0 = torch.randn(2, 20, 128, 128, generator=g).cuda()
cache = cla.window_cache8(2, 2, 128, window=250, sinks=4)
kw = dict(window=250, sinks=4)

def work():
    S = S0.clone()
    cla.window_cache8_write(k, v, *cache, **kw)
    return (cla.qk_norm_rope_fwd(q, k, w, w, f) + cla.qk_norm_rope_bwd(q, k, w, w, f, q, k)
            + (cla.window_attn_step8(q[:, :, 0], k[:, :, 0], v[:, :, 0], *cache, pos, **kw),
               cla.delta_step(q[:, :, :1], q[:, :, 1:2] * 0.1, q[:, :, 2:3], -gate[:, :, :1], gate[:, :, :1], S), S))

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
