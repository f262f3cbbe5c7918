"""The gated scan and the window attention as a hybrid stack uses them: a recurrent layer and a local attention layer,
trained on padded batches, prefilled and stepped; calls on several streams, captured, and side by side."""
import pytest
import torch

from tests import _mixers as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
B, T, H, K, d, W, N = 2, 300, 4, 2, 64, 90, 3
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
        return (torch.randn(*s, generator=g) * s[-2] ** -0.5).cuda()

    return dict(gates=w(D, 3 * D), qkv=w(D, (H + 2 * K) * d), lam=(torch.rand(D, generator=g) * 2 - 6).cuda())


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, cla, x, rg, ig, lam, lens):
        ck = cla.gated_scan_ckpt(x)
        h, hT = cla.gated_scan_fwd(x, rg, ig, lam, lens=lens, ckpt=ck)
        ctx.cla, ctx.lens = cla, lens
        ctx.save_for_backward(x, rg, ig, lam, ck)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, rg, ig, lam, ck = ctx.saved_tensors
        dx, dr, di, dlam, _ = ctx.cla.gated_scan_bwd(x, rg, ig, lam, None, dh.contiguous(), lens=ctx.lens, ckpt=ck)
        return None, dx, dr, di, dlam, None


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


def split(x):  # [B, T, (H + 2 K) d] -> views of q, k, v [B, heads, T, d]
    x = x.view(*x.shape[:-1], H + 2 * K, d)
    return [y.transpose(1, 2) for y in x.split((H, K, K), 2)]


def layers(x, p, scan, attend):
    """x -> recurrent layer -> local attention, a residual around each, in the type of x."""
    a, r, i = (x @ p["gates"].to(x.dtype)).split(D, -1)
    x = x + scan(a.contiguous(), r.contiguous(), i.contiguous())
    o = attend(*split(x @ p["qkv"].to(x.dtype)))
    return x + o.transpose(1, 2).reshape(x.shape)


def plain_scan(lam, lens):
    def f(x, r, i):
        h, out = 0.0, []
        a = torch.exp(-8 * torch.nn.functional.softplus(lam) * torch.sigmoid(r))
        b = torch.sqrt(1 - a * a) * torch.sigmoid(i) * x
        for t in range(x.shape[1]):
            h = a[:, t] * h + b[:, t]
            out.append(h)
        return torch.stack(out, 1) * (torch.arange(x.shape[1]) < lens[:, None])[..., None]

    return f


def plain_attend(lens):
    def f(q, k, v):
        see = R.visible(q.shape[2], W, N)
        k, v = (y.repeat_interleave(H // K, 1) for y in (k, v))
        o = torch.softmax((q @ k.transpose(2, 3) * d ** -0.5).masked_fill(~see, -float("inf")), 3) @ v
        return o * (torch.arange(q.shape[2]) < lens[:, None])[:, None, :, None]

    return f


def test_training_step_of_a_stack(cla):
    """Outputs and every weight's gradient against the 64-bit stack.  bf16 rounds each of about eight tensors on the way by
    2^-9 of its size (root mean square of a rounding by half a step of 2^-8), and errors pass through two layers: 2^-9 *
    sqrt(8) * 2, about 1.1%; 3% is allowed, in the 2-norm."""
    g = torch.Generator().manual_seed(1)
    x0 = torch.randn(B, T, D, generator=g).to(BF16)
    up = torch.randn(B, T, D, generator=g).to(BF16)
    lens = torch.tensor([T, 140], dtype=torch.int32)
    p = weights()
    live = (torch.arange(T) < lens[:, None])[..., None]
    names = ("x", "gates", "qkv", "lam")

    x = x0.cuda().requires_grad_()
    w = {n: v.clone().requires_grad_() for n, v in p.items()}
    y = layers(x, w, lambda a, r, i: Scan.apply(cla, a, r, i, w["lam"], lens.cuda()),
               lambda q, k, v: Window.apply(cla, q, k, v, lens.cuda()))
    got = torch.autograd.grad((y.float() * (up * live).cuda().float()).sum(), [x] + [w[n] for n in names[1:]])

    x64 = x0.double().requires_grad_()
    w64 = {n: v.cpu().double().to(torch.float64).requires_grad_() for n, v in p.items()}
    y64 = layers(x64, w64, plain_scan(w64["lam"], lens), plain_attend(lens))
    want = torch.autograd.grad((y64 * (up * live).double()).sum(), [x64] + [w64[n] for n in names[1:]])

    def near(name, a, b):
        a, b = a.detach().double().cpu(), b.detach()
        assert float((a - b).norm()) <= 0.03 * float(b.norm()), (name, float((a - b).norm() / b.norm()))

    near("y", y * live.cuda(), y64 * live)
    for n, a, b in zip(names, got, want):
        near(n, a, b)


def test_prefill_and_steps_are_the_forward(cla):
    """A prompt, then tokens one by one through both layers' states, against the stack over the whole sequence.  Both sides
    round at the same places; a step's sums come in another order, which can move a rounding by a step of 2^-8."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B, T, D, generator=g).to(BF16).cuda()
    p = weights(3)
    whole = layers(x, p, lambda a, r, i: cla.gated_scan_fwd(a, r, i, p["lam"])[0],
                   lambda q, k, v: cla.window_attn_fwd(q, k, v, window=W, sinks=N)[0])
    n = 250
    state = {}
    kc, vc = (torch.zeros(B, K, W + N, d, dtype=BF16, device="cuda") for _ in range(2))

    def scan(a, r, i):
        h, state["h"] = cla.gated_scan_fwd(a, r, i, p["lam"])
        return h

    def attend(q, k, v):
        cla.window_cache_write(k, v, kc, vc, window=W, sinks=N)
        return cla.window_attn_fwd(q, k, v, window=W, sinks=N)[0]

    y = [layers(x[:, :n], p, scan, attend)]
    pos = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for t in range(n, T):
        y.append(layers(
            x[:, t:t + 1], p,
            lambda a, r, i: cla.gated_scan_step(a[:, 0], r[:, 0], i[:, 0], p["lam"], state["h"])[:, None],
            lambda q, k, v: cla.window_attn_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], kc, vc, pos, window=W, sinks=N)[:, :, None]))
        pos += 1
    y = torch.cat(y, 1).float()
    assert float((y - whole.float()).abs().max()) <= 4 * 2.0 ** -7 * float(whole.float().abs().max())
    assert float((y - whole.float()).norm()) <= 2.0 ** -8 * float(whole.float().norm())


def test_window_attention_in_a_graph(cla):
    """Forward and backward captured while eager calls of the same inputs live, replayed on new inputs and lengths."""
    g = torch.Generator().manual_seed(5)

    def new(h):
        return torch.randn(B, h, T, d, generator=g).to(BF16).cuda()

    q, k, v, dO = new(H), new(K), new(K), new(H)
    lens = torch.tensor([T, 77], dtype=torch.int32).cuda()
    kw = dict(window=W, sinks=N, lens=lens)
    eager = cla.window_attn_fwd(q, k, v, **kw)
    s = torch.cuda.Stream()
    ws = [torch.empty(cla.window_attn_bwd_workspace_size(B, H, K, T, d, W, N), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, lse = cla.window_attn_fwd(q, k, v, workspace=ws[0], **kw)
        grads = cla.window_attn_bwd(q, k, v, o, lse, dO, workspace=ws[1], **kw)
    for n in (77, 0, 300):
        for x in (q, k, v, dO):
            x.copy_(new(x.shape[1]))
        lens[1] = n
        graph.replay()
        torch.cuda.synchronize()
        cla.check_status(ws[0])
        cla.check_status(ws[1])
        o1, lse1 = cla.window_attn_fwd(q, k, v, **kw)
        for a, b in zip((o, lse) + grads, (o1, lse1) + cla.window_attn_bwd(q, k, v, o1, lse1, dO, **kw)):
            assert torch.equal(a, b)
    del eager


def test_calls_on_two_streams_at_once(cla):
    """Two scans and two attentions in flight together, on workspaces of their own, give what they give alone."""
    g = torch.Generator().manual_seed(8)
    x, r, i, dh = (torch.randn(3, 3000, 256, generator=g).to(BF16).cuda() for _ in range(4))
    lam = torch.full((256,), -5.0, device="cuda")
    q, k, v, dO = (torch.randn(2, h, 2000, 128, generator=g).to(BF16).cuda() for h in (4, 2, 2, 4))

    def work(stream):
        h = cla.gated_scan_fwd(x, r, i, lam, stream=stream)
        b = cla.gated_scan_bwd(x, r, i, lam, None, dh, stream=stream)
        o = cla.window_attn_fwd(q, k, v, window=500, sinks=4, stream=stream)
        return h + b + o + cla.window_attn_bwd(q, k, v, *o, dO, window=500, sinks=4, stream=stream)

    want = work(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [work(streams[j % 3]) for j in range(9)]
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_memory_outlives_a_call_on_another_stream(cla):
    """Outputs and workspaces that the binding allocates are not given out again while the call's stream still waits."""
    g = torch.Generator().manual_seed(9)
    x, r, i, dh = (torch.randn(2, 2000, 256, generator=g).to(BF16).cuda() for _ in range(4))
    lam = torch.full((256,), -5.0, device="cuda")
    want = cla.gated_scan_bwd(x, r, i, lam, None, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = cla.gated_scan_bwd(x, r, i, lam, None, dh, stream=s)
    size = cla.gated_scan_workspace_size(2, 2000, 256)
    held = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del held
