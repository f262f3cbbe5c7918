"""Sliding-window attention with sinks against its 64-bit form: forward, backward, cache and step."""
import pytest
import torch

from tests import _mixers as R

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def inputs(B, H, K, T, d, dtype, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed)

    def rnd(h, s=1.0):
        return (torch.randn(B, h, T, d, generator=g) * s).to(dtype).cuda()

    return rnd(H, std), rnd(K), rnd(K), rnd(H)


def check(cla, q, k, v, dO, window, sinks, lens=None, scale=None, **out):
    ref = R.window(q, k, v, window, sinks, lens, scale, dO)
    kw = dict(window=window, sinks=sinks, lens=lens, scale=scale)
    o, lse = cla.window_attn_fwd(q, k, v, o=out.get("o"), **kw)
    got = dict(o=o, lse=lse)
    for n in ("o", "lse"):
        R.assert_within(n, got[n], *ref[n])
    got.update(zip(("dq", "dk", "dv"), cla.window_attn_bwd(q, k, v, o, lse, dO, dq=out.get("dq"), dk=out.get("dk"),
                                                           dv=out.get("dv"), **kw)))
    for n in ("dq", "dk", "dv"):
        R.assert_within(n, got[n], *ref[n])
    # a second run gives the same bits: sums are in a fixed order
    again = cla.window_attn_bwd(q, k, v, o, lse, dO, **kw)
    for n, x in zip(("dq", "dk", "dv"), again):
        assert torch.equal(x, got[n]), n
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window,sinks", [
    (1, 1, 0), (1, 5, 3), (2, 1, 1), (64, 64, 0), (127, 20, 4), (128, 128, 0), (129, 1, 0), (129, 1, 5), (130, 129, 1),
    (257, 100, 3), (300, 1000, 0), (384, 128, 128), (513, 127, 130), (640, 256, 16), (700, 65, 300), (500, 400, 1000)])
def test_masks(cla, T, window, sinks, d, dtype):
    check(cla, *inputs(1, 2, 1, T, d, dtype, T), window, sinks)


@pytest.mark.parametrize("B,H,K", [(1, 1, 1), (2, 4, 4), (3, 6, 2), (1, 8, 1), (2, 5, 1)])
def test_heads(cla, B, H, K):
    check(cla, *inputs(B, H, K, 200, 64, BF16), 70, 3)


@pytest.mark.parametrize("T,window,sinks,d", [(1500, 65, 4, 64), (1300, 10, 200, 128)])
def test_long_lists_of_the_sinks(cla, T, window, sinks, d):
    """Every later query sees the sinks: their gradients come from many more tiles than a window has."""
    lens = torch.tensor([T, 700], dtype=torch.int32).cuda()
    check(cla, *inputs(2, 4, 1, T, d, BF16), window, sinks, lens)


@pytest.mark.parametrize("H,K,T,window,sinks", [(2, 1, 200, 60, 1), (3, 3, 300, 1, 0), (1, 1, 130, 500, 0)])
def test_many_ragged_sequences(cla, H, K, T, window, sinks):
    """Batches of more sequences than a warp has lanes, empty ones in front, between and behind."""
    B = 71
    lens = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    lens[0] = lens[1] = lens[33] = lens[70] = 0
    check(cla, *inputs(B, H, K, T, 64, BF16), window, sinks, lens.cuda())
    check(cla, *inputs(B, H, K, T, 64, BF16), window, sinks, torch.zeros(B, dtype=torch.int32).cuda())


@pytest.mark.parametrize("B,H,K,T", [(0, 2, 1, 5), (2, 0, 0, 5), (2, 2, 1, 0)])
def test_nothing_to_do(cla, B, H, K, T):
    q, k, v, dO = inputs(B, H, K, T, 64, BF16)
    o, lse = cla.window_attn_fwd(q, k, v, window=4, sinks=1)
    grads = cla.window_attn_bwd(q, k, v, o, lse, dO, window=4, sinks=1)
    assert o.shape == q.shape and lse.shape == q.shape[:3] and [x.shape for x in grads] == [q.shape, k.shape, v.shape]


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16)])
def test_lengths(cla, d, dtype):
    """Padded rows: o 0, lse -inf, gradients 0, whatever they hold; a sequence of nothing; lengths out of range."""
    q, k, v, dO = inputs(6, 4, 2, 400, d, dtype)
    lens = torch.tensor([400, 0, 1, 128, 257, 9999], dtype=torch.int32).cuda()
    got = check(cla, q, k, v, dO, 150, 5, lens)
    assert float(got["o"][1].abs().max()) == 0 and bool((got["lse"][1] == -float("inf")).all())
    for x in (q, k, v, dO):
        for b, n in enumerate(lens.tolist()):
            x[b, :, max(0, n):] = float("nan") if b % 2 else float("inf")
    bad = check(cla, q, k, v, dO, 150, 5, lens)
    for n in got:
        assert torch.equal(got[n], bad[n]), n


def test_scale(cla):
    q, k, v, dO = inputs(1, 2, 2, 150, 64, BF16)
    for scale in (0.0, 1.0, -0.125):
        check(cla, q, k, v, dO, 60, 2, None, scale)


def test_large_logits(cla):
    """Logits in the hundreds: the running maximum moves, most weights vanish."""
    q, k, v, dO = inputs(1, 2, 1, 300, 64, BF16, 3, 40.0)
    check(cla, q, k, v, dO, 200, 4)


@pytest.mark.parametrize("T,window,sinks", [(1, 1, 0), (1, 50, 4), (200, 1, 0)])
def test_one_key_has_no_gradient(cla, T, window, sinks):
    """A query that sees one key gives it all its weight whatever the score: dq and dk are 0, not a rounding."""
    q, k, v, dO = inputs(2, 4, 2, T, 64, BF16)
    got = check(cla, q, k, v, dO, window, sinks)
    assert torch.equal(got["o"], v.repeat_interleave(2, 1))
    assert float(got["dq"].abs().max()) == 0 and float(got["dk"].abs().max()) == 0


def test_window_longer_than_any_sequence(cla):
    q, k, v, _ = inputs(2, 4, 2, 300, 64, BF16)
    want = cla.window_attn_fwd(q, k, v, window=300)
    for w, n in ((2 ** 62, 0), (5, 2 ** 62), (2 ** 31, 2 ** 31)):
        got = cla.window_attn_fwd(q, k, v, window=w, sinks=n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strided_views(cla):
    """q, k, v as slices of one projection [B, T, heads, d]; the output and gradients in that layout too."""
    B, H, K, T, d = 2, 4, 2, 150, 64
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, T, H + 2 * K, d, generator=g).to(BF16).cuda()
    q, k, v = (x.transpose(1, 2) for x in qkv.split((H, K, K), 2))
    grad = torch.full_like(qkv, float("nan"))
    dq, dk, dv = (x.transpose(1, 2) for x in grad.split((H, K, K), 2))
    o = torch.empty(B, T, H, d, dtype=BF16, device="cuda").transpose(1, 2)
    dO = torch.randn(B, T, H, d, generator=g).to(BF16).cuda().transpose(1, 2)
    got = check(cla, q, k, v, dO, 40, 3, o=o, dq=dq, dk=dk, dv=dv)
    assert got["o"].data_ptr() == o.data_ptr() and torch.isfinite(grad).all()
    dense = check(cla, *(x.contiguous() for x in (q, k, v, dO)), 40, 3)
    for n in got:
        assert torch.equal(got[n], dense[n]), n


def test_gradients_against_differences(cla):
    """Central differences of the 64-bit form along random directions, and of the kernel's own lse."""
    q, k, v, dO = inputs(1, 4, 2, 200, 64, F16)
    kw = dict(window=90, sinks=3)
    o, lse = cla.window_attn_fwd(q, k, v, **kw)
    grads = cla.window_attn_bwd(q, k, v, o, lse, dO, **kw)

    def loss(q, k, v):
        return float((R.window(q, k, v, 90, 3)["o"][0] * dO.double().cpu()).sum())

    base = [x.double().cpu() for x in (q, k, v)]
    for i, g in enumerate(grads):
        w = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        e = 1e-4
        num = (loss(*(b + e * w if j == i else b for j, b in enumerate(base)))
               - loss(*(b - e * w if j == i else b for j, b in enumerate(base)))) / (2 * e)
        terms = g.double().cpu() * w
        # each gradient within a few half steps of fp16, independent over the elements
        assert abs(num - float(terms.sum())) <= 8 * 2.0 ** -11 * float(terms.square().sum().sqrt()) + 1e-6 * float(terms.abs().sum())


# ------------------------------------------------------------------ the cache
@pytest.mark.parametrize("T,window,sinks", [(1, 1, 0), (3, 5, 2), (7, 5, 2), (8, 5, 2), (40, 5, 2), (300, 64, 4), (12, 100, 0),
                                            (50, 7, 60), (64, 1, 1)])
def test_cache_write(cla, T, window, sinks):
    B, K, d = 3, 2, 64
    _, k, v, _ = inputs(B, K, K, T, d, BF16)
    lens = torch.tensor([T, 0, (T + 1) // 2], dtype=torch.int32)
    for n in (None, lens.cuda()):
        kc, vc = (torch.randn(B, K, sinks + window, d).to(BF16).cuda() for _ in range(2))
        want = [kc.clone(), vc.clone()]
        for b in range(B):
            for p in range(T if n is None else int(lens[b])):
                j = R.slot(p, window, sinks)
                want[0][b, :, j], want[1][b, :, j] = k[b, :, p], v[b, :, p]
        cla.window_cache_write(k, v, kc, vc, window=window, sinks=sinks, lens=n)
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,H,K,d,window,sinks", [(1, 1, 1, 64, 1, 0), (4, 4, 2, 64, 30, 3), (5, 8, 1, 128, 200, 4),
                                                  (3, 6, 6, 128, 1500, 0), (2, 32, 2, 64, 5000, 16), (4, 5, 1, 64, 3, 100),
                                                  (2, 40, 1, 128, 130, 1), (1, 9, 1, 64, 33, 0), (9, 18, 9, 64, 3000, 2),
                                                  (1, 4, 1, 128, 20000, 0), (10, 22, 11, 128, 900, 5)])
def test_step(cla, B, H, K, d, window, sinks, dtype):
    g = torch.Generator().manual_seed(9)
    S = sinks + window

    def rnd(*s):
        return torch.randn(*s, generator=g).to(dtype).cuda()

    q, k, v, kc, vc = rnd(B, H, d) * 1.5, rnd(B, K, d), rnd(B, K, d), rnd(B, K, S, d), rnd(B, K, S, d)
    for pos in ([0, -1, S - 1, S, 3 * S + 5], [S // 2, 1, -7, sinks, 2 ** 31 - 1]):
        pos = torch.tensor((pos * 2)[:B], dtype=torch.int32)
        a, c = kc.clone(), vc.clone()
        for b, p in enumerate(pos.tolist()):  # what a slot that no token has reached holds is not used
            if 0 <= p < S:
                a[b, :, p:], c[b, :, p:] = float("nan"), float("nan")
        (ro, e), rk, rv = R.window_step(q, k, v, a, c, pos, sinks)
        o = cla.window_attn_step(q, k, v, a, c, pos.cuda(), window=window, sinks=sinks)
        R.assert_within("o", o, ro, e)
        assert torch.equal(a.view(torch.int16).cpu(), rk.view(torch.int16)) and torch.equal(c.view(torch.int16).cpu(), rv.view(torch.int16))


def test_step_strided(cla):
    """q, k, v as slices of one projection of the token."""
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(3, 8, 64, generator=g).to(BF16).cuda()
    q, k, v = qkv.split((4, 2, 2), 1)
    kc, vc = (torch.randn(3, 2, 20, 64, generator=g).to(BF16).cuda() for _ in range(2))
    pos = torch.tensor([3, 19, 50], dtype=torch.int32).cuda()
    k1, v1 = kc.clone(), vc.clone()
    o = cla.window_attn_step(q, k, v, kc, vc, pos, window=16, sinks=4)
    o1 = cla.window_attn_step(q.contiguous(), k.contiguous(), v.contiguous(), k1, v1, pos, window=16, sinks=4)
    assert torch.equal(o, o1) and torch.equal(kc, k1) and torch.equal(vc, v1)


def test_prefill_then_steps(cla):
    """A prompt through the forward and the cache, then tokens one by one: the forward over the whole sequence."""
    B, H, K, T, d, W, n = 2, 4, 2, 230, 64, 60, 3
    q, k, v, _ = inputs(B, H, K, T, d, BF16)
    ref = R.window(q, k, v, W, n)["o"]
    lens = torch.tensor([200, 37], dtype=torch.int32).cuda()
    kc, vc = (torch.full((B, K, W + n, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    cla.window_cache_write(k, v, kc, vc, window=W, sinks=n, lens=lens)
    pos = lens.clone()
    for _ in range(30):
        at = pos.long()
        b = torch.arange(B, device="cuda")
        o = cla.window_attn_step(q[b, :, at], k[b, :, at], v[b, :, at], kc, vc, pos, window=W, sinks=n)
        for i, p in enumerate(at.tolist()):
            R.assert_within("o", o[i], ref[0][i, :, p], ref[1][i, :, p])
        pos += 1


def test_step_in_a_graph(cla):
    """A captured step, replayed as the sequences grow: positions are read on the device."""
    B, H, K, d, W, n = 2, 8, 2, 128, 700, 4
    g = torch.Generator().manual_seed(6)

    def rnd(*s):
        return torch.randn(*s, generator=g).to(BF16).cuda()

    q, k, v, kc, vc = rnd(B, H, d), rnd(B, K, d), rnd(B, K, d), rnd(B, K, W + n, d), rnd(B, K, W + n, d)
    pos = torch.tensor([0, 640], dtype=torch.int32).cuda()
    kw = dict(window=W, sinks=n)
    k1, v1 = kc.clone(), vc.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        cla.window_attn_step(q, k, v, k1, v1, pos, **kw)
    s.synchronize()
    k1.copy_(kc), v1.copy_(vc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = cla.window_attn_step(q, k, v, k1, v1, pos, **kw)
    for _ in range(70):
        want = cla.window_attn_step(q, k, v, kc, vc, pos, **kw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        pos += 1
        q.copy_(rnd(B, H, d)), k.copy_(rnd(B, K, d)), v.copy_(rnd(B, K, d))
    assert torch.equal(kc, k1) and torch.equal(vc, v1)


# ------------------------------------------------------------------ status
def test_status_of_a_call(cla):
    """Each block of the attention's kernels records a timeout in an entry of its own behind the header's words: a call
    clears them all, whatever the workspace held and however few its blocks are, and check_status reads them."""
    q, k, v, dO = inputs(1, 2, 1, 100, 64, BF16)
    kw = dict(window=30, sinks=2)
    n = cla.window_attn_bwd_workspace_size(1, 2, 1, 100, 64, 30, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o, lse = cla.window_attn_fwd(q, k, v, **kw)
    for call in (lambda: cla.window_attn_fwd(q, k, v, workspace=ws, **kw),
                 lambda: cla.window_attn_bwd(q, k, v, o, lse, dO, workspace=ws, **kw)):
        for at in (96, 97, 96 + 151, 255):  # an entry, of a block that ran or of one that did not
            ws.fill_(255)
            call()
            cla.check_status(ws)
            ws[at] = 27
            with pytest.raises(cla.ClaError, match="site 27"):
                cla.check_status(ws)
    # calls that record elsewhere do not read what an earlier call's blocks left there
    a = torch.rand(1, 50, 8, device="cuda")
    big = torch.full((max(cla.scan_diag_workspace_size(1, 50, 8), 256),), 255, dtype=torch.uint8, device="cuda")
    cla.scan_diag_fwd(a, a, workspace=big)
    cla.check_status(big)


# ------------------------------------------------------------------ more items than blocks
@pytest.mark.parametrize("dtype,ragged,H,K,d", [(BF16, False, 8, 2, 128), (F16, True, 8, 2, 128), (BF16, True, 6, 2, 128),
                                                (F16, False, 8, 2, 64)])
def test_more_items_than_blocks(cla, dtype, ragged, H, K, d):
    """Blocks that take several items and lists one after the other (stages and parities in use again), every output
    compared: 4 sequences of 11 tiles."""
    lens = torch.tensor([1300, 700, 0, 1291], dtype=torch.int32).cuda() if ragged else None
    check(cla, *inputs(4, H, K, 1300, d, dtype, 7), 300, 5, lens)


def test_lse_against_differences(cla):
    """Central differences of the kernel's own lse along q: with v = k, o is sum P k, and d lse = scale o . dq."""
    q, k, _, _ = inputs(1, 4, 2, 200, 64, F16)
    w = torch.randn(q.shape, generator=torch.Generator().manual_seed(5)).cuda()
    up, down = (q + s * w for s in (0.03125, -0.03125))
    up, down = up.half(), down.half()
    kw = dict(window=90, sinks=3)
    o, _ = cla.window_attn_fwd(q, k, k, **kw)
    num = (cla.window_attn_fwd(up, k, k, **kw)[1].double() - cla.window_attn_fwd(down, k, k, **kw)[1].double()).cpu()
    q, k, o, up, down = (x.cpu().double() for x in (q, k, o, up, down))
    step = up - down
    ana = (o * step).sum(3) / 8
    mid = (up + down) / 2 - q
    # the logits of a row move by up to `reach` either way: a third derivative, the third moment of what moves by that,
    # is below its cube, of which the difference has a third (2 is allowed); up and down are rounded, so their middle is
    # off q by `mid`, which moves logits by `shift` and the derivative by the second moment, 2 reach shift; o and the P
    # in it are rounded by half a step of fp16 each; each lse is off by some 300 roundings of fp32 in its sums
    kk = k.repeat_interleave(2, 1)
    reach = (step / 2 @ kk.transpose(2, 3)).abs().amax(3) / 8
    shift = (mid @ kk.transpose(2, 3)).abs().amax(3) / 8
    bound = 2 * reach ** 3 + 2 * reach * shift + 2.1 * 2.0 ** -11 * (step.abs().sum(3) * kk.abs().amax((2, 3))[..., None]) / 8 + 300 * 2.0 ** -22
    assert bool(((num - ana).abs() <= bound).all()), float(((num - ana).abs() / bound).max())
