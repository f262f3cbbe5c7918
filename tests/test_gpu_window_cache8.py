"""The window cache in 8 bits against its 64-bit form: the prompts' write, and the step over it."""
import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def rnd(g, *s, dtype=torch.float32, std=1.0):
    return (torch.randn(*s, generator=g) * std).to(dtype).cuda()


def filled(g, B, K, S, d, pos, std=1.0):
    """(numbers, factors) of a cache whose slots below min(pos, S) hold tokens; NaN elsewhere."""
    num = torch.full((B, K, S, d), float("nan"), dtype=torch.float64)
    fac = torch.full((B, K, R.blocks(S)), float("nan"), dtype=torch.float64)
    for b, p in enumerate(pos.tolist()):
        n = min(max(p, 0), S)
        x = torch.randn(K, n, d, generator=g, dtype=torch.float64) * std
        for i in range(R.blocks(n)):
            at = slice(i * 64, min(n, i * 64 + 64))
            for h in range(K):
                y = x[h, at] * 4.0 ** ((i + h) % 5 - 2)
                fac[b, h, i] = R.factor(y)
                num[b, h, at] = R.rounded(y / fac[b, h, i])
    return num.float().to(E4M3).cuda(), fac.float().cuda()


def same(got, want):
    """Equal numbers: the cache's against 64 bits, NaN where no token is."""
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(torch.nan_to_num(got, nan=1e30), torch.nan_to_num(want, nan=1e30)), int((got != want).sum())


# ------------------------------------------------------------------ the write
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,window,sinks,d", [(1, 1, 0, 64), (3, 5, 2, 64), (8, 5, 2, 128), (40, 5, 2, 64), (300, 64, 4, 128),
                                              (64, 64, 0, 64), (65, 64, 0, 64), (12, 100, 0, 128), (50, 7, 60, 64), (130, 127, 1, 128),
                                              (500, 130, 70, 64), (200, 1000, 3, 64)])
def test_write(cla, T, window, sinks, d, dtype):
    B, K = 4, 2
    g = torch.Generator().manual_seed(T)
    k, v = rnd(g, B, K, T, d, dtype=dtype), rnd(g, B, K, T, d, dtype=dtype, std=30.0)
    for lens in (None, torch.tensor([T, 0, (T + 1) // 2, 99999], dtype=torch.int32)):
        kc, vc, ks, vs = cla.window_cache8(B, K, d, window=window, sinks=sinks)
        kc.view(torch.uint8).fill_(77), vs.fill_(3.0)
        want = [R.cache8_write(x, c, s, lens, window, sinks) for x, c, s in ((k, kc, ks), (v, vc, vs))]
        cla.window_cache8_write(k, v, kc, vc, ks, vs, window=window, sinks=sinks, lens=None if lens is None else lens.cuda())
        for got, ref in zip((kc, ks, vc, vs), want[0] + want[1]):
            same(got, ref)


def test_write_ranges(cla):
    """Blocks of zeros, of a type's smallest and largest, of one large number among small ones, around the steps of the
    factor; rows of one head do not touch another's factor."""
    B, K, T, d = 1, 6, 128, 64
    g = torch.Generator().manual_seed(2)
    for dtype in (BF16, F16):
        k = rnd(g, B, K, T, d, dtype=dtype)
        k[0, 0] = 0
        k[0, 1] *= torch.finfo(dtype).smallest_normal
        k[0, 2] = torch.finfo(dtype).max / 4
        k[0, 2, 3, 4] = torch.finfo(dtype).max
        k[0, 3, :64, 0], k[0, 3, 64:, 0] = 448.0, 450.0
        k[0, 4, 5, 6] = -3000.0
        kc, vc, ks, vs = cla.window_cache8(B, K, d, window=T)
        want = R.cache8_write(k, kc, ks, None, T, 0)
        cla.window_cache8_write(k, -k, kc, vc, ks, vs, window=T)
        same(kc, want[0]), same(ks, want[1]), same(vc, -want[0]), same(vs, want[1])


def test_write_what_is_not_finite(cla):
    """An infinity is the largest number, a NaN stays one and leaves its block's factor alone; others keep their bits."""
    g = torch.Generator().manual_seed(3)
    k = rnd(g, 1, 2, 128, 64, dtype=BF16)
    clean = cla.window_cache8(1, 2, 64, window=128)
    cla.window_cache8_write(k, k, *clean, window=128)
    k2 = k.clone()
    k2[0, 0, 3, 5] = float("nan")
    k2[0, 1, 70, 1], k2[0, 1, 70, 2] = float("inf"), -float("inf")
    got = cla.window_cache8(1, 2, 64, window=128)
    cla.window_cache8_write(k2, k, *got, window=128)
    a, b = got[0].float(), clean[0].float()
    assert torch.isnan(a[0, 0, 3, 5]) and float(a[0, 1, 70, 1]) == 448 and float(a[0, 1, 70, 2]) == -448
    assert torch.equal(got[2][0, 0], clean[2][0, 0]) and torch.equal(got[2][0, 1, :1], clean[2][0, 1, :1])
    a[0, 0, 3, 5] = b[0, 0, 3, 5]
    assert torch.equal(a[0, 0], b[0, 0]) and torch.equal(a[0, 1, :64], b[0, 1, :64])


def test_write_strided_and_nothing(cla):
    B, K, T, d = 2, 3, 90, 64
    g = torch.Generator().manual_seed(4)
    kv = rnd(g, B, T, 2 * K, d, dtype=F16)
    k, v = (x.transpose(1, 2) for x in kv.split((K, K), 2))
    a, b = (cla.window_cache8(B, K, d, window=70, sinks=2) for _ in range(2))
    cla.window_cache8_write(k, v, *a, window=70, sinks=2)
    cla.window_cache8_write(k.contiguous(), v.contiguous(), *b, window=70, sinks=2)
    for x, y in zip(a, b):
        assert torch.equal(x.float(), y.float())
    before = [x.clone() for x in a]
    cla.window_cache8_write(k[:, :, :0], v[:, :, :0], *a, window=70, sinks=2)
    cla.window_cache8_write(k, v, *a, window=70, sinks=2, lens=torch.tensor([0, -5], dtype=torch.int32).cuda())
    for x, y in zip(a, before):
        assert torch.equal(x.float(), y.float())


# ------------------------------------------------------------------ the step
def step(cla, g, B, H, K, d, window, sinks, dtype, pos, std=1.0, scale=None, new=1.0):
    S = sinks + window
    kc, ks = filled(g, B, K, S, d, pos)
    vc, vs = filled(g, B, K, S, d, pos, 3.0)
    q, k, v = rnd(g, B, H, d, dtype=dtype, std=1.5 * std), rnd(g, B, K, d, dtype=dtype, std=new), rnd(g, B, K, d, dtype=dtype, std=new)
    want = [R.cache8_put(x, c, s, pos, window, sinks) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    o, e = R.step8(q, *(torch.nan_to_num(x) for x in want[0] + want[1]), pos, scale)
    got = cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=window, sinks=sinks, scale=scale)
    for x, ref in zip((kc, ks, vc, vs), want[0] + want[1]):
        same(x, ref)
    M.assert_within("o", got, o, e)
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,H,K,d,window,sinks", [(1, 1, 1, 64, 1, 0), (4, 4, 2, 64, 30, 3), (5, 8, 1, 128, 200, 4),
                                                  (3, 6, 6, 128, 1500, 0), (2, 32, 2, 64, 5000, 16), (4, 5, 1, 64, 3, 100),
                                                  (2, 40, 1, 128, 130, 1), (1, 9, 1, 64, 33, 0), (9, 18, 9, 64, 3000, 2),
                                                  (1, 4, 1, 128, 20000, 0), (10, 22, 11, 128, 900, 5), (3, 3, 3, 64, 63, 1),
                                                  (3, 3, 3, 64, 64, 1), (2, 48, 2, 64, 700, 0), (1, 80, 1, 64, 3000, 5)])
def test_step(cla, B, H, K, d, window, sinks, dtype):
    g = torch.Generator().manual_seed(9)
    S = sinks + window
    for pos in ([0, -1, S - 1, S, 3 * S + 5], [S // 2, 1, -7, sinks, 2 ** 31 - 1], [63, 64, 65, 128, S + 63]):
        step(cla, g, B, H, K, d, window, sinks, dtype, torch.tensor((pos * 2)[:B], dtype=torch.int32))


@pytest.mark.parametrize("new", [0.0, 1e-6, 0.01, 100.0, 1e4])
def test_step_changes_the_factor(cla, new):
    """A token far larger or smaller than its block: the block's other numbers are rounded anew, or come back."""
    g = torch.Generator().manual_seed(11)
    pos = torch.tensor([0, 3, 64, 100, 130, 170, 4000, 4064, -1], dtype=torch.int32)
    step(cla, g, 9, 4, 2, 64, 150, 4, F16, pos, new=new)
    step(cla, g, 9, 4, 2, 128, 150, 4, BF16, pos, new=new)


def test_step_scales_and_large_logits(cla):
    g = torch.Generator().manual_seed(12)
    pos = torch.tensor([500, 20, 700], dtype=torch.int32)
    for scale in (0.0, 1.0, -0.125):
        step(cla, g, 3, 8, 2, 64, 600, 4, BF16, pos, scale=scale)
    step(cla, g, 3, 8, 2, 128, 600, 4, F16, pos, std=40.0)


def test_step_small_and_large_queries(cla):
    """Heads of queries of different sizes side by side, zeros among them: each is scaled by its own."""
    g = torch.Generator().manual_seed(13)
    B, H, K, d, W = 2, 8, 2, 64, 300
    pos = torch.tensor([250, 900], dtype=torch.int32)
    kc, ks = filled(g, B, K, W, d, pos)
    vc, vs = filled(g, B, K, W, d, pos)
    q, k, v = rnd(g, B, H, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16)
    q[:, 0] = 0
    q[:, 1] *= 1e-30
    q[:, 2] *= 1e-6
    q[:, 3, :-1] *= 2.0 ** -20
    q[:, 4] *= 1e4
    want = [R.cache8_put(x, c, s, pos, W, 0) for x, c, s in ((k, kc, ks), (v, vc, vs))]
    o, e = R.step8(q, *(torch.nan_to_num(x) for x in want[0] + want[1]), pos)
    M.assert_within("o", cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W), o, e)


def test_step_far_apart_factors(cla):
    """Blocks of values whose factors are far apart, keys that pick one or the other: the sums hold both."""
    g = torch.Generator().manual_seed(14)
    B, H, K, d, W = 1, 4, 1, 64, 256
    pos = torch.tensor([W - 1], dtype=torch.int32)
    for power in (-60, -20, 20, 60, 110):
        kc, ks = filled(g, B, K, W, d, pos)
        vc, vs = filled(g, B, K, W, d, pos)
        vs[:, :, 1] *= 2.0 ** power
        vs.clamp_(min=2.0 ** -64)
        q, k, v = rnd(g, B, H, d, dtype=BF16, std=4.0), rnd(g, B, K, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16)
        want = [R.cache8_put(x, c, s, pos, W, 0) for x, c, s in ((k, kc, ks), (v, vc, vs))]
        o, e = R.step8(q, *(torch.nan_to_num(x) for x in want[0] + want[1]), pos)
        M.assert_within("o", cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W), o, e)


def test_step_over_an_empty_cache_as_made(cla):
    """A new cache counts as zeros where the caller says it holds tokens; nothing is not a number."""
    cache = cla.window_cache8(2, 1, 64, window=100)
    x = torch.ones(2, 1, 64, dtype=BF16, device="cuda")
    o = cla.window_attn_step8(x, x, x, *cache, torch.tensor([0, 9], dtype=torch.int32).cuda(), window=100)
    want = torch.tensor([1.0, float(torch.tensor(8.0).exp() / (torch.tensor(8.0).exp() + 9))])
    torch.testing.assert_close(o.float().cpu(), want.view(2, 1, 1).expand(2, 1, 64), rtol=2 ** -7, atol=0)


def test_step_what_is_not_finite(cla):
    """A NaN in a key or a query reaches the heads that see it and no others, wherever its slot lies in the split of the work;
    one in a slot that no token has reached, or in a row without a sequence, reaches nothing."""
    g = torch.Generator().manual_seed(15)
    B, H, K, d, W = 3, 4, 2, 64, 3000
    pos = torch.tensor([2500, 100, -1], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, B, K, W, d, pos), filled(g, B, K, W, d, pos)
    q, k, v = rnd(g, B, H, d, dtype=F16), rnd(g, B, K, d, dtype=F16), rnd(g, B, K, d, dtype=F16)
    q[2], k[2] = float("nan"), float("inf")
    want = cla.window_attn_step8(q, k, v, kc.clone(), vc.clone(), ks.clone(), vs.clone(), pos.cuda(), window=W)
    assert bool(torch.isfinite(want).all()) and float(want[2].abs().max()) == 0
    for slot in (0, 63, 64, 1000, 2047, 2499):
        bad = kc.clone()
        bad.view(torch.uint8)[0, 1, slot, 5] = 0x7f
        got = cla.window_attn_step8(q, k, v, bad, vc.clone(), ks.clone(), vs.clone(), pos.cuda(), window=W)
        assert bool(torch.isnan(got[0, 2:]).all()) and torch.equal(got[0, :2], want[0, :2]) and torch.equal(got[1:], want[1:])
    bad = q.clone()
    bad[1, 1, 3] = float("nan")
    got = cla.window_attn_step8(bad, k, v, kc.clone(), vc.clone(), ks.clone(), vs.clone(), pos.cuda(), window=W)
    assert bool(torch.isnan(got[1, 1]).all())
    got[1, 1] = want[1, 1]
    assert torch.equal(got, want)


def test_step_beside_a_nan(cla):
    """A NaN that a block of the token holds does not count for its factor; the block's other numbers move as without it."""
    g = torch.Generator().manual_seed(16)
    pos = torch.tensor([40], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, 1, 1, 200, 64, pos), filled(g, 1, 1, 200, 64, pos)
    for new in (1e-3, 1.0, 500.0):
        q, k, v = rnd(g, 1, 2, 64, dtype=F16), rnd(g, 1, 1, 64, dtype=F16, std=new), rnd(g, 1, 1, 64, dtype=F16)
        a, b = ([x.clone() for x in (kc, vc, ks, vs)] for _ in range(2))
        a[0].view(torch.uint8)[0, 0, 7, 9], b[0].view(torch.uint8)[0, 0, 7, 9] = 0x7f, 0
        for x in (a, b):
            cla.window_attn_step8(q, k, v, *x, pos.cuda(), window=200)
        assert torch.equal(a[2][0, 0, :1], b[2][0, 0, :1])
        assert torch.isnan(a[0][0, 0, 7, 9].float())
        a[0].view(torch.uint8)[0, 0, 7, 9] = b[0].view(torch.uint8)[0, 0, 7, 9]
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))


def test_step_strided(cla):
    g = torch.Generator().manual_seed(4)
    qkv = rnd(g, 3, 8, 64, dtype=BF16)
    q, k, v = qkv.split((4, 2, 2), 1)
    pos = torch.tensor([3, 19, 50], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, 3, 2, 20, 64, pos), filled(g, 3, 2, 20, 64, pos)
    a, b = ([x.clone() for x in (kc, vc, ks, vs)] for _ in range(2))
    o = cla.window_attn_step8(q, k, v, *a, pos.cuda(), window=16, sinks=4)
    o1 = cla.window_attn_step8(q.contiguous(), k.contiguous(), v.contiguous(), *b, pos.cuda(), window=16, sinks=4)
    assert torch.equal(o, o1)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_prefill_then_steps(cla):
    """A prompt into the cache, then tokens one by one around it, against the 64-bit cache that goes the same way."""
    B, H, K, T, d, W, n = 2, 4, 2, 230, 64, 60, 3
    g = torch.Generator().manual_seed(8)
    q, k, v = rnd(g, B, H, T, d, dtype=F16), rnd(g, B, K, T, d, dtype=F16), rnd(g, B, K, T, d, dtype=F16)
    k = k * torch.logspace(-2, 2, T, device="cuda").half()[:, None]  # factors that grow, and shrink as the window moves on
    k[:, :, 150:] *= 0.01
    lens = torch.tensor([100, 37], dtype=torch.int32)
    cache = cla.window_cache8(B, K, d, window=W, sinks=n)
    ref = [R.cache8_write(x, c, s, lens, W, n) for x, c, s in ((k, cache[0], cache[2]), (v, cache[1], cache[3]))]
    cla.window_cache8_write(k, v, *cache, window=W, sinks=n, lens=lens.cuda())
    pos = lens.clone()
    b = torch.arange(B)
    for _ in range(130):
        q1, k1, v1 = (x[b.cuda(), :, pos.long().cuda()] for x in (q, k, v))
        ref = [R.cache8_put(x, *c, pos, W, n) for x, c in ((k1, ref[0]), (v1, ref[1]))]
        o = cla.window_attn_step8(q1, k1, v1, *cache, pos.cuda(), window=W, sinks=n)
        M.assert_within("o", o, *R.step8(q1, *ref[0], *ref[1], pos))
        pos += 1
    for x, y in zip(cache, (ref[0][0], ref[1][0], ref[0][1], ref[1][1])):
        same(x, y)


def test_near_the_attention_of_the_wide_cache(cla):
    """The step over 16 bits on the same tokens: off by what three mantissa bits are, 2^-4 of each key and value at most."""
    B, H, K, d, W = 3, 8, 2, 128, 500
    g = torch.Generator().manual_seed(21)
    k, v = rnd(g, B, K, W, d, dtype=BF16), rnd(g, B, K, W, d, dtype=BF16)
    q, k1, v1 = rnd(g, B, H, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16)
    pos = torch.full((B,), W, dtype=torch.int32, device="cuda")
    cache = cla.window_cache8(B, K, d, window=W)
    cla.window_cache8_write(k, v, *cache, window=W)
    o8 = cla.window_attn_step8(q, k1, v1, *cache, pos, window=W)
    kc, vc = k.clone(), v.clone()
    o16 = cla.window_attn_step(q, k1, v1, kc, vc, pos, window=W)
    # a logit moves by x = 2^-4 sum |q k| d^-1/2 at most, a weight by a factor of e^2x; values and the outputs' roundings
    x = 2 ** -4 * (q.float().view(B, K, 4, d).abs() @ kc.float().abs().transpose(2, 3)).max() * d ** -0.5
    far = float((2 * x).exp() - 1 + 2 ** -4 + 2 ** -7) * float(vc.float().abs().amax())
    assert float((o8.float() - o16.float()).abs().max()) <= far


def test_step_in_a_graph(cla):
    """A captured step, replayed as the sequences grow: positions and factors are read on the device."""
    B, H, K, d, W, n = 2, 8, 2, 128, 300, 4
    g = torch.Generator().manual_seed(6)
    q, k, v = rnd(g, B, H, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16)
    pos = torch.tensor([0, 280], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, B, K, W + n, d, pos), filled(g, B, K, W + n, d, pos)
    pos = pos.cuda()
    eager, static = [kc, vc, ks, vs], [x.clone() for x in (kc, vc, ks, vs)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = cla.window_attn_step8(q, k, v, *static, pos, window=W, sinks=n)
    for i in range(70):
        want = cla.window_attn_step8(q, k, v, *eager, pos, window=W, sinks=n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        pos += 1
        for x in (q, k, v):
            x.copy_(rnd(g, *x.shape, dtype=BF16, std=1 + i % 7))
    for a, b in zip(eager, static):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_repeats(cla):
    """The same call on the same cache gives the same bits: sums are in a fixed order, a block's numbers settle."""
    g = torch.Generator().manual_seed(7)
    B, H, K, d, W = 3, 12, 3, 64, 2000
    pos = torch.tensor([100, 1999, 7000], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, B, K, W, d, pos), filled(g, B, K, W, d, pos)
    q, k, v = rnd(g, B, H, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16, std=20.0), rnd(g, B, K, d, dtype=BF16)
    first = cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W)
    held = [x.clone() for x in (kc, vc, ks, vs)]
    for _ in range(5):
        assert torch.equal(first, cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W))
    for a, b in zip(held, (kc, vc, ks, vs)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_caches_of_more_than_31_bits(cla):
    """A cache of 2^32 bytes and more: the last sequence's slots and factors lie behind them.  Keys of zero weigh every slot
    alike; values are constant over a block."""
    B, K, d, W = 2, 1, 128, (1 << 24) + 1000
    pos = torch.tensor([W - 5, W + 64], dtype=torch.int32)
    kc, vc, ks, vs = cla.window_cache8(B, K, d, window=W)
    g = torch.Generator().manual_seed(1)
    val = torch.randint(0, 2, (B, K, R.blocks(W)), generator=g).double()
    rep = val.repeat_interleave(64, 2)[:, :, :W, None].cuda().to(torch.float32).to(E4M3)
    vc.view(torch.uint8).copy_(rep.view(torch.uint8).expand_as(vc))
    del rep
    ks.fill_(1.0), vs.fill_(2.0 ** -8)
    q, k, v = rnd(g, B, 2, d, dtype=F16), torch.zeros(B, K, d, dtype=F16, device="cuda"), rnd(g, B, K, d, dtype=F16)
    o = cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W)
    for b, p in enumerate(pos.tolist()):
        j, n = p % W, min(p + 1, W)
        mean = (val[b, 0].repeat_interleave(64)[:W][:n].sum() - val[b, 0, j // 64] * (p >= W)) / n * 2.0 ** -8
        # the token's own value is one of 2^24; a sum of 2^24 weights has 2^14 steps one after the other (16 blocks, 4 warps,
        # 16 slots at once), each off by a step of 2^-23 at most, and so has the one that divides; o by 2^-11
        torch.testing.assert_close(o[b].double().cpu(), mean.expand(2, d), rtol=2 ** -8 + 2 ** -11, atol=8 / n + 1e-7)
        f = R.factor(torch.cat((v[b, 0].double().cpu(), torch.tensor([2.0 ** -8]))))
        assert float(vs[b, 0, j // 64]) == f
        same(vc[b, 0, j], R.rounded(v[b, 0].double().cpu() / f))


@pytest.mark.parametrize("B,H,K,window", [(300, 2, 1, 100), (700, 1, 1, 63), (129, 2, 2, 200)])
def test_many_sequences(cla, B, H, K, window):
    """More sequences than a block has threads, most of them short or empty; and none at all."""
    g = torch.Generator().manual_seed(B)
    pos = torch.randint(-40, 2 * window, (B,), generator=g, dtype=torch.int32)
    pos[:3], pos[B - 2:] = -1, -5
    step(cla, g, B, H, K, 64, window, 2, BF16, pos)
    pos[:] = -1
    assert float(step(cla, g, B, H, K, 64, window, 2, BF16, pos).abs().max()) == 0
    pos[B // 2] = 70
    step(cla, g, B, H, K, 64, window, 2, BF16, pos)


@pytest.mark.parametrize("B,K", [(0, 1), (2, 0)])
def test_step_nothing_to_do(cla, B, K):
    cache = cla.window_cache8(B, K, 64, window=100)
    x = torch.zeros(B, K, 64, dtype=BF16, device="cuda")
    ws = torch.full((cla.window_attn_step8_workspace_size(B, K, K, 64, 100),), 255, dtype=torch.uint8, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    assert cla.window_attn_step8(x, x, x, *cache, pos, window=100, workspace=ws).shape == x.shape
    cla.check_status(ws)


def test_step_workspace(cla):
    """A workspace of the caller's, whatever it held and in use again; its status; one that is too small."""
    g = torch.Generator().manual_seed(17)
    B, H, K, d, W = 2, 6, 2, 64, 5000
    pos = torch.tensor([4000, 4999], dtype=torch.int32)
    (kc, ks), (vc, vs) = filled(g, B, K, W, d, pos), filled(g, B, K, W, d, pos)
    q, k, v = rnd(g, B, H, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16), rnd(g, B, K, d, dtype=BF16)
    want = cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W)
    n = cla.window_attn_step8_workspace_size(B, H, K, d, W)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(want, cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W, workspace=ws))
        cla.check_status(ws)
    with pytest.raises(ValueError, match="workspace"):
        cla.window_attn_step8(q, k, v, kc, vc, ks, vs, pos.cuda(), window=W, workspace=ws[:n - 1])
