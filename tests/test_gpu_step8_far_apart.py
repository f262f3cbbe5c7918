"""The 8-bit step over blocks of values whose factors lie far apart: every column within a bound of its own."""
import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
U = M.U

# (B, H, K, window): thread blocks of one block of slots each, joined; shares of several whole pairs; shares that cut pairs
SPLITS = [(1, 4, 1, 128), (2, 3, 1, 80), (100, 8, 4, 128), (3, 24, 2, 2000), (2, 40, 1, 700)]


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def columns(q, kc, ks, vc, vs, pos):
    """(o, bound) of a step over caches that hold the token already (64 bits).  What a column may be off by is a share of its
    own sum P |v|, with, for each slot, 2^-37 of the largest weight of its 16 slots.  Shares, with n slots: the logit's (its query's numbers off by
    2^-24 of the largest; d products in fp32; five roundings of its own), once for the weight and once, the largest, for the
    total; 2^-22 each for the weight's two parts and its power of two; 64 + n / 64 steps of 2^-23 for the sums of products and
    as many for the total; weights below 2^-110 of the largest may count as nothing."""
    ut, (B, H, d), K, S = M.half_step(q.dtype), q.shape, kc.shape[1], kc.shape[2]
    G = H // K
    o, e = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    for b, p in enumerate(pos.tolist()):
        n = min(p + 1, S)
        fk, fv = (f[b].repeat_interleave(64, 1)[:, :n].repeat_interleave(G, 0) for f in (ks, vs))
        ck, cv = (c[b, :, :n].repeat_interleave(G, 0) for c in (kc, vc))
        kk, vv = ck * fk[..., None], cv * fv[..., None]
        qq = q[b].double().cpu()
        x = (kk @ qq[..., None])[..., 0] * d ** -0.5
        xa = (kk.abs() @ qq.abs()[..., None])[..., 0] * d ** -0.5
        ex = U * ((d + 6) * xa + 6 * x.abs() + 16) + kk.abs().sum(2) * qq.abs().amax(1, keepdim=True) * d ** -0.5 * 2.0 ** -24
        P = torch.softmax(x, 1)
        tile = torch.nn.functional.pad(P, (0, -n % 16)).view(H, -1, 16).amax(2).repeat_interleave(16, 1)[:, :n]
        share = ex + ex.amax(1, keepdim=True) + 2 * 2.0 ** -22 + 2 * (n / 64 + 64) * 2 * U
        o[b] = (P[:, None] @ vv)[:, 0]
        e[b] = 1.01 * (((P * share + 2.0 ** -37 * tile + 2.0 ** -110)[:, None] @ vv.abs())[:, 0] + ut * o[b].abs()) + R._tiny(q.dtype)
    return o, e


def both(cla, q, k, v, window, pos):
    """The step over prompts of k and v up to the token at pos, and its 64-bit form: (got, o, bound)."""
    B, K, n, d = k.shape
    cache = cla.window_cache8(B, K, d, window=window)
    cla.window_cache8_write(k[:, :, :n - 1], v[:, :, :n - 1], *cache, window=window)
    held = [cache[0].double().cpu(), cache[2].double().cpu(), cache[1].double().cpu(), cache[3].double().cpu()]
    most = 448 * 2.0 ** 120  # what an infinity is held as
    kn, vn = (x[:, :, n - 1].double().cpu().clamp(-most, most) for x in (k, v))
    ref = R.cache8_put(kn, *held[:2], pos, window, 0) + R.cache8_put(vn, *held[2:], pos, window, 0)
    o, e = columns(q, *ref, pos)
    return cla.window_attn_step8(q, k[:, :, n - 1], v[:, :, n - 1], *cache, pos.cuda(), window=window), o, e


def inputs(B, H, K, n, d, dtype, seed, logits=0.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, H, d, generator=g) * logits
    k = torch.randn(B, K, n, d, generator=g) * (logits != 0)
    v = torch.randn(B, K, n, d, generator=g)
    return tuple(x.to(dtype).cuda() for x in (q, k, v))


@pytest.mark.parametrize("B,H,K,n", SPLITS)
@pytest.mark.parametrize("power", [78, 110, 125])
def test_zeros_beside_large_values(cla, B, H, K, n, power):
    """Slots of zeros weigh as much as others, whichever come first: the mean of 2^power and them."""
    q, k, v = inputs(B, H, K, n, 64, BF16, 1)
    pos = torch.full((B,), n - 1, dtype=torch.int32)
    for large in (slice(0, 64), slice(64, n)):
        v.zero_()
        v[:, :, large] = 2.0 ** power
        got, o, e = both(cla, q, k, v, n, pos)
        M.assert_within("o", got, o, e)
        share = len(range(n)[large]) / n
        torch.testing.assert_close(got.double().cpu(), torch.full_like(o, share * 2.0 ** power), rtol=2 ** -8 + 2 ** -12, atol=0)


@pytest.mark.parametrize("B,H,K,n", SPLITS)
@pytest.mark.parametrize("logits", [0.0, 1.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_an_infinity_in_one_column(cla, B, H, K, n, logits, dtype):
    """Held as the largest number, it takes the other numbers of its own block of 64 slots and key head with it, and what
    other blocks give in other columns stays."""
    q, k, v = inputs(B, H, K, n, 64, dtype, 2, logits)
    pos = torch.full((B,), n - 1, dtype=torch.int32)
    for slot in (0, n // 2, n - 2, n - 1):
        x = v.clone()
        x[:, 0, slot, 7] = float("inf")
        got, o, e = both(cla, q, k, x, n, pos)
        largest = torch.finfo(dtype).max
        o[..., 7] = torch.where(o[..., 7] > largest, float("inf"), o[..., 7])
        if dtype == BF16:  # about the largest number either is right
            e[..., 7] = torch.where(o[..., 7] > 0.99 * largest, float("inf"), e[..., 7])
            got[..., 7] = torch.where(o[..., 7].cuda() > 0.99 * largest, got[..., 7].clamp(max=largest), got[..., 7])
        M.assert_within("o", got, torch.nan_to_num(o, posinf=largest) if dtype == BF16 else o, e)


@pytest.mark.parametrize("B,H,K,n", SPLITS)
@pytest.mark.parametrize("logits", [0.0, 1.0])
@pytest.mark.parametrize("dtype,low,high", [(F16, -11, 13), (BF16, -10, 16), (BF16, -20, 60)])
def test_columns_that_only_small_blocks_hold(cla, B, H, K, n, logits, dtype, low, high):
    """A block of values 2^24 and more above the others in eight columns, with zeros in the rest: there the others decide."""
    q, k, v = inputs(B, H, K, n, 128, dtype, 3, logits)
    pos = torch.full((B,), n - 1, dtype=torch.int32)
    for large in (slice(0, 64), slice(64, min(n, 128)), slice(n - n % 64 if n % 64 else n - 64, n)):
        x = v * 2.0 ** low
        x[:, :, large] = 0
        x[:, :, large, 8:16] = v[:, :, large, 8:16] * 2.0 ** high
        M.assert_within("o", *both(cla, q, k, x, n, pos))


@pytest.mark.parametrize("B,H,K,n", SPLITS)
@pytest.mark.parametrize("below,high", [(30, 40), (45, 60), (60, 90)])
def test_small_weights_of_large_values(cla, B, H, K, n, below, high):
    """Slots whose weights are 2^-below of the others' and whose values are 2^high as large: they decide."""
    q, k, v = inputs(B, H, K, n, 64, BF16, 4)
    pos = torch.full((B,), n - 1, dtype=torch.int32)
    for large in (slice(0, 64), slice(64, n)):
        q.zero_(), k.zero_()
        q[..., 0] = 8.0
        k[:, :, large, 0] = -below * 0.6931
        k[..., 1] = torch.randn(k.shape[:3], generator=torch.Generator().manual_seed(5)).to(BF16).cuda()
        q[..., 1] = 4.0
        x = v.clone()
        x[:, :, large] *= 2.0 ** high
        M.assert_within("o", *both(cla, q, k, x, n, pos))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 16, 64, 128, 1600])
def test_a_score_of_minus_infinity(cla, n, dtype):
    """A token whose key is the largest number in the direction away from the query: its score is -inf in fp32 and its weight
    nothing, also where it is all that a tile holds."""
    B, H, K, d = 2, 4, 2, 64
    q = torch.zeros(B, H, d)
    q[..., 3] = -1000.0
    k, v = torch.zeros(B, K, n + 1, d), torch.ones(B, K, n + 1, d)
    k[:, :, n, 3], v[:, :, n] = float("inf"), 5.0
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    cache = cla.window_cache8(B, K, d, window=n + 1)
    cla.window_cache8_write(k[:, :, :n], v[:, :, :n], *cache, window=n + 1)
    pos = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got = cla.window_attn_step8(q, k[:, :, n], v[:, :, n], *cache, pos, window=n + 1)
    assert torch.equal(got, torch.ones_like(got))


@pytest.mark.parametrize("B,H,K,n", SPLITS)
def test_a_nan_of_no_weight(cla, B, H, K, n):
    """A NaN among the values reaches its column however small its slot's weight, whichever way the work is split."""
    q, k, v = (torch.zeros(B, h, m, 64, dtype=BF16, device="cuda") for h, m in ((H, 1), (K, n), (K, n)))
    q, pos = q[:, :, 0], torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    q[..., 0] = 8.0
    for slot in (5, 70):
        k.zero_(), v.fill_(1.0)
        k[:, :, slot // 64 * 64:slot // 64 * 64 + 64, 0] = -400.0
        v[:, :, slot, 9] = float("nan")
        cache = cla.window_cache8(B, K, 64, window=n)
        cla.window_cache8_write(k[:, :, :n - 1], v[:, :, :n - 1], *cache, window=n)
        got = cla.window_attn_step8(q, k[:, :, n - 1], v[:, :, n - 1], *cache, pos, window=n)
        assert bool(torch.isnan(got[..., 9]).all())
        got[..., 9] = 1.0
        assert torch.equal(got, torch.ones_like(got))
