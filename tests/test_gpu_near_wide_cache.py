"""The step over the 8-bit cache beside the one over 16 bits: as far apart as three mantissa bits are, and no further."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,H,K,d,W,n", [(3, 8, 2, 128, 500, 500), (2, 4, 4, 64, 300, 200), (2, 16, 1, 128, 3000, 7000)])
def test_near_the_attention_of_the_wide_cache(B, H, K, d, W, n, dtype):
    """A value is off by 2^-4 of itself at most, a logit by as much of each of its products: with signs that do not go together
    a head's output moves by 2^-4 (sum P^2 v^2)^1/2, and by 2^-4 (sum (q k)^2 / d)^1/2 of sum P^2 (v - o)^2's root, which for
    values and logits of size 1 is 2^-4 again.  The root mean square over a head's columns keeps within twice the sum of both."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as cla

    g = torch.Generator().manual_seed(W)

    def rnd(*s):
        return torch.randn(*s, generator=g).to(dtype).cuda()

    k, v, q, k1, v1 = rnd(B, K, n, d), rnd(B, K, n, d), rnd(B, H, d), rnd(B, K, d), rnd(B, K, d)
    pos = torch.full((B,), n, dtype=torch.int32, device="cuda")
    cache = cla.window_cache8(B, K, d, window=W)
    cla.window_cache8_write(k, v, *cache, window=W)
    o8 = cla.window_attn_step8(q, k1, v1, *cache, pos, window=W).double()
    kc, vc = (torch.zeros(B, K, W, d, dtype=dtype, device="cuda") for _ in range(2))
    cla.window_cache_write(k, v, kc, vc, window=W)
    o16 = cla.window_attn_step(q, k1, v1, kc, vc, pos, window=W).double()
    m = min(n + 1, W)
    kk, vv = (x[:, :, :m].double().repeat_interleave(H // K, 1) for x in (kc, vc))
    qk = q.double()[:, :, None] * kk * d ** -0.5
    P = torch.softmax(qk.sum(3), 2)[..., None]
    values = (P.square() * vv.square()).sum(2).mean(2).sqrt()
    logits = (P.square() * qk.square().sum(3, keepdim=True) * (vv - o16[:, :, None]).square()).sum(2).mean(2).sqrt()
    far = 2 * 2 ** -4 * (values + logits)
    off = (o8 - o16).square().mean(2).sqrt()
    size = o16.square().mean(2).sqrt()
    assert bool((far < 0.5 * size).all())  # neither zeros nor equal weights pass
    assert bool((off <= far).all()), float((off / far).max())
    assert float((off / far).min()) > 0.02  # 16 bits give something else
