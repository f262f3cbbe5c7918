"""The 8-bit step's weights keep fp32's accuracy for either type: values that cancel but for what their weights differ by."""
import pytest
import torch

from tests import _mixers as M

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,H,K,d,n", [(1, 4, 1, 64, 2), (2, 8, 2, 128, 64), (1, 16, 1, 64, 700), (3, 8, 1, 128, 5000),
                                       (90, 8, 4, 64, 256)])
def test_weights_that_nearly_cancel(cla, B, H, K, d, n, dtype):
    """Every other slot has the key 1 and the value 1, those between 9/8 and -1; query head h is (h + 1) 2^-9 in the same one
    place, so that a pair's weights differ by some 2^-12 of themselves, and what the head gives is that difference.

    Logits are single products of numbers of a few bits, exact, times the scale and log2 e.  Of the sum of all weights times
    |v|: a weight's two parts leave 2^-22 of it, its power of two 2^-22, and its logit (2^-5 at most, five roundings)
    nothing beside that; a product's sums over 16 slots, the warps' and the parts': n / 64 + 64 steps of 2^-23; the same for
    the total; the output half a step of itself.  One part of 11 bits would leave some 2^-12."""
    k = torch.zeros(B, K, n, d)
    k[..., 5] = 1.0
    k[:, :, 1::2, 5] = 1.125
    v = torch.ones(B, K, n, d)
    v[:, :, 1::2] = -1.0
    q = torch.zeros(B, H, d)
    q[..., 5] = (torch.arange(H) % (H // K) + 1) * 2.0 ** -9
    k, v, q = (x.to(dtype).cuda() for x in (k, v, q))
    cache = cla.window_cache8(B, K, d, window=n)
    cla.window_cache8_write(k[:, :, :n - 1], v[:, :, :n - 1], *cache, window=n)
    pos = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    got = cla.window_attn_step8(q, k[:, :, n - 1], v[:, :, n - 1], *cache, pos, window=n, scale=1.0)
    x = k[0, 0, :, 5].double().cpu() * q[0, :, 5].double().cpu()[:, None]
    want = (torch.softmax(x, 1) * v[0, 0, :, 0].double().cpu()).sum(1)[None, :, None].expand(B, H, d)
    e = M.half_step(dtype) * want.abs() + 3 * 2.0 ** -22 + 2 * (n / 64 + 64) * 2.0 ** -23
    assert float(e.max()) < 2.0 ** -3 * float(want.abs().max())  # a head's difference is well above what it may be off by
    M.assert_within("o", got, want, e)
