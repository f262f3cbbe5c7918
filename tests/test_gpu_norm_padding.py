"""Rows behind a sequence's length are 0 whatever the weights are."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d,rot,il", [(64, 64, False), (128, 32, False), (48, 16, True), (256, 0, False)])
def test_weights_that_are_not_finite(cla, d, rot, il, dtype):
    """A NaN and infinities among the weights reach the tokens of each sequence, and nothing behind them."""
    B, H, K, T = 4, 5, 2, 23
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, dq, dk = (torch.randn(B, h, T, d, generator=g, device="cuda").to(dtype) for h in (H, K, H, K))
    freq = torch.rand(rot // 2, generator=g, device="cuda") if rot else None
    lens = torch.tensor([T, 0, 7, -3], dtype=torch.int32, device="cuda")
    w = torch.ones(d, device="cuda")
    kw = dict(lens=lens, interleaved=il)
    clean = cla.qk_norm_rope_bwd(q, k, w, w, freq, dq, dk, **kw)
    w[3], w[d // 2], w[d - 1] = float("nan"), float("inf"), -float("inf")
    qo, ko = cla.qk_norm_rope_fwd(q, k, w, w, freq, **kw)
    got = cla.qk_norm_rope_bwd(q, k, w, w, freq, dq, dk, **kw)
    for x in (qo, ko, *got[:2]):
        for b, n in enumerate(lens.clamp(min=0).tolist()):
            assert bool((x[b, :, n:] == 0).all()), (b, n)
            assert n == 0 or bool(torch.isnan(x[b, :, :n]).any(-1).all())
    for a, b in zip(got[2:], clean[2:]):  # the weights' gradients do not depend on them
        assert torch.equal(a, b)
