"""A decay that underflows is not a reset: only a log decay of -inf drops what the state holds."""
import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("ld", [-103.0, -104.5, -150.0, -1e30, -INF])
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
def test_what_the_state_holds_stays(cla, ld, bad, T, dtype):
    """A column of the state with a NaN or an infinity stays without a number, the others are what they were without it; a
    reset drops it.  Finite states are as in 64 bits either way."""
    B, H, dk, dv = 2, 2, 64, 68
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(B, H, T, n, generator=g).to(dtype).cuda() for n in (dk, dk, dv))
    k = (k / 8).to(dtype)
    lds, beta = (torch.rand(B, H, T, generator=g).cuda() - 1 for _ in range(2))
    beta, S = beta + 1.5, torch.randn(B, H, dk, dv, generator=g).cuda()
    at = T // 2
    lds[1, 0, at] = ld
    ins = (q, k, v, lds, beta)
    (o, eo), (ST, eS) = R.delta(*ins, S)
    clean = S.clone()
    oc = cla.delta_step(*ins, clean)
    M.assert_within("o", oc, o, eo)
    M.assert_within("S", clean, ST, eS)
    S[1, 0, 9, 33] = bad
    ob = cla.delta_step(*ins, S)
    if ld == -INF:
        assert torch.equal(S[1, 0], clean[1, 0]) and torch.equal(ob[:, :, at:], oc[:, :, at:])
    else:
        assert not bool(torch.isfinite(S[1, 0, :, 33]).any()) and not bool(torch.isfinite(ob[1, 0, :, 33]).any())
    S[1, 0, :, 33], ob[1, 0, :, 33] = clean[1, 0, :, 33], oc[1, 0, :, 33]
    assert torch.equal(S, clean) and torch.equal(ob, oc)
