"""The gradients of the norm's weights against 64 bits, with a bound that follows the kernel's own chain of sums."""
import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = M.U


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def sums(x, g, freq=None, pos=None, lens=None, interleaved=False, eps=1e-6):
    """(dw, bound) in 64 bits on the tensors' device, a head at a time.  A term g n is off by the turn's 8 U of its pair's
    values and 21 U of itself (r: 17, three products); a lane adds 64 of them at most one after the other, and 5 rounds of
    lanes, in fp32; what follows has 48 bits or more, and the sum is rounded once."""
    B, h, T, d = x.shape
    rot = 0 if freq is None else 2 * freq.numel()
    cos = sin = None
    if rot:
        p = torch.arange(T, device=x.device).expand(B, T) if pos is None else pos
        angle = p.double()[:, None, :, None] * freq.double()
        cos, sin = torch.cos(angle), torch.sin(angle)
    dw, e = (torch.zeros(d, dtype=torch.float64, device=x.device) for _ in range(2))
    for i in range(h):
        z, up = x[:, i:i + 1].double(), g[:, i:i + 1].double()
        if lens is not None:
            live = (torch.arange(T, device=x.device) < lens[:, None])[:, None, :, None]
            z, up = torch.where(live, z, 0.0), torch.where(live, up, 0.0)
        n = z / torch.sqrt(z.square().mean(3, keepdim=True) + eps)
        terms = R._turned(up, cos, -sin if rot else None, rot, interleaved) * n
        dw += terms.sum((0, 1, 2))
        e += (U * (21 + 64 + 5) * terms.abs() + (U * 8 * R._pair_sum(up, rot, interleaved) * n.abs() if rot else 0)).sum((0, 1, 2))
    return dw, 1.01 * e + U * dw.abs() + 1e-37


def check(name, got, dw, e):
    """Within the bound, and the bound a small part of what there is."""
    assert float(e.max()) < 0.02 * float(dw.square().mean().sqrt()), name
    M.assert_within(name, got, dw, e)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,H,K,T,d,rot,il", [(2, 16, 4, 8000, 64, 64, False), (1, 3, 1, 40000, 32, 16, True),
                                              (3, 10, 5, 1531, 96, 48, True), (2, 4, 1, 3000, 256, 256, False),
                                              (1, 5, 2, 5000, 16, 0, False)])
def test_many_rows(cla, B, H, K, T, d, rot, il, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, dq, dk = (torch.randn(B, h, T, d, generator=g, device="cuda").to(dtype) for h in (H, K, H, K))
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").float() / rot) if rot else None
    pos = torch.randint(0, 100000, (B, T), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.tensor([T, T - 17, T // 2][:B], dtype=torch.int32, device="cuda")
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    _, _, dwq, dwk = cla.qk_norm_rope_bwd(q, k, w, w, freq, dq, dk, pos=pos, lens=lens, interleaved=il)
    check("dwq", dwq, *sums(q, dq, freq, pos, lens, il))
    check("dwk", dwk, *sums(k, dk, freq, pos, lens, il))


@pytest.mark.parametrize("d,H,rot", [(128, 256, 128), (256, 128, 0)])
def test_more_than_31_bits_of_elements(cla, d, H, rot):
    """Some 2300 rows a lane: no row is lost behind 2^31 elements, and rows that are all alike, whose sums in fp32 would drift
    in one direction, keep their bits."""
    T = 65536 + 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q, up = (torch.empty(1, H, T, d, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(2))
    k, w = torch.randn(1, 1, T, d, generator=g, device="cuda").to(BF16), torch.ones(d, device="cuda")
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").float() / rot) if rot else None
    dwq, dwk = cla.qk_norm_rope_bwd(q, k, w, w, freq, up, k)[2:]
    check("dwq", dwq, *sums(q, up, freq))
    check("dwk", dwk, *sums(k, k, freq))
    q.copy_(q[:, :1, :1].clone().expand_as(q))
    up.copy_(up[:, :1, :1].clone().expand_as(up))
    dwq = cla.qk_norm_rope_bwd(q, k, w, w, None, up, k)[2]
    dw, e = sums(q[:, :1, :1], up[:, :1, :1])
    M.assert_within("dwq of rows alike", dwq, dw * H * T, e * H * T)
