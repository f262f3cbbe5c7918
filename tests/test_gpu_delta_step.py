"""The delta rule token by token against its 64-bit form, and behind the chunked forward."""
import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def inputs(B, H, Hk, T, dk, dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g)

    k = rnd(B, Hk, T, dk)
    k = k / k.norm(dim=-1, keepdim=True)
    return (rnd(B, Hk, T, dk).to(dtype).cuda(), k.to(dtype).cuda(), rnd(B, H, T, dv).to(dtype).cuda(),
            -torch.rand(B, H, T, generator=g).cuda(), torch.rand(B, H, T, generator=g).cuda(), rnd(B, H, dk, dv).cuda())


def check(cla, args, lens=None):
    *ins, S = args
    (o, eo), (ST, eS) = R.delta(*ins, S, lens)
    S = S.clone()
    got = cla.delta_step(*ins, S, lens=lens)
    M.assert_within("o", got, o, eo)
    M.assert_within("S", S, ST, eS)
    return got, S


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,H,Hk,T,dk,dv", [(1, 1, 1, 1, 64, 64), (2, 4, 4, 1, 128, 128), (3, 6, 2, 1, 64, 192),
                                            (1, 5, 5, 3, 128, 4), (2, 3, 1, 7, 64, 36), (2, 2, 2, 20, 128, 68), (1, 2, 1, 1, 64, 1024),
                                            (40, 2, 1, 2, 64, 32), (1, 32, 16, 4, 128, 128)])
def test_shapes(cla, B, H, Hk, T, dk, dv, dtype):
    check(cla, inputs(B, H, Hk, T, dk, dv, dtype, T + dv))


def test_many_states(cla):
    """More blocks than the GPU holds at once."""
    check(cla, inputs(24, 32, 16, 1, 128, 128, BF16))


@pytest.mark.parametrize("B,H,T", [(0, 2, 3), (2, 0, 3), (2, 2, 0)])
def test_nothing_to_do(cla, B, H, T):
    *ins, S = inputs(B, H, H, T, 64, 64, BF16)
    before = S.clone()
    assert cla.delta_step(*ins, S).shape == (B, H, T, 64) and torch.equal(S, before)


def test_lengths(cla):
    """Tokens behind a sequence's length: o 0, the state of those before, whatever they hold; no token at all leaves the
    state's bits alone, NaN included."""
    args = inputs(6, 4, 2, 5, 64, 64, BF16)
    lens = torch.tensor([5, 0, 1, 3, 99, -4], dtype=torch.int32).cuda()
    o, S = check(cla, args, lens.clamp(0, 5))
    for x in args[:5]:
        for b, n in enumerate(lens.tolist()):
            x[b, :, max(n, 0):] = float("nan") if b % 2 else float("inf")
    S1 = args[5].clone()
    S1[1, 2, 3, 4] = float("nan")
    o1 = cla.delta_step(*args[:5], S1, lens=lens)
    assert torch.equal(o, o1) and float(o[1].abs().max()) == 0 and float(o[3, :, 3:].abs().max()) == 0
    assert torch.isnan(S1[1, 2, 3, 4])
    S1[1, 2, 3, 4] = S[1, 2, 3, 4]
    assert torch.equal(S1, S) and torch.equal(S1[5], args[5][5])


def test_decays(cla):
    """Decays of one, near none, and none: a log decay of -inf drops the state whatever it holds."""
    *ins, S = inputs(2, 2, 2, 4, 64, 64, F32)
    ins[3][:, 0] = 0.0
    ins[3][:, 1, 0] = -80.0
    ins[3][0, 1, 2] = -200.0
    check(cla, (*ins, S))
    ins[3][1, 1, 1] = -float("inf")
    o, ST = check(cla, (*ins, S))
    bad = S.clone()
    bad[1, 1, 5, 6], bad[1, 1, 0, 0] = float("nan"), float("inf")
    o1 = cla.delta_step(*ins, bad)
    assert torch.equal(o1[1, 1, 1:], o[1, 1, 1:]) and torch.equal(bad[1, 1], ST[1, 1])


def test_overwrite_stores_the_value_under_its_key(cla):
    """beta = 1 and a key of length one: reading with that key gives the value, whatever the state held."""
    *ins, S = inputs(3, 4, 4, 1, 128, 128, F32)
    ins[0] = ins[1].clone()
    ins[4].fill_(1.0)
    o = cla.delta_step(*ins, S)
    # two sums of 128 terms of the state each, states of size 1
    assert float((o - ins[2]).abs().max()) <= 40 * M.U * 128 ** 0.5 * 4


def test_strided(cla):
    """Slices of one projection [B, T, ...], gates [B, T, H], odd element offsets."""
    B, H, Hk, T, dk, dv = 2, 4, 2, 3, 64, 68
    g = torch.Generator().manual_seed(5)
    for dtype in (BF16, F32):
        flat = torch.randn(B * T * (2 * Hk * dk + H * dv) + 1, generator=g).to(dtype).cuda()
        mix = flat[1:].view(B, T, -1)
        q = mix[..., :Hk * dk].view(B, T, Hk, dk).transpose(1, 2)
        k = mix[..., Hk * dk:2 * Hk * dk].view(B, T, Hk, dk).transpose(1, 2)
        v = mix[..., 2 * Hk * dk:].view(B, T, H, dv).transpose(1, 2)
        k.mul_(0.1)
        gates = torch.rand(B, T, 2, H, generator=g).cuda()
        ld, be = -gates[:, :, 0].transpose(1, 2), gates[:, :, 1].transpose(1, 2)
        ld = torch.empty(B, T, H, device="cuda").transpose(1, 2).copy_(ld)
        S = torch.randn(B, H, dk, dv, generator=g).cuda()
        o, ST = check(cla, (q, k, v, ld, be, S))
        o1, ST1 = check(cla, tuple(x.contiguous() for x in (q, k, v, ld, be, S)))
        assert torch.equal(o, o1) and torch.equal(ST, ST1)
    with pytest.raises(cla.ClaError, match="stride 0 of k"):
        cla.delta_step(q, k[:, :1].expand(-1, Hk, -1, -1), v, ld, be, S)


def test_tokens_together_are_tokens_apart(cla):
    *ins, S = inputs(2, 4, 2, 6, 128, 64, BF16)
    S1 = S.clone()
    o = cla.delta_step(*ins, S)
    parts = [cla.delta_step(*(x[:, :, t:t + 1] for x in ins), S1) for t in range(6)]
    assert torch.equal(o, torch.cat(parts, 2)) and torch.equal(S, S1)


def test_behind_the_chunked_forward(cla):
    """A prompt through delta_fwd, then tokens one by one: the recurrence over the whole sequence.  The chunked forward's own
    error (its products round states and keys to bf16) decides: the bound of its tests, 2e-2 of the values' root mean
    square at most, carries through the state's contraction."""
    B, H, T, d, n = 2, 3, 100, 64, 90
    *ins, S = inputs(B, H, H, T, d, d, BF16, 3)
    (o, _), (ST, _) = R.delta(*ins, S)
    o0, state = cla.delta_fwd(*(x[:, :, :n].contiguous() for x in ins), S)
    got = [o0] + [cla.delta_step(*(x[:, :, t:t + 1] for x in ins), state) for t in range(n, T)]
    got = torch.cat(got, 2).double().cpu()
    assert float((got - o).abs().max()) <= 2e-2 * float(o.square().mean().sqrt()) * 4
    assert float((state.double().cpu() - ST).abs().max()) <= 2e-2 * float(ST.square().mean().sqrt()) * 4


def test_captured(cla):
    *ins, S = inputs(2, 4, 2, 2, 64, 64, BF16)
    lens = torch.tensor([2, 1], dtype=torch.int32).cuda()
    S1 = S.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = cla.delta_step(*ins, S1, lens=lens)
    for seed in range(4):
        want = cla.delta_step(*ins, S, lens=lens)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(S, S1)
        for a, b in zip(ins, inputs(2, 4, 2, 2, 64, 64, BF16, seed + 1)):
            a.copy_(b)
        lens.copy_(lens.flip(0))


def test_states_of_more_than_31_bits(cla):
    """States behind 2^31 elements are those of a call of their own."""
    B, H, dk, dv = 260, 512, 128, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    S = torch.empty(B, H, dk, dv, device="cuda").normal_(generator=g)
    *ins, _ = inputs(B, H, H, 1, dk, 4, BF16)
    v = torch.randn(B, H, 1, dv, device="cuda", generator=g).bfloat16()
    part = S[B - 1:].clone()
    o = cla.delta_step(ins[0], ins[1], v, ins[3], ins[4], S)
    o1 = cla.delta_step(*(x[B - 1:] for x in (ins[0], ins[1], v, ins[3], ins[4])), part)
    assert torch.equal(o[B - 1:], o1) and torch.equal(S[B - 1:], part)
