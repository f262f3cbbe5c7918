"""Norm and rotation of queries and keys against the 64-bit form: forward, backward, one token."""
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


def inputs(B, H, K, T, d, rot, dtype, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)

    def rnd(h, s=1.0):
        return (torch.randn(B, h, T, d, generator=g) * s).to(dtype).cuda()

    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    freq = (10000.0 ** (-torch.arange(0, rot, 2).float() / rot)).cuda() if rot else None
    return (rnd(H, std), rnd(K, std), wq.cuda(), wk.cuda(), freq), (rnd(H), rnd(K))


def check(cla, args, ups, out=None, grad=None, **kw):
    q, k, wq, wk, freq = args
    got = dict(zip(("qo", "ko"), cla.qk_norm_rope_fwd(*args, **(out or {}), **kw)))
    got.update(zip(("dq", "dk", "dwq", "dwk"), cla.qk_norm_rope_bwd(*args, *ups, **(grad or {}), **kw)))
    for n, x, w, up in (("q", q, wq, ups[0]), ("k", k, wk, ups[1])):
        ref = R.norm_rope(x, w, freq, g=up, **kw)
        M.assert_within(n + "o", got[n + "o"], *ref["o"])
        M.assert_within("d" + n, got["d" + n], *ref["dx"])
        if w is not None:
            M.assert_within("dw" + n, got["dw" + n], *ref["dw"])
    again = cla.qk_norm_rope_bwd(*args, *ups, **kw)
    for n, x in zip(("dq", "dk", "dwq", "dwk"), again):
        assert x is None or torch.equal(x, got[n]), n
    return got


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (16, 0), (32, 16), (48, 32), (64, 64), (80, 48), (96, 96), (128, 128), (128, 32),
                                   (144, 16), (240, 240), (256, 256), (256, 0)])
def test_head_sizes(cla, d, rot, interleaved, dtype):
    check(cla, *inputs(2, 3, 2, 37, d, rot, dtype, d + rot), interleaved=interleaved)


@pytest.mark.parametrize("B,H,K,T", [(1, 1, 1, 1), (1, 1, 0, 5), (2, 0, 3, 9), (3, 16, 4, 1), (1, 5, 1, 300), (2, 40, 8, 33),
                                     (70, 2, 1, 3)])
def test_shapes(cla, B, H, K, T):
    check(cla, *inputs(B, H, K, T, 64, 64, BF16, T))


@pytest.mark.parametrize("B,H,K,T,d", [(2, 16, 4, 8000, 64), (1, 3, 1, 40000, 32)])
def test_many_rows(cla, B, H, K, T, d):
    """More rows than the lanes of the grid: a block's lanes take several tokens, the weights' sums many rows."""
    check(cla, *inputs(B, H, K, T, d, d, BF16, 3))


@pytest.mark.parametrize("B,H,K,T", [(0, 2, 1, 5), (2, 2, 1, 0), (2, 0, 0, 4)])
def test_nothing_to_do(cla, B, H, K, T):
    args, ups = inputs(B, H, K, T, 64, 64, BF16)
    qo, ko = cla.qk_norm_rope_fwd(*args)
    dq, dk, dwq, dwk = cla.qk_norm_rope_bwd(*args, *ups)
    assert qo.shape == dq.shape == args[0].shape and ko.shape == dk.shape == args[1].shape
    assert float(dwq.abs().max()) == 0 and float(dwk.abs().max()) == 0


def test_workspace(cla):
    """A workspace of the caller's, whatever it held and in use again; its status; one that is too small."""
    n = cla.qk_norm_rope_bwd_workspace_size(2, 4, 2, 50, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for T in (50, 0, 50):
        args, ups = inputs(2, 4, 2, T, 64, 64, BF16)
        want = cla.qk_norm_rope_bwd(*args, *ups)
        for a, b in zip(want, cla.qk_norm_rope_bwd(*args, *ups, workspace=ws)):
            assert torch.equal(a, b)
        cla.check_status(ws)
        ws[100:].fill_(255)
    with pytest.raises(ValueError, match="workspace"):
        cla.qk_norm_rope_bwd(*args, *ups, workspace=ws[:n - 1])


@pytest.mark.parametrize("which", ["none", "q", "k"])
def test_weights_left_out(cla, which):
    (q, k, wq, wk, freq), ups = inputs(2, 3, 2, 20, 64, 32, BF16)
    args = (q, k, wq if which == "q" else None, wk if which == "k" else None, freq)
    got = check(cla, args, ups)
    assert (got["dwq"] is None) == (which != "q") and (got["dwk"] is None) == (which != "k")


def test_positions_and_lengths(cla):
    """Packed documents; padded rows: outputs and gradients 0 and out of the weights' sums, whatever they hold; lengths of
    nothing and out of range."""
    (q, k, wq, wk, freq), ups = inputs(5, 4, 2, 70, 64, 64, BF16)
    pos = (torch.arange(70) % 13).repeat(5, 1)
    pos[3] = -torch.arange(70) * 1000
    pos = pos.to(torch.int32).cuda()
    lens = torch.tensor([70, 0, 1, 33, 999], dtype=torch.int32).cuda()
    got = check(cla, (q, k, wq, wk, freq), ups, pos=pos, lens=lens)
    for x in (q, k, *ups):
        for b, n in enumerate(lens.tolist()):
            x[b, :, n:] = float("nan") if b % 2 else float("inf")
    pos[2, 1:] = 2 ** 31 - 1
    bad = check(cla, (q, k, wq, wk, freq), ups, pos=pos, lens=lens)
    for n in got:
        assert torch.equal(got[n], bad[n]), n
    assert float(got["qo"][1].abs().max()) == 0 and float(got["dk"][3, :, 33:].abs().max()) == 0


def test_far_positions(cla):
    """Angles stay exact over all 31 bits of a position: the turn of (1, 0) and (0, 1) against whole-number arithmetic."""
    freq = torch.tensor([1.0, 0.5, 0.1, 10000.0 ** -0.3, 1e-4, 3.0, 1e-9, 100.0], device="cuda")
    pos = [0, 1, -1, 7, 1000, 123457, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 30 - 5, 2 ** 31 - 1, -2 ** 31, 999999937]
    x = torch.zeros(1, 1, len(pos), 16, device="cuda")
    x[..., :8] = 1.0
    kw = dict(pos=torch.tensor([pos], dtype=torch.int32).cuda(), eps=1e-12)
    o, _ = cla.qk_norm_rope_fwd(x, x, None, None, freq, **kw)
    o = o[0, 0].double().cpu() / 2 ** 0.5  # mean square 1/2
    for t, p in enumerate(pos):
        for i, f in enumerate(freq.tolist()):
            c, s = R.angle_exact(p, f)
            # 7 roundings, and the angle's 2^-31 (1 + f) of a turn
            e = 12 * M.U + 2 ** -31 * (1 + f) * 6.3
            assert abs(float(o[t, i]) - c) <= e and abs(float(o[t, i + 8]) - s) <= e, (p, f)


def test_angles_densely(cla):
    """fp32 rows at many positions, in every eighth of a turn and at their borders: sines and cosines within the form's bound."""
    T = 30000
    args, ups = inputs(1, 1, 1, T, 16, 16, F32, 7)
    freq = torch.tensor([1.0, 0.7853981633974483, 1.5707963267948966, 3.141592653589793, 0.1, 6.283185307179586, 1e-3, 0.39269908],
                        device="cuda")
    g = torch.Generator().manual_seed(3)
    pos = torch.cat((torch.arange(T // 2), torch.randint(-(1 << 21), 1 << 21, (T - T // 2,), generator=g))).to(torch.int32)
    check(cla, args[:4] + (freq,), ups, pos=pos[None].cuda())


@pytest.mark.parametrize("B,T", [(5, 7), (3, 64), (2, 65), (40, 1), (3, 700)])
def test_groups_across_sequences(cla, B, T):
    """Groups of tokens that end one sequence and begin another, or several."""
    (q, k, wq, wk, freq), ups = inputs(B, 3, 1, T, 64, 64, BF16, B)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 5000, (B, T), generator=g, dtype=torch.int32).cuda()
    lens = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32).cuda()
    check(cla, (q, k, wq, wk, freq), ups, pos=pos, lens=lens)


def test_odd_frequencies(cla):
    """Negative, subnormal and vast frequencies: an angle of the other sign, none, and one that is some angle."""
    (q, k, wq, wk, _), _ = inputs(1, 2, 1, 9, 16, 0, F32)
    f = torch.tensor([0.3, 1e-3, 1.0, 0.7, 0.01, 2.0, 0.5, 0.2], device="cuda")
    a = cla.qk_norm_rope_fwd(q, k, wq, wk, -f)[0]
    b = cla.qk_norm_rope_fwd(q, k, wq, wk, f, pos=-torch.arange(9, dtype=torch.int32, device="cuda")[None])[0]
    assert torch.equal(a, b)
    none = cla.qk_norm_rope_fwd(q, k, wq, wk, torch.full_like(f, 1e-40))[0]
    M.assert_within("qo", none, *R.norm_rope(q, wq)["o"])
    vast = cla.qk_norm_rope_fwd(q, k, wq, wk, torch.full_like(f, 1e30))[0].double()
    # a turn keeps each pair's length
    n = R.norm_rope(q, wq)["o"][0]
    lens = [(x[..., :8] ** 2 + x[..., 8:] ** 2).cpu() for x in (vast, n.cuda())]
    torch.testing.assert_close(lens[0], lens[1], rtol=100 * M.U, atol=0)


def test_small_and_large_rows(cla):
    """Rows of zeros and of subnormals, where eps decides, and of values whose squares are near fp32's limits."""
    (q, k, wq, wk, freq), ups = inputs(1, 6, 1, 8, 64, 64, F32)
    q[:, 0] = 0
    q[:, 1] *= 1e-30
    q[:, 2] *= 1e-3
    q[:, 3] *= 1e17
    q[:, 4] = 0
    q[:, 4, :, 5] = 1e-20
    check(cla, (q, k, wq, wk, freq), ups)
    q, k = q.bfloat16(), k.bfloat16()
    check(cla, (q, k, wq, wk, freq), tuple(u.bfloat16() for u in ups), eps=1e-3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_and_in_place(cla, dtype):
    """Slices of one projection [B, T, heads, d], its gradient in that layout; over the inputs themselves."""
    B, H, K, T, d = 2, 4, 2, 50, 64
    (_, _, wq, wk, freq), ups = inputs(B, H, K, T, d, 32, dtype)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(B, T, H + 2 * K, d, generator=g).to(dtype).cuda()
    q, k, _ = (x.transpose(1, 2) for x in qkv.split((H, K, K), 2))
    grad = torch.full_like(qkv, 7.0)
    dq, dk, rest = (x.transpose(1, 2) for x in grad.split((H, K, K), 2))
    qo, ko = (torch.empty(B, T, h, d, dtype=dtype, device="cuda").transpose(1, 2) for h in (H, K))
    got = check(cla, (q, k, wq, wk, freq), ups, dict(qo=qo, ko=ko), dict(dq=dq, dk=dk))
    dense = check(cla, (q.contiguous(), k.contiguous(), wq, wk, freq), ups)
    for n in got:
        assert torch.equal(got[n], dense[n]), n
    assert bool((rest == 7).all()) and got["qo"].data_ptr() == qo.data_ptr()
    # expanded inputs are refused
    with pytest.raises(cla.ClaError, match="stride 0 of q"):
        cla.qk_norm_rope_fwd(q[:, :1].expand(-1, 3, -1, -1), k, wq, wk, freq)
    up = tuple(u.clone() for u in ups)
    a, b, *_ = cla.qk_norm_rope_bwd(q, k, wq, wk, freq, *up, dq=up[0], dk=up[1])
    assert a is up[0] and torch.equal(a, got["dq"]) and torch.equal(b, got["dk"])
    v = qkv[:, :, H + K:].clone()
    a, b = cla.qk_norm_rope_fwd(q, k, wq, wk, freq, qo=q, ko=k)
    assert a is q and torch.equal(q, got["qo"]) and torch.equal(k, got["ko"]) and torch.equal(qkv[:, :, H + K:], v)


def test_misaligned_views(cla):
    (q, k, wq, wk, freq), _ = inputs(1, 2, 1, 5, 64, 64, BF16)
    flat = torch.zeros(q.numel() + 8, dtype=BF16, device="cuda")
    off = flat[1:1 + q.numel()].view(q.shape)
    with pytest.raises(cla.ClaError, match="misaligned"):
        cla.qk_norm_rope_fwd(off, k, wq, wk, freq)
    wide = torch.zeros(1, 2, 5, 68, dtype=BF16, device="cuda")[..., :64]
    with pytest.raises(cla.ClaError, match="stride"):
        cla.qk_norm_rope_fwd(wide, k, wq, wk, freq)


def test_step(cla):
    """One token a sequence: what the whole sequence's call gives at its position; slices of a projection, in place."""
    B, H, K, T, d = 3, 4, 2, 30, 128
    (q, k, wq, wk, freq), _ = inputs(B, H, K, T, d, 64, BF16)
    for il in (False, True):
        qo, ko = cla.qk_norm_rope_fwd(q, k, wq, wk, freq, interleaved=il)
        pos = torch.tensor([0, 29, 7], dtype=torch.int32).cuda()
        b = torch.arange(B, device="cuda")
        mix = torch.cat((q[b, :, pos.long()], k[b, :, pos.long()]), 1)
        a, c = cla.qk_norm_rope_step(mix[:, :H], mix[:, H:], wq, wk, freq, pos, interleaved=il)
        assert a.shape == (B, H, d) and torch.equal(a, qo[b, :, pos.long()]) and torch.equal(c, ko[b, :, pos.long()])
        q1, k1 = mix[:, :H], mix[:, H:]
        a, c = cla.qk_norm_rope_step(q1, k1, wq, wk, freq, pos, interleaved=il, qo=q1, ko=k1)
        assert a is q1 and torch.equal(mix, torch.cat((qo[b, :, pos.long()], ko[b, :, pos.long()]), 1))


def test_gradients_against_differences(cla):
    """Central differences of the 64-bit form along random directions."""
    (q, k, wq, wk, freq), (up, upk) = inputs(2, 3, 1, 20, 64, 64, F32)
    dq, _, dwq, _ = cla.qk_norm_rope_bwd(q, k, wq, wk, freq, up, upk)

    def loss(x, w):
        return float((R.norm_rope(x, w, freq)["o"][0] * up.double().cpu()).sum())

    q, wq = q.double().cpu(), wq.double().cpu()
    for got, which in ((dq, 0), (dwq, 1)):
        s = torch.randn(got.shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
        e = 1e-5
        a, b = ((q + e * s, wq), (q - e * s, wq)) if which == 0 else ((q, wq + e * s), (q, wq - e * s))
        num = (loss(*a) - loss(*b)) / (2 * e)
        terms = got.double().cpu() * s
        assert abs(num - float(terms.sum())) <= 1e-6 * float(terms.abs().sum())


def test_captured(cla):
    """Forward and backward in a graph, replayed on new inputs, positions and lengths."""
    args, ups = inputs(2, 4, 2, 40, 64, 64, BF16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1)
    lens = torch.tensor([40, 11], dtype=torch.int32).cuda()
    kw = dict(pos=pos, lens=lens)
    cla.qk_norm_rope_fwd(*args, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = cla.qk_norm_rope_fwd(*args, **kw) + cla.qk_norm_rope_bwd(*args, *ups, **kw)
    for seed in (5, 6):
        new, up = inputs(2, 4, 2, 40, 64, 64, BF16, seed)
        for a, b in zip(args + ups, new + up):
            a.copy_(b)
        pos.add_(1000), lens.fill_(17 + seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, cla.qk_norm_rope_fwd(*args, **kw) + cla.qk_norm_rope_bwd(*args, *ups, **kw)):
            assert torch.equal(a, b)


def test_more_than_31_bits_of_elements(cla):
    """Rows behind 2^31 elements of q are the rows of a call of their own."""
    T, H, d = 65536 + 64, 256, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.empty(1, H, T, d, dtype=BF16, device="cuda").normal_(generator=g)
    (_, k, wq, wk, freq), _ = inputs(1, 1, 1, T, d, 128, BF16)
    qo, ko = cla.qk_norm_rope_fwd(q, k, wq, wk, freq)
    dq, _, dwq, _ = cla.qk_norm_rope_bwd(q, k, wq, wk, freq, q, k)
    pos = torch.arange(T - 50, T, dtype=torch.int32, device="cuda")[None]
    part = (q[:, H - 2:, T - 50:].contiguous(), k[:, :, T - 50:].contiguous())
    a, b = cla.qk_norm_rope_fwd(*part, wq, wk, freq, pos=pos)
    assert torch.equal(qo[:, H - 2:, T - 50:], a) and torch.equal(ko[:, :, T - 50:], b)
    c = cla.qk_norm_rope_bwd(*part, wq, wk, freq, *part, pos=pos)[0]
    assert torch.equal(dq[:, H - 2:, T - 50:], c)
    assert bool(torch.isfinite(dwq).all())
