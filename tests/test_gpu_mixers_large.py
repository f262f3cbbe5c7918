"""The gated scan and the window attention on tensors of more than 2^31 elements: the last tokens, which lie behind that
many, against the 64-bit forms of a slice that holds all they depend on."""
import pytest
import torch

from tests import _mixers as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def rnd(seed, *s, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(s, dtype=BF16, device="cuda").normal_(0, std, generator=g)


def tail_within(name, x, ref, n):
    """The last n tokens (second last axis) of x against those of the slice's reference."""
    r, e = ref
    R.assert_within(name, x[..., -n:, :], r[..., -n:, :], e.expand_as(r)[..., -n:, :])


@pytest.mark.parametrize("heads_last", [False, True])
def test_window_attention(cla, heads_last):
    H, T, d, W = 32, (1 << 19) + 77, 128, 200

    def make(seed, h, std=1.0):
        return rnd(seed, 1, T, h, d, std=std).transpose(1, 2) if heads_last else rnd(seed, 1, h, T, d, std=std)

    q, k, v, dO = make(1, H, 1.5), make(2, 1), make(3, 1), make(4, H)
    assert q.numel() > 1 << 31
    o, lse = cla.window_attn_fwd(q, k, v, window=W, o=torch.empty_like(q))
    dq, dk, dv = cla.window_attn_bwd(q, k, v, o, lse, dO, window=W, dq=torch.empty_like(q))
    cut = lambda x: x[:, :, -2 * W:].contiguous()
    ref = R.window(cut(q), cut(k), cut(v), W, 0, dO=cut(dO))
    for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        tail_within(n, x, ref[n], W)
    R.assert_within("lse", lse[:, :, -W:], ref["lse"][0][..., -W:], ref["lse"][1].expand_as(ref["lse"][0])[..., -W:])


def test_window_step(cla):
    B, H, K, d, W, n = 65, 8, 8, 128, 1 << 15, 4
    kc, vc = rnd(1, B, K, W + n, d), rnd(2, B, K, W + n, d)
    assert kc.numel() > 1 << 31
    q, k, v = rnd(3, B, H, d, std=1.5), rnd(4, B, K, d), rnd(5, B, K, d)
    pos = torch.full((B,), -1, dtype=torch.int32)
    pos[-1] = 3 * W + 1000
    at = n + (3 * W + 1000 - n) % W
    (ro, e), rk, rv = R.window_step(q[-1:], k[-1:], v[-1:], kc[-1:], vc[-1:], pos[-1:], n)
    o = cla.window_attn_step(q, k, v, kc, vc, pos.cuda(), window=W, sinks=n)
    R.assert_within("o", o[-1:], ro, e)
    assert torch.equal(kc[-1].cpu(), rk[0]) and torch.equal(vc[-1, :, at].cpu(), v[-1].cpu())
    assert float(o[:-1].abs().max()) == 0


def test_cache_write(cla):
    B, K, T, d, W, n = 66, 8, 300, 128, 1 << 15, 4
    kc, vc = (torch.zeros(B, K, W + n, d, dtype=BF16, device="cuda") for _ in range(2))
    k, v = rnd(1, B, K, T, d), rnd(2, B, K, T, d)
    cla.window_cache_write(k, v, kc, vc, window=W, sinks=n)
    assert torch.equal(kc[-1, :, :T], k[-1]) and torch.equal(vc[-1, :, :T], v[-1]) and float(kc[-1, :, T:].abs().max()) == 0


def test_gated_scan(cla):
    T, D, n = (1 << 20) + 77, 2048, 200
    x, r, i, dh = rnd(1, 1, T, D), rnd(2, 1, T, D, std=1.5), rnd(3, 1, T, D, std=1.5), rnd(4, 1, T, D)
    assert x.numel() > 1 << 31
    lam = torch.zeros(D, device="cuda")  # a fully open gate leaves e^-5.5: a hundred steps leave nothing
    ck = cla.gated_scan_ckpt(x)
    ws = torch.empty(cla.gated_scan_workspace_size(1, T, D), dtype=torch.uint8, device="cuda")
    h, hT = cla.gated_scan_fwd(x, r, i, lam, ckpt=ck, workspace=ws)
    cla.check_status(ws)
    dx, dr, di, _, _ = cla.gated_scan_bwd(x, r, i, lam, None, dh, ckpt=ck, workspace=ws)
    cla.check_status(ws)
    cut = lambda t: t[:, -n:].contiguous()
    ref = R.gated(cut(x), cut(r), cut(i), lam, dh=cut(dh))
    for name, y in (("h", h), ("dx", dx), ("drgate", dr), ("digate", di)):
        tail_within(name, y, ref[name], n // 2)
    R.assert_within("hT", hT, *ref["hT"])


def test_list_of_a_million_steps(cla):
    """One key head for 128 query heads: the list of the sinks' tile has 2^20 steps, over all of which its stores wait.
    Queries, keys and values of 0 leave P = 1 / n_t (n_t: the keys that t sees) and dv_s = sum of dO_t / n_t over the
    queries that see s."""
    H, T, d, W = 128, 1 << 20, 64, 12800
    zeros = torch.zeros(1, H, T, d, dtype=BF16, device="cuda")  # q and o
    kv = torch.zeros(1, 1, T, d, dtype=BF16, device="cuda")
    dO = torch.empty(1, H, T, d, dtype=BF16, device="cuda").uniform_(0.5, 1.5, generator=torch.Generator(device="cuda").manual_seed(1))
    t = torch.arange(T, device="cuda")
    seen = ((t + 1).clamp(max=W) + (t >= W)).double()
    lse = seen.log().float().expand(1, H, T).contiguous()
    ws = torch.empty(cla.window_attn_bwd_workspace_size(1, H, 1, T, d, W, 1), dtype=torch.uint8, device="cuda")
    dq, dk, dv = cla.window_attn_bwd(zeros, kv, kv, zeros, lse, dO, window=W, sinks=1, workspace=ws)
    cla.check_status(ws)
    assert not dq.any() and not dk.any() and torch.isfinite(dv).all()
    share = torch.stack([dO[0, :, :, c].sum(0, dtype=torch.float64) for c in range(d)], 1) / seen[:, None]
    run = torch.cat([share.new_zeros(1, d), share.cumsum(0)])
    want = run[(t + W).clamp(max=T)] - run[t]
    # P: the log's and the exponential's roundings and half a step of bf16; fp32 sums of 101 x 128 steps of 8 products
    # each, every one off by at most a step of the sum so far (all terms are positive); dv's own half step
    bound = want * (1.01 * (2.0 ** -8 + 64 * 2.0 ** -24) + 101 * 128 * 8 * 2.0 ** -23 + 2.0 ** -8)
    R.assert_within("dv", dv[0, 0, 1:], want[1:], bound[1:])


def test_gated_scan_sums(cla):
    """dlam, whose terms come from more than 2^31 elements, and dh0: resets every 1024 tokens make the documents
    independent, so that the 64-bit form takes four channels of them as a batch."""
    T, D, n, C = (1 << 20) + 77, 2048, 1024, 4
    x, r, i, dh = rnd(1, 1, T, D), rnd(2, 1, T, D, std=1.5), rnd(3, 1, T, D, std=1.5), rnd(4, 1, T, D)
    lam = torch.linspace(-8, 0, D, device="cuda").roll(D // 2 - 2)
    h0 = torch.ones(1, D, device="cuda")
    reset = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    reset[:, n::n] = True
    at = D // 2 - 4  # channels at the ends and the middle of lam's range
    _, _, _, dlam, dh0 = cla.gated_scan_bwd(x, r, i, lam, h0, dh, reset=reset)
    docs = (T + n - 1) // n

    def cut(v):
        v = torch.nn.functional.pad(v[0, :, at:at + C], (0, 0, 0, docs * n - T))
        return v.reshape(docs, n, C).contiguous()

    first = torch.zeros(docs, n, dtype=torch.bool)
    first[1:, 0] = True
    h = torch.zeros(docs, C)
    h[0] = 1.0
    lens = torch.full((docs,), n)
    lens[-1] = T - (docs - 1) * n
    ref = R.gated(cut(x), cut(r), cut(i), lam[at:at + C], h, first, lens, dh=cut(dh))
    R.assert_within("dlam", dlam[at:at + C], *ref["dlam"])
    R.assert_within("dh0", dh0[0, at:at + C], ref["dh0"][0][0], ref["dh0"][1][0])
