"""The gated scan against its 64-bit form: forward, backward and the one-token step."""
import pytest
import torch

from tests import _mixers as R

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import chunkwise_linear_attention_gb300 as m

    m.lib()
    return m


def inputs(B, T, D, dtype, seed=0, state=True):
    g = torch.Generator().manual_seed(seed)

    def rnd(*s, std=1.0, dt=dtype):
        return (torch.randn(*s, generator=g) * std).to(dt).cuda()

    a = torch.rand(D, generator=g) * 0.099 + 0.9
    t = dict(x=rnd(B, T, D), rgate=rnd(B, T, D, std=1.5), igate=rnd(B, T, D, std=1.5),
             lam=torch.log(torch.expm1(-torch.log(a) / 8)).cuda(), h0=rnd(B, D, dt=F32) if state else None)
    return t, rnd(B, T, D), rnd(B, D, dt=F32) if state else None


def check(cla, t, dh, dhT, reset=None, lens=None, c=8.0):
    B, T, D = t["x"].shape
    ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"], reset, lens, c, dh, dhT)
    kw = dict(reset=reset, lens=lens, c=c)
    args = (t["x"], t["rgate"], t["igate"], t["lam"], t["h0"])
    ck = cla.gated_scan_ckpt(t["x"])
    ws = torch.empty(max(256, cla.gated_scan_workspace_size(B, T, D)), dtype=torch.uint8, device="cuda")
    h, hT = cla.gated_scan_fwd(*args, ckpt=ck, workspace=ws, **kw)
    if B * D:
        cla.check_status(ws)
    got = dict(h=h, hT=hT)
    names = ("dx", "drgate", "digate", "dlam", "dh0")
    saved = cla.gated_scan_bwd(*args, dh, dhT, ckpt=ck, workspace=ws, **kw)
    if B * D:
        cla.check_status(ws)
    rebuilt = cla.gated_scan_bwd(*args, dh, dhT, **kw)
    for n, x, y in zip(names, saved, rebuilt):
        assert torch.equal(x, y), n
        got[n] = x
    for n, x in got.items():
        R.assert_within(n, x, *ref[n])
    # without a checkpoint the forward is the same, and so is a second run of all of it
    h2, hT2 = cla.gated_scan_fwd(*args, **kw)
    assert torch.equal(h, h2) and torch.equal(hT, hT2)
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 1, 64), (2, 2, 7), (1, 63, 64), (3, 64, 20), (2, 65, 128), (1, 128, 31),
                                   (2, 300, 96), (1, 1000, 40), (5, 129, 260), (1, 4100, 8)])
def test_sizes(cla, B, T, D, dtype):
    check(cla, *inputs(B, T, D, dtype))


@pytest.mark.parametrize("B,T,D", [(0, 5, 8), (2, 0, 8), (2, 5, 0)])
def test_nothing_to_do(cla, B, T, D):
    check(cla, *inputs(B, T, D, BF16))


def test_no_state(cla):
    check(cla, *inputs(2, 200, 48, F32, state=False))


@pytest.mark.parametrize("dtype,D", [(F32, 33), (BF16, 64), (F16, 10)])
def test_resets_and_lengths(cla, dtype, D):
    t, dh, dhT = inputs(4, 400, D, dtype)
    g = torch.Generator().manual_seed(5)
    reset = torch.rand(4, 400, generator=g) < 0.02
    reset[0, 0] = reset[1, 63] = reset[1, 64] = reset[2, 399] = True
    lens = torch.tensor([400, 0, 65, 1], dtype=torch.int32).cuda()
    check(cla, t, dh, dhT, reset.cuda(), lens)
    check(cla, t, dh, dhT, reset.to(torch.uint8).cuda())
    check(cla, t, dh, dhT, None, lens)


def test_lengths_are_clamped(cla):
    t, dh, dhT = inputs(3, 70, 16, F32)
    check(cla, t, dh, dhT, None, torch.tensor([-5, 1000, 70], dtype=torch.int32).cuda())


def test_extreme_gates(cla):
    """Gates from closed to open (to +-100 and infinite), decays from 1 to far below the smallest float."""
    t, dh, dhT = inputs(2, 150, 24, F32)
    g = torch.Generator().manual_seed(2)
    pick = torch.randint(0, 8, (2, 150, 24), generator=g).cuda()
    far = torch.tensor([-float("inf"), -100.0, -30.0, -5.0, 0.0, 30.0, 100.0, float("inf")], device="cuda")
    t["rgate"], t["igate"] = far[pick], far[(pick * 3 + 1) % 8]
    t["lam"] = torch.linspace(-40, 60, 24, device="cuda")
    ref = R.gated(t["x"], t["rgate"].clamp(-1e4, 1e4), t["igate"].clamp(-1e4, 1e4), t["lam"], t["h0"], None, None, 8.0, dh, dhT)
    args = (t["x"], t["rgate"], t["igate"], t["lam"], t["h0"])
    got = dict(zip(("h", "hT"), cla.gated_scan_fwd(*args)))
    got.update(zip(("dx", "drgate", "digate", "dlam", "dh0"), cla.gated_scan_bwd(*args, dh, dhT)))
    for n, x in got.items():
        # the error bounds of closed gates grow with |gate|: the values at +-100 are below 1e-30 of the others
        R.assert_within(n, x, ref[n][0], ref[n][1].clamp(max=2e-5 * float(ref[n][0].abs().max())) + 1e-5 * ref[n][0].abs() + 1e-12)


def test_nothing_passes_a_reset(cla):
    """NaN and infinity before a reset, or behind a length, reach nothing on its other side."""
    t, dh, dhT = inputs(2, 200, 16, F32)
    reset = torch.zeros(2, 200, dtype=torch.bool)
    reset[:, 100] = True
    lens = torch.tensor([200, 150], dtype=torch.int32).cuda()
    bad = {n: (v.clone() if v is not None else None) for n, v in t.items()}
    bad["x"][:, 40] = float("nan")
    bad["x"][:, 90, ::2] = float("inf")
    bad["rgate"][:, 70, 1::2] = float("nan")
    for n in ("x", "rgate", "igate"):
        bad[n][1, 150:] = float("nan")
    bdh = dh.clone()
    bdh[1, 150:] = float("nan")
    kw = dict(reset=reset.cuda(), lens=lens)
    names = ("x", "rgate", "igate", "lam", "h0")
    h, hT = cla.gated_scan_fwd(*(bad[n] for n in names), **kw)
    h1, hT1 = cla.gated_scan_fwd(*(t[n] for n in names), **kw)
    assert torch.equal(h[:, 100:], h1[:, 100:]) and torch.equal(hT, hT1)
    assert not torch.isfinite(h[:, 90:100]).all()
    g, g1 = (cla.gated_scan_bwd(*(s[n] for n in names), u, dhT, **kw) for s, u in ((bad, bdh), (t, dh)))
    for y, y1 in zip(g[:3], g1[:3]):
        assert torch.equal(y[:, 100:], y1[:, 100:])
    bdh = dh.clone()
    bdh[:, 120] = float("nan")  # and in the gradients' direction
    g = cla.gated_scan_bwd(*(t[n] for n in names), bdh, dhT, **kw)
    for y, y1 in zip(g[:3], g1[:3]):
        assert torch.equal(y[:, :100], y1[:, :100])
    assert torch.equal(g[4], g1[4])


def test_gradients_against_differences(cla):
    """Central differences of the forward in fp32: step e, error of the loss about 1e-6 of its terms."""
    t, dh, dhT = inputs(2, 70, 12, F32)
    names = ("x", "rgate", "igate", "lam", "h0")
    grads = dict(zip(("x", "rgate", "igate", "lam", "h0"), cla.gated_scan_bwd(*(t[n] for n in names), dh, dhT)))

    def loss(s):
        h, hT = cla.gated_scan_fwd(*(s[n] for n in names))
        return float((h.double() * dh.double()).sum() + (hT.double() * dhT.double()).sum())

    e = 1e-2
    for n in names:
        v = torch.randn(t[n].shape, generator=torch.Generator().manual_seed(7)).cuda()
        up, down = (dict(t, **{n: t[n] + s * e * v}) for s in (1, -1))
        num = (loss(up) - loss(down)) / (2 * e)
        ana = float((grads[n].double() * v.double()).sum())
        scale = float((grads[n].double() * v.double()).abs().sum())
        # third derivatives are of the order of the terms themselves: e^2 of them, and the rounding 1e-6 / e
        assert abs(num - ana) <= (2 * e * e + 1e-6 / e) * scale, (n, num, ana)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (8, 1024), (33, 100), (0, 8)])
def test_step(cla, B, D, dtype):
    t, _, _ = inputs(B, 1, D, dtype)
    reset = torch.arange(B) % 3 == 1
    for rs in (None, reset.cuda()):
        ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"], None if rs is None else rs[:, None])
        h = t["h0"].clone()
        y = cla.gated_scan_step(t["x"][:, 0], t["rgate"][:, 0], t["igate"][:, 0], t["lam"], h, reset=rs)
        R.assert_within("y", y, ref["h"][0][:, 0], ref["h"][1][:, 0])
        R.assert_within("h", h, *ref["hT"])


def test_step_at_odd_addresses(cla):
    """Rows that are not aligned for four elements at once; what lies around them stays as it was."""
    t, _, _ = inputs(5, 1, 64, BF16)
    ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"])

    def moved(v):
        buf = torch.full((v.numel() + 8,), 7.0, dtype=v.dtype, device="cuda")
        buf[1:1 + v.numel()] = v.reshape(-1)
        return buf, buf[1:1 + v.numel()].view(v.shape)

    (_, x), (_, r), (_, i) = (moved(t[n][:, 0].contiguous()) for n in ("x", "rgate", "igate"))
    (hb, h), (yb, y) = moved(t["h0"]), moved(torch.zeros_like(t["x"][:, 0]))
    assert cla.gated_scan_step(x, r, i, t["lam"], h, y=y) is y
    R.assert_within("y", y, ref["h"][0][:, 0], ref["h"][1][:, 0])
    R.assert_within("h", h, *ref["hT"])
    for buf, n in ((hb, h.numel()), (yb, y.numel())):
        assert float(buf[0]) == 7 and bool((buf[1 + n:] == 7).all())


def test_steps_continue_a_forward(cla):
    t, _, _ = inputs(3, 100, 64, BF16)
    ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"])
    _, h = cla.gated_scan_fwd(*(t[n][:, :90].contiguous() for n in ("x", "rgate", "igate")), t["lam"], t["h0"])
    for s in range(90, 100):
        y = cla.gated_scan_step(*(t[n][:, s].contiguous() for n in ("x", "rgate", "igate")), t["lam"], h)
        R.assert_within("y", y, ref["h"][0][:, s], ref["h"][1][:, s])
    R.assert_within("h", h, *ref["hT"])


def test_in_a_graph_and_on_a_stream(cla):
    """Captured once, replayed on new inputs; two captured graphs on workspaces of their own."""
    t, dh, dhT = inputs(2, 500, 64, BF16)
    names = ("x", "rgate", "igate", "lam", "h0")
    s = torch.cuda.Stream()
    static = {n: t[n].clone() for n in names}
    ws = [torch.empty(cla.gated_scan_workspace_size(2, 500, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ck = cla.gated_scan_ckpt(static["x"])
        cla.gated_scan_fwd(*static.values(), ckpt=ck, workspace=ws[0])
        cla.gated_scan_bwd(*static.values(), dh, dhT, ckpt=ck, workspace=ws[1])
    s.synchronize()
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            if k == 0:
                outs.append(cla.gated_scan_fwd(*static.values(), ckpt=ck, workspace=ws[0]))
            else:
                outs.append(cla.gated_scan_bwd(*static.values(), dh, dhT, ckpt=ck, workspace=ws[1]))
        graphs.append(g)
    for seed in (11, 12):
        t2, _, _ = inputs(2, 500, 64, BF16, seed)
        for n in names:
            static[n].copy_(t2[n])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = cla.gated_scan_fwd(*(t2[n] for n in names)) + cla.gated_scan_bwd(*(t2[n] for n in names), dh, dhT)
        for x, y in zip(outs[0] + outs[1], want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_only_a_reset_drops_what_is_not_finite(cla, dtype):
    """Decays whose product underflows carry a NaN or an infinity on, with a reset mask as without one, as far as the next
    reset and no further; in the gradients' direction too."""
    t, dh, dhT = inputs(2, 700, 16, dtype)
    t["lam"] = torch.zeros(16, device="cuda")  # open gates leave e^-5.5 a step: 20 steps are below the smallest float
    t["rgate"] = t["rgate"] + 2
    names = ("x", "rgate", "igate", "lam", "h0")
    reset = torch.zeros(2, 700, dtype=torch.bool)
    reset[0, 500] = True
    bad = dict(t, x=t["x"].clone())
    bad["x"][:, 5, ::2], bad["x"][:, 5, 1::2] = float("nan"), float("inf")
    good = cla.gated_scan_fwd(*(t[n] for n in names), reset=reset.cuda())
    h, hT = cla.gated_scan_fwd(*(bad[n] for n in names), reset=reset.cuda())
    assert not torch.isfinite(h[0, 5:500]).any() and not torch.isfinite(h[1, 5:]).any() and not torch.isfinite(hT[1]).any()
    assert torch.equal(h[0, 500:], good[0][0, 500:]) and torch.equal(hT[0], good[1][0]) and torch.equal(h[:, :5], good[0][:, :5])
    bdh = dh.clone()
    bdh[:, 690, ::2], bdh[:, 690, 1::2] = float("nan"), float("inf")
    want = cla.gated_scan_bwd(*(t[n] for n in names), dh, dhT, reset=reset.cuda())
    got = cla.gated_scan_bwd(*(t[n] for n in names), bdh, dhT, reset=reset.cuda())
    assert not torch.isfinite(got[0][0, 500:691]).any() and not torch.isfinite(got[0][1, :691]).any()
    assert not torch.isfinite(got[4][1]).any() and torch.equal(got[4][0], want[4][0])
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x[0, :500], y[0, :500]) and torch.equal(x[:, 691:], y[:, 691:])


@pytest.mark.parametrize("B,D", [(97, 40), (120, 33), (128, 64), (306, 5120), (700, 5120), (300, 3000)])
def test_rows_of_dlam(cla, B, D):
    """Every sequence of two steps leaves a row for dlam: up to 128 are added in one step, more in shares whose rows are
    taken 128 at a time (5120 channels: two shares, 153 and 350 rows; 3000: four, of 75)."""
    t, dh, dhT = inputs(B, 2, D, F32)
    ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"], None, None, 8.0, dh, dhT)
    got = cla.gated_scan_bwd(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"], dh, dhT)
    R.assert_within("dlam", got[3], *ref["dlam"])
    R.assert_within("dh0", got[4], *ref["dh0"])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("which", ["inputs", "outputs", "all"])
def test_odd_addresses(cla, dtype, off, which):
    """Rows of a multiple of four channels at addresses that are not one of four elements; what lies around the outputs
    stays as it was."""
    B, T, D = 2, 150, 36
    t, dh, dhT = inputs(B, T, D, dtype)
    bufs = []

    def moved(v, now):
        buf = torch.full((v.numel() + 16,), 7.0, dtype=v.dtype, device="cuda")
        at = off if now else 8
        view = buf[at:at + v.numel()].view(v.shape)
        view.copy_(v)
        bufs.append((buf, at, v.numel()))
        return view

    x, r, i, g = (moved(v, which != "outputs") for v in (t["x"], t["rgate"], t["igate"], dh))
    h, dx, dr, di = (moved(torch.zeros_like(t["x"]), which != "inputs") for _ in range(4))
    ck = cla.gated_scan_ckpt(x)
    reset = torch.zeros(B, T, dtype=torch.bool)
    reset[1, 70] = True
    for rs in (None, reset.cuda()):
        ref = R.gated(t["x"], t["rgate"], t["igate"], t["lam"], t["h0"], rs, None, 8.0, dh, dhT)
        _, hT = cla.gated_scan_fwd(x, r, i, t["lam"], t["h0"], reset=rs, h=h, ckpt=ck)
        _, _, _, dlam, dh0 = cla.gated_scan_bwd(x, r, i, t["lam"], t["h0"], g, dhT, reset=rs, dx=dx, drgate=dr, digate=di, ckpt=ck)
        for n, v in dict(h=h, hT=hT, dx=dx, drgate=dr, digate=di, dlam=dlam, dh0=dh0).items():
            R.assert_within(n, v, *ref[n])
        for buf, at, n in bufs:
            assert bool((buf[:at] == 7).all()) and bool((buf[at + n:] == 7).all())
