"""Refusals of the gated scan's and the window attention's entry points, and their size queries: on the host, without
a GPU; and the tests' own 64-bit gradients against automatic differentiation."""
import ctypes

import pytest
import torch

from tests import _mixers as R

P = ctypes.c_void_p
A, ODD, WS = P(1 << 20), P((1 << 20) + 2), P(1 << 21)
ODD1 = P((1 << 20) + 1)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from chunkwise_linear_attention_gb300 import build

    build.build()
    import chunkwise_linear_attention_gb300 as cla

    return cla.lib()


def gfwd(lib, x=A, lam=A, h0=None, h=A, c=8.0, dtype=1, B=2, T=100, D=64, ws=WS, n=BIG, ck=None, lens=None):
    return lib.cla_gated_scan_fwd(x, A, A, lam, h0, None, lens, h, None, ck, c, dtype, B, T, D, ws, n, None)


def gbwd(lib, dx=A, dh=A, lam=A, dtype=1, c=8.0, B=2, T=100, D=64, ws=WS, n=BIG, ck=None):
    return lib.cla_gated_scan_bwd(A, A, A, lam, None, None, None, ck, dh, None, dx, A, A, None, None, c, dtype, B, T, D, ws,
                                  n, None)


@pytest.mark.parametrize("call", [gfwd, gbwd])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(D=-1), 1), (dict(c=0.0), 1), (dict(c=-1.0), 1), (dict(c=float("nan")), 1),
    (dict(c=float("inf")), 1), (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(lam=None), 1), (dict(lam=ODD), 1),
    (dict(ck=ODD), 1), (dict(ws=None), 5), (dict(ws=ODD), 5), (dict(n=100), 5), (dict(B=1 << 20, D=1 << 20), 2),
    (dict(T=1 << 31), 2)])
def test_gated_scan_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.cla_last_error_message()


def test_gated_scan_pointers(lib):
    assert gfwd(lib, x=None) == 1 and gfwd(lib, h=None) == 1 and gfwd(lib, x=ODD1) == 1 and gfwd(lib, x=ODD, dtype=0) == 1
    assert gfwd(lib, h0=ODD) == 1 and gfwd(lib, lens=ODD) == 1 and gbwd(lib, dx=None) == 1 and gbwd(lib, dh=ODD1) == 1
    step = lambda h=A, y=A, dtype=1, B=2, D=8, c=8.0: lib.cla_gated_scan_step(A, A, A, A, None, h, y, c, dtype, B, D, None)
    assert step(h=None) == 1 and step(y=None) == 1 and step(h=ODD) == 1 and step(dtype=7) == 2 and step(B=-1) == 1
    assert step(c=0.0) == 1 and step(B=0) == 0


def test_gated_scan_sizes(lib):
    assert lib.cla_gated_scan_ckpt_elems(3, 129, 10) == 3 * 5 * 10
    assert lib.cla_gated_scan_ckpt_elems(3, 0, 10) == 0 and lib.cla_gated_scan_ckpt_elems(-1, 5, 5) == 0
    assert lib.cla_gated_scan_workspace_size(2, 100, 64) >= 256 and lib.cla_gated_scan_workspace_size(2, -1, 64) == 0


def _arr(s):
    return None if s is None else (ctypes.c_int64 * len(s))(*s)


def wfwd(lib, q=A, o=A, lse=A, lens=None, scale=0.1, window=16, sinks=2, dtype=1, B=2, H=4, K=2, T=100, d=64, strides=None,
         ws=WS, n=BIG):
    return lib.cla_window_attn_fwd(q, A, A, lens, o, lse, scale, window, sinks, dtype, B, H, K, T, d, _arr(strides), ws, n,
                                   None)


def wbwd(lib, q=A, o=A, lse=A, lens=None, scale=0.1, window=16, sinks=2, dtype=1, B=2, H=4, K=2, T=100, d=64, strides=None,
         ws=WS, n=BIG):
    s = None if strides is None else list(strides) + [H * T * d, T * d, d] * 4
    return lib.cla_window_attn_bwd(q, A, A, lens, o, lse, A, A, A, A, scale, window, sinks, dtype, B, H, K, T, d, _arr(s), ws,
                                   n, None)


def wstep(lib, q=A, o=A, lse=A, lens=A, scale=0.1, window=16, sinks=2, dtype=1, B=2, H=4, K=2, T=1, d=64, strides=None):
    s = None if strides is None else [x for i in range(3) for x in strides[3 * i:3 * i + 2]]
    return lib.cla_window_attn_step(q, A, A, lse, A, lens, o, scale, window, sinks, dtype, B, H, K, d, _arr(s), None)


COMMON = [(dict(B=-1), 1), (dict(H=-4), 1), (dict(K=-2), 1), (dict(H=5), 1), (dict(K=0), 1), (dict(window=0), 1),
          (dict(window=-3), 1), (dict(sinks=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
          (dict(dtype=0), 2), (dict(dtype=9), 2), (dict(d=32), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(q=None), 1),
          (dict(o=None), 1), (dict(lse=None), 1), (dict(q=ODD), 1), (dict(lens=ODD), 1), (dict(B=1 << 20, H=1 << 20), 2),
          (dict(strides=[64 * 400, 0, 64] * 4), 1), (dict(strides=[64 * 400, 65, 64] * 4), 1),
          (dict(strides=[-64, 64, 64] * 4), 1)]


@pytest.mark.parametrize("call,kw,status", [(c, kw, st) for c in (wfwd, wbwd, wstep) for kw, st in COMMON] + [
    (wfwd, dict(T=-1), 1), (wbwd, dict(T=-1), 1), (wfwd, dict(T=1 << 31), 2), (wfwd, dict(ws=None), 5), (wfwd, dict(n=255), 5), (wbwd, dict(ws=None), 5), (wbwd, dict(ws=ODD), 5),
    (wbwd, dict(n=64), 5), (wstep, dict(lens=None), 1),
    (wfwd, dict(strides=[64 * 400, 64 * 100, 0] * 4), 1), (wfwd, dict(strides=[64 * 400, 64 * 100, 4] * 4), 1),
    (wstep, dict(window=1 << 60), 2), (wstep, dict(sinks=1 << 60), 2)])
def test_window_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.cla_last_error_message()


@pytest.mark.parametrize("call", [wfwd, wbwd, wstep])
def test_window_heads_without_queries(lib, call):
    """Key heads that no query reads: their gradients and cache slots would be nobody's to write."""
    assert call(lib, H=0, K=2) == 1
    if call is wstep:  # the others' empty calls clear their workspace on the GPU
        assert call(lib, H=0, K=0) == 0


def test_window_sizes_at_the_limits(lib):
    # a tile more a head than B H T / 128 counts
    assert wfwd(lib, B=1 << 15, H=1 << 15, K=1, T=129) == 2 and wbwd(lib, B=1 << 15, H=1 << 15, K=1, T=129) == 2
    # a window or sinks longer than any sequence are every token
    assert lib.cla_window_attn_workspace_size(2, 4, 2, 100, 64, (1 << 63) - 1, (1 << 63) - 1) == 256
    assert (lib.cla_window_attn_bwd_workspace_size(2, 4, 2, 1000, 64, (1 << 63) - 1, 0)
            == lib.cla_window_attn_bwd_workspace_size(2, 4, 2, 1000, 64, 1000, 0))
    big = (1 << 63) - 1
    assert wstep(lib, B=0, window=big, sinks=big) == 2 and wstep(lib, window=(1 << 31) - 512, sinks=1) == 2
    assert lib.cla_window_cache_write(A, A, None, A, A, big, big, 1, 0, 1, 5, 64, None, None) == 2


def test_window_cache_refusals(lib):
    f = lambda k=A, kc=A, w=8, n=1, dtype=1, B=1, K=1, T=5, d=64, s=None: lib.cla_window_cache_write(
        k, A, None, kc, A, w, n, dtype, B, K, T, d, _arr(s), None)
    for kw, st in [(dict(k=None), 1), (dict(kc=None), 1), (dict(kc=ODD), 1), (dict(w=0), 1), (dict(n=-1), 1), (dict(dtype=0), 2),
                   (dict(d=80), 2), (dict(B=-1), 1), (dict(T=-1), 1), (dict(s=[64, 64, 0] * 2), 1), (dict(w=1 << 60), 2)]:
        assert f(**kw) == st, kw
    assert f(B=0) == 0 and f(T=0) == 0


def test_window_sizes(lib):
    assert lib.cla_window_attn_bwd_workspace_size(2, 4, 2, 100, 64, 16, 2) >= 256 + 2 * 4 * 100 * 4
    assert lib.cla_window_attn_workspace_size(2, 4, 2, 100, 64, 16, 2) == 256
    assert lib.cla_window_attn_workspace_size(2, 4, 2, 100, 65, 16, 2) == 0
    assert lib.cla_window_attn_bwd_workspace_size(2, 4, 3, 100, 64, 16, 2) == 0


def test_binding_refusals():
    import chunkwise_linear_attention_gb300 as cla

    x, lam = torch.zeros(2, 4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        cla.gated_scan_fwd(x, x, x, lam)
    with pytest.raises(ValueError, match="rgate must be"):
        cla.gated_scan_fwd(x, x.double(), x, lam)
    with pytest.raises(ValueError, match="lam must have shape"):
        cla.gated_scan_fwd(x, x, x, lam[:4])
    with pytest.raises(ValueError, match="reset must be"):
        cla.gated_scan_fwd(x, x, x, lam, reset=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="x must be one of"):
        cla.gated_scan_step(x[:, 0].double(), x[:, 0], x[:, 0], lam, x[:, 0])
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cla.window_attn_fwd(q, q, q, window=4)
    with pytest.raises(ValueError, match="q must be one of"):
        cla.window_attn_fwd(q.float(), q, q, window=4)
    with pytest.raises(ValueError, match="v must have shape"):
        cla.window_attn_fwd(q, q, q[:, :1], window=4)
    with pytest.raises(ValueError, match="kcache must have shape"):
        cla.window_attn_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], q, q, torch.zeros(1, dtype=torch.int32), window=4, sinks=1)


# ------------------------------------------------------------------ the 64-bit forms themselves
def test_gated_form_against_autograd():
    g = torch.Generator().manual_seed(0)
    B, T, D = 2, 30, 5
    x, rg, ig, dh = (torch.randn(B, T, D, generator=g, dtype=torch.float64) for _ in range(4))
    lam, h0, dhT = torch.randn(D, generator=g, dtype=torch.float64) - 4, torch.randn(B, D, generator=g, dtype=torch.float64), torch.randn(B, D, generator=g, dtype=torch.float64)
    reset = torch.rand(B, T, generator=g) < 0.1
    lens = torch.tensor([30, 21])
    leaves = [v.clone().requires_grad_() for v in (x, rg, ig, lam, h0)]
    xs, rs, is_, ls, s = leaves
    a = torch.exp(-8 * torch.nn.functional.softplus(ls) * torch.sigmoid(rs))
    m = torch.sqrt(1 - a * a)
    out = []
    for t in range(T):
        n = torch.where(reset[:, t, None], torch.sigmoid(is_[:, t]) * xs[:, t],
                        a[:, t] * s + m[:, t] * torch.sigmoid(is_[:, t]) * xs[:, t])
        on = (t < lens)[:, None]
        s = torch.where(on, n, s)
        out.append(torch.where(on, n, 0.0))
    h = torch.stack(out, 1)
    grads = torch.autograd.grad((h * dh).sum() + (s * dhT).sum(), leaves)
    ref = R.gated(x, rg, ig, lam, h0, reset, lens, 8.0, dh, dhT)
    for n, v in zip(("h", "hT", "dx", "drgate", "digate", "dlam", "dh0"), (h, s) + grads):
        torch.testing.assert_close(ref[n][0], v.detach(), rtol=1e-9, atol=1e-11)


def test_window_form_against_autograd():
    g = torch.Generator().manual_seed(0)
    B, H, K, T, d = 2, 4, 2, 40, 64
    q, dO = (torch.randn(B, H, T, d, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(B, K, T, d, generator=g, dtype=torch.float64) for _ in range(2))
    lens = torch.tensor([40, 17])
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out = []
    for b in range(B):
        n = int(lens[b])
        qq, kk, vv = (x[b, :, :n] for x in leaves)
        kk, vv = kk.repeat_interleave(2, 0), vv.repeat_interleave(2, 0)
        x = (qq @ kk.transpose(1, 2) / 8).masked_fill(~R.visible(n, 7, 2), -float("inf"))
        out.append(torch.nn.functional.pad(torch.softmax(x, 2) @ vv, (0, 0, 0, T - n)))
    o = torch.stack(out)
    grads = torch.autograd.grad((o * dO).sum(), leaves)
    ref = R.window(q, k, v, 7, 2, lens, None, dO)
    for n, x in zip(("o", "dq", "dk", "dv"), (o,) + grads):
        torch.testing.assert_close(ref[n][0], x.detach(), rtol=1e-9, atol=1e-11)


@pytest.mark.parametrize("window,sinks", [(2 ** 64 + 5, 0), (4.5, 0), (8, 2 ** 63), (8, 0.25), (-2 ** 63 - 1, 0)])
def test_binding_counts(lib, window, sinks):
    """Windows and sinks that 64 bits cannot hold, or that are not whole, are not cut to some other number."""
    import chunkwise_linear_attention_gb300 as cla

    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: cla.window_attn_workspace_size(1, 2, 2, 4, 64, window, sinks),
                 lambda: cla.window_attn_bwd_workspace_size(1, 2, 2, 4, 64, window, sinks),
                 lambda: cla.window_attn_fwd(q, q, q, window=window, sinks=sinks),
                 lambda: cla.window_cache_write(q, q, q, q, window=window, sinks=sinks),
                 lambda: cla.window_attn_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], q, q, torch.zeros(1, dtype=torch.int32),
                                              window=window, sinks=sinks)):
        with pytest.raises(ValueError, match="a whole number"):
            call()
    assert cla.window_attn_workspace_size(1, 2, 2, 4, 64, 8.0, 2 ** 63 - 1) == 256
