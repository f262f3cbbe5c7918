"""Refusals of the norm and rotation, the 8-bit window cache and the delta rule's steps, on the host; and the tests' own
64-bit forms against automatic differentiation, differences and the other forms of the same thing."""
import ctypes
import math

import pytest
import torch

from tests import _mixers as M
from tests import _serving as R

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


def _arr(s):
    return None if s is None else (ctypes.c_int64 * len(s))(*s)


def nfwd(lib, q=A, k=A, w=A, freq=A, pos=None, lens=None, qo=A, ko=A, eps=1e-6, rot=64, dtype=1, B=2, H=4, K=2, T=10, d=64, s=None):
    return lib.cla_qk_norm_rope_fwd(q, k, w, w, freq, pos, lens, qo, ko, eps, rot, 0, dtype, B, H, K, T, d, _arr(s), None)


def nbwd(lib, q=A, k=A, w=A, freq=A, pos=None, lens=None, qo=A, ko=A, eps=1e-6, rot=64, dtype=1, B=2, H=4, K=2, T=10, d=64, s=None,
         dw=A, ws=WS, n=BIG):
    s = None if s is None else list(s) + list(s[:6])
    return lib.cla_qk_norm_rope_bwd(q, k, w, w, freq, pos, lens, qo, ko, A, A, dw, dw, eps, rot, 0, dtype, B, H, K, T, d, _arr(s),
                                    ws, n, None)


@pytest.mark.parametrize("call", [nfwd, nbwd])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(H=-1), 1), (dict(K=-1), 1), (dict(T=-1), 1), (dict(d=-16), 1), (dict(rot=-16), 1), (dict(rot=80), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dtype=3), 2),
    (dict(dtype=-1), 2), (dict(d=0, rot=0), 2), (dict(d=72), 2), (dict(d=272), 2), (dict(rot=24), 2), (dict(q=None), 1),
    (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(freq=None), 1), (dict(q=ODD), 1), (dict(ko=ODD), 1),
    (dict(w=ODD), 1), (dict(freq=ODD), 1), (dict(pos=ODD), 1), (dict(lens=ODD), 1), (dict(B=1 << 20, T=1 << 20), 2),
    (dict(H=1 << 20), 2), (dict(B=1 << 16, T=1 << 14, H=1 << 10), 2), (dict(B=1 << 40, T=1 << 40, H=0, K=0), 2),
    (dict(s=[640, 64, 0] * 4), 1), (dict(s=[640, 64, -64] * 4), 1), (dict(s=[640, 68, 64] * 4), 1),
    (dict(s=[1 << 39, 64, 64] * 4), 1)])
def test_norm_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.cla_last_error_message()


def test_norm_workspace(lib):
    for kw, st in [(dict(ws=None), 5), (dict(ws=ODD), 5), (dict(n=100), 5), (dict(dw=ODD), 1)]:
        assert nbwd(lib, **kw) == st, kw
    assert lib.cla_qk_norm_rope_bwd_workspace_size(2, 4, 2, 10, 64) >= 256 + 2 * 64 * 4
    assert lib.cla_qk_norm_rope_bwd_workspace_size(2, 4, 2, 10, 65) == 0
    assert lib.cla_qk_norm_rope_bwd_workspace_size(-2, 4, 2, 10, 64) == 0
    assert nfwd(lib, B=0) == 0 and nfwd(lib, H=0, K=0) == 0 and nfwd(lib, T=0, q=None, k=None, qo=None, ko=None, freq=None) == 0


def cwrite(lib, q=A, kc=A, ks=A, lens=None, pos=None, o=None, scale=None, window=100, sinks=2, dtype=1, B=2, H=None, K=2, T=10, d=64,
           s=None):
    return lib.cla_window_cache8_write(q, A, lens, kc, A, ks, A, window, sinks, dtype, B, K, T, d, _arr(s), None)


def cstep(lib, q=A, kc=A, ks=A, lens=A, o=A, scale=0.1, window=100, sinks=2, dtype=1, B=2, H=4, K=2, T=1, d=64, s=None,
          ws=WS, nbytes=BIG):
    s = None if s is None else [x for x in s[:2]] * 3
    return lib.cla_window_attn_step8(q, A, A, kc, A, ks, A, lens, o, scale, window, sinks, dtype, B, H, K, d, _arr(s), ws, nbytes,
                                     None)


@pytest.mark.parametrize("call", [cwrite, cstep])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(K=-2), 1), (dict(window=0), 1), (dict(sinks=-1), 1), (dict(dtype=0), 2), (dict(dtype=9), 2),
    (dict(d=32), 2), (dict(d=256), 2), (dict(q=None), 1), (dict(kc=None), 1), (dict(ks=None), 1), (dict(q=ODD), 1),
    (dict(kc=ODD), 1), (dict(ks=ODD), 1), (dict(lens=ODD), 1), (dict(window=1 << 60), 2), (dict(sinks=1 << 60), 2),
    (dict(window=(1 << 31) - 512, sinks=1), 2), (dict(B=1 << 20, K=1 << 10, H=1 << 10), 2), (dict(s=[640, 68, 64] * 2), 1),
    (dict(s=[640, -64, 64] * 2), 1), (dict(B=1 << 12, window=1 << 26, sinks=0), 2)])
def test_cache8_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status
    assert lib.cla_last_error_message()


def test_cache8_calls(lib):
    for kw in (dict(H=5), dict(H=0), dict(K=0), dict(H=-4), dict(scale=float("nan")), dict(scale=float("inf")), dict(o=None),
               dict(lens=None), dict(o=ODD)):
        assert cstep(lib, **kw) == 1, kw
    assert cstep(lib, ws=None) == 5 and cstep(lib, ws=ODD) == 5 and cstep(lib, nbytes=1000) == 5
    assert cstep(lib, H=1 << 26, K=1) == 2 and cstep(lib, H=1 << 16, K=1) == 2
    assert lib.cla_window_attn_step8_workspace_size(2, 4, 2, 64, 100, 2) > 256 + 8 * 2 * 66 * 4
    assert lib.cla_window_attn_step8_workspace_size(0, 0, 0, 64, 100, 2) >= 256
    assert lib.cla_window_attn_step8_workspace_size(2, 4, 3, 64, 100, 2) == 0
    assert cwrite(lib, T=-1) == 1 and cwrite(lib, T=1 << 31) == 2
    assert cwrite(lib, B=0) == 0 and cwrite(lib, T=0) == 0 and cstep(lib, B=0, ws=None) == 5


def dstep(lib, q=A, v=A, ld=A, beta=A, lens=None, S=A, o=A, dtype=1, B=2, H=4, Hk=2, T=3, dk=64, dv=64, s=None):
    return lib.cla_delta_step(q, A, v, ld, beta, lens, S, o, dtype, B, H, Hk, T, dk, dv, _arr(s), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(H=-4), 1), (dict(Hk=-1), 1), (dict(T=-1), 1), (dict(dk=-64), 1), (dict(dv=-4), 1), (dict(H=5), 1),
    (dict(H=0), 1), (dict(Hk=0), 1), (dict(dtype=3), 2), (dict(dk=32), 2), (dict(dk=256), 2), (dict(dv=66), 2), (dict(dv=0), 2),
    (dict(q=None), 1), (dict(v=None), 1), (dict(ld=None), 1), (dict(beta=None), 1), (dict(S=None), 1), (dict(o=None), 1),
    (dict(q=ODD1), 1), (dict(q=ODD, dtype=0), 1), (dict(ld=ODD), 1), (dict(lens=ODD), 1), (dict(S=ODD), 1), (dict(o=ODD), 1),
    (dict(B=1 << 20, H=1 << 12, Hk=1), 2), (dict(T=1 << 31), 2), (dict(T=65537), 2), (dict(dv=1 << 40), 2), (dict(s=[64, 64, 0] * 5), 1),
    (dict(s=[64, -1, 64] * 5), 1)])
def test_delta_step_refusals(lib, kw, status):
    assert dstep(lib, **kw) == status
    assert lib.cla_last_error_message()


def test_delta_step_nothing(lib):
    assert dstep(lib, B=0) == 0 and dstep(lib, T=0, S=None, o=None) == 0 and dstep(lib, H=0, Hk=0) == 0


def test_binding_refusals(lib):
    import chunkwise_linear_attention_gb300 as cla

    bf = torch.bfloat16
    q, k, w, f = torch.zeros(1, 4, 8, 64, dtype=bf), torch.zeros(1, 2, 8, 64, dtype=bf), torch.ones(64), torch.ones(32)
    kc, vc, ks, vs = cla.window_cache8(1, 2, 64, window=100, sinks=4, device="cpu")
    assert kc.dtype == torch.float8_e4m3fn and kc.shape == (1, 2, 104, 64) and ks.shape == (1, 2, 2)
    pos = torch.zeros(1, dtype=torch.int32)

    def raises(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    raises("CUDA", cla.qk_norm_rope_fwd, q, k, w, w, f)
    raises("wk must have shape", cla.qk_norm_rope_fwd, q, k, w, w[:32], f)
    raises("k must be torch.bfloat16", cla.qk_norm_rope_fwd, q, k.float(), w, w, f)
    raises("q must be one of", cla.qk_norm_rope_fwd, q.double(), k, w, w, f)
    raises("freq must be torch.float32", cla.qk_norm_rope_fwd, q, k, w, w, f.double())
    raises("freq must have 1 dim", cla.qk_norm_rope_fwd, q, k, w, w, f[None])
    raises("pos must have shape", cla.qk_norm_rope_fwd, q, k, w, w, f, pos=torch.zeros(8, dtype=torch.int32))
    raises("qo must have shape", cla.qk_norm_rope_fwd, q, k, w, w, f, qo=k)
    raises("q must have 3 dim", cla.qk_norm_rope_step, q, k[:, :, 0], w, w, f, pos)
    raises("CUDA", cla.qk_norm_rope_step, q[:, :, 0], k[:, :, 0], w, w, f, pos)
    raises("pos must have shape", cla.qk_norm_rope_step, q[:, :, 0], k[:, :, 0], w, w, f, pos.repeat(2))
    raises("dko must have shape", cla.qk_norm_rope_bwd, q, k, w, w, f, q, q)
    raises("dwq must be torch.float32", cla.qk_norm_rope_bwd, q, k, w, w, f, q, k, dwq=w.double())
    raises("CUDA", cla.window_cache8_write, k, k, kc, vc, ks, vs, window=100, sinks=4)
    raises("kcache must be torch.float8_e4m3fn", cla.window_cache8_write, k, k, kc.view(torch.uint8), vc, ks, vs, window=100, sinks=4)
    raises("kcache must have shape", cla.window_cache8_write, k, k, kc, vc, ks, vs, window=99, sinks=4)
    raises("vscale must have shape", cla.window_cache8_write, k, k, kc, vc, ks, vs[:, :, :1], window=100, sinks=4)
    one = (q[:, :, 0], k[:, :, 0], k[:, :, 0])
    raises("CUDA", cla.window_attn_step8, *one, kc, vc, ks, vs, pos, window=100, sinks=4)
    raises("kscale must be torch.float32", cla.window_attn_step8, *one, kc, vc, ks.double(), vs, pos, window=100, sinks=4)
    raises("a whole number", cla.window_attn_step8, *one, kc, vc, ks, vs, pos, window=100.5, sinks=4)
    raises("a whole number", cla.window_cache8, 1, 2, 64, window=2 ** 64)
    g, S = torch.zeros(1, 4, 8), torch.zeros(1, 4, 64, 64)
    v = torch.zeros(1, 4, 8, 64, dtype=bf)
    raises("CUDA", cla.delta_step, k, k, v, g, g, S)
    raises("S must have shape", cla.delta_step, k, k, v, g, g, S[:, :2])
    raises("S must be torch.float32", cla.delta_step, k, k, v, g, g, S.to(bf))
    raises("beta must have shape", cla.delta_step, k, k, v, g, g[:, :2], S)
    raises("v must be torch.bfloat16", cla.delta_step, k, k, v.float(), g, g, S)
    raises("k must have shape", cla.delta_step, k, q, v, g, g, S)


# ------------------------------------------------------------------ the 64-bit forms themselves
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_form_against_autograd_and_differences(interleaved):
    g = torch.Generator().manual_seed(0)
    B, h, T, d, rot = 2, 3, 5, 32, 16
    x, up = (torch.randn(B, h, T, d, generator=g, dtype=torch.float64) for _ in range(2))
    w, freq = torch.randn(d, generator=g, dtype=torch.float64), torch.rand(rot // 2, generator=g).float()
    pos = torch.randint(-50, 50, (B, T), generator=g, dtype=torch.int32)
    lens = torch.tensor([5, 3])

    def f(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-3).sqrt() * w
        ang = pos[:, None, :, None].double() * freq.double()
        out = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = torch.cos(ang[..., i]), torch.sin(ang[..., i])
            out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        return out * (torch.arange(T) < lens[:, None])[:, None, :, None]

    leaves = [v.clone().requires_grad_() for v in (x, w)]
    y = f(*leaves)
    gx, gw = torch.autograd.grad(y, leaves, up)
    ref = R.norm_rope(x, w, freq, pos, lens, 1e-3, interleaved, up)
    for n, v in (("o", y.detach()), ("dx", gx), ("dw", gw)):
        torch.testing.assert_close(ref[n][0], v, rtol=1e-10, atol=1e-12)
    step = torch.randn(x.shape, generator=g, dtype=torch.float64)
    num = float(((f(x + 1e-5 * step, w) - f(x - 1e-5 * step, w)) * up).sum()) / 2e-5
    assert abs(num - float((ref["dx"][0] * step).sum())) <= 1e-7 * max(1.0, abs(num))


def test_angles_of_whole_numbers():
    for pos, f in ((0, 1.0), (1, 0.5), (-7, 0.25), (1000, 0.625), (12345, 1.0), (3, -2.0)):
        c, s = R.angle_exact(pos, f)
        assert abs(c - math.cos(pos * f)) < 1e-11 and abs(s - math.sin(pos * f)) < 1e-11, (pos, f)


def test_rounding_is_the_types():
    """The grid's rounding against torch's conversion, over every fp16 number up to 448."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.float().to(torch.float8_e4m3fn).double()
    assert torch.equal(R.rounded(x.double()), want)
    for top, e in ((0.0, -64), (448.0, 0), (448.5, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7501, -7), (2.0 ** -80, -64)):
        assert R.factor(torch.tensor([top, -top / 3])) == 2.0 ** e


def test_delta_form_against_the_oracle():
    import numpy as np
    import oracle

    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(2, 2, 7, 8, generator=g, dtype=torch.float64) for _ in range(3))
    ld, be = -torch.rand(2, 2, 7, generator=g, dtype=torch.float64), torch.rand(2, 2, 7, generator=g, dtype=torch.float64)
    S = torch.randn(2, 2, 8, 8, generator=g, dtype=torch.float64)
    (o, _), (ST, _) = R.delta(q, k, v, ld, be, S)
    ro, rS = oracle.delta_fwd(*(x.numpy() for x in (q, k, v, ld, be, S)))
    np.testing.assert_allclose(o.numpy(), ro, rtol=0, atol=1e-12)
    np.testing.assert_allclose(ST.numpy(), rS, rtol=0, atol=1e-12)


def test_cache8_forms_agree():
    """Tokens put one by one hold what the prompt's write holds, where blocks only fill up and nothing is subnormal."""
    g = torch.Generator().manual_seed(1)
    k = torch.randn(1, 2, 60, 64, generator=g).half()
    k = torch.where(k.abs() < 0.25, k.sign() * 0.25 + 0.25 * (k == 0), k)  # no number is rounded twice to different steps
    kc, ks = torch.zeros(1, 2, 104, 64, dtype=torch.float64), torch.zeros(1, 2, 2, dtype=torch.float64)
    want = R.cache8_write(k, kc, ks, None, 100, 4)
    for p in range(60):
        kc, ks = R.cache8_put(k[:, :, p], kc, ks, torch.tensor([p]), 100, 4)
    assert torch.equal(kc, want[0]) and torch.equal(ks, want[1])
    q = torch.randn(1, 4, 64, generator=g).half()
    o, _ = R.step8(q, kc, ks, kc, ks, torch.tensor([59]))
    held = (kc * ks.repeat_interleave(64, 2)[:, :, :104, None])[:, :, :60].repeat_interleave(2, 1)
    x = torch.einsum("bhd,bhsd->bhs", q.double(), held) / 8
    torch.testing.assert_close(o, torch.einsum("bhs,bhsd->bhd", torch.softmax(x, 2), held), rtol=1e-10, atol=1e-12)
    assert M.slot(103, 100, 4) == 103 and M.slot(104, 100, 4) == 4
