"""Plain 64-bit forms of the norm and rotation of queries and keys, of the 8-bit window cache and of the delta rule token
by token, with error bounds.

As in tests/_mixers.py, every bound is a running one: U is half a step of fp32, half_step(t) of the tensors' type, and each
value's bound adds, with absolute values in the place of signed terms, what each rounding on the way to it can contribute.
"""
import math
from fractions import Fraction

import torch

from tests._mixers import U, half_step, slot

BLOCK = 64


def _tiny(dtype):
    """What a rounding below the type's normal range can be off by, and the smallest fp32 normal."""
    return torch.finfo(dtype).smallest_normal * 2 * half_step(dtype) + 1e-37


# ------------------------------------------------------------------ norm and rotation
def _pairs(y, rot, interleaved):
    return (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])


def _turned(y, cos, sin, rot, interleaved):
    if not rot:
        return y
    a, b = _pairs(y, rot, interleaved)
    a, b = a * cos - b * sin, b * cos + a * sin
    front = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((front, y[..., rot:]), -1)


def _pair_sum(y, rot, interleaved):
    """|a| + |b| at both places of each pair, |y| elsewhere."""
    if not rot:
        return y.abs()
    a, b = (v.abs() for v in _pairs(y, rot, interleaved))
    front = torch.stack((a + b, a + b), -1).flatten(-2) if interleaved else torch.cat((a + b, a + b), -1)
    return torch.cat((front, y[..., rot:].abs()), -1)


def norm_rope(x, w=None, freq=None, pos=None, lens=None, eps=1e-6, interleaved=False, g=None):
    """{name: (value, bound)} of one of q and k, [B, heads, T, d].  Bounds, in units of U: a sum of d squares, 16 in a lane and
    4 rounds of shuffles: 22, half of it in r, with the mean's product, eps, and 4 for the reciprocal root: 17; r, x and w's
    products: 20.  A sine or cosine: the angle's 24 bits in half turns, pi / 2, 2^-31 of a turn, and 2 of its own: 5; the
    turn adds 3 of its terms."""
    dt, ut, tiny = x.dtype, half_step(x.dtype), _tiny(x.dtype)
    x = x.double().cpu()
    B, h, T, d = x.shape
    live = torch.ones(B, 1, T, 1, dtype=torch.bool)
    if lens is not None:
        live = (torch.arange(T)[None] < lens.cpu()[:, None])[:, None, :, None]
    x = torch.where(live, x, 0.0)
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double().cpu()
    rot = 0 if freq is None else 2 * freq.numel()
    cos = sin = None
    if rot:
        p = torch.arange(T).expand(B, T) if pos is None else pos.cpu().view(B, T)
        angle = p.double()[:, None, :, None] * freq.double().cpu()
        cos, sin = torch.cos(angle), torch.sin(angle)
    r = 1 / torch.sqrt(x.square().mean(3, keepdim=True) + eps)
    n = x * r
    zero = torch.zeros((), dtype=torch.float64)

    def kept(v, e):
        return torch.where(live, v, 0.0), torch.where(live, 1.01 * e + ut * v.abs() + tiny, zero)

    y = n * w
    val = {"o": kept(_turned(y, cos, sin, rot, interleaved), U * 28 * _pair_sum(y, rot, interleaved))}
    if g is None:
        return val
    g = torch.where(live, g.double().cpu(), 0.0)
    eg = U * 8 * _pair_sum(g, rot, interleaved)
    g = _turned(g, cos, -sin if rot else None, rot, interleaved)
    gw, egw = g * w, eg * w.abs() + U * (g * w).abs()
    m = (gw * n).mean(3, keepdim=True)
    em = (egw * n.abs()).mean(3, keepdim=True) + U * (22 + 40) * (gw * n).abs().mean(3, keepdim=True)
    dx = r * (gw - n * m)
    val["dx"] = kept(dx, r * (egw + n.abs() * em + U * 24 * (gw.abs() + (n * m).abs())))
    terms = g * n
    # rows are added one after the other in a lane, then over lanes, warps and blocks
    val["dw"] = (terms.sum((0, 1, 2)),
                 1.01 * ((eg * n.abs()).sum((0, 1, 2)) + U * (20 + B * h * T + 40) * terms.abs().sum((0, 1, 2))) + 1e-37)
    return val


PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)


def angle_exact(pos, freq):
    """(cos, sin) of pos freq, a whole number and a float of any size, from fractions."""
    angle = pos * Fraction(freq)
    x = float(angle - 2 * PI * round(angle / (2 * PI)))
    return math.cos(x), math.sin(x)


# ------------------------------------------------------------------ the cache in 8 bits
def _grid():
    return torch.tensor([math.ldexp(m + 8 * (e > 0), max(e, 1) - 10) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64)


GRID = _grid()


def rounded(x):
    """The e4m3 numbers nearest to x (64 bits, at most 448), the even one of two."""
    a = x.abs().contiguous()
    hi = torch.searchsorted(GRID, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - GRID[lo], GRID[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(GRID[pick], x)


def factor(x):
    """The factor of a block that holds x."""
    top = float(x.abs().max()) if x.numel() else 0.0
    e = -64
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def blocks(S):
    return -(-S // BLOCK)


def cache8_write(k, kc, ks, lens, window, sinks):
    """(kcache, kscale) in 64 bits after a prompt's keys (or values)."""
    kc, ks = kc.double().cpu().clone(), ks.double().cpu().clone()
    B, K, T, d = k.shape
    S = sinks + window
    for b in range(B):
        x, n = {}, T if lens is None else min(max(int(lens[b]), 0), T)
        for p in range(n):
            x[slot(p, window, sinks)] = p
        for i in range(blocks(S)):
            held = [j for j in range(i * BLOCK, min(S, (i + 1) * BLOCK)) if j in x]
            if not held:
                continue
            val = k[b, :, [x[j] for j in held]].double().cpu()
            for h in range(K):
                f = factor(val[h])
                ks[b, h, i], kc[b, h, held] = f, rounded(val[h] / f)
    return kc, ks


def cache8_put(x, kc, ks, pos, window, sinks):
    """(kcache, kscale) in 64 bits after one token's keys (or values) x [B, K, d]."""
    kc, ks = kc.double().cpu().clone(), ks.double().cpu().clone()
    S = sinks + window
    for b, p in enumerate(pos.tolist()):
        if p < 0:
            continue
        j = slot(p, window, sinks)
        i, n = j // BLOCK, min(p + 1, S)
        lo, hi = i * BLOCK, min((i + 1) * BLOCK, n)
        for h in range(kc.shape[1]):
            val = kc[b, h, lo:hi] * ks[b, h, i]
            val[j - lo] = x[b, h].double().cpu()
            f = factor(val)
            ks[b, h, i], kc[b, h, lo:hi] = f, rounded(val / f)
    return kc, ks


def step8(q, kc, ks, vc, vs, pos, scale=None):
    """(o, bound) of a step over caches that hold the token already (64 bits).  Bounds: queries are fp16 with their head's
    largest in [1, 2): 2^-24 of the largest each; a logit is a sum of d exact products in fp32; a weight with v's factor is
    rounded to fp16, by 2^-11 of itself or 2^-32 of the largest such; the logarithms and powers of two: 2^-21."""
    ut, (B, H, d), K, S = half_step(q.dtype), q.shape, kc.shape[1], kc.shape[2]
    G = H // K
    scale = d ** -0.5 if scale is None else scale
    o, e = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    for b, p in enumerate(pos.tolist()):
        if p < 0:
            continue
        m = min(p + 1, S)
        fk, fv = (f[b].repeat_interleave(BLOCK, 1)[:, :m].repeat_interleave(G, 0) for f in (ks, vs))
        ck, cv = (c[b, :, :m].repeat_interleave(G, 0) for c in (kc, vc))
        kk, vv = ck * fk[..., None], cv * fv[..., None]
        qq = q[b].double().cpu()
        x = (kk @ qq[..., None])[..., 0] * scale
        xa = (kk.abs() @ qq.abs()[..., None])[..., 0] * abs(scale)
        xq = kk.abs().sum(2) * qq.abs().amax(1, keepdim=True) * abs(scale) * 2.0 ** -24
        P = torch.softmax(x, 1)
        ex = U * ((d + 6) * xa + 2 * x.abs() + fv.log().abs() + 16) + xq
        eP = ex + ex.amax(1, keepdim=True) + U * (32 + 4 * m ** 0.5)
        o[b] = (P[:, None] @ vv)[:, 0]
        e[b] = 1.01 * (((P * (eP + 2.0 ** -11))[:, None] @ vv.abs())[:, 0] + ut * o[b].abs()
                       + 2.0 ** -32 * (P * fv).amax(1, keepdim=True) * cv.abs().sum(1)) + _tiny(q.dtype)
    return o, e


# ------------------------------------------------------------------ the delta rule
def delta(q, k, v, log_decay, beta, S, lens=None):
    """((o, bound), (S, bound)) in 64 bits.  Bounds, in units of U: a decay: 4; sums over dk rows, dk / 16 in a thread, two
    rounds of shuffles, four warps: dk / 16 + 8."""
    q, k, v, ld, beta, S = (x.double().cpu() for x in (q, k, v, log_decay, beta, S))
    B, H, T, dv = v.shape
    G = H // q.shape[1]
    q, k = (x.repeat_interleave(G, 1) for x in (q, k))
    n = q.shape[3] / 16 + 8
    E = torch.zeros_like(S)
    o, eo = torch.zeros(B, H, T, dv, dtype=torch.float64), torch.zeros(B, H, T, dv, dtype=torch.float64)
    live = torch.ones(B, T, dtype=torch.bool) if lens is None else torch.arange(T)[None] < lens.cpu()[:, None]
    for t in range(T):
        on = live[:, t, None, None, None]
        a, be = torch.exp(ld[:, :, t, None, None]), beta[:, :, t, None, None]
        kt, qt, vt = k[:, :, t, :, None], q[:, :, t, :, None], v[:, :, t, None]
        aS = torch.where(a == 0, 0.0, a * S)
        EA = torch.where(a == 0, 0.0, a * E + 5 * U * aS.abs())
        p, pa = (kt * aS).sum(2, keepdim=True), (kt * aS).abs().sum(2, keepdim=True)
        ep = (kt.abs() * EA).sum(2, keepdim=True) + n * U * pa
        u = be * (vt - p)
        eu = be.abs() * (ep + U * (vt.abs() + pa)) + 2 * U * u.abs()
        new = aS + kt * u
        En = EA + kt.abs() * eu + 2 * U * (aS.abs() + (kt * u).abs())
        qk = (qt * kt).sum(2, keepdim=True)
        eqk = n * U * (qt * kt).abs().sum(2, keepdim=True)
        y = (qt * aS).sum(2, keepdim=True)
        ot = y + qk * u
        et = ((qt.abs() * EA).sum(2, keepdim=True) + n * U * (qt * aS).abs().sum(2, keepdim=True) + qk.abs() * eu + eqk * u.abs()
              + 2 * U * (y.abs() + (qk * u).abs()))
        S, E = torch.where(on, new, S), torch.where(on, En, E)
        o[:, :, t], eo[:, :, t] = torch.where(on, ot, 0.0)[:, :, 0], torch.where(on, 1.01 * et + 1e-37, 0.0)[:, :, 0]
    return (o, eo), (S, 1.01 * E + 1e-37 * (E > 0))
