"""Plain 64-bit forms of the gated scan and of window attention, with error bounds.

Every bound is a running one: u is half a step of fp32 (2^-24), ut half a step of the tensors' type
(torch.finfo(t).eps / 2), and each value's bound adds, with absolute values in the place of signed terms, what
each rounding on the way to it can contribute.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_within(name, x, r, bound):
    x, r, bound = x.detach().double().cpu(), r.double().cpu(), bound.double().cpu()
    assert x.shape == r.shape, (name, x.shape, r.shape)
    if r.numel() == 0:
        return
    same = x == r  # equal infinities
    assert bool((torch.isfinite(x) | same).all()), f"{name}: non-finite values"
    over = torch.where(same, -1.0, (x - r).abs() - bound)
    i = int(over.argmax())
    assert float(over.max()) <= 0, (
        f"{name}[{i}]: {x.reshape(-1)[i].item()} against {r.reshape(-1)[i].item()}, "
        f"allowed {bound.expand_as(r).reshape(-1)[i].item():.3e}, "
        f"worst ratio {float(((x - r).abs() / bound.clamp(min=1e-300))[~same].max()):.3g}")


# ------------------------------------------------------------------ gated scan
def gated(x, rg, ig, lam, h0=None, reset=None, lens=None, c=8.0, dh=None, dhT=None):
    """{name: (value, bound)} in 64 bits.  Bounds, in units of u:
    a sigmoid: its exponential's argument is rounded (|g|), the exponential (2), sum, reciprocal and products (6);
    L: the gate's, softplus (4), two products: |rg| + 16;  a = e^L: |L| times L's, and 3 for the power;
    1 - a: L's (|L| a / (1 - a) <= 1) and 4;  m: half of that and of 1 + a's, and 3 for the root."""
    dt = x.dtype
    x, rg, ig, lam = (v.double().cpu() for v in (x, rg, ig, lam))
    B, T, D = x.shape
    z = torch.zeros(B, D, dtype=torch.float64)
    h0 = z if h0 is None else h0.double().cpu()
    live = torch.ones(B, T, 1, dtype=torch.bool)
    if lens is not None:
        live = (torch.arange(T)[None] < lens.cpu().clamp(0, T)[:, None])[..., None]
    rs = torch.zeros(B, T, 1, dtype=torch.bool) if reset is None else reset.cpu().bool()[..., None]
    x, rg, ig = (torch.where(live, v, 0.0) for v in (x, rg, ig))
    sp = torch.where(lam > 0, lam, 0.0) + torch.log1p(torch.exp(-lam.abs()))
    r, i = torch.sigmoid(rg), torch.sigmoid(ig)
    L = -c * sp * r
    a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
    kL = rg.abs() + 16
    ki = ig.abs() + 8
    ka = L.abs() * kL + 3
    km = (kL + 8) / 2 + 3
    a_, m_ = torch.where(rs, 0.0, a), torch.where(rs, 1.0, m)
    a_ = torch.where(live, a_, 1.0)
    w = i * x
    b = torch.where(live, m_ * w, 0.0)
    kb = km + ki + 3
    hs, Hs, Es = [h0], [h0.abs()], [z]
    for t in range(T):
        h = torch.where(a_[:, t] == 0, 0.0, a_[:, t] * hs[-1]) + b[:, t]
        H = a_[:, t] * Hs[-1] + b[:, t].abs()
        E = a_[:, t] * Es[-1] + U * ((ka[:, t] + 4) * a_[:, t] * Hs[-1] + (kb[:, t] + 2) * b[:, t].abs())
        E = torch.where(live[:, t], E, Es[-1])
        hs.append(h), Hs.append(H), Es.append(E)
    none = [torch.empty(B, 0, D, dtype=torch.float64)]
    h, E = (torch.cat([v[:, None] for v in s[1:]] + none, 1) for s in (hs, Es))
    ut = half_step(dt)
    zero = torch.zeros((), dtype=torch.float64)
    # what lies below the type's smallest normal is rounded to its smallest step
    tiny = torch.finfo(dt).smallest_normal * 2 * ut
    val = {"h": (torch.where(live, h, 0.0), torch.where(live, ut * h.abs() + 1.01 * E + tiny, zero)),
           "hT": (hs[-1], Es[-1] + 1e-38)}
    if dh is None:
        return val
    g = torch.where(live, dh.double().cpu(), 0.0)
    carry = z if dhT is None else dhT.double().cpu()
    cabs, cerr = carry.abs(), z
    hb, Hb, Eb = (torch.empty(B, T, D, dtype=torch.float64) for _ in range(3))
    for t in range(T - 1, -1, -1):
        hb[:, t], Hb[:, t], Eb[:, t] = g[:, t] + carry, g[:, t].abs() + cabs, cerr + U * (g[:, t].abs() + cabs)
        at = a_[:, t]
        k = torch.where(live[:, t], ka[:, t] + 4, 0.0)
        carry, cabs, cerr = at * hb[:, t], at * Hb[:, t], at * (Eb[:, t] + U * k * Hb[:, t])
    before, Eh = (torch.cat([v[:, None] for v in s[:-1]] + none, 1) for s in (hs, Es))
    Lm = torch.where(m > 0, L / m, 0.0)
    p1 = torch.where(rs, 0.0, before * a * L)
    p2 = torch.where(rs, 0.0, a * a * Lm * w)
    G = hb * (p1 - p2)
    EG = Eb * (p1.abs() + p2.abs()) + hb.abs() * (torch.where(rs, 0.0, Eh * a * L.abs())
                                                  + U * ((ka + kL + 6) * p1.abs() + (2 * ka + kL + km + ki + 8) * p2.abs()))
    E1 = Eb + U * 3 * Hb

    def put(name, v, e):
        v = torch.where(live, v, 0.0)
        val[name] = (v, torch.where(live, ut * v.abs() + 1.01 * e + tiny, zero))

    put("dx", hb * m_ * i, E1 * m_ * i + U * (km + ki + 3) * (hb * m_ * i).abs())
    put("digate", hb * m_ * w * (1 - i), E1 * m_ * w.abs() * (1 - i) + U * (km + 2 * ki + 5) * (hb * m_ * w).abs() * (1 - i))
    put("drgate", G * (1 - r), EG * (1 - r) + U * (kL + 3) * (G * (1 - r)).abs())
    slope = torch.sigmoid(lam) / sp
    G, EG = torch.where(live, G, 0.0), torch.where(live, EG, 0.0)
    n = math.log2(max(2, B * T)) + 64  # partial sums of 64 terms, then few rows
    val["dlam"] = (G.sum((0, 1)) * slope, (EG.sum((0, 1)) + U * (n + 12) * G.abs().sum((0, 1))) * slope + 1e-38)
    val["dh0"] = (carry, cerr + U * 2 * cabs + 1e-38)
    return val


# ------------------------------------------------------------------ window attention
def visible(T, window, sinks):
    t, s = torch.arange(T)[:, None], torch.arange(T)[None]
    return (s <= t) & ((t - s < window) | (s < sinks))


def window(q, k, v, window, sinks, lens=None, scale=None, dO=None):
    """{name: (value, bound)} in 64 bits.  Bounds: a logit is a sum of d exact products in fp32, (d + 4) u of its
    absolute terms, which is what P is off by (twice with lse's); P, dS, o are rounded to the type before or after a
    product: ut of their absolute terms; delta is formed from the rounded o."""
    dt, ut = q.dtype, half_step(q.dtype)
    q, k, v = (x.double().cpu() for x in (q, k, v))
    B, H, T, d = q.shape
    K = k.shape[1]
    G = H // K
    scale = d ** -0.5 if scale is None else scale
    n = torch.full((B,), T) if lens is None else lens.cpu().clamp(0, T).long()
    ok = torch.arange(T)[None] < n[:, None]  # [B, T]
    q = torch.where(ok[:, None, :, None], q, 0.0)
    k, v = (torch.where(ok[:, None, :, None], x, 0.0) for x in (k, v))
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    see = (visible(T, window, sinks)[None] & ok[:, :, None])[:, None]
    x = (q @ kk.transpose(2, 3) * scale).masked_fill(~see, -math.inf)
    xa = (q.abs() @ kk.abs().transpose(2, 3) * abs(scale)).masked_fill(~see, 0.0)
    lse = torch.logsumexp(x, 3) if T else torch.empty(B, H, 0, dtype=torch.float64)
    P = torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0)[..., None])
    top = xa.amax(3, keepdim=True) if T else xa
    eP = U * (2 * (d + 4) * (xa + top) + 2 * x.masked_fill(~see, 0.0).abs() + 32)  # relative
    o = P @ vv
    tiny = torch.finfo(dt).smallest_normal * 2 * ut
    # P itself may be rounded below the type's normal range (fp16): half its smallest step each
    Psub = see.double() * (tiny / 2)
    eo = (P * (1.01 * ut + eP) + Psub) @ vv.abs() + ut * o.abs() + tiny
    live = ok[:, None, :, None]
    zero = torch.zeros((), dtype=torch.float64)
    val = {"o": (o, torch.where(live, 1.01 * eo, zero)),
           "lse": (lse, torch.where(ok[:, None], (eP.amax(3) if T else lse * 0) + 4 * U * lse.abs().nan_to_num(posinf=0, neginf=0), zero))}
    if dO is None:
        return val
    g = torch.where(live, dO.double().cpu(), 0.0)
    delta = (g * o).sum(3, keepdim=True)
    edelta = (g.abs() * 1.01 * eo).sum(3, keepdim=True) + U * (d + 4) * (g.abs() * o.abs()).sum(3, keepdim=True)
    dP = g @ vv.transpose(2, 3)
    dPa = g.abs() @ vv.abs().transpose(2, 3)
    dS = P * (dP - delta)
    edS = dS.abs() * (1.01 * ut + eP) + P * (U * (d + 4) * dPa + edelta) * 1.01 + Psub * (1 + (dP - delta).abs())

    def heads(y):
        return y.view(B, K, G, T, d).sum(2)

    dq = dS @ kk * scale
    val["dq"] = (dq, torch.where(live, 1.01 * (edS @ kk.abs() * abs(scale) + ut * dq.abs() + tiny), zero))
    dk = heads(dS.transpose(2, 3) @ q * scale)
    val["dk"] = (dk, torch.where(live, 1.01 * (heads(edS.transpose(2, 3) @ q.abs() * abs(scale)) + ut * dk.abs() + tiny), zero))
    dv = heads(P.transpose(2, 3) @ g)
    val["dv"] = (dv, torch.where(live, 1.01 * (heads((P * (1.01 * ut + eP) + Psub).transpose(2, 3) @ g.abs()) + ut * dv.abs() + tiny), zero))
    return val


def slot(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


def window_step(q, k, v, kc, vc, pos, sinks, scale=None):
    """((o, bound), kcache, vcache) of one token; caches [B, Hkv, sinks + window, d]."""
    ut, (B, H, d), K, S = half_step(q.dtype), q.shape, k.shape[1], kc.shape[2]
    kc, vc = kc.cpu().clone(), vc.cpu().clone()
    o, e = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    scale = d ** -0.5 if scale is None else scale
    for b, p in enumerate(pos.tolist()):
        if p < 0:
            continue
        j = slot(p, S - sinks, sinks)
        kc[b, :, j], vc[b, :, j] = k[b].cpu(), v[b].cpu()
        m = min(p + 1, S)
        kk, vv = (c[b, :, :m].double().repeat_interleave(H // K, 0) for c in (kc, vc))
        qq = q[b].double().cpu()[:, None]
        x = (qq @ kk.transpose(1, 2))[:, 0] * scale
        xa = (qq.abs() @ kk.abs().transpose(1, 2))[:, 0] * abs(scale)
        P = torch.softmax(x, 1)
        eP = U * (2 * (d + 4) * (xa + xa.amax(1, keepdim=True)) + 32 + 4 * m ** 0.5)
        o[b] = (P[:, None] @ vv)[:, 0]
        e[b] = 1.01 * (((P * eP)[:, None] @ vv.abs())[:, 0] + ut * o[b].abs()) + torch.finfo(q.dtype).smallest_normal * 2 * ut
    return (o, e), kc, vc
