"""The gated scan and the sliding-window attention with sinks: their cases, plain forms and 64-bit values.

Gated scan, over [B, T, D]:  r = sigmoid(rgate), i = sigmoid(igate), L = -c softplus(lam) r, a = e^L,
m = sqrt(1 - a^2), h_t = a_t h_{t-1} + m_t i_t x_t.  A reset starts afresh (a = 0, m = 1); tokens behind a
sequence's length keep the state, and have output and gradients of zero.

Window attention, over [B, H, T, d] with shared key heads: token t sees s <= t with t - s < window or s < sinks.
Its cache holds sinks + window slots: token p in slot p (p < sinks), else in sinks + (p - sinks) % window.
"""
import math

import torch

own = False

C_GATE = 8.0
_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _g(name, op, B, T, D, dtype, reset=False, ragged=False):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "dtype": dtype, "reset": reset, "ragged": ragged}


def _w(name, op, B, H, Hkv, T, d, window, sinks, dtype, ragged=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "T": T, "d": d, "window": window, "sinks": sinks,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # serving, one token for a few sequences: a launch's latency
        _g("gated step 8x1024", "gated_step", 8, 1, 1024, "bf16"),
        # serving, one token for a full batch of a wide layer
        _g("gated step 512x4096", "gated_step", 512, 1, 4096, "bf16"),
        # serving, a long prompt from a state
        _g("gated prefill 1x65536x1024", "gated_prefill", 1, 65536, 1024, "bf16"),
        # training, the shape of the benchmark's diagonal scan
        _g("gated train 8x4096x1024", "gated_train", 8, 4096, 1024, "bf16"),
        # training in 32 bits: packed documents in a padded batch, odd sizes
        _g("gated train fp32 3x2531x777", "gated_train", 3, 2531, 777, "fp32", True, True),
        # serving, a long prompt, and the cache that the next tokens read
        _w("window prefill 32768", "window_prefill", 1, 32, 8, 32768, 128, 1024, 4, "bf16"),
        # serving, short padded prompts of odd sizes
        _w("window prefill 3x257", "window_prefill", 3, 8, 2, 257, 64, 100, 3, "fp16", True),
        # training, the shape of the benchmark's constant-decay attention
        _w("window train 4x16x8192 d64", "window_train", 4, 16, 16, 8192, 64, 512, 0, "bf16"),
        # training, shared key heads and a wide window
        _w("window train 2x16x8192 d128", "window_train", 2, 16, 4, 8192, 128, 2048, 16, "bf16"),
        # training, a padded batch of odd sizes
        _w("window train 2x6x1531 d64", "window_train", 2, 6, 3, 1531, 64, 300, 7, "fp16", True),
        # serving, one token for a few sequences, some of them shorter than the window
        _w("window step 4x16 w1024", "window_step", 4, 16, 4, 1, 128, 1024, 4, "bf16", True),
        # serving, one token for a full batch with a wide window
        _w("window step 64x32 w4096", "window_step", 64, 32, 8, 1, 128, 4096, 4, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_step", "gated_prefill", "gated_train", "window_prefill", "window_train", "window_step"])
    if op == "gated_step":
        return _unnamed(_g("", op, _log(rng, 1, 512), 1, _log(rng, 16, 4096), rng.choice(["bf16", "fp16", "fp32"]),
                           rng.random() < 0.3))
    if op.startswith("gated"):
        T, D = _log(rng, 1, 65536), _log(rng, 16, 4096)
        D = D if rng.random() < 0.4 else max(16, D // 64 * 64)
        B = _log(rng, 1, max(1, min(16, 33_000_000 // (T * D))))
        return _unnamed(_g("", op, B, min(T, 33_000_000 // D), D, rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                           rng.random() < 0.3, rng.random() < 0.3))
    Hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    H = Hkv * rng.choice([1, 2, 4])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    sinks = rng.choice([0, 1, 4, 16, rng.randint(1, 64)])
    if op == "window_step":
        window = _log(rng, 1, 4096)
        return _unnamed(_w("", op, _log(rng, 1, 64), H, Hkv, 1, d, window, sinks, dtype, rng.random() < 0.5))
    T = _log(rng, 1, 16384)
    window = _log(rng, 1, 2048)
    most = 2 * 16 * 8192 * 2048
    window = min(window, most // (H * T))
    B = _log(rng, 1, max(1, min(8, most // (H * T * max(64, min(window, T))))))
    return _unnamed(_w("", op, B, H, Hkv, T, d, window, sinks, dtype, rng.random() < 0.4))


def _unnamed(c):
    del c["name"]
    return c


def _lens(c):
    """Ragged batches: the first sequence full, the others shorter by even steps, down to almost nothing."""
    B, T = c["B"], c["T"]
    return [max(1, T - (T * b) // B) for b in range(B)]


def _pos(c):
    """Tokens before the step: every sequence beyond its window, or, ragged, spread from none at all."""
    B, S = c["B"], c["sinks"] + c["window"]
    return [(2 * S * b) // B if c["ragged"] else S + 37 * b for b in range(B)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _T[c["dtype"]]

    def rnd(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"].startswith("gated"):
        B, T, D = c["B"], c["T"], c["D"]
        shape = (B, D) if c["op"] == "gated_step" else (B, T, D)
        s["x"], s["rgate"], s["igate"] = rnd(*shape), rnd(*shape, std=1.5), rnd(*shape, std=1.5)
        # decays at an open gate between 0.9 and 0.999, as such layers are initialised
        a = torch.rand(D, generator=g, device="cuda") * 0.099 + 0.9
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / C_GATE))
        s["h0"] = rnd(B, D, dtype=torch.float32)
        s["reset"] = s["lens"] = None
        if c["reset"]:
            s["reset"] = torch.rand(shape[:-1], generator=g, device="cuda") < 1.0 / 200
        if c["ragged"]:
            s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        if c["op"] == "gated_train":
            s["dh"], s["dhT"] = rnd(*shape), rnd(B, D, dtype=torch.float32)
        return s
    B, H, Hkv, T, d = (c[n] for n in ("B", "H", "Hkv", "T", "d"))
    S = c["sinks"] + c["window"]
    if c["op"] == "window_step":
        s["q"], s["k"], s["v"] = rnd(B, H, d, std=1.5), rnd(B, Hkv, d), rnd(B, Hkv, d)
        s["kcache"], s["vcache"] = rnd(B, Hkv, S, d), rnd(B, Hkv, S, d)
        s["pos"] = torch.tensor(_pos(c), dtype=torch.int32, device="cuda")
        return s
    s["q"], s["k"], s["v"] = rnd(B, H, T, d, std=1.5), rnd(B, Hkv, T, d), rnd(B, Hkv, T, d)
    s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
    if c["op"] == "window_train":
        s["do"] = rnd(B, H, T, d)
    else:
        s["kcache"] = torch.zeros(B, Hkv, S, d, dtype=t, device="cuda")
        s["vcache"] = torch.zeros(B, Hkv, S, d, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import chunkwise_linear_attention_gb300 as cla

    c = s["case"]
    if c["op"] == "gated_step":
        y = cla.gated_scan_step(s["x"], s["rgate"], s["igate"], s["lam"], s["h0"], reset=s["reset"])
        return y, s["h0"]
    if c["op"] == "gated_prefill":
        return cla.gated_scan_fwd(s["x"], s["rgate"], s["igate"], s["lam"], s["h0"], reset=s["reset"], lens=s["lens"])
    if c["op"] == "gated_train":
        ck = cla.gated_scan_ckpt(s["x"])
        h, hT = cla.gated_scan_fwd(s["x"], s["rgate"], s["igate"], s["lam"], s["h0"], reset=s["reset"], lens=s["lens"],
                                   ckpt=ck)
        return (h, hT) + cla.gated_scan_bwd(s["x"], s["rgate"], s["igate"], s["lam"], s["h0"], s["dh"], s["dhT"],
                                            reset=s["reset"], lens=s["lens"], ckpt=ck)
    w, n = c["window"], c["sinks"]
    if c["op"] == "window_step":
        o = cla.window_attn_step(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["pos"], window=w, sinks=n)
        return o, s["kcache"], s["vcache"]
    o, lse = cla.window_attn_fwd(s["q"], s["k"], s["v"], window=w, sinks=n, lens=s["lens"])
    if c["op"] == "window_prefill":
        cla.window_cache_write(s["k"], s["v"], s["kcache"], s["vcache"], window=w, sinks=n, lens=s["lens"])
        return o, lse, s["kcache"], s["vcache"]
    return (o, lse) + cla.window_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], window=w, sinks=n, lens=s["lens"])


def _run_plain(s):
    return {"gated_step": _plain_gated_step, "gated_prefill": _plain_gated, "gated_train": _plain_gated,
            "window_step": _plain_window_step, "window_prefill": _plain_window, "window_train": _plain_window}[
        s["case"]["op"]](s)


def _gates(s, x, rgate, igate, reset):
    """(r, i, L, a, m) in 32 bits; 1 - a^2 as -expm1(2 L), which keeps its digits where a is near 1."""
    r, i = torch.sigmoid(rgate.float()), torch.sigmoid(igate.float())
    L = -C_GATE * torch.logaddexp(s["lam"], torch.zeros_like(s["lam"])) * r
    a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
    if reset is not None:
        a, m = a.masked_fill(reset[..., None], 0.0), m.masked_fill(reset[..., None], 1.0)
    return r, i, L, a, m


def _plain_gated_step(s):
    _, i, _, a, m = _gates(s, s["x"], s["rgate"], s["igate"], s["reset"])
    h = a * s["h0"] + m * i * s["x"].float()
    s["h0"].copy_(h)
    return h.to(s["x"].dtype), s["h0"]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 from zero, by doubling the distance that is composed."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat((b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]), 1)
        a = torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1)
        n *= 2
    return b


def _plain_gated(s):
    c, x, reset, lens = s["case"], s["x"].float(), s["reset"], s["lens"]
    r, i, L, a, m = _gates(s, x, s["rgate"], s["igate"], reset)
    u = i * x
    b = m * u
    ok = None
    if lens is not None:
        ok = (torch.arange(c["T"], device=x.device) < lens[:, None])[..., None]
        a, b = torch.where(ok, a, 1.0), torch.where(ok, b, 0.0)
    h = _scan(a, torch.cat((b[:, :1] + a[:, :1] * s["h0"][:, None], b[:, 1:]), 1))
    hT = h[:, -1].clone()
    out = h if ok is None else torch.where(ok, h, 0.0)
    out = out.to(s["x"].dtype)
    if c["op"] == "gated_prefill":
        return out, hT
    g = s["dh"].float()
    g = g if ok is None else torch.where(ok, g, 0.0)
    g = torch.cat((g[:, :-1], g[:, -1:] + s["dhT"][:, None]), 1)
    after = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    hb = _scan(after.flip(1), g.flip(1)).flip(1)
    before = torch.cat((s["h0"][:, None], h[:, :-1]), 1)
    gl = hb * (before * a * L - a * a * torch.where(m > 0, L / m, 0.0) * u)
    if reset is not None:
        gl = gl.masked_fill(reset[..., None], 0.0)
    dx, di, dr = hb * m * i, hb * m * u * (1 - i), gl * (1 - r)
    if ok is not None:
        dx, di, dr, gl = (torch.where(ok, v, 0.0) for v in (dx, di, dr, gl))
    slope = torch.sigmoid(s["lam"]) / torch.logaddexp(s["lam"], torch.zeros_like(s["lam"]))
    dlam = gl.sum((0, 1), dtype=torch.float64).float() * slope
    t = s["x"].dtype
    return out, hT, dx.to(t), dr.to(t), di.to(t), dlam, a[:, 0] * hb[:, 0]


def _plain_window(s):
    """The band in blocks of C >= window tokens: a block of queries sees its own block of keys and the one before it;
    the sinks that the window has left behind come as further columns."""
    c = s["case"]
    B, H, K, T, d, W = (c[n] for n in ("B", "H", "Hkv", "T", "d", "window"))
    G, n = H // K, min(c["sinks"], c["T"])
    C = min(max(W, 64), T)
    nb = -(-T // C)
    scale = d ** -0.5
    dev = s["q"].device

    def padded(x, front):
        return torch.nn.functional.pad(x.float(), (0, 0, front, nb * C - T))

    def rows(x):  # [B, H, T, d] -> [B, K, nb, G * C, d]
        return padded(x, 0).view(B, K, G, nb, C, d).transpose(2, 3).reshape(B, K, nb, G * C, d)

    def heads(x):  # and back
        return x.view(B, K, nb, G, C, -1).transpose(2, 3).reshape(B, H, nb * C, -1)[:, :, :T]

    def pairs(x):  # [B, K, T, d] -> [B, K, nb, 2 * C, d]
        x = padded(x, C).view(B, K, nb + 1, C, d)
        return torch.cat((x[:, :, :-1], x[:, :, 1:]), 3)

    q, k, v = rows(s["q"]), pairs(s["k"]), pairs(s["v"])
    ks, vs = s["k"][:, :, None, :n].float(), s["v"][:, :, None, :n].float()
    t = torch.arange(nb * C, device=dev).view(nb, 1, C, 1)
    u = (torch.arange(nb, device=dev)[:, None] - 1) * C + torch.arange(2 * C, device=dev)
    u = u.view(nb, 1, 1, 2 * C)
    z = torch.arange(n, device=dev)
    lens = s["lens"] if s["lens"] is not None else torch.full((1,), T, device=dev)
    live = t < lens.view(-1, 1, 1, 1, 1)
    see = torch.cat(((u >= 0) & (u <= t) & (t - u < W), t - z >= W), 3) & live
    see = see[:, None].expand(-1, -1, -1, G, -1, -1).reshape(see.shape[0], 1, nb, G * C, 2 * C + n)
    x = torch.cat((q @ k.transpose(3, 4), q @ ks.transpose(3, 4)), 4).mul_(scale).masked_fill_(~see, -math.inf)
    top = x.amax(4, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    lse = torch.log(total) + top
    p = p.div_(torch.where(total > 0, total, 1.0))
    of = p[..., :2 * C] @ v + p[..., 2 * C:] @ vs
    o, e = heads(of).to(s["q"].dtype), heads(lse)[..., 0].contiguous()
    if c["op"] == "window_prefill":
        for name in ("k", "v"):
            _plain_write(s[name], s[name + "cache"], c, s["lens"])
        return o, e, s["kcache"], s["vcache"]
    g = rows(s["do"])
    delta = (g * of).sum(4, keepdim=True)
    ds = torch.cat((g @ v.transpose(3, 4), g @ vs.transpose(3, 4)), 4).sub_(delta).mul_(p).mul_(scale)
    dq = heads(ds[..., :2 * C] @ k + ds[..., 2 * C:] @ ks)
    g = torch.where(live[:, None].expand(-1, -1, -1, G, -1, -1).reshape(live.shape[0], 1, nb, G * C, 1), g, 0.0)

    def keys(w, y):  # w^T y, the two blocks of each pair added up where they overlap, and the sinks'
        z = w[..., :2 * C].transpose(3, 4) @ y
        z = torch.nn.functional.pad(z[:, :, 1:, :C], (0, 0, 0, 0, 0, 1)) + z[:, :, :, C:]
        z = z.reshape(B, K, nb * C, d)[:, :, :T]
        z[:, :, :n] += (w[..., 2 * C:].transpose(3, 4) @ y).sum(2)
        return z

    dt = s["q"].dtype
    return o, e, dq.to(dt), keys(ds, q).to(dt), keys(p, g).to(dt)


def _plain_write(x, cache, c, lens):
    W, n, T = c["window"], c["sinks"], c["T"]
    lens = lens if lens is not None else torch.full((c["B"],), T, device=x.device, dtype=torch.int32)
    j = torch.arange(n + W, device=x.device)
    turn = torch.div(lens[:, None] - 1 - j, W, rounding_mode="floor").clamp(min=0)
    p = torch.where(j < n, j, j + W * turn)  # the last token that this slot has had
    at = p.clamp(max=T - 1)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
    cache.copy_(torch.where((p < lens[:, None])[:, None, :, None], x.gather(2, at), cache))


def _plain_window_step(s):
    c = s["case"]
    B, H, K, d, W, n = (c[m] for m in ("B", "H", "Hkv", "d", "window", "sinks"))
    pos = s["pos"].long()
    at = torch.where(pos < n, pos, n + (pos - n) % W)[:, None, None, None].expand(-1, K, 1, d)
    s["kcache"].scatter_(2, at, s["k"][:, :, None])
    s["vcache"].scatter_(2, at, s["v"][:, :, None])
    see = torch.arange(n + W, device=pos.device) < (pos + 1)[:, None]
    q = s["q"].float().view(B, K, H // K, d)
    x = (q @ s["kcache"].float().transpose(2, 3) * d ** -0.5).masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(3, keepdim=True))
    o = (p / p.sum(3, keepdim=True)) @ s["vcache"].float()
    return o.view(B, H, d).to(s["q"].dtype), s["kcache"], s["vcache"]


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(T, W, n):
    """Pairs (t, s) of a sequence of T tokens that the mask leaves."""
    band = T * (T + 1) // 2 if T <= W else W * (W + 1) // 2 + (T - W) * W
    return band + sum(max(0, T - W - j) for j in range(min(n, T)))


def work(case):
    c = case
    e = torch.empty(0, dtype=_T[c["dtype"]]).element_size()
    if c["op"].startswith("gated"):
        n = (sum(_lens(c)) if c["ragged"] else c["B"] * c["T"]) * c["D"]
        full, state = c["B"] * c["T"] * c["D"], 4 * c["B"] * c["D"]
        once = 3 * e * n + e * full + 2 * state + 4 * c["D"]
        if c["op"] != "gated_train":
            return {"bytes": once, "flops": 20 * n}
        return {"bytes": once + 4 * e * n + 3 * e * full + 3 * state + 4 * c["D"], "flops": 60 * n}
    B, H, K, T, d, W, n = (c[m] for m in ("B", "H", "Hkv", "T", "d", "window", "sinks"))
    if c["op"] == "window_step":
        seen = sum(min(p + 1, n + W) for p in _pos(c))
        return {"bytes": e * d * (2 * K * seen + 2 * B * H + 2 * B * K), "flops": 4 * d * (H // K) * K * seen}
    lens = _lens(c) if c["ragged"] else [T] * B
    pairs, used = H * sum(_seen(m, W, n) for m in lens), sum(lens)
    io = e * d * (H * used + 2 * K * used + H * B * T) + 4 * H * B * T
    if c["op"] == "window_prefill":
        return {"bytes": io + 2 * e * d * K * sum(min(m, n + W) for m in lens), "flops": 4 * d * pairs}
    return {"bytes": io + e * d * (H * used + (H + 2 * K) * B * T), "flops": 14 * d * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        return (_exact_gated if case["op"].startswith("gated") else _exact_window)(case, s)


def _exact_gated(c, s):
    """Token by token, from the definition; the gradients by walking back, derivatives through a itself."""
    step = c["op"] == "gated_step"
    x, rg, ig = ((s[n][:, None] if step else s[n]).double() for n in ("x", "rgate", "igate"))
    B, T, D = x.shape
    lam, h = s["lam"].double(), s["h0"].double()
    sp = torch.log1p(torch.exp(-lam.abs())) + lam.clamp(min=0)
    r, i = 1 / (1 + torch.exp(-rg)), 1 / (1 + torch.exp(-ig))
    a = torch.exp(-C_GATE * sp * r)
    m = torch.sqrt(-torch.expm1(-2 * C_GATE * sp * r))
    keep = torch.ones(B, T, 1, dtype=torch.float64, device=x.device)
    if s["reset"] is not None:
        keep = 1 - s["reset"].double().view(B, T, 1)
    live = torch.ones(B, T, 1, dtype=torch.bool, device=x.device)
    if s["lens"] is not None:
        live = (torch.arange(T, device=x.device)[None] < s["lens"][:, None])[..., None]
    a1 = torch.where(live, a * keep, 1.0)
    m1 = m * keep + (1 - keep)
    b1 = torch.where(live, m1 * i * x, 0.0)
    hs = torch.empty(B, T + 1, D, dtype=torch.float64, device=x.device)
    hs[:, 0] = h
    for t in range(T):
        torch.addcmul(b1[:, t], a1[:, t], hs[:, t], out=hs[:, t + 1])
    out, hT = torch.where(live, hs[:, 1:], 0.0), hs[:, T]
    if step:
        return out[:, 0], hT
    if c["op"] == "gated_prefill":
        return out, hT
    g = torch.where(live, s["dh"].double(), 0.0)
    hb = torch.empty_like(g)
    carry = s["dhT"].double()
    for t in range(T - 1, -1, -1):
        torch.add(g[:, t], carry, out=hb[:, t])
        carry = a1[:, t] * hb[:, t]
    db = torch.where(live, hb, 0.0)
    da = db * (hs[:, :-1] - a / m * i * x) * keep  # a's own gradient, m's part included
    dx, di = db * m1 * i, db * m1 * x * i * (1 - i)
    dL = da * a
    dr = dL * (-C_GATE * sp) * r * (1 - r)
    dlam = (dL * (-C_GATE) * r).sum((0, 1)) / (1 + torch.exp(-lam))
    return out, hT, dx, dr, di, dlam, carry


def _exact_window(c, s):
    """A strip of queries at a time against the keys that any of them sees; gradients by automatic differentiation."""
    B, H, K, T, d, W, n = (c[m] for m in ("B", "H", "Hkv", "T", "d", "window", "sinks"))
    if c["op"] == "window_step":
        kc, vc = s["kcache"].double(), s["vcache"].double()
        out = torch.empty(B, H, d, dtype=torch.float64, device=kc.device)
        for b, p in enumerate(_pos(c)):
            j = p if p < n else n + (p - n) % W
            kc[b, :, j], vc[b, :, j] = s["k"][b].double(), s["v"][b].double()
            m = min(p + 1, n + W)
            x = torch.einsum("kgd,ksd->kgs", s["q"][b].double().view(K, H // K, d), kc[b, :, :m]) / math.sqrt(d)
            out[b] = torch.einsum("kgs,ksd->kgd", torch.softmax(x, 2), vc[b, :, :m]).reshape(H, d)
        return out, kc, vc
    lens = _lens(c) if c["ragged"] else [T] * B
    train = c["op"] == "window_train"
    q, k, v = (s[m].double() for m in ("q", "k", "v"))
    o, lse = torch.zeros_like(q), torch.full((B, H, T), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v)) if train else (None, None, None)
    R = max(16, min(512, W))
    for b in range(B):
        for t0 in range(0, lens[b], R):
            t1 = min(t0 + R, lens[b])
            lo = max(0, t0 - W + 1)
            e = min(n, lo)  # sinks in front of the strip's band
            sel = torch.cat((torch.arange(e, device=q.device), torch.arange(lo, t1, device=q.device)))
            tt = torch.arange(t0, t1, device=q.device)[:, None]
            see = (sel <= tt) & ((tt - sel < W) | (sel < n))
            qq = q[b, :, t0:t1].view(K, H // K, t1 - t0, d).detach().requires_grad_(train)
            kk, vv = (y[b][:, sel].detach().requires_grad_(train) for y in (k, v))
            x = torch.einsum("kgtd,ksd->kgts", qq, kk) / math.sqrt(d)
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, 3)
            y = torch.einsum("kgts,ksd->kgtd", torch.exp(x - z[..., None]), vv)
            o[b, :, t0:t1], lse[b, :, t0:t1] = y.detach().reshape(H, -1, d), z.detach().reshape(H, -1)
            if train:
                up = s["do"][b, :, t0:t1].double().view_as(y)
                gq, gk, gv = torch.autograd.grad(y, (qq, kk, vv), up)
                dq[b, :, t0:t1] = gq.reshape(H, -1, d)
                dk[b].index_add_(1, sel, gk)
                dv[b].index_add_(1, sel, gv)
    if train:
        return o, lse, dq, dk, dv
    for b in range(B):
        for p in list(range(min(n, lens[b]))) + list(range(max(n, lens[b] - W), lens[b])):
            j = p if p < n else n + (p - n) % W
            s["kcache"][b, :, j], s["vcache"][b, :, j] = s["k"][b, :, p], s["v"][b, :, p]
    return o, lse, s["kcache"].double(), s["vcache"].double()
