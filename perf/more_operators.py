"""Norm and rotation of queries and keys, the rolling cache in 8 bits, the delta rule token by token: their cases, plain
forms and 64-bit values.

Norm and rotation, a row x of d values of head h of token t:  n = x / sqrt(mean(x^2) + eps), y = w n, and the pairs
(i, i + rot / 2) of y's first rot values (or (2i, 2i + 1), interleaved) turned by the angle pos_t freq_i.

8-bit cache of window attention: token p in slot p (p < sinks), else in sinks + (p - sinks) % window, as e4m3 numbers of
a factor for every 64 slots of a key head: the smallest power of two, 2^-64 at least, under which what the block
holds stays within 448.  A step puts its token into its slot, its block's factor becomes that of what the block then
holds, and it attends over the cache's values.

Delta rule:  u = beta (v - a S^T k),  S = a S + k u^T,  o = S^T q,  a = exp(log_decay), tokens in order.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 64
_T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _n(name, op, B, H, Hkv, T, d, rot, dtype, interleaved=False, packed=False, ragged=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "T": T, "d": d, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "packed": packed, "ragged": ragged}


def _c(name, op, B, H, Hkv, T, d, window, sinks, dtype, ragged=False):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "T": T, "d": d, "window": window, "sinks": sinks,
            "dtype": dtype, "ragged": ragged}


def _d(name, B, H, Hk, T, dk, dv, dtype, ragged=False):
    return {"name": name, "op": "delta_step", "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv, "dtype": dtype,
            "ragged": ragged}


def listed():
    return [
        # serving, one token for a few sequences at far positions: a launch's latency
        _n("norm step 4x16", "norm_step", 4, 16, 4, 1, 128, 128, "bf16"),
        # serving, a long prompt
        _n("norm prefill 1x32x32768", "norm_prefill", 1, 32, 8, 32768, 128, 128, "bf16"),
        # training, the shape of the benchmark's constant-decay attention
        _n("norm train 4x16x8192 d64", "norm_train", 4, 16, 16, 8192, 64, 64, "bf16"),
        # training, packed documents in a padded batch, half of an odd head rotated, neighbours as pairs
        _n("norm train 3x10x1531 d96", "norm_train", 3, 10, 5, 1531, 96, 48, "fp16", True, True, True),
        # serving, the prompts of a batch into the cache
        _c("cache8 write 16x8192", "cache8_write", 16, 8, 8, 8192, 128, 4096, 4, "bf16"),
        # serving, short padded prompts of odd sizes
        _c("cache8 write 5x777 d64", "cache8_write", 5, 3, 3, 777, 64, 300, 7, "fp16", True),
        # serving, one token for a few sequences, some of them shorter than the window
        _c("cache8 step 4x16 w1024", "cache8_step", 4, 16, 4, 1, 128, 1024, 4, "bf16", True),
        # serving, one token for a full batch with a wide window
        _c("cache8 step 64x32 w4096", "cache8_step", 64, 32, 8, 1, 128, 4096, 4, "bf16"),
        # serving, few long sequences
        _c("cache8 step 2x32 w65536", "cache8_step", 2, 32, 4, 1, 128, 65536, 0, "fp16"),
        # serving, one token for a few sequences
        _d("delta step 4x16", 4, 16, 16, 1, 128, 128, "bf16"),
        # serving, one token for a full batch, key heads shared
        _d("delta step 64x32", 64, 32, 16, 1, 128, 128, "bf16"),
        # serving, drafts of a few tokens, of which each sequence takes some
        _d("delta step 24x12x5 d64", 24, 12, 4, 5, 64, 192, "fp16", True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_step", "norm_prefill", "norm_train", "cache8_write", "cache8_step", "delta_step"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "delta_step":
        Hk, dk = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128])
        H, dv = Hk * rng.choice([1, 2, 3]), rng.choice([64, 128, 128, 4 * rng.randint(4, 64)])
        B = _log(rng, 1, max(1, min(256, 33_000_000 // (H * dk * dv))))
        return _unnamed(_d("", B, H, Hk, rng.choice([1, 1, 1, rng.randint(2, 8)]), dk, dv,
                           rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.random() < 0.3))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 5])
    if op.startswith("norm"):
        d = rng.choice([64, 128, 128, 256, 16 * rng.randint(1, 16)])
        rot = rng.choice([d, d, 16 * rng.randint(0, d // 16)])
        dtype = rng.choice([dtype, dtype, "fp32"])
        most = (30_000_000 if dtype == "fp32" else 60_000_000) // ((H + Hkv) * d)
        T = 1 if op == "norm_step" else _log(rng, 1, min(65536, most))
        B = _log(rng, 1, max(1, min(512 if T == 1 else 16, most // T)))
        more = T > 1
        return _unnamed(_n("", op, B, H, Hkv, T, d, rot, dtype, rng.random() < 0.3, more and rng.random() < 0.3,
                           more and rng.random() < 0.3))
    d, sinks = rng.choice([64, 128]), rng.choice([0, 1, 4, 16, rng.randint(1, 100)])
    most = (2_000_000 if op == "cache8_step" else 500_000) // Hkv  # slots, or tokens, of all sequences together
    window = _log(rng, 1, 65536 if op == "cache8_step" else 8192)
    B = _log(rng, 1, max(1, min(64, most // (window + sinks))))
    T = 1 if op == "cache8_step" else _log(rng, 1, max(1, min(16384, most // B)))
    return _unnamed(_c("", op, B, H if op == "cache8_step" else Hkv, Hkv, T, d, window, sinks, dtype, rng.random() < 0.5))


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


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _T[c["dtype"]]

    def rnd(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def lens():
        return torch.tensor(_lens(c), dtype=torch.int32, device="cuda") if c["ragged"] else None

    s = {"case": c}
    B, H, T = c["B"], c["H"], c["T"]
    if c["op"] == "delta_step":
        Hk, dk, dv = c["Hk"], c["dk"], c["dv"]
        # q, k, v as a convolution leaves them, tokens first; keys and queries of length one
        mix = rnd(B, T, 2 * Hk * dk + H * dv, dtype=torch.float32)
        for x in mix[..., :2 * Hk * dk].view(B, T, 2 * Hk, dk).unbind(2):
            x.div_(x.norm(dim=-1, keepdim=True))
        mix = mix.to(t)
        s["q"], s["k"] = mix[..., :2 * Hk * dk].view(B, T, 2, Hk, dk).permute(2, 0, 3, 1, 4)
        s["v"] = mix[..., 2 * Hk * dk:].view(B, T, H, dv).transpose(1, 2)
        s["log_decay"] = -torch.rand(B, T, H, generator=g, device="cuda").mul_(0.3).transpose(1, 2)
        s["beta"] = torch.sigmoid(rnd(B, T, H, dtype=torch.float32)).transpose(1, 2)
        s["S"] = rnd(B, H, dk, dv, std=0.3, dtype=torch.float32)
        s["lens"] = lens()
        return s
    K, d = c["Hkv"], c["d"]
    if c["op"].startswith("norm"):
        # slices of one projection [B, T, heads, d]
        qkv = rnd(B, T, H + 2 * K, d, std=2.0)
        s["q"], s["k"] = (x.transpose(1, 2) for x in (qkv[:, :, :H], qkv[:, :, H:H + K]))
        s["wq"], s["wk"] = (1 + 0.2 * rnd(d, dtype=torch.float32) for _ in range(2))
        s["freq"] = None
        if c["rot"]:
            s["freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float32) / c["rot"])
        s["pos"], s["lens"] = None, lens()
        if c["op"] == "norm_step":
            s["q"], s["k"] = s["q"][:, :, 0], s["k"][:, :, 0]
            s["pos"] = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda", dtype=torch.int32)
        elif c["packed"]:  # documents of about 200 tokens, each from position 0
            at = torch.arange(T, device="cuda").expand(B, T)
            first = torch.rand(B, T, generator=g, device="cuda") < 1.0 / 200
            s["pos"] = (at - torch.where(first, at, 0).cummax(1).values).to(torch.int32)
        if c["op"] == "norm_train":
            s["dqo"], s["dko"] = rnd(B, H, T, d), rnd(B, K, T, d)
        return s
    S = c["sinks"] + c["window"]
    nb = -(-S // BLOCK)
    if c["op"] == "cache8_write":
        kv = rnd(B, T, 2 * K, d)
        s["k"], s["v"] = (x.transpose(1, 2) for x in (kv[:, :, :K], kv[:, :, K:]))
        for n in ("k", "v"):
            s[n + "cache"] = torch.zeros(B, K, S, d, device="cuda").to(_E4M3)
            s[n + "scale"] = torch.zeros(B, K, nb, device="cuda")
        s["lens"] = lens()
        return s
    qkv = rnd(B, H + 2 * K, d)
    s["q"], s["k"], s["v"] = qkv[:, :H] * 1.5, qkv[:, H:H + K], qkv[:, H + K:]
    s["pos"] = torch.tensor(_pos(c), dtype=torch.int32, device="cuda")
    held = (torch.arange(S, device="cuda") < s["pos"][:, None])[:, None, :, None]
    for n in ("k", "v"):
        x = torch.where(held, rnd(B, K, S, d, dtype=torch.float32), 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, nb * BLOCK - S)).view(B, K, nb, BLOCK, d)
        f = _factor(x.abs().amax((3, 4)))
        s[n + "cache"] = (x / f[..., None, None]).to(_E4M3).view(B, K, nb * BLOCK, d)[:, :, :S].contiguous()
        s[n + "scale"] = f
    return s


def _factor(top):
    """The smallest power of two, 2^-64 at least, of which 448 is not below `top`."""
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1, and 448 = 7/8 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875), -64).clamp(min=-64)
    return ((e + 127) << 23).view(torch.float32)


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import chunkwise_linear_attention_gb300 as cla

    c = s["case"]
    if c["op"] == "delta_step":
        return cla.delta_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["S"], lens=s["lens"]), s["S"]
    if c["op"].startswith("norm"):
        qk, kw = (s["q"], s["k"], s["wq"], s["wk"], s["freq"]), {"eps": EPS, "interleaved": c["interleaved"]}
        if c["op"] == "norm_step":
            return cla.qk_norm_rope_step(*qk, s["pos"], **kw)
        kw.update(pos=s["pos"], lens=s["lens"])
        out = cla.qk_norm_rope_fwd(*qk, **kw)
        return out if c["op"] == "norm_prefill" else out + cla.qk_norm_rope_bwd(*qk, s["dqo"], s["dko"], **kw)
    cache, kw = (s["kcache"], s["vcache"], s["kscale"], s["vscale"]), {"window": c["window"], "sinks": c["sinks"]}
    if c["op"] == "cache8_write":
        cla.window_cache8_write(s["k"], s["v"], *cache, lens=s["lens"], **kw)
        return cache
    return (cla.window_attn_step8(s["q"], s["k"], s["v"], *cache, s["pos"], **kw),) + cache


def _run_plain(s):
    op = s["case"]["op"]
    return {"d": _plain_delta, "n": _plain_norm, "c": _plain_write if op == "cache8_write" else _plain_step}[op[0]](s)


def _plain_norm(s):
    c = s["case"]
    step, rot = c["op"] == "norm_step", c["rot"]
    B, T, h = c["B"], c["T"], c["rot"] // 2
    q, k = ((x[:, :, None] if step else x).float() for x in (s["q"], s["k"]))
    dev, t = q.device, s["q"].dtype
    pos = torch.arange(T, device=dev).expand(B, T) if s["pos"] is None else s["pos"].view(B, T)
    cos = sin = None
    if rot:
        angle = pos[:, None, :, None].double() * s["freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    live = None
    if s["lens"] is not None:
        live = (torch.arange(T, device=dev) < s["lens"][:, None])[:, None, :, None]

    def turn(y, sin):
        if not rot:
            return y
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            front = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :h], y[..., h:rot]
            front = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((front, y[..., rot:]), -1)

    def keep(y):
        return (y if live is None else torch.where(live, y, 0.0)).to(t)

    out, normed = [], []
    for x, w in ((q, s["wq"]), (k, s["wk"])):
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        normed.append((x * r, r))
        out.append(keep(turn(x * r * w, sin)))
    if step:
        return tuple(y[:, :, 0] for y in out)
    if c["op"] == "norm_prefill":
        return tuple(out)
    dx, dw = [], []
    for (n, r), w, up in zip(normed, (s["wq"], s["wk"]), (s["dqo"], s["dko"])):
        g = turn(up.float(), -sin if rot else None)
        g = g if live is None else torch.where(live, g, 0.0)
        gn = g * n
        dw.append(gn.sum((0, 1, 2), dtype=torch.float64).float())
        dx.append(keep(r * (g * w - n * (gn * w).mean(-1, keepdim=True))))
    return tuple(out + dx + dw)


def _plain_write(s):
    c = s["case"]
    B, K, T, d, W, n = (c[m] for m in ("B", "Hkv", "T", "d", "window", "sinks"))
    S = n + W
    nb = -(-S // BLOCK)
    dev = s["k"].device
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), T, device=dev, dtype=torch.int32)
    j = torch.arange(S, device=dev)
    turn = torch.div(lens[:, None] - 1 - j, W, rounding_mode="floor").clamp(min=0)
    p = torch.where(j < n, j, j + W * turn)  # the last token that falls on this slot
    held = (p < lens[:, None])[:, None, :, None]
    at = p.clamp(max=T - 1)[:, None, :, None].expand(-1, K, -1, d)
    for m in ("k", "v"):
        x = torch.where(held, s[m].gather(2, at).float(), 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, nb * BLOCK - S)).view(B, K, nb, BLOCK, d)
        any_ = torch.nn.functional.pad(held[:, :, :, 0], (0, nb * BLOCK - S)).view(B, 1, nb, BLOCK).any(3)
        f = torch.where(any_, _factor(x.abs().amax((3, 4))), s[m + "scale"])
        code = (x / torch.where(any_, f, 1.0)[..., None, None]).to(_E4M3).view(B, K, nb * BLOCK, d)[:, :, :S]
        s[m + "scale"].copy_(f)
        bits = s[m + "cache"].view(torch.uint8)
        bits.copy_(torch.where(held, code.view(torch.uint8), bits))
    return s["kcache"], s["vcache"], s["kscale"], s["vscale"]


def _plain_step(s):
    c = s["case"]
    B, H, K, d, W, n = (c[m] for m in ("B", "H", "Hkv", "d", "window", "sinks"))
    S, pos = n + W, s["pos"].long()
    mine = torch.where(pos < n, pos, n + (pos - n) % W)
    j = (mine // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device=pos.device)  # the slots of the token's block
    held = ((j < (pos + 1)[:, None]) & (j < S))[:, None, :, None]
    new = (j == mine[:, None])[:, None, :, None]
    at = j.clamp(max=S - 1)[:, None, :, None].expand(-1, K, -1, d)
    blk = (mine // BLOCK)[:, None, None].expand(-1, K, 1)
    val = []
    for m in ("k", "v"):
        bits = s[m + "cache"].view(torch.uint8)
        old = bits.gather(2, at)
        x = old.view(_E4M3).float() * s[m + "scale"].gather(2, blk)[..., None]
        x = torch.where(new, s[m][:, :, None].float(), torch.where(held, x, 0.0))
        f = _factor(x.abs().amax((2, 3)))[..., None]
        code = torch.where(held, (x / f[..., None]).to(_E4M3).view(torch.uint8), old)
        # what would lie behind the cache's last slot writes the block's first one once more
        inside = torch.where(j < S, j, j[:, :1])[:, None, :, None].expand(-1, K, -1, d)
        bits.scatter_(2, inside, torch.where((j < S)[:, None, :, None], code, code[:, :, :1]))
        s[m + "scale"].scatter_(2, blk, f)
        val.append(s[m + "cache"].float() * s[m + "scale"].repeat_interleave(BLOCK, 2)[:, :, :S, None])
    see = torch.arange(S, device=pos.device) < (pos + 1)[:, None]
    q = s["q"].float().view(B, K, H // K, d)
    x = (q @ val[0].transpose(2, 3) * d ** -0.5).masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(3, keepdim=True))
    o = (p / p.sum(3, keepdim=True)) @ val[1]
    return o.view(B, H, d).to(s["q"].dtype), s["kcache"], s["vcache"], s["kscale"], s["vscale"]


def _plain_delta(s):
    c = s["case"]
    G, S = c["H"] // c["Hk"], s["S"]
    q, k = (s[m].float().repeat_interleave(G, 1) for m in ("q", "k"))
    v, a, beta = s["v"].float(), torch.exp(s["log_decay"]), s["beta"]
    live = None
    if s["lens"] is not None:
        live = (torch.arange(c["T"], device=q.device) < s["lens"][:, None])[:, None, :, None]
    h, out = S, []
    for t in range(c["T"]):
        ah = a[:, :, t, None, None] * h
        u = beta[:, :, t, None] * (v[:, :, t] - (ah * k[:, :, t, :, None]).sum(2))
        new = ah + k[:, :, t, :, None] * u[:, :, None]
        o = (new * q[:, :, t, :, None]).sum(2)
        if live is not None:
            new, o = torch.where(live[:, :, t, None], new, h), torch.where(live[:, :, t], o, 0.0)
        h = new
        out.append(o)
    S.copy_(h)
    return torch.stack(out, 2), S


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = torch.empty(0, dtype=_T[c["dtype"]]).element_size()
    B, H, T = c["B"], c["H"], c["T"]
    used = sum(_lens(c)) if c["ragged"] else B * T
    if c["op"] == "delta_step":
        state, io = B * H * c["dk"] * c["dv"], e * used * (2 * c["Hk"] * c["dk"] + H * c["dv"])
        return {"bytes": 8 * state + io + 4 * B * T * H * c["dv"] + 8 * used * H, "flops": 7 * used * H * c["dk"] * c["dv"]}
    K, d = c["Hkv"], c["d"]
    if c["op"].startswith("norm"):
        n, full = used * (H + K) * d, B * T * (H + K) * d
        once = e * (n + full) + 8 * d + 2 * c["rot"] + (4 * used if c["op"] == "norm_step" or c["packed"] else 0)
        if c["op"] != "norm_train":
            return {"bytes": once, "flops": 8 * n}
        return {"bytes": once + e * (2 * n + full) + 8 * d, "flops": 25 * n}
    S = c["sinks"] + c["window"]
    if c["op"] == "cache8_write":
        kept = sum(min(m, S) for m in (_lens(c) if c["ragged"] else [T] * B))
        return {"bytes": 2 * K * kept * d * (e + 1) + 8 * K * kept // BLOCK, "flops": 4 * K * kept * d}
    # one slot's write and its block's factors are what a step changes
    seen = sum(min(p + 1, S) for p in _pos(c))
    return {"bytes": 2 * K * d * seen + 8 * K * -(-seen // BLOCK) + e * d * (2 * B * H + 2 * B * K) + 2 * B * K * d,
            "flops": 4 * d * H * seen}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        return {"d": _exact_delta, "n": _exact_norm, "c": _exact_cache}[case["op"][0]](case, s)


def _exact_norm(c, s):
    """Pairs as complex numbers; gradients by automatic differentiation."""
    step, train, rot = c["op"] == "norm_step", c["op"] == "norm_train", c["rot"]
    B, T = c["B"], c["T"]
    dev = s["q"].device
    pos = torch.arange(T, device=dev).repeat(B, 1) if s["pos"] is None else s["pos"].reshape(B, T)
    lens = torch.tensor(_lens(c) if c["ragged"] else [T] * B, device=dev)
    live = (torch.arange(T, device=dev)[None] < lens[:, None])[:, None, :, None].double()
    outs, dxs, dws = [], [], []
    for n, w in (("q", s["wq"]), ("k", s["wk"])):
        x = (s[n][:, :, None] if step else s[n]).double().detach().requires_grad_(train)
        w = w.double().detach().requires_grad_(train)
        y = x / torch.sqrt(x.pow(2).sum(3, keepdim=True) / c["d"] + EPS) * w
        if rot:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                               pos.double()[:, None, :, None] * s["freq"].double())
            z = y[..., :rot]
            z = z.unflatten(3, (rot // 2, 2)) if c["interleaved"] else z.unflatten(3, (2, rot // 2)).transpose(3, 4)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.flatten(3) if c["interleaved"] else z.transpose(3, 4).flatten(3)
            y = torch.cat((z, y[..., rot:]), 3)
        y = y * live
        if train:
            dx, dw = torch.autograd.grad(y, (x, w), s["d" + n + "o"].double())
            dxs.append(dx)
            dws.append(dw)
        y = y.detach()
        outs.append(y[:, :, 0] if step else y)
    return tuple(outs + dxs + dws)


def _nearest(x):
    """The e4m3 numbers nearest to x, the even one of two: by looking them up among all of them."""
    grid = [math.ldexp(m + 8 * (e > 0), max(e, 1) - 10) for e in range(16) for m in range(8)]
    grid = torch.tensor(grid[:127], dtype=torch.float64, device=x.device)
    a = x.abs()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[pick], x)


def _exact_blocks(x):
    """(numbers, factors) of what blocks hold, [..., block, slot, d]."""
    top = x.abs().amax((-2, -1))
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -80) / 448)).long()
    f = ((e + 1023) << 52).view(torch.float64)  # or twice, or half that
    f = torch.where(top > 448 * f, 2 * f, torch.where(top <= 224 * f, f / 2, f)).clamp(min=2.0 ** -64)
    return _nearest(x / f[..., None, None]), f


def _exact_cache(c, s):
    B, H, K, T, d, W, n = (c[m] for m in ("B", "H", "Hkv", "T", "d", "window", "sinks"))
    S = n + W
    cache = {m: s[m + "cache"].double() for m in ("k", "v")}
    scale = {m: s[m + "scale"].double() for m in ("k", "v")}
    dev = s["k"].device
    if c["op"] == "cache8_write":
        for b, m in enumerate(_lens(c) if c["ragged"] else [T] * B):
            p = torch.cat((torch.arange(min(n, m)), torch.arange(min(m, max(n, m - W)), m))).to(dev)
            j = torch.where(p < n, p, n + (p - n) % W)
            m = min(m, S)
            i = -(-m // BLOCK)
            for name in ("k", "v"):
                x = torch.zeros(K, i * BLOCK, d, dtype=torch.float64, device=dev)
                x[:, j] = s[name][b][:, p].double()
                x, scale[name][b, :, :i] = _exact_blocks(x.view(K, i, BLOCK, d))
                cache[name][b, :, :m] = x.view(K, i * BLOCK, d)[:, :m]
        return cache["k"], cache["v"], scale["k"], scale["v"]
    out = torch.empty(B, H, d, dtype=torch.float64, device=dev)
    for b, p in enumerate(_pos(c)):
        j = p if p < n else n + (p - n) % W
        i, m = j // BLOCK, min(p + 1, S)
        lo, hi = i * BLOCK, min((i + 1) * BLOCK, m)
        val = {}
        for name in ("k", "v"):
            x = cache[name][b, :, lo:hi] * scale[name][b, :, i, None, None]
            x[:, j - lo] = s[name][b].double()
            cache[name][b, :, lo:hi], scale[name][b, :, i] = _exact_blocks(x)
            val[name] = cache[name][b, :, :m] * scale[name][b][:, torch.arange(m, device=dev) // BLOCK, None]
        x = torch.einsum("kgd,ksd->kgs", s["q"][b].double().view(K, H // K, d), val["k"]) / math.sqrt(d)
        out[b] = torch.einsum("kgs,ksd->kgd", torch.softmax(x, 2), val["v"]).reshape(H, d)
    return out, cache["k"], cache["v"], scale["k"], scale["v"]


def _exact_delta(c, s):
    """The state's transition as the matrix a (I - beta k k^T), token by token, one sequence after the other."""
    B, H, G, T = c["B"], c["H"], c["H"] // c["Hk"], c["T"]
    o = torch.zeros(B, H, T, c["dv"], dtype=torch.float64, device=s["S"].device)
    S = s["S"].double()
    one = torch.eye(c["dk"], dtype=torch.float64, device=s["S"].device)
    for b, m in enumerate(_lens(c) if c["ragged"] else [T] * B):
        for t in range(m):
            q, k = (s[n][b, :, t].double().repeat_interleave(G, 0) for n in ("q", "k"))
            beta, a = s["beta"][b, :, t, None, None].double(), s["log_decay"][b, :, t, None, None].double().exp()
            move = a * (one - beta * k[:, :, None] * k[:, None])
            S[b] = move @ S[b] + beta * k[:, :, None] * s["v"][b, :, t, None].double()
            o[b, :, t] = (q[:, None] @ S[b])[:, 0]
    return o, S
