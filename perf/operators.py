"""Measured cases of the exact-attention operators: rotary positions, dense
attention forward, dense attention forward + backward, and dense attention of
one new token per sequence over a paged key-value cache.

``run`` computes them in their plain form (elementary torch operations in 32
bits, angles in 64, rounded once at the end), or with ``own = True`` through
this package's entry points.  ``exact`` restates each in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _rotary(name, B, H, Hkv, N, d, dtype, axes, layout, inverse, positions, scaling="none",
            factor=1.0, token_major=False):
    return dict(name=name, kind="rotary", B=B, H=H, Hkv=Hkv, N=N, d=d, dtype=dtype, axes=axes,
                layout=layout, inverse=inverse, positions=positions, scaling=scaling,
                factor=factor, token_major=token_major)


def _attn(name, kind, B, H, Hkv, Nq, Nk, d, dtype, causal=False, ragged=False,
          token_major=False):
    return dict(name=name, kind=kind, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype,
                causal=causal, ragged=ragged, token_major=token_major)


def _decode(name, B, H, Hkv, L, page, d, dtype, ragged, head_major=False):
    return dict(name=name, kind="decode", B=B, H=H, Hkv=Hkv, L=L, page=page, d=d, dtype=dtype,
                ragged=ragged, head_major=head_major)


def listed():
    return [
        # one new token per sequence at far positions, before a decode call: latency
        _rotary("rotary token", 32, 12, 12, 1, 128, "bf16", "128", "half", False, "far", "parts",
                8.0),
        # 480p latent in raster order, three axes, part of the head, fp32 activations
        _rotary("rotary 480p", 1, 12, 12, 4680, 128, "f32", "32,32,32", "interleaved", False,
                "3,30,52"),
        # gradients of the rotated q and k of a 720p latent
        _rotary("rotary 720p backward", 1, 12, 12, 75600, 128, "bf16", "44,42,42", "half", True,
                "21,45,80"),
        # ViT-B layer left dense: 196 patches and the class token
        _attn("fwd vit", "fwd", 32, 12, 12, 197, 197, 64, "bf16"),
        # one new 30x52 frame over the three frames in hand (two earlier, itself), shared heads
        _attn("fwd frame", "fwd", 1, 12, 4, 1560, 4680, 128, "bf16", token_major=True),
        # the longest sequence of the sweep
        _attn("fwd 16k", "fwd", 1, 12, 12, 16384, 16384, 64, "bf16"),
        # finetuning step of a dense layer in 32 bits, the sweep's 1K
        _attn("train 1k f32", "train", 1, 12, 12, 1024, 1024, 64, "f32"),
        # padded batch of texts in a causal layer with shared heads, token-major projections
        _attn("train padded causal", "train", 4, 16, 4, 2000, 2000, 128, "bf16", True, True,
              True),
        # finetuning step of a dense layer on the 480p latent
        _attn("train 480p", "train", 1, 12, 12, 4680, 4680, 128, "bf16"),
        # one short sequence: latency
        _decode("decode one", 1, 12, 12, 1000, 16, 64, "bf16", False),
        # a batch of requests of every length, shared heads
        _decode("decode ragged", 64, 16, 4, 8192, 64, 128, "bf16", True),
        # two very long sequences: few rows, split over the cache
        _decode("decode long", 2, 32, 8, 131072, 128, 128, "bf16", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "fwd", "train", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 4, 5])
    if kind == "rotary":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        B = _log(rng, 1, 16)
        layout = rng.choice(["half", "interleaved"])
        inverse = rng.random() < 0.5
        tm = rng.random() < 0.5
        top = max(2, int(1.2e8 / (B * (H + Hkv) * d)))
        if rng.random() < 0.5:  # a (f, h, w) latent, three axes
            a = d // 3 // 2 * 2
            part = rng.choice([f"{d - 2 * a},{a},{a}", f"{a},{a},{a}"])
            h, w = rng.randint(5, 45), rng.randint(5, 80)
            f = max(1, min(_log(rng, 1, 24), top // (h * w)))
            case = _rotary("", B if f * h * w <= top else 1, H, Hkv, f * h * w, d, dtype, part,
                           layout, inverse, f"{f},{h},{w}", token_major=tm)
        else:
            rot = rng.choice([d, d // 4 * 2, 16])
            scaling = rng.choice(["none", "linear", "ntk", "parts"])
            factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.5, 32.0])
            case = _rotary("", B, H, Hkv, min(_log(rng, 1, 40000), top), d, dtype, str(rot),
                           layout, inverse, rng.choice(["range", "far"]), scaling, factor, tm)
    elif kind in ("fwd", "train"):
        d = rng.choice([64, 64, 128, 128, 32, 80, 96, 40])
        B = _log(rng, 1, 8)
        most = 1.6e9 if dtype == "bf16" else 6e7  # query-key pairs over all heads
        if kind == "train":
            most /= 3.6
        top = int(math.sqrt(most / (B * H)))
        # (the gradients of q and k are zero where a row sees one key: nothing to compare)
        Nk = _log(rng, 17 if kind == "train" else 1, min(16384, 2 * top))
        square = kind == "train" or rng.random() < 0.5
        Nq = min(Nk, top) if square else _log(rng, 1, max(1, min(top, int(most / (B * H * Nk)))))
        if square:
            Nk = Nq
        causal = rng.random() < 0.5
        ragged = rng.random() < 0.4
        case = _attn("", kind, B, H, Hkv, Nq, Nk, d, dtype, causal, ragged, rng.random() < 0.5)
    else:
        d = rng.choice([64, 128, 128, 80, 96])
        B = _log(rng, 1, 128)
        size = 2 if dtype == "bf16" else 4
        top = int(1.0e9 / (B * Hkv * d * size * 2))
        L = _log(rng, 1, max(2, min(131072, top)))
        case = _decode("", B, H, Hkv, L, rng.choice([1, 8, 16, 24, 64, 128, 256]), d, dtype,
                       rng.random() < 0.6, rng.random() < 0.5)
        if L > 20000 and case["page"] < 16:
            case["page"] = 16
    del case["name"]
    return case


def _lens(count, top):
    """`count` lengths spread over 0 .. top (one empty, one full, where there are two or more)."""
    if count == 1:
        return [top - top // 5]
    return [top * b // (count - 1) for b in range(count)]


def _pairs(c):
    """Query-key pairs that one head of every sequence of the batch computes, summed."""
    lens = _lens(c["B"], c["Nk"]) if c["ragged"] else [c["Nk"]] * c["B"]
    if not c["causal"]:
        return sum(lens) * c["Nq"]
    shift, total = c["Nk"] - c["Nq"], 0
    for n in lens:
        # sum over i of min(n, i + shift + 1), shift >= 0 here or rows before -shift see nothing
        lo = max(0, -shift)
        full = min(max(n - 1 - shift, lo), c["Nq"])  # rows below `full` see i + shift + 1 keys
        total += (full - lo) * shift + (full * (full + 1) - lo * (lo + 1)) // 2
        total += (c["Nq"] - full) * n
    return total


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] == "rotary":
        n = c["B"] * (c["H"] + c["Hkv"]) * c["N"] * c["d"]
        axes = len(c["axes"].split(","))
        return {"bytes": 2 * n * e + 4 * axes * c["N"], "flops": 3 * n}
    if c["kind"] == "decode":
        keys = sum(_lens(c["B"], c["L"])) if c["ragged"] else c["B"] * c["L"]
        io = 2 * c["B"] * c["H"] * c["d"] * e + c["B"] * c["H"] * 4
        return {"bytes": 2 * keys * c["Hkv"] * c["d"] * e + io + 4 * -(-keys // c["page"]),
                "flops": 4 * keys * c["H"] * c["d"]}
    q = c["B"] * c["H"] * c["Nq"] * c["d"] * e
    kv = c["B"] * c["Hkv"] * c["Nk"] * c["d"] * e
    lse = c["B"] * c["H"] * c["Nq"] * 4
    fl = 2 * c["H"] * c["d"] * _pairs(c)
    if c["kind"] == "fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * fl}
    # q, k, v, dout read; out, dq, dk, dv written; seven products of the pairs
    return {"bytes": 4 * q + 4 * kv, "flops": 7 * fl}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _heads(g, B, H, N, d, dtype, token_major):
    if token_major:
        return torch.randn(B, N, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    return torch.randn(B, H, N, d, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["kind"] == "rotary":
        tm = c["token_major"]
        s["q"] = _heads(g, c["B"], c["H"], c["N"], c["d"], dtype, tm)
        s["k"] = _heads(g, c["B"], c["Hkv"], c["N"], c["d"], dtype, tm)
        if c["positions"] == "range":
            p = torch.arange(c["N"], device="cuda")[None]
        elif c["positions"] == "far":  # each sequence somewhere in a long context
            at = torch.randint(0, 1000000, (c["B"], 1, 1), generator=g, device="cuda")
            p = at + torch.arange(c["N"], device="cuda")
        else:  # raster order of a (f, h, w) latent
            f, h, w = (int(x) for x in c["positions"].split(","))
            grid = torch.meshgrid(*(torch.arange(n, device="cuda") for n in (f, h, w)),
                                  indexing="ij")
            p = torch.stack([x.reshape(-1) for x in grid])
        s["positions"] = p.to(torch.int32).contiguous()
        s["axes"] = tuple(int(x) for x in c["axes"].split(","))
        return s
    if c["kind"] == "decode":
        B, ps, L = c["B"], c["page"], c["L"]
        lens = _lens(B, L) if c["ragged"] else [L] * B
        order = torch.randperm(B, generator=g, device="cuda")
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)[order].contiguous()
        per = -(-L // ps)
        pages = B * per
        s["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(B, per)
        s["q"] = torch.randn(B, c["H"], c["d"], generator=g, device="cuda").to(dtype)
        caches = []
        for _ in range(2):
            if c["head_major"]:
                x = torch.empty(pages, c["Hkv"], ps, c["d"], device="cuda", dtype=dtype)
            else:
                x = torch.empty(pages, ps, c["Hkv"], c["d"], device="cuda", dtype=dtype)
            x.normal_(generator=g)
            caches.append(x if c["head_major"] else x.transpose(1, 2))
        s["k"], s["v"] = caches
        return s
    tm = c["token_major"]
    s["q"] = _heads(g, c["B"], c["H"], c["Nq"], c["d"], dtype, tm)
    s["k"] = _heads(g, c["B"], c["Hkv"], c["Nk"], c["d"], dtype, tm)
    s["v"] = _heads(g, c["B"], c["Hkv"], c["Nk"], c["d"], dtype, tm)
    s["lens"] = None
    if c["ragged"]:
        order = torch.randperm(c["B"], generator=g, device="cuda")
        lens = torch.tensor(_lens(c["B"], c["Nk"]), device="cuda", dtype=torch.int32)
        s["lens"] = lens[order].contiguous()
    if c["kind"] == "train":
        s["dout"] = _heads(g, c["B"], c["H"], c["Nq"], c["d"], dtype, tm)
    return s


SCALING_ORIGINAL = 4096.0  # context that the scaled positions were trained on
SCALING_SLOW, SCALING_FAST = 1.0, 32.0  # turns over it between which "parts" blends


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _frequencies(axes, scaling, factor, device):
    """Angular frequency of each rotated pair (64 bits), axis after axis, and the magnitude."""
    n = torch.tensor(axes, device=device, dtype=torch.float64)
    r = torch.cat([torch.arange(a // 2, device=device, dtype=torch.float64) for a in axes])
    width = torch.repeat_interleave(n, (n / 2).to(torch.int64))
    base = torch.full_like(width, 10000.0)
    if scaling == "ntk":
        base = base * factor ** (width / (width - 2).clamp(min=1))
    f = base ** (-2 * r / width)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        turns = SCALING_ORIGINAL * f / (2 * math.pi)
        keep = ((turns - SCALING_SLOW) / (SCALING_FAST - SCALING_SLOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f, 0.1 * math.log(factor) + 1 if scaling == "parts" else 1.0


def _pair_channels(axes, layout, device):
    """Channels of the first and second member of each rotated pair, axis after axis."""
    n = torch.tensor(axes, device=device)
    half = n // 2
    axis = torch.repeat_interleave(torch.arange(len(axes), device=device), half)
    start = (torch.cumsum(n, 0) - n)[axis]
    r = torch.arange(int(sum(axes)) // 2, device=device) - (torch.cumsum(half, 0) - half)[axis]
    if layout == "interleaved":
        return axis, start + 2 * r, start + 2 * r + 1
    return axis, start + r, start + r + half[axis]


def _plain_rotary(s):
    c, p = s["case"], s["positions"]
    f, mag = _frequencies(s["axes"], c["scaling"], c["factor"], p.device)
    axis, first, second = _pair_channels(s["axes"], c["layout"], p.device)
    p = p if p.dim() == 3 else p[None]
    angle = p[:, axis].transpose(1, 2).to(torch.float64) * f  # (B or 1, N, pairs)
    cos = (torch.cos(angle) * mag).to(torch.float32)[:, None]
    sin = (torch.sin(angle) * mag).to(torch.float32)[:, None]
    sin = -sin if c["inverse"] else sin

    def turn(x):
        y = x.float()
        a, b = y[..., first], y[..., second]
        z = y.clone()
        z[..., first] = a * cos - b * sin
        z[..., second] = b * cos + a * sin
        return z.to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _by_group(x, Hkv):
    """(B, H, ...) as (B, Hkv, H / Hkv, ...): query heads beside the head they share."""
    return x.reshape(x.shape[0], Hkv, x.shape[1] // Hkv, *x.shape[2:])


def _visible(c, lens, device):
    j = torch.arange(c["Nk"], device=device)
    ok = None
    if lens is not None:
        ok = (j < lens[:, None])[:, None, None, None, :]
    if c["causal"]:
        i = torch.arange(c["Nq"], device=device)[:, None]
        low = j <= i + (c["Nk"] - c["Nq"])
        ok = low if ok is None else ok & low
    return ok


def _softmax(S, ok):
    """Probabilities over the visible keys (a row without one: zeros) and log-sum-exp."""
    if ok is not None:
        S = S.masked_fill(~ok, -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = torch.exp(S - m)
    z = P.sum(-1, keepdim=True)
    lse = (m + torch.log(z)).squeeze(-1)
    return P.div_(torch.where(z == 0, torch.ones_like(z), z)), lse


def _plain_fwd(s):
    c = s["case"]
    Hkv, sc = c["Hkv"], 1 / math.sqrt(c["d"])
    q, k, v = _by_group(s["q"].float(), Hkv), s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    P, lse = _softmax(torch.matmul(q, k.transpose(-1, -2)) * sc, _visible(c, s["lens"], q.device))
    out = torch.matmul(P, v)
    return (out.flatten(1, 2).to(s["q"].dtype), lse.flatten(1, 2)), (q, k, v, P, out)


def _plain_train(s):
    c = s["case"]
    (out, lse), (q, k, v, P, o) = _plain_fwd(s)
    sc = 1 / math.sqrt(c["d"])
    do = _by_group(s["dout"].float(), c["Hkv"])
    dv = torch.matmul(P.transpose(-1, -2), do).sum(2)
    dS = torch.matmul(do, v.transpose(-1, -2))
    dS = dS.sub_((do * o).sum(-1, keepdim=True)).mul_(P).mul_(sc)
    dq = torch.matmul(dS, k).flatten(1, 2)
    dk = torch.matmul(dS.transpose(-1, -2), q).sum(2)
    return out, dq.to(out.dtype), dk.to(out.dtype), dv.to(out.dtype)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    table = s["table"].long()

    def gather(x):  # (B, Hkv, keys, d)
        return x[table].transpose(1, 2).reshape(B, Hkv, -1, d).float()

    q = _by_group(s["q"].float(), Hkv)
    S = torch.matmul(q, gather(s["k"]).transpose(-1, -2)) / math.sqrt(d)
    ok = torch.arange(S.shape[-1], device=S.device) < s["lens"][:, None, None, None]
    P, lse = _softmax(S, ok)
    v = gather(s["v"]).masked_fill(~ok.reshape(B, 1, -1, 1), 0)
    return torch.matmul(P, v).flatten(1, 2).to(s["q"].dtype), lse.flatten(1, 2)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _scaling(c):
    if c["scaling"] == "none":
        return None
    if c["scaling"] == "parts":
        return ("parts", c["factor"], SCALING_ORIGINAL, SCALING_SLOW, SCALING_FAST)
    return (c["scaling"], c["factor"])


def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        from structured_sub_quadratic_b200 import api

        c = s["case"]
        if kind == "rotary":
            return api.monarch_attn_rotary(s["q"], s["k"], s["positions"], axis_dims=s["axes"],
                                           interleaved=c["layout"] == "interleaved",
                                           scaling=_scaling(c), inverse=c["inverse"])
        if kind == "decode":
            return api.monarch_attn_dense_decode(s["q"], s["k"], s["v"], s["table"], s["lens"])
        out, lse = api.monarch_attn_dense_fwd(s["q"], s["k"], s["v"], causal=c["causal"],
                                              k_lens=s["lens"])
        if kind == "fwd":
            return out, lse
        return (out, *api.monarch_attn_dense_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"],
                                                 causal=c["causal"], k_lens=s["lens"]))
    if kind == "rotary":
        return _plain_rotary(s)
    if kind == "decode":
        return _plain_decode(s)
    return _plain_fwd(s)[0] if kind == "fwd" else _plain_train(s)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_rotary(s):
    c, axes, p = s["case"], s["axes"], s["positions"].double()
    if p.dim() == 2:
        p = p.unsqueeze(0)
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        at = 0
        for a, n in enumerate(axes):
            part = y[..., at:at + n]
            z = torch.view_as_complex(
                (part.reshape(*part.shape[:-1], n // 2, 2) if c["layout"] == "interleaved" else
                 torch.stack([part[..., :n // 2], part[..., n // 2:]], -1)).contiguous())
            w, mag = [], 1.0
            for r in range(n // 2):
                th = 10000.0 ** (-2.0 * r / n)
                if c["scaling"] == "linear":
                    th /= c["factor"]
                elif c["scaling"] == "ntk":
                    th = (10000.0 * c["factor"] ** (n / max(n - 2, 1))) ** (-2.0 * r / n)
                elif c["scaling"] == "parts":
                    turns = th * SCALING_ORIGINAL / (2 * math.pi)
                    g = min(1.0, max(0.0, (turns - SCALING_SLOW) / (SCALING_FAST - SCALING_SLOW)))
                    th = (1 - g) * th / c["factor"] + g * th
                    mag = 1 + 0.1 * math.log(c["factor"])
                w.append(th)
            ang = p[:, a, :, None] * torch.tensor(w, device=y.device, dtype=torch.float64)
            ang = -ang if c["inverse"] else ang
            z = z * torch.polar(torch.full_like(ang, mag), ang)[:, None]
            y[..., at:at + n] = (torch.view_as_real(z).flatten(-2) if c["layout"] == "interleaved"
                                 else torch.cat([z.real, z.imag], -1))
            at += n
        outs.append(y)
    return tuple(outs)


def _exact_attention(s):
    c = s["case"]
    B, H, Nq, Nk, d = c["B"], c["H"], c["Nq"], c["Nk"], c["d"]
    rep, train = H // c["Hkv"], c["kind"] == "train"
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.zeros(B, H, Nq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, H, Nq), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = (torch.zeros(x.shape, device="cuda", dtype=torch.float64) for x in (q, k, v))
    i = torch.arange(Nq, device="cuda")[:, None]
    lens = [Nk] * B if s["lens"] is None else s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        first = 0  # the first query that sees a key
        if c["causal"]:
            first = min(Nq, max(0, Nq - Nk))
        if n == 0 or first == Nq:
            continue
        hide = None
        if c["causal"]:
            hide = torch.arange(n, device="cuda")[None] > i[first:] + (Nk - Nq)
        for h in range(H):
            qq, kk, vv = (x.double().requires_grad_(train)
                          for x in (q[b, h, first:], k[b, h // rep, :n], v[b, h // rep, :n]))
            with torch.set_grad_enabled(train):
                S = (qq @ kk.T) / math.sqrt(d)
                if hide is not None:
                    S = S.masked_fill(hide, -math.inf)
                o = torch.softmax(S, -1) @ vv
                lse[b, h, first:] = torch.logsumexp(S.detach(), -1)
            out[b, h, first:] = o.detach()
            if train:
                gq, gk, gv = torch.autograd.grad(o, (qq, kk, vv), s["dout"][b, h, first:].double())
                dq[b, h, first:] = gq
                dk[b, h // rep, :n] += gk
                dv[b, h // rep, :n] += gv
    return (out, dq, dk, dv) if train else (out, lse)


def _exact_decode(s):
    c = s["case"]
    B, H, d, ps = c["B"], c["H"], c["d"], c["page"]
    rep = H // c["Hkv"]
    out = torch.zeros(B, H, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, device="cuda", dtype=torch.float64)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // ps)].long()
        k = torch.cat(list(s["k"][pages].double()), 1)[:, :n]  # (Hkv, n, d)
        v = torch.cat(list(s["v"][pages].double()), 1)[:, :n]
        for h in range(H):
            S = (k[h // rep] @ s["q"][b, h].double()) / math.sqrt(d)
            out[b, h] = torch.softmax(S, 0) @ v[h // rep]
            lse[b, h] = torch.logsumexp(S, 0)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rotary":
        return _exact_rotary(s)
    return _exact_decode(s) if kind == "decode" else _exact_attention(s)
