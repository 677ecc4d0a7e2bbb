"""Cases of the operators around the span cache: token log-probabilities (and the surprisal that
marks span boundaries), rotary positions, and the 4-bit cache with its append, read-back and
attention.  Plain forms are elementary torch; with ``own`` the calls are the framework's."""

import math

import torch

own = False

DEV = "cuda"
PAGE, TILE, TILE_BYTES, PAGE_BYTES = 64, 16, 2304, 9216
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "f32": 4}


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the next token of one sequence, with five alternatives to show beside it: latency
        dict(name="logprobs 1x32000 top5", op="logprobs", rows=1, vocab=32000, top=5, dtype="bf16", scale=1.0),
        # one decode step of a served batch that asks for twenty alternatives
        dict(name="logprobs 48x128000 top20", op="logprobs", rows=48, vocab=128000, top=20, dtype="bf16", scale=1.0),
        # 32-bit logits of an evaluation, an odd vocabulary, a temperature
        dict(name="logprobs 257x50021 f32 top3", op="logprobs", rows=257, vocab=50021, top=3, dtype="f32", scale=0.75),
        # the boundary signal of a prefill chunk, in the layout the span build takes
        dict(name="surprisal 1x4096x128000", op="surprisal", batch=1, ctx=4096, vocab=128000, dtype="bf16"),
        # one decode step, batch 1, 32 query and 8 KV heads: latency
        dict(name="rope 1x1 32/8", op="rope", batch=1, ctx=1, hq=32, hkv=8, dim=128, rot=128, dtype="bf16",
             interleaved=False, scaling="banded", factor=8.0, base=500000.0, start=131000),
        # a ragged decode batch, part of the head, adjacent pairs, by-parts scaling
        dict(name="rope 16x3 28/4 part", op="rope", batch=16, ctx=3, hq=28, hkv=4, dim=128, rot=64, dtype="fp16",
             interleaved=True, scaling="parts", factor=4.0, base=10000.0, start=60000),
        # a prefill: q in place of the projection's layout, k into the layout of the span build
        dict(name="rope 1x32768 32/8", op="rope", batch=1, ctx=32768, hq=32, hkv=8, dim=128, rot=128, dtype="bf16",
             interleaved=False, scaling="none", factor=1.0, base=500000.0, start=0),
        # one decode step of a batch: a token's K and V into the 4-bit cache, and what it then holds
        dict(name="kv4 store 16x1", op="store", batch=16, ctx=1, hkv=4, start=4000, dtype="bf16"),
        # a prefill into the 4-bit cache, and its K and V read back for the span build
        dict(name="kv4 store 1x32768", op="store", batch=1, ctx=32768, hkv=8, start=0, dtype="bf16"),
        # draft tokens of a few short conversations
        dict(name="kv4 attention 4x2000 q3", op="attention", batch=4, ctx=2000, hq=32, hkv=8, nq=3, ragged=True, dtype="bf16"),
        # one long context, the shape of the headline decode step
        dict(name="kv4 attention 1x131072", op="attention", batch=1, ctx=131072, hq=32, hkv=8, nq=1, ragged=False, dtype="bf16"),
        # a batch of long contexts, seven query heads to a KV head
        dict(name="kv4 attention 16x65536", op="attention", batch=16, ctx=65536, hq=28, hkv=4, nq=1, ragged=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "surprisal", "rope", "rope", "store", "store", "attention", "attention", "attention"])
    if op == "logprobs":
        vocab = _log(rng, 50, 160000)
        rows = _log(rng, 1, max(2, min(2000, 100_000_000 // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, top=min(vocab, rng.randint(0, 32)), dtype=rng.choice(["bf16", "fp16", "f32"]),
                    scale=rng.choice([1.0, 0.5, 0.75, 1.25]))
    if op == "surprisal":
        vocab = _log(rng, 500, 160000)
        batch, dtype = rng.randint(1, 4), rng.choice(["bf16", "fp16", "f32"])
        return dict(op=op, batch=batch, ctx=_log(rng, 2, max(3, min(4000, 800_000_000 // SIZE[dtype] // vocab // batch))), vocab=vocab,
                    dtype=dtype)
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([64, 96, 128, 128, 192, 256])
        batch = rng.randint(1, 16)
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        hq = hkv * rng.choice([1, 2, 4, 7])
        return dict(op=op, batch=batch, ctx=_log(rng, 1, max(2, min(30000, 120_000_000 // (hq + hkv) // dim) // batch)), hq=hq, hkv=hkv, dim=dim, rot=rot,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "f32"]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "parts", "banded"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), start=_log(rng, 1, 1000000))
    if op == "store":
        batch = rng.randint(1, 16)
        return dict(op=op, batch=batch, ctx=_log(rng, 1, 30000 // batch), hkv=rng.choice([1, 2, 4, 8]), start=rng.choice([0, rng.randint(1, 5000)]),
                    dtype=rng.choice(["bf16", "fp16"]))
    hkv = rng.choice([1, 2, 4, 8])
    batch, nq = rng.randint(1, 24), rng.choice([1, 1, 1, 2, 4, 7])
    return dict(op=op, batch=batch, ctx=_log(rng, 1, 2_000_000 // batch // hkv // nq), hq=hkv * rng.choice([1, 2, 4, 7, 8]), hkv=hkv, nq=nq,
                ragged=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "fp16"]))


# ---------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pages_of(c):
    """(pages of one sequence, pages of the pool): a few more than the sequences fill."""
    mp = -(-(c.get("start", 0) + c["ctx"]) // PAGE)
    return mp, c["batch"] * mp + 3


def _table(c, g):
    mp, n = _pages_of(c)
    return torch.randperm(n, generator=g, device=DEV)[: c["batch"] * mp].to(torch.int32).view(c["batch"], mp).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    if c["op"] in ("logprobs", "surprisal"):
        shape = (c["rows"],) if c["op"] == "logprobs" else (c["batch"], c["ctx"])
        logits = torch.empty(*shape, c["vocab"], dtype=DT[c["dtype"]], device=DEV).normal_(0, 2.5, generator=g)
        tok = torch.randint(0, c["vocab"], shape, generator=g, device=DEV)
        # the token that comes is a likely one: its logit stands out by up to ten
        at = tok if c["op"] == "logprobs" else torch.roll(tok, -1, 1)
        up = torch.rand(*shape, 1, generator=g, device=DEV) * 10
        logits.scatter_(-1, at[..., None], (torch.gather(logits, -1, at[..., None]).float() + up).to(logits.dtype))
        s.update(logits=logits, tokens=tok)
    elif c["op"] == "rope":
        B, T = c["batch"], c["ctx"]
        s["q"] = torch.randn(B, T, c["hq"], c["dim"], generator=g, device=DEV).to(DT[c["dtype"]])
        s["k"] = torch.randn(B, T, c["hkv"], c["dim"], generator=g, device=DEV).to(DT[c["dtype"]])
        first = c["start"] - torch.randint(0, max(1, c["start"] // 2 + 1), (B, 1), generator=g, device=DEV) if B > 1 else c["start"]
        s["pos"] = (torch.arange(T, device=DEV)[None] + first).to(torch.int32).contiguous()
    elif c["op"] == "store":
        B, T, H = c["batch"], c["ctx"], c["hkv"]
        # keys: a few channels stand out, and have a mean of their own; values: plain
        ch = torch.where(torch.rand(H, 128, generator=g, device=DEV) < 0.05, 6.0, 1.0)
        mean = torch.randn(H, 128, generator=g, device=DEV) * ch
        s["k"] = (torch.randn(B, T, H, 128, generator=g, device=DEV) * ch + mean).to(DT[c["dtype"]])
        s["v"] = torch.randn(B, T, H, 128, generator=g, device=DEV).to(DT[c["dtype"]])
        s["table"] = _table(c, g)
        s["pages"] = torch.zeros(_pages_of(c)[1], H, PAGE_BYTES, dtype=torch.uint8, device=DEV)
        s["pos0"] = torch.full((B,), c["start"], dtype=torch.int32, device=DEV)
    else:
        B, H = c["batch"], c["hkv"]
        n = _pages_of(c)[1]
        s["table"] = _table(c, g)
        pages = torch.randint(0, 256, (n, H, PAGE // TILE, TILE_BYTES), dtype=torch.uint8, generator=g, device=DEV)
        sz = torch.rand(n, H, PAGE // TILE, 64, 2, generator=g, device=DEV)  # (token, group): scale and zero point
        sz[..., 0] = sz[..., 0] * 0.25 + 0.1
        sz[..., 1] = sz[..., 1] * 0.6 - 8 * sz[..., 0]
        pages[..., 2048:] = sz.to(torch.bfloat16).view(torch.uint8).view(n, H, PAGE // TILE, 256)
        s["pages"] = pages.view(n, H, PAGE_BYTES)
        s["q"] = torch.randn(B, c["nq"], c["hq"], 128, generator=g, device=DEV).to(DT[c["dtype"]])
        lens = torch.full((B,), c["ctx"], dtype=torch.int32, device=DEV)
        if c["ragged"] and B > 1:  # one full-length sequence, the others from half of it up
            less = torch.rand(B, generator=g, device=DEV) * (c["ctx"] // 2)
            lens = lens - less.to(torch.int32) * (torch.arange(B, device=DEV) > 0)
        s["lens"] = lens.to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------------------------- the plain forms
def _logprob_parts(logits, scale):
    x = logits.float() * scale
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    tot = e.sum(-1)
    return x, m[..., 0], e, tot


def _plain_logprobs(s):
    c, logits = s["c"], s["logits"]
    x, m, e, tot = _logprob_parts(logits, c["scale"])
    ln = torch.log(tot)
    lse = m + ln
    tok = torch.gather(x, -1, s["tokens"][:, None])[:, 0]
    ent = ln - (e * (x - m[:, None])).sum(-1) / tot
    out = {"logprob": tok - lse, "lse": lse, "entropy": ent}
    if c["top"]:
        b = (logits.float() + 0.0).view(torch.int32).to(torch.int64)
        key = torch.where(b < 0, -(b & 0x7FFFFFFF), b) * (1 << 32) + (c["vocab"] - torch.arange(c["vocab"], device=DEV))
        ids = torch.topk(key, c["top"], -1).indices
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = torch.gather(x, -1, ids) - lse[:, None]
    return out


def _plain_surprisal(s):
    x, m, _, tot = _logprob_parts(s["logits"][:, :-1], 1.0)
    tok = torch.gather(x, -1, s["tokens"][:, 1:, None])[..., 0]
    H = m + torch.log(tot) - tok
    return torch.cat([torch.zeros_like(H[:, :1]), H], 1)


def _inv_freq(c):
    """Angles per position of the rotated pairs, 64 bits, and the factor on the result."""
    d, base, f, orig = c["rot"], c["base"], c["factor"], 8192.0
    i = torch.arange(0, d, 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "ntk" and d > 2:
        base = base * f ** (d / (d - 2.0))
    inv, m = base ** (-i / d), 1.0
    if c["scaling"] == "linear":
        inv = inv / f
    elif c["scaling"] == "parts":
        lo = math.floor(d * math.log(orig / (32.0 * 2 * math.pi)) / (2 * math.log(base)))
        hi = math.ceil(d * math.log(orig / (1.0 * 2 * math.pi)) / (2 * math.log(base)))
        lo, hi = max(lo, 0), min(hi, d - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        inv = inv / f * ramp + inv * (1 - ramp)
        m = 0.1 * math.log(f) + 1.0 if f > 1 else 1.0
    elif c["scaling"] == "banded":
        wave = 2 * math.pi / inv
        t = ((orig / wave - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        inv = (1 - t) * inv / f + t * inv
    return inv, m


def _rotated(x, cos, sin, c, m):
    r = c["rot"]
    h = x[..., :r]
    a, b = (h[..., 0::2], h[..., 1::2]) if c["interleaved"] else (h[..., : r // 2], h[..., r // 2 :])
    u, v = (a * cos - b * sin) * m, (b * cos + a * sin) * m
    rot = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([rot, x[..., r:]], -1)


def _plain_rope(s):
    c = s["c"]
    inv, m = _inv_freq(c)
    ang = s["pos"].double()[..., None] * inv
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    q, k = (_rotated(s[n].float(), cos, sin, c, m).to(s[n].dtype) for n in "qk")
    return {"q": q, "k": k.transpose(1, 2).contiguous()}


def _plain_store(s):
    out = {}
    for n in "kv":
        x = s[n].float().unflatten(-1, (2, 64))
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        z = lo.to(torch.bfloat16)  # the largest bf16 at or below the smallest value
        z = torch.where(z.float() > lo, torch.nextafter(z, torch.full_like(z, -math.inf)), z).float()
        sc = ((hi - z) / 15).to(torch.bfloat16).float()
        code = torch.where(sc > 0, torch.round((x - z) / torch.where(sc > 0, sc, 1.0)).clamp(0, 15), 0.0)
        out[n] = (z + sc * code).flatten(-2).to(torch.bfloat16).transpose(1, 2).contiguous()
    return out


def _unpacked(s, dt):
    """K and V [B][Hkv][T][128] that the pages of each sequence stand for."""
    c = s["c"]
    B, H = c["batch"], c["hkv"]
    p = s["pages"][s["table"].long()]  # [B][np][Hkv][page]
    p = p.transpose(1, 2).reshape(B, H, -1, TILE_BYTES)

    def nibbles(b):
        return torch.stack([b & 15, b >> 4], -1)

    nt = p.shape[2]
    k = nibbles(p[..., :1024].reshape(B, H, nt, 16, 4, 2, 2, 4))  # token, quarter, group, word, byte, nibble
    k = k.permute(0, 1, 2, 3, 5, 4, 6, 7, 8).reshape(B, H, nt * 16, 2, 64).to(dt)
    v = nibbles(p[..., 1024:2048].reshape(B, H, nt, 2, 8, 4, 2, 2, 2, 2))  # half, dims, pair, group, word, parity, byte, nibble
    v = v.permute(0, 1, 2, 3, 5, 8, 6, 4, 7, 9, 10).reshape(B, H, nt * 16, 2, 64).to(dt)
    w = p[..., 2048:].contiguous().view(torch.bfloat16).to(dt).reshape(B, H, nt, 2, 4, 2, 2, 2, 2)  # K/V, pair, half, parity, group, (s, z)
    w = w.permute(3, 0, 1, 2, 5, 4, 6, 7, 8).reshape(2, B, H, nt * 16, 2, 2)
    k, v = (w[i, ..., 1:] + w[i, ..., :1] * x for i, x in ((0, k), (1, v)))
    return k.reshape(B, H, nt * 16, 128)[:, :, : c["ctx"]], v.reshape(B, H, nt * 16, 128)[:, :, : c["ctx"]]


def _plain_attention(s):
    c = s["c"]
    B, H, nq, G = c["batch"], c["hkv"], c["nq"], c["hq"] // c["hkv"]
    k, v = _unpacked(s, torch.float32)
    q = s["q"].float().view(B, nq, H, G, 128).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, 128)
    x = (q @ k.transpose(-1, -2)).view(B, H, nq, G, -1) * (1 / math.sqrt(128.0))
    last = s["lens"][:, None] - nq + torch.arange(nq, device=DEV)[None]  # the last key each query sees
    seen = torch.arange(c["ctx"], device=DEV) <= last[:, None, :, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - torch.where(m > -math.inf, m, 0.0)), 0.0)
    tot = e.sum(-1, keepdim=True)
    o = (e / torch.where(tot > 0, tot, 1.0)).view(B, H, nq * G, -1) @ v
    o = o.view(B, H, nq, G, 128).permute(0, 2, 1, 3, 4).reshape(B, nq, c["hq"], 128)
    lse = (m + torch.log(tot))[..., 0].permute(0, 2, 1, 3).reshape(B, nq, c["hq"])
    return {"out": o, "lse": lse}


# ---------------------------------------------------------------------------------- the framework's calls
def _kept(s, sk):
    """What a program makes once and keeps: configuration, workspace, plan, cache handle."""
    if "kept" not in s:
        c = s["c"]
        if c["op"] in ("logprobs", "surprisal"):
            s["kept"] = sk.Workspace(sk.Config(1, 1, 1, 0, 0, 64))
        elif c["op"] == "rope":
            s["kept"] = sk.RopePlan(c["rot"], base=c["base"], interleaved=c["interleaved"], scaling=c["scaling"], factor=c["factor"],
                                    original_context=8192)
        else:
            cfg = sk.Config(c["batch"], c.get("hq", c["hkv"]), c["hkv"], 0, 0, 64)
            s["kept"] = cfg, sk.Kv4Cache(cfg, s["pages"], s["table"]), sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=c.get("nq", 1))
    return s["kept"]


def _own(s):
    import decode_attention_span_gb300 as sk

    c, h = s["c"], _kept(s, sk)
    if c["op"] == "logprobs":
        r = sk.token_logprobs(s["logits"], s["tokens"], h, n_top=c["top"], scale=c["scale"])
        out = {"logprob": r.logprob, "lse": r.lse, "entropy": r.entropy}
        if c["top"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    if c["op"] == "surprisal":
        return sk.surprisal(s["logits"], s["tokens"], h)
    if c["op"] == "rope":
        k = torch.empty(c["batch"], c["hkv"], c["ctx"], c["dim"], dtype=s["k"].dtype, device=DEV)
        q, _ = sk.rope(h, s["q"], s["k"], s["pos"], k_out=k.transpose(1, 2))
        return {"q": q, "k": k}
    cfg, cache, ws = h
    if c["op"] == "store":
        sk.kv4_append(cfg, cache, s["k"], s["v"], s["pos0"], ws)
        k, v = sk.kv4_read(cfg, cache, s["pos0"], c["ctx"], ws)
        return {"k": k, "v": v}
    o, lse = sk.kv4_attention(cfg, cache, s["q"], s["lens"], 1 / math.sqrt(128.0), ws)
    return {"out": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"logprobs": _plain_logprobs, "surprisal": _plain_surprisal, "rope": _plain_rope, "store": _plain_store,
            "attention": _plain_attention}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------- what a pass needs, and its exact answer
def work(case):
    c = case
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * SIZE[c["dtype"]] + c["rows"] * (8 + 12 + 8 * c["top"]), "flops": 6 * n}
    if c["op"] == "surprisal":
        n = c["batch"] * (c["ctx"] - 1) * c["vocab"]
        return {"bytes": n * SIZE[c["dtype"]] + c["batch"] * c["ctx"] * 12, "flops": 4 * n}
    if c["op"] == "rope":
        n = c["batch"] * c["ctx"] * (c["hq"] + c["hkv"])
        return {"bytes": n * c["dim"] * 2 * SIZE[c["dtype"]] + c["batch"] * c["ctx"] * 4, "flops": 3 * n * c["rot"]}
    rows = c["batch"] * c["ctx"] * c["hkv"]
    if c["op"] == "store":  # K and V in, their 4-bit form out and in again, K and V out
        return {"bytes": rows * (512 + 144 + 144 + 512), "flops": rows * 256 * 6}
    if c["ragged"] and c["batch"] > 1:
        rows = int(rows * (1 + 0.75 * (c["batch"] - 1)) / c["batch"])
    return {"bytes": rows * 144 + c["batch"] * c["nq"] * c["hq"] * (256 + 512 + 4), "flops": rows * (c["hq"] // c["hkv"]) * c["nq"] * 4 * 128}


def _exact_logits(x, tok, scale, chunk=64):
    """(logprob, lse, entropy) of rows in 64 bits, a few rows at a time."""
    got = []
    for i in range(0, x.shape[0], chunk):
        p = torch.log_softmax(x[i : i + chunk].double() * scale, -1)
        y = x[i : i + chunk].double() * scale
        got.append((p.gather(-1, tok[i : i + chunk, None])[:, 0], torch.logsumexp(y, -1), -(p.exp() * p).sum(-1)))
    return [torch.cat(t) for t in zip(*got)]


def _exact_freq(c):
    """The angle of each pair from its definition, one pair at a time, and the factor on the result."""
    d, f, orig, got = c["rot"], c["factor"], 8192, []
    for p in range(d // 2):
        base = c["base"] * (f ** (d / (d - 2)) if c["scaling"] == "ntk" and d > 2 else 1)
        a = math.exp(-2 * p / d * math.log(base))
        turns = orig * a / (2 * math.pi)  # how often the pair goes round in the original context
        if c["scaling"] == "linear":
            a /= f
        elif c["scaling"] == "banded":  # below one turn: stretched; above four: as it was; between: mixed
            keep = min(max((turns - 1) / 3, 0), 1)
            a = a * keep + a / f * (1 - keep)
        elif c["scaling"] == "parts":  # from the pair of 32 turns to the pair of one turn
            at = [d / 2 * math.log(orig / (2 * math.pi * n), c["base"]) for n in (32, 1)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
            slow = min(max((p - lo) / max(hi - lo, 0.001), 0), 1)
            a = a * (1 - slow) + a / f * slow
        got.append(a)
    return got, 1 + math.log(f) / 10 if c["scaling"] == "parts" and f > 1 else 1.0


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "logprobs":
        lp, lse, ent = _exact_logits(s["logits"], s["tokens"], c["scale"])
        out = {"logprob": lp, "lse": lse, "entropy": ent}
        if c["top"]:
            v, i = torch.sort(s["logits"].double() + 0.0, dim=-1, descending=True, stable=True)
            out["top_ids"] = i[:, : c["top"]].to(torch.int32)
            out["top_logprobs"] = v[:, : c["top"]] * c["scale"] - lse[:, None]
        return out
    if c["op"] == "surprisal":
        B, T = c["batch"], c["ctx"]
        lp = _exact_logits(s["logits"][:, :-1].reshape(B * (T - 1), -1), s["tokens"][:, 1:].reshape(-1), 1.0)[0]
        return torch.cat([torch.zeros(B, 1, dtype=torch.float64, device=DEV), -lp.view(B, T - 1)], 1)
    if c["op"] == "rope":
        inv, m = _exact_freq(c)
        inv = torch.tensor(inv, dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.full_like(inv, m).expand(*s["pos"].shape, -1).contiguous(), s["pos"].double()[..., None] * inv)[:, :, None]
        out = {}
        for n in "qk":
            x, r = s[n].double(), c["rot"]
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * turn
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2 : r].contiguous()) * turn
                y = torch.cat([z.real, z.imag], -1)
            out[n] = torch.cat([y, x[..., r:]], -1)
        out["k"] = out["k"].transpose(1, 2).contiguous()
        return out
    if c["op"] == "store":  # what the 4 bits stand for: z + s n, with z and s as bf16 by definition
        out = {}
        for n in "kv":
            x = s[n].double().reshape(*s[n].shape[:3], 2, 64)
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            z = lo.to(torch.bfloat16)
            z = torch.where(z.double() > lo, torch.nextafter(z, torch.full_like(z, -math.inf)), z).double()
            sc = ((hi - z) / 15).to(torch.bfloat16).double()
            code = torch.floor((x - z) / sc.clamp_min(1e-300) + 0.5)
            even = torch.where((x - z) / sc.clamp_min(1e-300) + 0.5 == code, torch.floor(code / 2) * 2, code)  # halves go to the even code
            out[n] = (z + sc * even.clamp(0, 15) * (sc > 0)).reshape(s[n].shape).transpose(1, 2).contiguous()
        return out
    B, H, nq, G = c["batch"], c["hkv"], c["nq"], c["hq"] // c["hkv"]
    if B * c["ctx"] * c["hq"] * nq > 2**26:
        return None
    out = torch.zeros(B, nq, c["hq"], 128, dtype=torch.float64, device=DEV)
    lse = torch.full((B, nq, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    # key j of the sequence sits in tile j // 16 of its pages, at row j % 16
    j = torch.arange(c["ctx"], device=DEV)
    r = j % 16
    d = torch.arange(128, device=DEV)
    kat = r[:, None] * 64 + (d % 64 // 16) * 16 + (d // 64) * 8 + (d % 16) // 2
    vat = 1024 + (r // 8 * 512)[:, None] + (d % 64 // 8) * 64 + (r % 8 // 2 * 16)[:, None] + (d // 64) * 8 + (d % 8 // 4) * 4 + (r % 2 * 2)[:, None] + (d % 4) // 2
    pat = 1024 + (r % 8 // 2 * 16 + (r // 8 * 2 + r % 2) * 4)[:, None] + d // 64 * 2
    lens = s["lens"].tolist()
    for b in range(B):
        tiles = s["pages"][s["table"][b].long()].view(-1, H, 4, TILE_BYTES).transpose(0, 1).reshape(H, -1, TILE_BYTES)[:, j // 16]
        par = tiles.view(torch.bfloat16).double()
        for h in range(H):
            kv = []
            for at, off in ((kat, 0), (vat, 64)):
                code = (tiles[h].gather(1, at).long() >> (d % 2 * 4)) & 15
                kv.append(par[h].gather(1, pat + off + 1) + par[h].gather(1, pat + off) * code)
            for t in range(nq):
                n = lens[b] - nq + 1 + t
                if n <= 0:
                    continue
                x = s["q"][b, t, h * G : h * G + G].double() @ kv[0][:n].T / math.sqrt(128.0)
                out[b, t, h * G : h * G + G] = torch.softmax(x, -1) @ kv[1][:n]
                lse[b, t, h * G : h * G + G] = torch.logsumexp(x, -1)
    return {"out": out, "lse": lse}
