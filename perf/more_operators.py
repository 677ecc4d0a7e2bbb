"""Cases of the operators of a step with drafted tokens: attention of a tree of drafted tokens over
the 4-bit cache and keeping the branch that is accepted, and the log-probabilities of tokens from a
model's last states without keeping logits, with their gradient.  Plain forms are elementary torch;
with ``own`` the calls are the framework's."""

import math
import random

import torch

own = False

DEV = "cuda"
PAGE, TILE, TILE_BYTES, PAGE_BYTES = 64, 16, 2304, 9216
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the next token of one sequence: its log-probability, straight from the last state (latency)
        dict(name="score 1x32000 d4096", op="score", rows=1, vocab=32000, dim=4096, dtype="bf16", scale=1.0),
        # drafted tokens of a served batch, scored before any is accepted
        dict(name="score 128x128000 d4096", op="score", rows=128, vocab=128000, dim=4096, dtype="bf16", scale=1.0),
        # an evaluation at a temperature: odd numbers of rows and tokens, a narrow model
        dict(name="score 1003x50021 d1000 f16", op="score", rows=1003, vocab=50021, dim=1000, dtype="fp16", scale=0.75),
        # the boundary signal of a prefill chunk, in the layout the span build takes
        dict(name="surprisal 1x8192x128000 d4096", op="surprisal", batch=1, ctx=8192, vocab=128000, dim=4096, dtype="bf16"),
        # a training step's loss with its gradients: a few short rows
        dict(name="train 96x32000 d1024", op="train", rows=96, vocab=32000, dim=1024, dtype="bf16"),
        # odd sizes, f16
        dict(name="train 1021x50021 d2000 f16", op="train", rows=1021, vocab=50021, dim=2000, dtype="fp16"),
        # a full micro-batch against a large vocabulary
        dict(name="train 4096x128000 d4096", op="train", rows=4096, vocab=128000, dim=4096, dtype="bf16"),
        # one short conversation, a small tree: latency
        dict(name="tree 1x2000 n16", op="tree", batch=1, ctx=2000, hq=32, hkv=8, nodes=16, dtype="bf16"),
        # a served batch, seven query heads to a KV head, lengths and trees of their own
        dict(name="tree 8x16384 n26 f16", op="tree", batch=8, ctx=16384, hq=28, hkv=4, nodes=26, dtype="fp16"),
        # one long context, the widest tree
        dict(name="tree 1x131072 n64", op="tree", batch=1, ctx=131072, hq=32, hkv=8, nodes=64, dtype="bf16"),
        # the accepted branch of one sequence, moved up behind the prefix and read back
        dict(name="keep 1x16", op="keep", batch=1, ctx=4000, hkv=8, nodes=16, most=4),
        # of a large batch of wide trees
        dict(name="keep 256x64", op="keep", batch=256, ctx=1000, hkv=8, nodes=64, most=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "surprisal", "train", "train", "tree", "tree", "tree", "keep"])
    if op in ("score", "surprisal", "train"):
        vocab, dim = _log(rng, 300, 160000), 8 * _log(rng, 8, 800)
        most = max(2, min(8192, 300_000_000 // vocab, int((1.0 if op == "train" else 2.0) * 10**12) // vocab // dim))
        c = dict(op=op, vocab=vocab, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        if op == "surprisal":
            batch = rng.randint(1, 4)
            return dict(c, batch=batch, ctx=max(2, _log(rng, 2, max(3, most)) // batch))
        if op == "train":
            return dict(c, rows=_log(rng, 1, most))
        return dict(c, rows=_log(rng, 1, most), scale=rng.choice([1.0, 0.5, 0.75, 1.25]))
    hkv = rng.choice([1, 2, 4, 8])
    if op == "keep":
        nodes = rng.randint(2, 64)
        return dict(op=op, batch=_log(rng, 1, 256), ctx=_log(rng, 1, 2000), hkv=hkv, nodes=nodes, most=rng.randint(1, max(1, nodes // 2)))
    batch, nodes = rng.randint(1, 16), rng.choice([1, 2, 5, 8, 16, 25, 32, 48, 61, 64])
    return dict(op=op, batch=batch, ctx=_log(rng, 1, max(2, min(100_000, 30_000_000 // nodes // batch // hkv, 2_000_000 // batch // hkv))), hq=hkv * rng.choice([1, 2, 4, 7, 8]),
                hkv=hkv, nodes=nodes, dtype=rng.choice(["bf16", "bf16", "fp16"]))


# ---------------------------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _states(c, g):
    """Last states, the vocabulary matrix and the tokens: logits spread by 2.5, the token that comes
    stands out by up to ten."""
    shape = (c["batch"], c["ctx"]) if c["op"] == "surprisal" else (c["rows"],)
    V, D = c["vocab"], c["dim"]
    w = torch.empty(V, D, dtype=DT[c["dtype"]], device=DEV).normal_(0, 2.5 / math.sqrt(D), generator=g)
    tok = torch.randint(0, V, shape, generator=g, device=DEV)
    at = torch.roll(tok, -1, 1) if c["op"] == "surprisal" else tok
    x = torch.randn(*shape, D, generator=g, device=DEV)
    up = torch.rand(*shape, 1, generator=g, device=DEV) * 10
    row = w[at].float()
    x = (x + up * row / (row * row).sum(-1, keepdim=True)).to(DT[c["dtype"]])
    if c["op"] == "train":  # one row in twenty is padding
        tok = torch.where(torch.rand(shape, generator=g, device=DEV) < 0.05, -1, tok)
    return {"states": x, "weight": w, "tokens": tok}


def _lengths(c, g):
    """Tokens before the drafted ones: the full length, in a batch less of it for most sequences."""
    less = torch.rand(c["batch"], generator=g, device=DEV) * (c["ctx"] // 2)
    return (c["ctx"] - less.to(torch.int32) * (torch.arange(c["batch"], device=DEV) > 0)).to(torch.int32).contiguous()


def _pages(c, g):
    """A pool of pages in any order: codes of any value, scales and zero points as an append leaves them."""
    B, H = c["batch"], c["hkv"]
    mp = -(-(c["ctx"] + c["nodes"]) // PAGE)
    n = B * mp + 3
    pages = torch.randint(0, 256, (n, H, PAGE // TILE, TILE_BYTES), dtype=torch.uint8, generator=g, device=DEV)
    sz = torch.rand(n, H, PAGE // TILE, 64, 2, generator=g, device=DEV)
    sz[..., 0] = sz[..., 0] * 0.25 + 0.1
    sz[..., 1] = sz[..., 1] * 0.6 - 8 * sz[..., 0]
    pages[..., 2048:] = sz.to(torch.bfloat16).view(torch.uint8).view(n, H, PAGE // TILE, 256)
    table = torch.randperm(n, generator=g, device=DEV)[: B * mp].to(torch.int32).view(B, mp).contiguous()
    return {"pages": pages.view(n, H, PAGE_BYTES), "table": table}


def _trees(c, seed):
    """Bit j of mask[b][i]: drafted token j is i itself or one of its ancestors."""
    rng, masks = random.Random(seed), []
    for _ in range(c["batch"]):
        m = []
        for i in range(c["nodes"]):
            up = rng.randint(max(-1, i - 12), i - 1)
            m.append((m[up] if up >= 0 else 0) | 1 << i)
        masks.append([x - (1 << 64) if x >> 63 else x for x in m])
    return torch.tensor(masks, dtype=torch.int64, device=DEV)


def _branches(c, seed):
    """The drafted tokens that are kept, in order, and how many.  A token that moves comes from behind
    the places that are filled, so that a pass can be made again on what it leaves."""
    rng, keep, n = random.Random(seed), [], []
    for _ in range(c["batch"]):
        k = rng.randint(0, c["most"])
        same = rng.randint(0, k)
        far = sorted(rng.sample(range(k, c["nodes"]), min(k - same, c["nodes"] - k)))
        row = list(range(k - len(far))) + far
        keep.append(row + [0] * (c["most"] - k))
        n.append(k)
    return torch.tensor(keep, dtype=torch.int32, device=DEV), torch.tensor(n, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    if c["op"] in ("score", "surprisal", "train"):
        s.update(_states(c, g))
        if c["op"] == "train":
            n = max(1, int((s["tokens"] >= 0).sum()))
            s["grad"] = torch.full((c["rows"],), -1.0 / n, device=DEV)  # of the mean of -log p
        return s
    s.update(_pages(c, g))
    s["first"] = _lengths(c, g)
    if c["op"] == "tree":
        s["q"] = torch.randn(c["batch"], c["nodes"], c["hq"], 128, generator=g, device=DEV).to(DT[c["dtype"]])
        s["mask"] = _trees(c, seed)
    else:
        s["keep"], s["n_keep"] = _branches(c, seed)
        s["k"], s["v"] = (torch.zeros(c["batch"], c["hkv"], c["most"], 128, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    return s


# ---------------------------------------------------------------------------------- the plain forms
def _logits(s, scale):
    c = s["c"]
    return (s["states"].view(-1, c["dim"]).float() @ s["weight"].float().T) * scale


def _logprob_parts(x, tok):
    """(log p of the tokens, log-sum-exp) of rows of logits."""
    m = x.amax(-1, keepdim=True)
    tot = torch.exp(x - m).sum(-1)
    at = torch.gather(x, -1, tok.clamp(min=0)[:, None])[:, 0]
    lse = m[:, 0] + torch.log(tot)
    return torch.where(tok >= 0, at - m[:, 0] - torch.log(tot), 0.0), lse


def _plain_score(s):
    lp, lse = _logprob_parts(_logits(s, s["c"]["scale"]), s["tokens"])
    return {"logprob": lp, "lse": lse}


def _plain_surprisal(s):
    c = s["c"]
    lp, _ = _logprob_parts(_logits(s, 1.0), torch.roll(s["tokens"], -1, 1).view(-1))
    return torch.cat([torch.zeros(c["batch"], 1, device=DEV), -lp.view(c["batch"], -1)[:, :-1]], 1)


def _plain_train(s):
    x, tok = _logits(s, 1.0), s["tokens"]
    lp, lse = _logprob_parts(x, tok)
    g = torch.where(tok >= 0, s["grad"], 0.0)[:, None]
    d = torch.exp(x - lse[:, None]) * -g
    d.scatter_add_(1, tok.clamp(min=0)[:, None], g)
    return {"logprob": lp, "lse": lse, "d_states": (d @ s["weight"].float()).to(s["states"].dtype),
            "d_weight": (d.T @ s["states"].float()).to(s["weight"].dtype)}


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
    return tuple((w[i, ..., 1:] + w[i, ..., :1] * x).reshape(B, H, nt * 16, 128) for i, x in ((0, k), (1, v)))


def _plain_tree(s):
    c = s["c"]
    B, H, n, G = c["batch"], c["hkv"], c["nodes"], c["hq"] // c["hkv"]
    k, v = (x[:, :, : c["ctx"] + n] for x in _unpacked(s, torch.float32))
    q = s["q"].float().view(B, n, H, G, 128).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, 128)
    x = (q @ k.transpose(-1, -2)).view(B, H, n, G, -1) * (1 / math.sqrt(128.0))
    at = torch.arange(c["ctx"] + n, device=DEV)[None] - s["first"][:, None]  # the drafted token that a key is
    bit = s["mask"][:, :, None] >> at.clamp(0, 63)[:, None] & 1
    seen = ((at < 0)[:, None] | ((at < n)[:, None] & (bit == 1)))[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    tot = e.sum(-1, keepdim=True)
    o = (e / torch.where(tot > 0, tot, 1.0)).view(B, H, n * G, -1) @ v
    o = o.view(B, H, n, G, 128).permute(0, 2, 1, 3, 4).reshape(B, n, c["hq"], 128)
    lse = (m + torch.log(tot))[..., 0].permute(0, 2, 1, 3).reshape(B, n, c["hq"])
    return {"out": o, "lse": lse}


def _plain_keep(s):
    """The kept tokens' values, in order; zero behind them."""
    c = s["c"]
    pos = s["first"][:, None] + s["keep"]
    tile = torch.gather(s["table"].long(), 1, pos.long() // PAGE)
    t = {"c": dict(c, batch=c["batch"] * c["most"]), "pages": s["pages"], "table": tile.view(-1, 1)}
    got, row = _unpacked(t, torch.float32), (pos.long() % PAGE).view(-1, 1, 1, 1).expand(-1, c["hkv"], 1, 128)
    held = (torch.arange(c["most"], device=DEV)[None] < s["n_keep"][:, None])[:, None, :, None]
    out = {}
    for name, x in zip("kv", got):
        x = torch.gather(x, 2, row).view(c["batch"], c["most"], c["hkv"], 128).transpose(1, 2)
        out[name] = torch.where(held, x, 0.0).to(torch.bfloat16).contiguous()
    return out


# ---------------------------------------------------------------------------------- the framework's calls
def _kept(s, sk):
    """What a program makes once and keeps: configuration, workspace, cache handle."""
    if "kept" not in s:
        c = s["c"]
        if c["op"] in ("score", "surprisal", "train"):
            rows = c["batch"] * c["ctx"] if c["op"] == "surprisal" else c["rows"]
            s["kept"] = sk.StatesWorkspace(rows, c["vocab"], c["dim"], backward=c["op"] == "train")
        else:
            cfg = sk.Config(c["batch"], c.get("hq", c["hkv"]), c["hkv"], 0, 0, 64)
            s["kept"] = cfg, sk.Kv4Cache(cfg, s["pages"], s["table"]), sk.Workspace(cfg, which=sk.SEKV_CALL_KV4, ctx_len=c["nodes"])
    return s["kept"]


def _own(s):
    import decode_attention_span_gb300 as sk

    c, h = s["c"], _kept(s, sk)
    if c["op"] == "score":
        r = sk.states_logprobs(s["states"], s["weight"], s["tokens"], h, scale=c["scale"])
        return {"logprob": r.logprob, "lse": r.lse}
    if c["op"] == "surprisal":
        return sk.states_surprisal(s["states"], s["weight"], s["tokens"], h)
    if c["op"] == "train":
        r = sk.states_logprobs(s["states"], s["weight"], s["tokens"], h)
        dx, dw = sk.states_logprobs_backward(s["states"], s["weight"], s["tokens"], r.lse, s["grad"], h)
        return {"logprob": r.logprob, "lse": r.lse, "d_states": dx, "d_weight": dw}
    cfg, cache, ws = h
    if c["op"] == "tree":
        o, lse = sk.kv4_tree_attention(cfg, cache, s["q"], s["first"], s["mask"], 1 / math.sqrt(128.0), ws)
        return {"out": o, "lse": lse}
    sk.kv4_keep(cfg, cache, s["first"], s["keep"], s["n_keep"], ws)
    k, v = sk.kv4_read(cfg, cache, s["first"], c["most"], ws, n_valid=s["n_keep"], out=(s["k"], s["v"]))
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"score": _plain_score, "surprisal": _plain_surprisal, "train": _plain_train, "tree": _plain_tree, "keep": _plain_keep}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------- what a pass needs, and its exact answer
def work(case):
    c = case
    if c["op"] in ("score", "surprisal", "train"):
        n, V, D = c.get("rows", c.get("batch", 1) * c.get("ctx", 1)), c["vocab"], c["dim"]
        both = (n + V) * D * 2
        # the gradient needs the logits' product, which the loss made, and two more
        return {"bytes": both * (2 if c["op"] == "train" else 1) + n * 16, "flops": n * V * D * (6 if c["op"] == "train" else 2)}
    if c["op"] == "keep":  # a kept token's codes and scales in and out, and its values
        n = c["batch"] * c["hkv"] * c["most"] // 2
        return {"bytes": n * (144 * 2 + 512), "flops": n * 256 * 2}
    rows = c["batch"] * (c["ctx"] + c["nodes"]) * c["hkv"]
    if c["batch"] > 1:
        rows = int(rows * (1 + 0.75 * (c["batch"] - 1)) / c["batch"])
    return {"bytes": rows * 144 + c["batch"] * c["nodes"] * c["hq"] * (256 + 512 + 4), "flops": rows * (c["hq"] // c["hkv"]) * c["nodes"] * 4 * 128}


def _exact_states(s):
    c = s["c"]
    D, V = c["dim"], c["vocab"]
    x, w = s["states"].reshape(-1, D), s["weight"].double()
    tok = (torch.roll(s["tokens"], -1, 1) if c["op"] == "surprisal" else s["tokens"]).reshape(-1)
    lp, lse, dx = [], [], []
    dw = torch.zeros(V, D, dtype=torch.float64, device=DEV) if c["op"] == "train" else None
    for i in range(0, x.shape[0], 512):
        h, t = x[i : i + 512].double(), tok[i : i + 512]
        y = torch.nn.functional.linear(h, w) * c.get("scale", 1.0)
        p = torch.log_softmax(y, -1)
        lse.append(torch.logsumexp(y, -1))
        lp.append(torch.where(t < 0, 0.0, p[torch.arange(len(t), device=DEV), t]))
        if dw is not None:
            p = p.exp()
            p[torch.arange(len(t), device=DEV), t] -= 1
            p *= torch.where(t < 0, 0.0, -s["grad"][i : i + 512].double())[:, None]
            dx.append(p @ w)
            dw.addmm_(p.T, h)
    return torch.cat(lp), torch.cat(lse), torch.cat(dx) if dx else None, dw


def _exact_places():
    """Of row r of a tile and dimension d: the byte of K's code, of V's, and the 16-bit word of the scale."""
    r, d = torch.arange(16, device=DEV)[:, None], torch.arange(128, device=DEV)[None]
    kat = r * 64 + d % 64 // 16 * 16 + d // 64 * 8 + d % 16 // 2
    vat = 1024 + r // 8 * 512 + d % 64 // 8 * 64 + r % 8 // 2 * 16 + d // 64 * 8 + d % 8 // 4 * 4 + r % 2 * 2 + d % 4 // 2
    pat = 1024 + r % 8 // 2 * 16 + (r // 8 * 2 + r % 2) * 4 + d // 64 * 2
    return (kat, pat), (vat, pat + 64)


def _exact_rows(s, b, h, pos):
    """K and V of the tokens `pos` of a sequence, in 64 bits."""
    tiles = s["pages"][s["table"][b].long()[pos // PAGE], h].view(-1, PAGE // TILE, TILE_BYTES)
    tiles = tiles[torch.arange(len(pos), device=DEV), pos % PAGE // TILE]
    par, odd, got = tiles.view(torch.bfloat16).double(), torch.arange(128, device=DEV) % 2, []
    for at, sz in _exact_places():
        code = (tiles.gather(1, at[pos % TILE]).long() >> (odd * 4)) & 15
        got.append(par.gather(1, sz[pos % TILE] + 1) + par.gather(1, sz[pos % TILE]) * code)
    return got


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("score", "surprisal", "train"):
        if work(c)["flops"] * (4 / 3 if c["op"] == "train" else 1) > 6e12:
            return None
        s = prepare(case, seed)
        lp, lse, dx, dw = _exact_states(s)
        if c["op"] == "surprisal":
            return torch.cat([torch.zeros(c["batch"], 1, dtype=torch.float64, device=DEV), -lp.view(c["batch"], -1)[:, :-1]], 1)
        return {"logprob": lp, "lse": lse} if dw is None else {"logprob": lp, "lse": lse, "d_states": dx, "d_weight": dw}
    if c["op"] == "tree" and c["batch"] * c["ctx"] * c["hq"] * c["nodes"] > 2**27:
        return None
    s = prepare(case, seed)
    B, H, n, first = c["batch"], c["hkv"], c["nodes"], s["first"].tolist()
    if c["op"] == "keep":
        out = {x: torch.zeros(B, H, c["most"], 128, dtype=torch.float64, device=DEV) for x in "kv"}
        many = s["n_keep"].tolist()
        for b in range(B):
            pos = (first[b] + s["keep"][b, : many[b]]).long()
            for h in range(H):
                out["k"][b, h, : many[b]], out["v"][b, h, : many[b]] = _exact_rows(s, b, h, pos)
        return out
    G = c["hq"] // H
    out = torch.zeros(B, n, c["hq"], 128, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        bits = [[m >> j & 1 == 1 for j in range(n)] for m in s["mask"][b].tolist()]
        hidden = torch.cat([torch.zeros(n, first[b], dtype=torch.bool, device=DEV), ~torch.tensor(bits, device=DEV)], 1)
        for h in range(H):
            k, v = _exact_rows(s, b, h, torch.arange(first[b] + n, device=DEV))
            x = torch.einsum("igd,td->igt", s["q"][b, :, h * G : h * G + G].double(), k) / math.sqrt(128.0)
            x.masked_fill_(hidden[:, None], -math.inf)
            out[b, :, h * G : h * G + G] = torch.softmax(x, -1) @ v
            lse[b, :, h * G : h * G + G] = torch.logsumexp(x, -1)
    return {"out": out, "lse": lse}
