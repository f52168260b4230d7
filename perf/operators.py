"""The operators between the verify GEMMs of one speculative-decoding step, as
cases to measure: attention of the verify rows over a paged key-value cache,
the head norm / rotary / cache append before it, and the penalties, biases and
grammar masks on the verify logits after the LM head.

`own` selects the side: False computes every case in elementary torch
operations, True calls this repository's entry points (include/vw4.h).
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One sequence, one new token, a short chat: the smallest attention call of
        # plain decoding; launch and load latency are all there is.
        dict(name="attn_one_token", op="attn", B=1, R=1, Hq=24, Hkv=4, D=256, page=16, kv="bf16",
             order="nhd", lo=517, hi=517, window=0, sinks=0),
        # A handful of sequences verifying 7 drafts each on the dense layer's heads
        # (6144 = 24 x 256 query, 1024 = 4 x 256 key columns), ragged contexts.
        dict(name="attn_verify8", op="attn", B=4, R=8, Hq=24, Hkv=4, D=256, page=64, kv="bf16",
             order="nhd", lo=1000, hi=9001, window=0, sinks=0),
        # A decode batch over long 8-bit caches, one token each.
        dict(name="attn_decode_long8", op="attn", B=32, R=1, Hq=32, Hkv=8, D=128, page=64,
             kv="e4m3", order="hnd", lo=2000, hi=32768, window=0, sinks=0),
        # The widest verify batch (16 rows) with 8 query heads a key head: 128 rows share a key.
        dict(name="attn_verify16_wide", op="attn", B=8, R=16, Hq=32, Hkv=4, D=128, page=32,
             kv="bf16", order="hnd", lo=3001, hi=16384, window=0, sinks=0),
        # A local layer: a window of 1024 and 4 first tokens that stay visible, 8-bit cache.
        dict(name="attn_window", op="attn", B=64, R=4, Hq=24, Hkv=4, D=256, page=16, kv="e4m3",
             order="nhd", lo=300, hi=20000, window=1024, sinks=4),
        # The rows of one sequence's verify batch into a bf16 cache, partial rotation.
        dict(name="append_one_seq", op="append", B=1, R=8, Hq=24, Hkv=4, D=256, page=16, kv="bf16",
             order="nhd", lo=4001, hi=4001, rot=64, pairs="half", norm=True, x="f32"),
        # The accept sweep's 256 sequences with 8 drafts each, into an 8-bit cache.
        dict(name="append_sweep", op="append", B=256, R=9, Hq=24, Hkv=4, D=256, page=16, kv="e4m3",
             order="hnd", lo=64, hi=600, rot=256, pairs="half", norm=True, x="f32"),
        # One sequence's 8 verify rows of the widest LM head: penalties and a few biases.
        dict(name="logits_one_seq", op="logits", B=1, R=8, V=262144, hist=2048, bias=32, mask=0.0),
        # A small batch with an odd vocabulary, every row under a grammar.
        dict(name="logits_odd", op="logits", B=5, R=3, V=32003, hist=301, bias=3, mask=0.5),
        # A batch where every row carries a grammar mask.
        dict(name="logits_grammar", op="logits", B=64, R=5, V=151936, hist=4096, bias=16, mask=0.3),
        # The accept sweep: 256 sequences, 8 drafts, every row penalized.
        dict(name="logits_sweep", op="logits", B=256, R=9, V=151936, hist=1024, bias=8, mask=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "logits"])
    if op == "logits":
        B, R = _log(rng, 1, 256), rng.randint(1, 9)
        V = rng.choice([_log(rng, 1000, 262144), 32000, 151936, 262144])
        B = max(1, min(B, 256 * 9 * 151936 // (R * V)))
        return dict(op=op, B=B, R=R, V=V, hist=_log(rng, 1, 8192), bias=rng.randint(0, 64),
                    mask=rng.choice([0.0, 0.01, 0.5, 0.9]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    D = rng.choice([64, 128, 256])
    c = dict(op=op, B=_log(rng, 1, 256), R=rng.randint(1, 16), Hq=Hkv * G, Hkv=Hkv, D=D,
             page=rng.choice([8, 16, 32, 64, 128]), kv=rng.choice(["bf16", "e4m3"]),
             order=rng.choice(["nhd", "hnd"]))
    if op == "append":
        c["B"] = min(c["B"], 256 * 9 // c["R"])
        c["lo"] = rng.randint(c["R"], 64)
        c["hi"] = _log(rng, c["lo"], 600)
        c.update(rot=rng.choice([0, D // 4, D // 2, D]), pairs=rng.choice(["half", "adjacent"]),
                 norm=rng.random() < 0.6, x=rng.choice(["f32", "bf16"]))
        return c
    if rng.random() < 0.5:
        c["R"] = 1
    hi = _log(rng, 17, 65536)
    c["B"] = max(1, min(c["B"], int(5e8) // (hi * Hkv * D)))
    c["lo"] = _log(rng, max(1, hi // 16), hi)
    c["hi"] = hi
    c["window"] = rng.choice([0, 0, _log(rng, 16, 8192)])
    c["sinks"] = rng.choice([0, 4, 33]) if c["window"] else 0
    return c


def _lens(c):
    """The cache lengths of a case's sequences, spread over [lo, hi]."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [max(1, round(lo * (hi / lo) ** ((b + 1) / B))) for b in range(B)]


def _seen(n, R, window, sinks):
    """(tokens that some verify row sees, sum over the rows of the tokens each sees)."""
    some, pairs = 0, 0
    for i in range(R):
        p = n - R + i
        if p < 0:
            continue
        if window == 0:
            pairs += p + 1
        else:
            lo = max(0, p - window + 1)
            pairs += p + 1 - lo + min(sinks, lo)
    first = max(0, n - R)
    lo = max(0, first - window + 1) if window else 0
    some = n - lo + min(sinks, lo)
    return some, pairs


def work(case):
    c = case
    if c["op"] == "logits":
        rows = c["B"] * c["R"]
        b = rows * c["V"] * 8.0 + rows * ((c["V"] + 15) // 16) * 4.0 + c["B"] * c["hist"] * 4.0
        b += c["B"] * c["bias"] * 8.0 + c["B"] * (c["R"] - 1) * 4.0
        if c["mask"]:
            b += rows * ((c["V"] + 31) // 32) * 4.0
        return {"bytes": b, "flops": rows * c["V"] * 2.0}
    es = 2 if c["kv"] == "bf16" else 1
    rows = c["B"] * c["R"]
    if c["op"] == "append":
        xs = 4 if c["x"] == "f32" else 2
        heads = c["Hq"] + 2 * c["Hkv"]
        b = rows * c["D"] * (heads * xs + c["Hq"] * 2.0 + 2.0 * c["Hkv"] * es) + c["B"] * 4.0
        return {"bytes": b, "flops": rows * c["D"] * heads * 6.0}
    some, pairs, pages = 0, 0, 0
    for n in _lens(c):
        s, p = _seen(n, c["R"], c["window"], c["sinks"])
        some, pairs, pages = some + s, pairs + p, pages + -(-s // c["page"])
    b = some * c["Hkv"] * c["D"] * 2.0 * es + rows * c["Hq"] * (c["D"] * 4.0 + 4.0)
    return {"bytes": b + pages * 4.0 + c["B"] * 4.0, "flops": pairs * c["Hq"] * c["D"] * 4.0}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _cache(c, g, seed, fill):
    """Pages in a random order; the tokens of a sequence are where its table says."""
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    cpu = torch.Generator().manual_seed(seed)
    n = torch.tensor(_lens(c))[torch.randperm(c["B"], generator=cpu)]
    per = (n + page - 1) // page
    total, cols = int(per.sum()), int(per.max())
    ids = torch.randperm(total, generator=cpu)
    table = torch.full((c["B"], cols), -1, dtype=torch.int64)
    at = torch.cumsum(per, 0) - per
    col = torch.arange(cols)[None, :]
    inside = col < per[:, None]
    table[inside] = ids[(at[:, None] + col)[inside]]
    shape = (total, page, Hkv, D) if c["order"] == "nhd" else (total, Hkv, page, D)
    pages = []
    for _ in range(2):
        t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        t.normal_(generator=g) if fill else t.zero_()
        if c["kv"] == "e4m3":
            # unit values stored under scales near 1/32: well inside the range of 448
            t = (t * 32).to(torch.float8_e4m3fn)
        pages.append(t if c["order"] == "nhd" else t.transpose(1, 2))
    scales = [None, None]
    if c["kv"] == "e4m3":
        scales = [(torch.rand(Hkv, device=DEV, generator=g) * 0.5 + 0.75) / 32 for _ in range(2)]
    return dict(k=pages[0], v=pages[1], table=table.to(torch.int32).to(DEV),
                lens=n.to(torch.int32).to(DEV), k_scale=scales[0], v_scale=scales[1])


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["op"] == "attn":
        s.update(_cache(c, g, seed, True))
        # queries about twice unit size: the softmax leans on some tokens, as after training
        s["q"] = (torch.randn(c["B"], c["R"], c["Hq"], c["D"], device=DEV, generator=g) * 2).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(c["D"])
    elif c["op"] == "append":
        s.update(_cache(c, g, seed, False))
        heads = c["Hq"] + 2 * c["Hkv"]
        x = torch.randn(c["B"] * c["R"], heads * c["D"], device=DEV, generator=g)
        s["x"] = x if c["x"] == "f32" else x.to(torch.bfloat16)
        j = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
        s["inv_freq"] = 1e6 ** (-2 * j / max(1, c["rot"]))
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"] = torch.randn(c["D"], device=DEV, generator=g) * 0.1 + 1
            s["k_norm"] = torch.randn(c["D"], device=DEV, generator=g) * 0.1 + 1
    else:
        B, R, V = c["B"], c["R"], c["V"]
        s["logits"] = torch.randn(B, R, V, device=DEV, generator=g) * 3

        def ids(*shape):  # token ids with a long tail: low ids are frequent
            u = torch.rand(*shape, device=DEV, generator=g, dtype=torch.float64)
            return (torch.exp(u * math.log(V)) - 1).long().clamp(0, V - 1).to(torch.int32)
        s["drafts"] = ids(B, R - 1)
        s["history"] = ids(B, c["hist"])
        u = torch.rand(2, B, device=DEV, generator=g)
        s["hist_len"] = (c["hist"] * (0.5 + 0.5 * u[0])).ceil().to(torch.int32).clamp(max=c["hist"])
        s["prompt_len"] = (s["hist_len"] * u[1]).to(torch.int32)
        u = torch.rand(3, B, device=DEV, generator=g)
        s["repetition"], s["presence"], s["frequency"] = 1 + u[0] * 0.3, u[1], u[2] * 0.5
        s["bias_ids"] = s["bias_vals"] = None
        if c["bias"]:  # distinct ids: a stride over the vocabulary
            first = torch.randint(0, V, (B, 1), device=DEV, generator=g)
            step = torch.arange(c["bias"], device=DEV) * max(1, V // (c["bias"] + 1))
            s["bias_ids"] = ((first + step) % V).to(torch.int32)
            s["bias_vals"] = torch.randn(B, c["bias"], device=DEV, generator=g) * 4
        s["mask"] = None
        if c["mask"]:  # allowed tokens come in runs of 64 ids, and single ones between them
            W = (V + 31) // 32
            run = torch.rand(B, R, (W + 1) // 2, device=DEV, generator=g) < c["mask"]
            words = torch.where(run.repeat_interleave(2, -1)[..., :W], -1, 0)
            one = torch.rand(B, R, W, device=DEV, generator=g) < 0.02
            bit = torch.randint(0, 31, (B, R, W), device=DEV, generator=g)
            words = words | torch.where(one, torch.ones_like(bit) << bit, 0)
            s["mask"] = words.to(torch.int32)
    if own:
        s["call"], s["out"] = _bind(s)
    return s


def _bind(s):
    """The handle that an engine keeps next to its buffers: the argument block of one call,
    with the output buffers and the workspace.  A call does all of the work."""
    import speculative_decode_verification_w4_gb300 as vw4
    c = s["case"]
    if c["op"] == "logits":
        out = torch.empty_like(s["logits"])
        bm = torch.empty(c["B"], c["R"], (c["V"] + 15) // 16, device=DEV)
        call = vw4.PreparedLogits(
            s["logits"], s["drafts"], history=s["history"], hist_len=s["hist_len"],
            prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
            frequency=s["frequency"], bias_ids=s["bias_ids"], bias_vals=s["bias_vals"],
            mask=s["mask"], out=out, block_max=bm)
        return call, (out, bm)
    cache = vw4.KVCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])
    q = torch.empty(c["B"], c["R"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
    if c["op"] == "append":
        call = vw4.PreparedAppend(s["x"], cache, s["lens"], c["R"], c["Hq"], inv_freq=s["inv_freq"],
                                  adjacent=c["pairs"] == "adjacent", q_norm=s["q_norm"],
                                  k_norm=s["k_norm"], eps=1e-6, q_out=q)
        return call, (q, s["k"], s["v"])
    lse = torch.empty(c["B"], c["R"], c["Hq"], device=DEV)
    call = vw4.PreparedAttn(s["q"], cache, s["lens"], scale=s["scale"], window=c["window"],
                            sinks=c["sinks"], out=q, lse=lse)
    return call, (q, lse)


def run(state):
    if own:
        state["call"]()
        return state["out"]
    return {"attn": _attn, "append": _append, "logits": _logits}[state["case"]["op"]](state)


# -------------------------------------------------------------- plain forms
def _attn(s):
    c = s["case"]
    B, R, Hq, Hkv, D, page = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page"))
    G, L = Hq // Hkv, s["table"].shape[1] * page
    rows = s["table"].clamp(min=0).long()

    def tokens(pages, scale):  # [B, Hkv, L, D] in 32 bits
        t = pages[rows].float().reshape(B, L, Hkv, D).transpose(1, 2)
        return t if scale is None else t * scale[None, :, None, None]
    q = s["q"].float().reshape(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    j = torch.arange(L, device=DEV)[None, None, :]
    p = (s["lens"][:, None] - R + torch.arange(R, device=DEV)[None, :])[:, :, None]
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    seen = seen[:, None, :, None, :]  # [B, 1, R, 1, L]
    sc = (q @ tokens(s["k"], s["k_scale"]).transpose(-1, -2) * s["scale"]).reshape(B, Hkv, R, G, L)
    sc = torch.where(seen, sc, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isinf(m), 0.0, m))
    z = e.sum(-1, keepdim=True)
    v = torch.where(seen.any(2).transpose(-1, -2), tokens(s["v"], s["v_scale"]), 0.0)
    o = (e.reshape(B, Hkv, R * G, L) @ v).reshape(B, Hkv, R, G, D)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (m + torch.log(z))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(torch.bfloat16)
    return o, lse.permute(0, 2, 1, 3).reshape(B, R, Hq)


def _append(s):
    c = s["case"]
    B, R, Hq, Hkv, D, page, rot = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page", "rot"))
    x = s["x"].float().reshape(B, R, Hq + 2 * Hkv, D)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    pos = (s["lens"][:, None] - R + torch.arange(R, device=DEV)[None, :]).long()  # [B, R]
    angle = pos[..., None].double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]

    def turn(t, w):
        if w is not None:
            t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        if rot == 0:
            return t
        h = rot // 2
        a, b = (t[..., :h], t[..., h:rot]) if c["pairs"] == "half" else (t[..., 0:rot:2], t[..., 1:rot:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([a, b], -1) if c["pairs"] == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([r, t[..., rot:]], -1)
    q, k = turn(q, s["q_norm"]), turn(k, s["k_norm"])
    at = torch.gather(s["table"].long(), 1, pos.clamp(min=0) // page), pos.clamp(min=0) % page
    keep = pos >= 0
    for t, pages, scale in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        if scale is not None:
            t = (t / scale[:, None]).clamp(-448, 448)
        pages[at[0][keep], at[1][keep]] = t[keep].to(pages.dtype)
    return q.to(torch.bfloat16), s["k"], s["v"]


def _logits(s):
    c = s["case"]
    B, R, V = c["B"], c["R"], c["V"]
    i = torch.arange(c["hist"], device=DEV)[None, :]
    ids = s["history"].long()
    valid = (i < s["hist_len"][:, None]).int()
    made = valid * (i >= s["prompt_len"][:, None]).int()
    zero = torch.zeros(B, V, dtype=torch.int32, device=DEV)
    known = zero.scatter_add(1, ids, valid)[:, None, :]
    count = zero.scatter_add(1, ids, made)[:, None, :]
    if R > 1:  # row i also counts drafts 0 .. i - 1
        before = torch.zeros(B, R, V, dtype=torch.int32, device=DEV)
        tri = torch.ones(R, R - 1, dtype=torch.int32, device=DEV).tril(-1)[None].expand(B, R, R - 1)
        before.scatter_add_(2, s["drafts"].long()[:, None, :].expand(B, R, R - 1), tri.contiguous())
        known, count = known + before, count + before
    x = s["logits"]
    r = s["repetition"][:, None, None]
    x = torch.where(known > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_ids"] is not None:
        bias = torch.zeros(B, V, device=DEV)
        bias.scatter_(1, s["bias_ids"].long(), s["bias_vals"])
        x = x + bias[:, None, :]
    if s["mask"] is not None:
        v = torch.arange(V, device=DEV)
        x = torch.where((s["mask"][:, :, v >> 5] >> (v & 31)) & 1 == 1, x, float("-inf"))
    pad = torch.full((B, R, -V % 16), float("-inf"), device=DEV)
    return x, torch.cat([x, pad], -1).reshape(B, R, -1, 16).amax(-1)


# ---------------------------------------------------------- 64-bit definition
def exact(case, seed):
    global own
    mine, own = own, False
    s = prepare(case, seed)
    own = mine
    f = {"attn": _exact_attn, "append": _exact_append, "logits": _exact_logits}[case["op"]]
    return f(case, s)


def _exact_attn(c, s):
    B, R, Hq, Hkv, D, page = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, R, Hq), float("-inf"), dtype=torch.float64, device=DEV)
    lens, table = s["lens"].tolist(), s["table"].tolist()
    for b in range(B):
        n = lens[b]
        used = torch.tensor(table[b][:-(-n // page)], device=DEV)
        k = s["k"][used].double().flatten(0, 1)[:n]
        v = s["v"][used].double().flatten(0, 1)[:n]
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        for i in range(R):
            p = n - R + i
            if p < 0:
                continue
            lo = max(0, p - c["window"] + 1) if c["window"] else 0
            sel = list(range(min(c["sinks"], lo))) if lo else []
            ki = torch.cat([k[:len(sel)], k[lo:p + 1]]) if sel else k[lo:p + 1]
            vi = torch.cat([v[:len(sel)], v[lo:p + 1]]) if sel else v[lo:p + 1]
            q = s["q"][b, i].double().reshape(Hkv, G, D)
            a = torch.einsum("hgd,thd->hgt", q, ki) / math.sqrt(D)
            top = a.max(-1, keepdim=True).values
            w = (a - top).exp()
            tot = w.sum(-1, keepdim=True)
            out[b, i] = torch.einsum("hgt,thd->hgd", w / tot, vi).reshape(Hq, D)
            lse[b, i] = (top + tot.log()).reshape(Hq)
    return out, lse


def _exact_append(c, s):
    B, R, Hq, Hkv, D, page, rot = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page", "rot"))
    K, V = s["k"].double(), s["v"].double()
    Q = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=DEV)
    X = s["x"].double()
    b, i = torch.meshgrid(torch.arange(B, device=DEV), torch.arange(R, device=DEV), indexing="ij")
    b, i = b.flatten(), i.flatten()
    p = s["lens"].long()[b] - R + i
    ok = p >= 0
    heads = X.view(B * R, Hq + 2 * Hkv, D)
    M = torch.eye(D, dtype=torch.float64, device=DEV).repeat(B * R, 1, 1)
    for j in range(rot // 2):
        t = p.double() * s["inv_freq"][j]
        u, w = (j, j + rot // 2) if c["pairs"] == "half" else (2 * j, 2 * j + 1)
        M[:, u, u], M[:, u, w], M[:, w, u], M[:, w, w] = t.cos(), -t.sin(), t.sin(), t.cos()

    def normed(h, w):
        if w is None:
            return h
        return h / ((h ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
    q = torch.einsum("nij,nhj->nhi", M, normed(heads[:, :Hq], s["q_norm"]))
    k = torch.einsum("nij,nhj->nhi", M, normed(heads[:, Hq:Hq + Hkv], s["k_norm"]))
    v = heads[:, Hq + Hkv:]
    Q[b, i] = q
    pages = s["table"].long()[b, (p.clamp(min=0) // page)]
    for src, dst, scale in ((k, K, s["k_scale"]), (v, V, s["v_scale"])):
        if scale is not None:
            src = (src / scale.double()[:, None]).clamp(-448, 448)
        dst[pages[ok], (p % page)[ok]] = src[ok]
    return Q, K, V


def _exact_logits(c, s):
    B, R, V = c["B"], c["R"], c["V"]
    X = s["logits"].double()
    hist, drafts = s["history"].long(), s["drafts"].long()
    hl, pl = s["hist_len"].tolist(), s["prompt_len"].tolist()
    rep, pre, fre = (s[k].double() for k in ("repetition", "presence", "frequency"))
    for b in range(B):
        for i in range(R):
            tokens = torch.cat([hist[b, :hl[b]], drafts[b, :i]])
            ids, n = torch.unique(torch.cat([hist[b, pl[b]:hl[b]], drafts[b, :i]]), return_counts=True)
            u = torch.unique(tokens)
            l = X[b, i, u]
            X[b, i, u] = torch.where(l > 0, l / rep[b], l * rep[b])
            X[b, i, ids] -= fre[b] * n + pre[b]
    if s["bias_ids"] is not None:
        bi = s["bias_ids"].long()[:, None, :].expand(B, R, c["bias"])
        X.scatter_add_(2, bi, s["bias_vals"].double()[:, None, :].expand(B, R, c["bias"]))
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=DEV)) & 1
        X[bits.flatten(-2)[..., :V] == 0] = -math.inf
    M = X.new_full((B, R, (V + 15) // 16), -math.inf)
    for k in range(16):
        t = X[..., k::16]
        M[..., :t.shape[-1]] = torch.maximum(M[..., :t.shape[-1]], t)
    return X, M
