"""A paged key-value cache held in 4 bits, and what else a speculative-decoding step
does with its cache and its committed tokens, as cases to measure:

  append4   head norm, rotation and rounding of the verify rows into the 4-bit cache,
            then the new rows read back (a read returns what the cache stands for)
  attn4     attention of the verify rows over the 4-bit cache
  read4     tokens of the 4-bit cache as bf16 keys and values
  pages     lengths after an accept, pages for the next rows, their slots
  logprobs  log probabilities of the committed tokens, entropy, best alternatives

`own` selects the side: False computes every case in elementary torch operations,
True calls this repository's entry points (include/vw4.h).

The 4-bit format is nvfp4: e2m1 values, the even element of a pair in the low nibble,
an e4m3 scale for each 16 elements of a head, one fp32 scale a head.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One sequence, one new token, a short chat: the smallest call of plain decoding.
        dict(name="attn4_one_token", op="attn4", B=1, R=1, Hq=24, Hkv=4, D=256, page=16,
             order="nhd", lo=517, hi=517, window=0, sinks=0),
        # A handful of sequences verifying 7 drafts each on the dense layer's heads, ragged.
        dict(name="attn4_verify8", op="attn4", B=4, R=8, Hq=24, Hkv=4, D=256, page=64,
             order="nhd", lo=1000, hi=9001, window=0, sinks=0),
        # A decode batch over long caches, one token each: where 4 bits pay the most.
        dict(name="attn4_decode_long", op="attn4", B=32, R=1, Hq=32, Hkv=8, D=128, page=64,
             order="hnd", lo=2000, hi=32768, window=0, sinks=0),
        # A local layer: a window of 1024 and 4 first tokens that stay visible.
        dict(name="attn4_window", op="attn4", B=64, R=4, Hq=24, Hkv=4, D=256, page=16,
             order="nhd", lo=300, hi=20000, window=1024, sinks=4),
        # The rows of one sequence's verify batch, partial rotation.
        dict(name="append4_one_seq", op="append4", B=1, R=8, Hq=24, Hkv=4, D=256, page=16,
             order="nhd", lo=4001, hi=4001, rot=64, pairs="half", norm=True, x="f32"),
        # The accept sweep's 256 sequences with 8 drafts each.
        dict(name="append4_sweep", op="append4", B=256, R=9, Hq=24, Hkv=4, D=256, page=16,
             order="hnd", lo=64, hi=600, rot=256, pairs="half", norm=True, x="f32"),
        # The context of two short chats as contiguous rows, for a pass over a prompt's chunk.
        dict(name="read4_short", op="read4", B=2, n=517, Hkv=4, D=256, page=16, order="nhd",
             lo=300, hi=700),
        # Long contexts of a batch, read back for a pass that takes bf16 rows.
        dict(name="read4_long", op="read4", B=16, n=8192, Hkv=8, D=128, page=64, order="hnd",
             lo=4000, hi=9000),
        # The step of a small batch after its accept: most sequences stay on their pages.
        dict(name="pages_step", op="pages", B=16, R=8, page=16, lo=100, hi=5000, new=0.0, prompt=1),
        # A full server: 4096 places, of which an eighth ended and an eighth take a new prompt.
        dict(name="pages_prompts", op="pages", B=4096, R=9, page=16, lo=64, hi=4096, new=0.125,
             prompt=8192),
        # One sequence's 8 verify rows of the widest LM head, 20 alternatives.
        dict(name="logprobs_one_seq", op="logprobs", B=1, R=8, V=262144, top=20, keep=1.0,
             x="f32", masked=0.0),
        # The accept sweep: 256 sequences with 8 drafts, whose committed rows are read.
        dict(name="logprobs_sweep", op="logprobs", B=256, R=9, V=151936, top=5, keep=0.6,
             x="f32", masked=0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn4", "attn4", "append4", "read4", "pages", "logprobs"])
    if op == "logprobs":
        B, R = _log(rng, 1, 256), rng.randint(1, 9)
        V = rng.choice([_log(rng, 1000, 262144), 32003, 151936, 262144])
        B = max(1, min(B, 256 * 9 * 151936 // (2 * R * V)))
        return dict(op=op, B=B, R=R, V=V, top=rng.randint(0, 32), keep=rng.choice([0.3, 0.6, 1.0]),
                    x=rng.choice(["f32", "f32", "bf16"]), masked=rng.choice([0.0, 0.5, 0.99]))
    if op == "pages":
        lo = _log(rng, 1, 2000)
        return dict(op=op, B=_log(rng, 1, 4096), R=rng.randint(1, 16),
                    page=rng.choice([8, 16, 32, 64, 128]), lo=lo, hi=_log(rng, lo, 4096),
                    new=rng.choice([0.0, 0.02, 0.1]), prompt=_log(rng, 16, 8192))
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 256])
    c = dict(op=op, B=_log(rng, 1, 256), Hkv=Hkv, D=D, page=rng.choice([8, 16, 32, 64, 128]),
             order=rng.choice(["nhd", "hnd"]))
    if op == "read4":
        c["n"] = _log(rng, 1, 8192)
        c["B"] = max(1, min(c["B"], 16 * 8192 * 8 * 128 // (c["n"] * Hkv * D)))
        c["hi"] = _log(rng, max(1, c["n"] // 2), 2 * c["n"])
        c["lo"] = _log(rng, max(1, c["hi"] // 4), c["hi"])
        return c
    c.update(R=rng.randint(1, 16), Hq=Hkv * rng.choice([1, 2, 3, 4, 6, 8]))
    if op == "append4":
        c["B"] = max(1, min(c["B"], 256 * 9 // c["R"]))
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
    """The lengths of a case's sequences, spread over [lo, hi]."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [max(1, round(lo * (hi / lo) ** ((b + 1) / B))) for b in range(B)]


def _seen(n, R, window, sinks):
    """(tokens that some verify row sees, sum over the rows of the tokens each sees)."""
    pairs = 0
    for i in range(R):
        p = n - R + i
        if p < 0:
            continue
        lo = max(0, p - window + 1) if window else 0
        pairs += p + 1 - lo + min(sinks, lo)
    first = max(0, n - R)
    lo = max(0, first - window + 1) if window else 0
    return n - lo + min(sinks, lo), pairs


def work(case):
    c = case
    if c["op"] == "logprobs":
        rows = c["B"] * c["R"] * c["keep"]
        b = rows * (c["V"] * (4.0 if c["x"] == "f32" else 2.0) + 20 + 8 * c["top"])
        return {"bytes": b, "flops": rows * c["V"] * 4.0}
    if c["op"] == "pages":
        new = c["B"] * c["new"]
        rows = (c["B"] - 2 * new) * c["R"] + new * c["prompt"] / max(1.0, math.log(c["prompt"]))
        moved = rows / c["page"] + new * (c["lo"] + c["hi"]) / 2 / c["page"]
        return {"bytes": c["B"] * 36.0 + rows * 8.0 + moved * 8.0, "flops": rows * 2.0}
    token = c["Hkv"] * c["D"] * 2 * (0.5 + 1 / 16)  # bytes of a token's keys and values
    if c["op"] == "read4":
        there = sum(min(c["n"], n) for n in _lens(c))
        b = there * token + c["B"] * c["n"] * c["Hkv"] * c["D"] * 4.0 + c["B"] * 8.0
        return {"bytes": b, "flops": there * c["Hkv"] * c["D"] * 4.0}
    rows = c["B"] * c["R"]
    if c["op"] == "append4":
        xs = 4 if c["x"] == "f32" else 2
        heads = c["Hq"] + 2 * c["Hkv"]
        b = rows * (c["D"] * (heads * xs + c["Hq"] * 2.0) + token) + c["B"] * 4.0
        # the rows read back
        b += rows * (token + c["Hkv"] * c["D"] * 4.0)
        return {"bytes": b, "flops": rows * c["D"] * heads * 6.0}
    some, pairs, pages = 0, 0, 0
    for n in _lens(c):
        s, p = _seen(n, c["R"], c["window"], c["sinks"])
        some, pairs, pages = some + s, pairs + p, pages + -(-s // c["page"])
    b = some * token + rows * c["Hq"] * (c["D"] * 4.0 + 4.0)
    return {"bytes": b + pages * 4.0 + c["B"] * 4.0, "flops": pairs * c["Hq"] * c["D"] * 4.0}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _pages(c, seed):
    """Lengths, and a block table of pages in a random order."""
    cpu = torch.Generator().manual_seed(seed)
    n = torch.tensor(_lens(c))[torch.randperm(c["B"], generator=cpu)]
    per = (n + c["page"] - 1) // c["page"]
    total, cols = int(per.sum()), int(per.max())
    ids = torch.randperm(total, generator=cpu)
    table = torch.full((c["B"], cols), -1, dtype=torch.int64)
    at = torch.cumsum(per, 0) - per
    col = torch.arange(cols)[None, :]
    inside = col < per[:, None]
    table[inside] = ids[(at[:, None] + col)[inside]]
    return n, table, total


def _cache(c, g, seed, fill):
    """A cache of unit normal values under head scales near 1/32, in 4 bits."""
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    n, table, total = _pages(c, seed)
    s = dict(table=table.to(torch.int32).to(DEV), lens=n.to(torch.int32).to(DEV))
    for name in ("k", "v"):
        s[name + "_scale"] = (torch.rand(Hkv, device=DEV, generator=g) * 0.5 + 0.75) / 32
        codes = torch.zeros(total, Hkv, page, D // 2, dtype=torch.uint8, device=DEV)
        blocks = torch.zeros(total, Hkv, page, D // 16, device=DEV)
        if fill:
            x = torch.randn(total, Hkv, page, D, device=DEV, generator=g)
            codes, blocks = _encode(x.div_(s[name + "_scale"][:, None, None]))
        codes = codes.transpose(1, 2)  # the logical order: page, token, head, bytes
        s[name] = codes.contiguous() if c["order"] == "nhd" else codes
        s[name + "_blocks"] = blocks.to(torch.float8_e4m3fn)
    return s


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["op"] == "attn4":
        s.update(_cache(c, g, seed, True))
        # queries about twice unit size: the softmax leans on some tokens, as after training
        q = torch.randn(c["B"], c["R"], c["Hq"], c["D"], device=DEV, generator=g)
        s["q"], s["scale"] = (q * 2).to(torch.bfloat16), 1.0 / math.sqrt(c["D"])
    elif c["op"] == "read4":
        s.update(_cache(c, g, seed, True))
        # the last n tokens of the longer sequences, all of the shorter ones
        s["first"] = (s["lens"] - c["n"]).clamp(min=0)
    elif c["op"] == "append4":
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
    elif c["op"] == "pages":
        B, R, page = c["B"], c["R"], c["page"]
        n, table, used = _pages(dict(c, lo=c["lo"] + R, hi=c["hi"] + R), seed)
        n = n.to(DEV)
        wide = -(-(max(c["hi"], c["prompt"]) + 2 * R) // page)
        s["held"] = ((n + page - 1) // page).to(torch.int32)
        # the first places are free for new prompts, spread over 1 .. prompt; the next have ended
        k = int(B * c["new"])
        place = torch.randperm(B, device=DEV, generator=g)
        fresh, ended = place < k, (place >= k) & (place < 2 * k)
        prompt = c["prompt"] ** ((place + 1) / max(k, 1)).clamp(max=1)
        s["held"] = torch.where(fresh, 0, s["held"])
        # a step has verified R rows a sequence, of which the accept kept 1 .. R
        s["lens"] = torch.where(fresh, 0, n - R).to(torch.int32)
        kept = torch.randint(1, R + 1, (B,), device=DEV, generator=g)
        s["accepted"] = torch.where(fresh, 0, kept).to(torch.int32)
        s["grow"] = torch.where(fresh, prompt.round().int(), torch.where(ended, 0, R)).to(torch.int32)
        s["ended"] = ended.to(torch.int32)
        s["rows"] = int(s["grow"].sum())
        spare = B * (2 * R // page + 2) + k * (c["prompt"] // page + 1)
        ids = torch.randperm(used + spare, device=DEV, generator=g)
        s["table"] = torch.full((B, wide), -1, dtype=torch.int32, device=DEV)
        table = table.to(DEV)
        s["table"][:, :table.shape[1]] = torch.where(table >= 0, ids[table.clamp(min=0)], -1)
        s["free"] = torch.full((used + spare,), -1, dtype=torch.int32, device=DEV)
        s["free"][:spare] = ids[used:]
        s["free_count"] = torch.tensor([spare], dtype=torch.int32, device=DEV)
    else:
        B, R, V = c["B"], c["R"], c["V"]
        x = torch.randn(B, R, V, device=DEV, generator=g) * 3
        if c["masked"]:  # tokens that a grammar forbids, the same ones in every row
            x.masked_fill_(torch.rand(V, device=DEV, generator=g) < c["masked"], -math.inf)
        s["logits"] = x if c["x"] == "f32" else x.to(torch.bfloat16)
        # the committed tokens: the largest logits of a few random ids
        some = torch.randint(0, V, (B, R, 64), device=DEV, generator=g)
        pick = torch.gather(s["logits"].float(), 2, some).argmax(-1, keepdim=True)
        s["tokens"] = torch.gather(some, 2, pick)[..., 0].to(torch.int32)
        s["length"] = None
        if c["keep"] < 1:
            u = torch.rand(B, device=DEV, generator=g)
            s["length"] = (u * (2 * c["keep"] * R - 1)).round().to(torch.int32).clamp(0, R - 1) + 1
    if own:
        s["calls"], s["out"] = _bind(s)
    return s


def _bind(s):
    """The handles that an engine keeps next to its buffers: the argument blocks of its calls,
    with the output buffers and the workspaces.  A call does all of the work."""
    import speculative_decode_verification_w4_gb300 as vw4
    c = s["case"]
    if c["op"] == "pages":
        call = vw4.PreparedAdvance(
            s["table"], c["page"], s["lens"], s["held"], s["free"], s["free_count"], s["rows"],
            accepted=s["accepted"], ended=s["ended"], grow=s["grow"],
            slots=torch.full((s["rows"],), -1, dtype=torch.int64, device=DEV))
        return (call,), (call.lens, call.held, call.free_count, s["free"], s["table"],
                         call.seq_lens, call.row_start, call.slots)
    if c["op"] == "logprobs":
        B, R, n = c["B"], c["R"], c["top"]
        out = dict(logprob=torch.zeros(B, R, device=DEV), lse=torch.zeros(B, R, device=DEV),
                   entropy=torch.zeros(B, R, device=DEV),
                   rank=torch.zeros(B, R, dtype=torch.int32, device=DEV))
        if n:
            out.update(top_ids=torch.zeros(B, R, n, dtype=torch.int32, device=DEV),
                       top_logprobs=torch.zeros(B, R, n, device=DEV))
        call = vw4.PreparedLogprobs(s["logits"], s["tokens"], length=s["length"], top=n,
                                    scale=1 / 0.8, **out)
        return (call,), tuple(out.values())
    cache = vw4.KVCache4(s["k"], s["v"], s["k_blocks"], s["v_blocks"], s["table"], s["k_scale"],
                         s["v_scale"])
    if c["op"] == "read4":
        call = vw4.PreparedRead(cache, s["lens"], c["n"], first=s["first"])
        return (call,), (call.k, call.v)
    q = torch.empty(c["B"], c["R"], c["Hq"], c["D"], dtype=torch.bfloat16, device=DEV)
    if c["op"] == "append4":
        call = vw4.PreparedAppend(s["x"], cache, s["lens"], c["R"], c["Hq"], inv_freq=s["inv_freq"],
                                  adjacent=c["pairs"] == "adjacent", q_norm=s["q_norm"],
                                  k_norm=s["k_norm"], eps=1e-6, q_out=q)
        back = vw4.PreparedRead(cache, s["lens"], c["R"])
        return (call, back), (q, back.k, back.v)
    lse = torch.empty(c["B"], c["R"], c["Hq"], device=DEV)
    call = vw4.PreparedAttn(s["q"], cache, s["lens"], scale=s["scale"], window=c["window"],
                            sinks=c["sinks"], out=q, lse=lse)
    return (call,), (q, lse)


def run(state):
    if own:
        for call in state["calls"]:
            call()
        return state["out"]
    return {"attn4": _attn, "append4": _append, "read4": _read, "pages": _advance,
            "logprobs": _logprobs}[state["case"]["op"]](state)


# -------------------------------------------------------------- plain forms
def _encode(t):
    """t [..., D] (head scale already divided out) -> nibbles u8 [..., D/2], block scales
    [..., D/16] (e4m3 values, in t's type).  Nearest, ties to even, in both."""
    t = t.clamp(-2688.0, 2688.0).unflatten(-1, (-1, 16))
    a = (t.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0)
    step = torch.exp2(torch.frexp(a)[1].clamp(min=-5).to(t.dtype) - 4)  # of 4 significant bits
    b = torch.round(a / step) * step
    x = t / torch.where(b > 0, b, 1.0)
    m = x.abs()
    h = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = torch.where(b > 0, (torch.round(m / h) * h).clamp(max=6.0), 0.0)
    # 0, .5, 1, 1.5, 2, 3, 4, 6 -> 0 .. 7
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code | torch.where(t < 0, 8, 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), b[..., 0]


def _values(codes, blocks):
    """What nibbles [..., D/2] under block scales [..., D/16] stand for, in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return (lut[nib.int()].unflatten(-1, (-1, 16)) * blocks.float()[..., None]).flatten(-2)


def _tokens(s, name, page, at):
    """Tokens of the cache, [..., Hkv, D] for page ids and places in the page [...]."""
    return _values(s[name][page, at], s[name + "_blocks"][page, :, at]) * s[name + "_scale"][:, None]


def _attn(s):
    c = s["case"]
    B, R, Hq, Hkv, D, page = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page"))
    G, L = Hq // Hkv, s["table"].shape[1] * page
    rows = s["table"].clamp(min=0).long()

    def tokens(name):  # [B, Hkv, L, D] in 32 bits
        codes = s[name][rows].transpose(2, 3)  # [B, cols, Hkv, page, D/2]
        t = _values(codes, s[name + "_blocks"][rows]).transpose(1, 2).reshape(B, Hkv, L, D)
        return t * s[name + "_scale"][None, :, None, None]
    q = s["q"].float().reshape(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    j = torch.arange(L, device=DEV)[None, None, :]
    p = (s["lens"][:, None] - R + torch.arange(R, device=DEV)[None, :])[:, :, None]
    seen = j <= p
    if c["window"]:
        seen = seen & ((j > p - c["window"]) | (j < c["sinks"]))
    seen = seen[:, None, :, None, :]  # [B, 1, R, 1, L]
    sc = (q @ tokens("k").transpose(-1, -2) * s["scale"]).reshape(B, Hkv, R, G, L)
    sc = torch.where(seen, sc, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isinf(m), 0.0, m))
    z = e.sum(-1, keepdim=True)
    v = torch.where(seen.any(2).transpose(-1, -2), tokens("v"), 0.0)
    o = (e.reshape(B, Hkv, R * G, L) @ v).reshape(B, Hkv, R, G, D)
    o = torch.where(z > 0, o / z, 0.0)
    lse = (m + torch.log(z))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(torch.bfloat16)
    return o, lse.permute(0, 2, 1, 3).reshape(B, R, Hq)


def _append(s):
    c = s["case"]
    B, R, Hq, Hkv, D, page, rot = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page", "rot"))
    x = s["x"].float().reshape(B, R, Hq + 2 * Hkv, D)
    # keys and values in 64 bits: next to a border of 4 bits, 32 decide at random
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv].double(), x[:, :, Hq + Hkv:].double()
    pos = (s["lens"][:, None] - R + torch.arange(R, device=DEV)[None, :]).long()  # [B, R]
    angle = (pos[..., None].double() * s["inv_freq"])[:, :, None]

    def turn(t, w):
        if w is not None:
            t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        if rot == 0:
            return t
        h, cos, sin = rot // 2, angle.cos().to(t.dtype), angle.sin().to(t.dtype)
        a, b = (t[..., :h], t[..., h:rot]) if c["pairs"] == "half" else (t[..., 0:rot:2], t[..., 1:rot:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([a, b], -1) if c["pairs"] == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([r, t[..., rot:]], -1)
    q, k = turn(q, s["q_norm"]), turn(k, s["k_norm"])
    pg = torch.gather(s["table"].long(), 1, pos.clamp(min=0) // page)
    at = pos.clamp(min=0) % page

    def put(name, t):
        codes, blocks = _encode(t / s[name + "_scale"].double()[:, None])
        s[name][pg, at] = codes
        s[name + "_blocks"][pg, :, at] = blocks.float().to(torch.float8_e4m3fn)
        return _tokens(s, name, pg, at).to(torch.bfloat16)
    return q.to(torch.bfloat16), put("k", k), put("v", v)


def _read(s):
    c = s["case"]
    pos = s["first"].long()[:, None] + torch.arange(c["n"], device=DEV)
    live = (pos < s["lens"][:, None])[..., None, None]
    pos = pos.clamp(max=s["table"].shape[1] * c["page"] - 1)
    pg = torch.gather(s["table"].long(), 1, pos // c["page"]).clamp(min=0)
    at = pos % c["page"]
    return (torch.where(live, _tokens(s, "k", pg, at), 0.0).to(torch.bfloat16),
            torch.where(live, _tokens(s, "v", pg, at), 0.0).to(torch.bfloat16))


def _advance(s):
    c = s["case"]
    page, table, free = c["page"], s["table"], s["free"]
    ended = s["ended"] > 0
    lens = torch.where(ended, 0, s["lens"] + s["accepted"])
    # the pages of ended sequences go back to the end of the free list
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    back = torch.where(ended, s["held"], 0)
    at = s["free_count"] + torch.cumsum(back, 0) - back
    spot = torch.where(col < back[:, None], at[:, None] + col, free.numel()).long()
    room = torch.cat([free, free[:1]]).scatter(0, spot.flatten(), table.flatten())
    free.copy_(room[:-1])
    count = s["free_count"] + back.sum()
    # pages for the next rows, from its end on, in the order of the sequences
    held = torch.where(ended, 0, s["held"])
    need = ((lens + s["grow"] + page - 1) // page - held).clamp(min=0)
    taken = torch.cumsum(need, 0) - need
    inside = (col >= held[:, None]) & (col < (held + need)[:, None])
    spot = (count - 1 - taken[:, None] - (col - held[:, None])).clamp(0, free.numel() - 1).long()
    table.copy_(torch.where(inside, free[spot], table))
    start = torch.cumsum(s["grow"], 0) - s["grow"]
    # every row's sequence, its position, its slot
    b = torch.repeat_interleave(torch.arange(c["B"], device=DEV), s["grow"], output_size=s["rows"])
    pos = lens[b] + torch.arange(s["rows"], device=DEV) - start[b]
    slots = table[b, pos // page].long() * page + pos % page
    start = torch.cat([start, start[-1:] + s["grow"][-1:]])
    return (lens.to(torch.int32), (held + need).to(torch.int32), (count - need.sum()).to(torch.int32),
            free, table, (lens + s["grow"]).to(torch.int32), start.to(torch.int32), slots)


def _logprobs(s):
    c = s["case"]
    B, R, V, n = c["B"], c["R"], c["V"], c["top"]
    live = torch.ones(B, R, dtype=torch.bool, device=DEV)
    if s["length"] is not None:
        live = torch.arange(R, device=DEV) < s["length"][:, None]
    x = s["logits"].float()
    t = s["tokens"].long()[..., None]
    y = x * (1 / 0.8)
    m = y.amax(-1, keepdim=True)
    d = y - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    entropy = torch.log(z) - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / z
    xt = torch.gather(x, 2, t)
    before = (x > xt) | ((x == xt) & (torch.arange(V, device=DEV) < t))
    zero = torch.zeros((), device=DEV)
    out = [torch.where(live, (torch.gather(y, 2, t) - lse)[..., 0], zero),
           torch.where(live, lse[..., 0], zero), torch.where(live, entropy[..., 0], zero),
           torch.where(live, 1 + before.sum(-1), 0).to(torch.int32)]
    if n:
        # the largest first, equal ones by their index: one 64-bit key for both
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32
        top, _ = torch.topk(key + (2 ** 31 - torch.arange(V, device=DEV)), n, -1)
        ids = 2 ** 31 - (top & 0xFFFFFFFF)
        lp = torch.gather(y, 2, ids) - lse
        ids = torch.where(torch.isinf(lp), -1, ids)
        out += [torch.where(live[..., None], ids, 0).to(torch.int32),
                torch.where(live[..., None], lp, zero)]
    return tuple(out)


# ---------------------------------------------------------- 64-bit definition
def exact(case, seed):
    global own
    mine, own = own, False
    s = prepare(case, seed)
    own = mine
    f = {"attn4": _exact_attn, "append4": _exact_append, "read4": _exact_read,
         "pages": _exact_pages, "logprobs": _exact_logprobs}[case["op"]]
    return f(case, s)


def _exact_values(s, name, pages):
    """[pages, page, Hkv, D] in 64 bits."""
    codes, sc = s[name][pages], s[name + "_blocks"][pages].double().transpose(1, 2)
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=DEV)
    for half in (0, 1):
        c = (codes >> (4 * half)).int() & 15
        e, f = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(e == 0, f / 2, (1 + f / 2) * torch.pow(2.0, e.double() - 1))
        out[..., half::2] = torch.where(c >= 8, -mag, mag)
    return out * sc.repeat_interleave(16, -1) * s[name + "_scale"].double()[:, None]


def _exact_attn(c, s):
    B, R, Hq, Hkv, D, page = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, R, Hq), float("-inf"), dtype=torch.float64, device=DEV)
    lens, table = s["lens"].tolist(), s["table"].tolist()
    for b in range(B):
        n = lens[b]
        used = torch.tensor(table[b][:-(-n // page)], device=DEV)
        k = _exact_values(s, "k", used).flatten(0, 1)[:n]
        v = _exact_values(s, "v", used).flatten(0, 1)[:n]
        for i in range(R):
            p = n - R + i
            if p < 0:
                continue
            lo = max(0, p - c["window"] + 1) if c["window"] else 0
            first = min(c["sinks"], lo)
            ki, vi = torch.cat([k[:first], k[lo:p + 1]]), torch.cat([v[:first], v[lo:p + 1]])
            q = s["q"][b, i].double().reshape(Hkv, G, D)
            a = torch.einsum("hgd,thd->hgt", q, ki) / math.sqrt(D)
            top = a.max(-1, keepdim=True).values
            w = (a - top).exp()
            tot = w.sum(-1, keepdim=True)
            out[b, i] = torch.einsum("hgt,thd->hgd", w / tot, vi).reshape(Hq, D)
            lse[b, i] = (top + tot.log()).reshape(Hq)
    return out, lse


def _exact_append(c, s):
    B, R, Hq, Hkv, D, rot = (c[k] for k in ("B", "R", "Hq", "Hkv", "D", "rot"))
    X = s["x"].double().view(B * R, Hq + 2 * Hkv, D)
    p = (s["lens"].long()[:, None] - R + torch.arange(R, device=DEV)).flatten()
    M = torch.eye(D, dtype=torch.float64, device=DEV).repeat(B * R, 1, 1)
    for j in range(rot // 2):
        t = p.double() * s["inv_freq"][j]
        u, w = (j, j + rot // 2) if c["pairs"] == "half" else (2 * j, 2 * j + 1)
        M[:, u, u], M[:, u, w], M[:, w, u], M[:, w, w] = t.cos(), -t.sin(), t.sin(), t.cos()

    def normed(h, w):
        if w is None:
            return h
        return h / ((h ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
    q = torch.einsum("nij,nhj->nhi", M, normed(X[:, :Hq], s["q_norm"]))
    k = torch.einsum("nij,nhj->nhi", M, normed(X[:, Hq:Hq + Hkv], s["k_norm"]))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    # the values of e4m3 that are not negative, largest 448; borders half way between
    fine = torch.arange(0, 127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()

    def nearest(x, values):  # ties to the even index, whose last bit is 0
        mid = (values[1:] + values[:-1]) / 2
        lo, hi = torch.searchsorted(mid, x, right=False), torch.searchsorted(mid, x, right=True)
        return values[torch.where(lo % 2 == 0, lo, hi)]

    def held(t, g):
        t = (t / g.double()[:, None]).view(B * R, Hkv, D // 16, 16)
        b = nearest(t.abs().amax(-1) / 6, fine)[..., None]
        v = torch.where(b > 0, nearest(t.abs() / torch.where(b > 0, b, 1.0), grid), 0.0) * b
        v = torch.where(t < 0, -v, v).view(B * R, Hkv, D) * g.double()[:, None]
        return v.view(B, R, Hkv, D)
    return q.view(B, R, Hq, D), held(k, s["k_scale"]), held(X[:, Hq + Hkv:], s["v_scale"])


def _exact_read(c, s):
    B, n, page = c["B"], c["n"], c["page"]
    out = [torch.zeros(B, n, c["Hkv"], c["D"], dtype=torch.float64, device=DEV) for _ in range(2)]
    for b, (length, first) in enumerate(zip(s["lens"].tolist(), s["first"].tolist())):
        used = s["table"][b, :-(-length // page)].long()
        for t, name in zip(out, ("k", "v")):
            v = _exact_values(s, name, used).flatten(0, 1)[first:min(length, first + n)]
            t[b, :len(v)] = v
    return tuple(out)


def _exact_pages(c, s):
    page, B = c["page"], c["B"]
    lens, held, acc, ended, grow = (s[k].tolist() for k in ("lens", "held", "accepted", "ended", "grow"))
    table, stack = s["table"].tolist(), s["free"].tolist()
    top = int(s["free_count"])
    for b in range(B):
        lens[b] += acc[b]
        if ended[b]:
            for p in table[b][:held[b]]:
                stack[top] = p
                top += 1
            lens[b] = held[b] = 0
    start, slots = [0], []
    for b in range(B):
        while held[b] * page < lens[b] + grow[b]:
            top -= 1
            table[b][held[b]] = stack[top]
            held[b] += 1
        slots += [table[b][j // page] * page + j % page for j in range(lens[b], lens[b] + grow[b])]
        start.append(len(slots))
    return tuple(torch.tensor(t, device=DEV) for t in (
        lens, held, [top], stack, table, [n + g for n, g in zip(lens, grow)], start, slots))


def _exact_logprobs(c, s):
    B, R, n = c["B"], c["R"], c["top"]
    out = [torch.zeros(B, R, dtype=torch.float64, device=DEV) for _ in range(3)]
    rank = torch.zeros(B, R, dtype=torch.int64, device=DEV)
    ids = torch.zeros(B, R, n, dtype=torch.int64, device=DEV)
    lps = torch.zeros(B, R, n, dtype=torch.float64, device=DEV)
    for b in range(B):
        r = R if s["length"] is None else int(s["length"][b])
        x, t = s["logits"][b, :r].double(), s["tokens"][b, :r].long()[:, None]
        lp = torch.log_softmax(x / 0.8, -1)
        p = lp.exp()
        out[0][b, :r] = lp.gather(1, t)[:, 0]
        out[1][b, :r] = torch.logsumexp(x / 0.8, -1)
        out[2][b, :r] = -torch.where(p > 0, p * lp, 0.0).sum(-1)
        val, order = torch.sort(x, dim=-1, descending=True, stable=True)
        rank[b, :r] = (order == t).int().argmax(-1) + 1
        ids[b, :r] = torch.where(torch.isinf(val[:, :n]), -1, order[:, :n])
        lps[b, :r] = lp.gather(1, order[:, :n])
    return (*out, rank, ids, lps) if n else (*out, rank)
