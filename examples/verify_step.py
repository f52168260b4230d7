"""One speculative-decoding loop on random 4-bit weights: how the calls of this
library follow one another in a step.

    qkv = verify_gemm_w4(x)           -> packed rows of every verify token
    verify_rope_append(qkv)           -> rotated queries; keys and values into the cache
    verify_attn(q)                    -> the verify rows over the paged cache
    verify_gemm_w4(attention)         -> output projection        (per layer, to here)
    verify_gemm_w4_blockmax(x)        -> logits of the LM head and their block maxima
    process_logits(logits)            -> penalties, biases and the grammar's mask
    accept_rejection_blockmax(logits) -> committed tokens
    token_logprobs(logits, tokens)    -> their log probabilities, and the best alternatives
    advance_pages(accepted)           -> lengths, and pages for the next step's rows

A step verifies the token committed last and Kd drafts of every sequence: R = Kd
+ 1 rows at the end of the cache.  Rejected drafts leave their keys and values
behind the new length, where the next step's rows overwrite them.  The drafts
come from a table of logits by the token before (a stand-in for a draft model).
Pages come from one pool, as the sequences grow; the caches hold bf16, e4m3 or
(kv="nvfp4") 4 bits a value.

Run it on a GPU:  python examples/verify_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decode_verification_w4_gb300 as vw4  # noqa: E402


class Linear4:
    """A random nvfp4 weight [N, K] with outputs of about unit size."""

    def __init__(self, N, K, g):
        self.q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        self.scales = torch.ones((N, K // 16), device="cuda").to(torch.float8_e4m3fn)
        self.args = (vw4.FMT_NVFP4, self.q, self.scales, 0.35 * K ** -0.5)

    def __call__(self, x):
        return vw4.verify_gemm_w4(*self.args, x)


def rms_norm(x):
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class VerifyLoop:
    """The model's state and the sequences being decoded; step() commits 1 .. Kd + 1
    tokens to each."""

    def __init__(self, prompts, Kd=3, layers=2, hidden=1024, Hq=8, Hkv=2, D=128, V=4000, page=16,
                 max_len=256, kv=torch.bfloat16, window=0, sinks=0, allowed=None, seed=0):
        B = len(prompts)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.Kd, self.R, self.V, self.D = B, Kd, Kd + 1, V, D
        self.Hq, self.hidden, self.window, self.sinks = Hq, hidden, window, sinks
        self.embed = torch.randn(V, hidden, device="cuda", generator=g)
        self.qkv = [Linear4((Hq + 2 * Hkv) * D, hidden, g) for _ in range(layers)]
        self.proj = [Linear4(hidden, Hq * D, g) for _ in range(layers)]
        self.head = Linear4(V, hidden, g)
        self.draft_table = torch.randn(V, V, device="cuda", generator=g)
        self.inv_freq = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        self.head_norm = torch.ones(D, device="cuda")
        # the pages of one pool, in any order, go to the sequences as they grow
        cols = -(-max_len // page)
        self.page, pages = page, B * cols
        self.free = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(B, dtype=torch.int32, device="cuda")
        if kv == "nvfp4":
            scale = torch.full((Hkv,), 1 / 64, device="cuda")
            self.caches = [vw4.KVCache4(
                *(torch.zeros(pages, page, Hkv, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)),
                *(torch.zeros(pages, Hkv, page, D // 16, device="cuda").to(torch.float8_e4m3fn)
                  for _ in range(2)), self.table, scale, scale) for _ in range(layers)]
        else:
            scale = torch.full((Hkv,), 1 / 32, device="cuda") if kv == torch.float8_e4m3fn else None
            self.caches = [vw4.KVCache(torch.zeros(pages, page, Hkv, D, device="cuda").to(kv),
                                       torch.zeros(pages, page, Hkv, D, device="cuda").to(kv),
                                       self.table, scale, scale) for _ in range(layers)]
        # all tokens so far: the prompt, then what was committed
        self.history = torch.zeros((B, max_len), dtype=torch.int32, device="cuda")
        self.length = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        self.prompt_len = self.length.clone()
        for b, p in enumerate(prompts):
            self.history[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        self.repetition = torch.full((B,), 1.1, device="cuda")
        self.presence = torch.full((B,), 0.2, device="cuda")
        self.frequency = torch.full((B,), 0.1, device="cuda")
        # a grammar of one state: a bit a token, the same mask for every row
        self.mask = self.mask_row = None
        if allowed is not None:
            bits = torch.zeros((V + 31) // 32 * 32, dtype=torch.int64)
            bits[allowed] = 1
            words = (bits.view(-1, 32) << torch.arange(32)).sum(-1)
            self.mask = (words - ((words >> 31) << 32)).to(torch.int32).view(1, -1).cuda()
            self.mask_row = torch.zeros((B, self.R), dtype=torch.int32, device="cuda")
        self.steps = 0
        self.logprobs = None  # of the last step's tokens
        self.graphs = None
        # the prompts, but for their last tokens, which the first step verifies
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.seq_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.advance(grow=self.length + self.Kd)
        for i in range(0, int(self.length.max()) - 1):
            n = torch.minimum(self.length - 1, torch.tensor(i + 1, device="cuda")).to(torch.int32)
            self.layers(self.history.gather(1, (n - 1).clamp(min=0).long()[:, None]), n)

        self.cached.copy_(self.length - 1)

    def advance(self, accepted=None, grow=None):
        """Lengths of the caches after accepted more tokens, pages for R (or grow) more rows."""
        vw4.advance_pages(self.table, self.page, self.cached, self.held, self.free, self.free_count,
                          R=self.R, accepted=accepted, grow=grow, lens_out=self.cached,
                          held_out=self.held, free_count_out=self.free_count, seq_lens=self.seq_lens)

    def layers(self, tokens, seq_lens):
        """The rows of tokens [B, R] at the end of caches of seq_lens tokens -> [B * R, hidden]."""
        R = tokens.shape[1]
        x = self.embed[tokens.long().flatten()]
        for qkv, proj, cache in zip(self.qkv, self.proj, self.caches):
            q = vw4.verify_rope_append(qkv(rms_norm(x)), cache, seq_lens, R, self.Hq,
                                       inv_freq=self.inv_freq, q_norm=self.head_norm,
                                       k_norm=self.head_norm)
            a = vw4.verify_attn(q, cache, seq_lens, window=self.window, sinks=self.sinks)
            x = x + proj(a.view(self.B * R, self.Hq * self.D))
        return x

    def draft(self):
        """Kd drafts a sequence and the logits that each was drawn from."""
        token = self.history.gather(1, self.length.long()[:, None] - 1)
        g = torch.Generator(device="cuda").manual_seed(1000 + self.steps)
        drafts, logits = [token[:, :0]], []
        for _ in range(self.Kd):
            logits.append(self.draft_table[token[:, 0].long()])
            p = torch.softmax(logits[-1].double(), -1)
            token = torch.multinomial(p, 1, generator=g).to(torch.int32)
            drafts.append(token)
        return torch.cat(drafts, 1), torch.stack(logits, 1) if logits else None

    def verify(self, drafts):
        """-> processed logits [B, R, V] of the last token and the drafts, their block maxima."""
        B, R, V = self.B, self.R, self.V
        last = self.history.gather(1, self.length.long()[:, None] - 1)
        rows = torch.cat([last, drafts], 1)
        x = self.layers(rows, self.seq_lens)
        logits, bmax = vw4.verify_gemm_w4_blockmax(*self.head.args, rms_norm(x))
        logits, bmax = logits.view(B, R, V), bmax.view(B, R, -1)
        vw4.process_logits(logits, drafts, history=self.history, hist_len=self.length,
                           prompt_len=self.prompt_len, repetition=self.repetition,
                           presence=self.presence, frequency=self.frequency, mask=self.mask,
                           mask_index=self.mask_row, out=logits, block_max=bmax)
        return logits, bmax

    def step(self):
        """-> tokens [B, Kd + 1] and how many of them are committed [B].  After capture(): the
        same from two graphs, in tensors that the next step overwrites."""
        drafts, draft_logits = self.draft()
        if self.graphs is None:
            out = self.commit(drafts, draft_logits)
        else:
            before, after, rows, scored, kept, logprobs = self.graphs
            rows[0].copy_(drafts)
            if draft_logits is not None:
                rows[1].copy_(draft_logits)
            before.replay()
            # the accept itself is launched: a graph would hold the offset of its random numbers
            for to, made in zip(kept, self.accept(*rows, *scored)):
                to.copy_(made)
            after.replay()
            out, self.logprobs = kept, logprobs
        self.steps += 1
        return out

    def commit(self, drafts, draft_logits):
        """The step after its drafts, on the device and in place.  (Captured whole, every replay
        would draw the random numbers of the captured step's offset: see capture.)"""
        scored = self.score(drafts, draft_logits)
        tokens, n = self.accept(drafts, draft_logits, *scored)
        self.logprobs = self.keep(scored[0], tokens, n)
        return tokens, n

    def score(self, drafts, draft_logits):
        """-> the verify rows' logits and block maxima, and the drafts' block maxima."""
        logits, bmax = self.verify(drafts)
        draft_bmax = None
        if self.Kd:  # the draft's logits as they are; the call fills in their block maxima
            draft_bmax = torch.empty(self.B, self.Kd, bmax.shape[2], device="cuda")
            vw4.process_logits(draft_logits, drafts[:, 1:].contiguous(), out=draft_logits,
                               block_max=draft_bmax)
        return logits, bmax, draft_bmax

    def accept(self, drafts, draft_logits, logits, bmax, draft_bmax):
        return vw4.accept_rejection_blockmax(logits, bmax, draft_logits, draft_bmax, drafts,
                                             temperature=1.0, top_p=1.0, seed=7, offset=self.steps)

    def keep(self, logits, tokens, n):
        """The committed tokens into the history, pages for what follows -> their log probabilities."""
        logprobs = vw4.token_logprobs(logits, tokens, length=n, top=4)
        at = self.length.long()[:, None] + torch.arange(self.R, device="cuda")
        keep = torch.arange(self.R, device="cuda") < n[:, None]
        old = self.history.gather(1, at)
        self.history.scatter_(1, at, torch.where(keep, tokens, old))
        self.length += n
        self.advance(accepted=n)
        return logprobs

    def capture(self):
        """From now on (after a first step) a step replays what lies before and behind its accept
        from graphs.  The accept takes its random numbers' offset from the host, so that it stays
        a launch of its own."""
        drafts, draft_logits = self.draft()
        rows = drafts.clone(), None if draft_logits is None else draft_logits.clone()
        kept = (torch.zeros(self.B, self.R, dtype=torch.int32, device="cuda"),
                torch.zeros(self.B, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        before, after = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(before):
            scored = self.score(*rows)
        with torch.cuda.graph(after):
            logprobs = self.keep(scored[0], *kept)
        self.graphs = before, after, rows, scored, kept, logprobs


def main():
    loop = VerifyLoop([[5, 17, 300, 42], [9, 9, 1234]], kv="nvfp4",
                      allowed=torch.arange(0, 4000, 2))
    for k in range(8):
        tokens, n = loop.step()
        if k == 0:
            loop.capture()
        print("committed", [tokens[b, :n[b]].tolist() for b in range(loop.B)], "of log probability",
              [[round(x, 2) for x in loop.logprobs.logprob[b, :n[b]].tolist()] for b in range(loop.B)])
    if vw4.vw4_get_device_status():
        raise SystemExit("the device reported an error")


if __name__ == "__main__":
    main()
