"""A small decoder that serves a batch with drafted tokens, on synthetic weights.

Prompts of different lengths go through in one chunk each; then every step
feeds each sequence's last token and a few drafted ones, and keeps what the
model's probabilities allow.  All products are of ternary weights in the
rotated basis, and the operators between them stay in it:

  tb_block_norm       residual, norm and both rotations between two products
  tb_ternary_gemm     queries, keys and values of 128-wide heads stay rotated:
                      scores do not change, and the output projection takes
                      rotated inputs
  tb_paged_append     the new keys and values into the pages of the cache
  tb_paged_append_rotary  (--rotary) the same with positions: queries and keys are
                      rotated back for them, and into the products' basis again,
                      where a cache of few bits loses least
  tb_paged_attention  the new tokens over their sequence's pages
  tb_token_probs      the target's probabilities: penalties of tokens that a
                      sequence has had, tokens that are not allowed, temperature
  tb_verify_draft     which drafts are kept, and the token drawn after them

The drafter is the model without its layers: it draws from what the last
token's embedding alone gives.  A draft that is not kept leaves its key and
value in the cache; the next step's tokens are written over them.

  python examples/speculative_decode.py [--steps 32] [--max-draft 4] [--cache bf16|fp8|int4] [--rotary 10000]
                                        [--repeats 1.1] [--presence 0.5] [--frequency 0.2]
"""

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ternary_weights_hadamard_amd import tb  # noqa: E402

HEAD_DIM = 128


@dataclass
class Config:
    layers: int = 2
    channels: int = 512
    heads: int = 4
    heads_kv: int = 2
    hidden: int = 1024
    vocab: int = 1031
    page: int = 16
    cache: str = "bf16"
    temperature: float = 0.5
    sure: float = 0.05  # the drafter stops where its likeliest token has less
    rotary: float = 0.0  # base of the rotary positions' frequencies; 0: no positions
    repeats: float = 1.0  # penalties, of tokens in the sequence, and of its
    presence: float = 0.0  # generated ones: once, and
    frequency: float = 0.0  # for each time
    banned: tuple = ()  # tokens that are never drawn


class Decoder:
    """Weights, a pool of cache pages and the state of a batch of sequences."""

    def __init__(self, config, batch, max_tokens, seed=0, device="cuda"):
        c = self.config = config
        self.device = device
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=gen, device=device)  # noqa: E731
        ternary = lambda n, k: tb.tb_quantize_pack(normal(n, k) * k ** -0.5)[::2]  # noqa: E731  (codes, scales)
        ones = lambda: torch.ones(c.channels, device=device)  # noqa: E731
        self.embedding = normal(c.vocab, c.channels)
        self.head = normal(c.vocab, c.channels) * c.channels ** -0.5
        self.layers = [dict(norm=ones(), qkv=ternary((c.heads + 2 * c.heads_kv) * HEAD_DIM, c.channels),
                            out=ternary(c.channels, c.heads * HEAD_DIM), norm2=ones(),
                            up=ternary(c.hidden, c.channels), gate=ternary(c.hidden, c.channels),
                            down=ternary(c.channels, c.hidden)) for _ in range(c.layers)]
        self.last_norm = ones()

        # Pages are handed out in any order; a sequence keeps a table of its own.
        each = -(-max_tokens // c.page)
        kind = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}[c.cache]
        wide = HEAD_DIM // 2 if c.cache == "int4" else HEAD_DIM  # two 4-bit codes a byte
        self.max_tokens, pages = each * c.page, batch * each
        scale8 = None if c.cache != "fp8" else torch.full((c.heads_kv,), 1.0 / 32, device=device)
        for layer in self.layers:
            layer["k"] = torch.zeros((pages, c.heads_kv, c.page, wide), device=device).to(kind)
            layer["v"] = torch.zeros((pages, c.heads_kv, wide, c.page), device=device).to(kind)
            layer["scales"] = dict(k_scale=scale8, v_scale=scale8)
            if c.cache == "int4":  # a scale and an offset for each position and head
                half = lambda *shape: torch.zeros(shape, dtype=torch.float16, device=device)  # noqa: E731
                layer["scales"] = dict(k_scale=half(pages, c.heads_kv, c.page, 2), v_scale=half(pages, c.heads_kv, 2, c.page))
        order = torch.randperm(pages, generator=gen, device=device)
        self.table = order.view(batch, each).to(torch.int32)
        self.freq = tb.tb_rotary_frequencies(HEAD_DIM, c.rotary)[0].to(device) if c.rotary else None
        self.params = torch.tensor([[c.temperature, c.repeats, c.presence, c.frequency]] * batch, device=device)
        self.mask = None
        if c.banned:
            allowed = torch.ones(-(-c.vocab // 32) * 32, dtype=torch.int64)
            allowed[list(c.banned)] = 0
            words = (allowed.view(-1, 32) << torch.arange(32)).sum(1)
            self.mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)[None].to(device)
        self.tokens = [[] for _ in range(batch)]
        self.prompt = [0] * batch
        self.random = torch.Generator(device=device).manual_seed(seed + 1)

    def _ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def forward(self, new):
        """Logits [tokens, vocab] of each sequence's tokens `new`, which follow
        the `held` ones whose keys and values are in the cache."""
        c = self.config
        cu = [0]
        for n in new:
            cu.append(cu[-1] + len(n))
        ends = [held + len(n) for held, n in zip(self.held(), new)]
        if max(ends) > self.max_tokens:
            raise ValueError(f"a sequence of {max(ends)} tokens: there is room for {self.max_tokens}")
        max_q = max(len(n) for n in new)
        where = (self.table, self._ints(cu), self._ints(ends))
        h = self.embedding[torch.tensor([t for n in new for t in n], device=self.device)]
        _, z = tb.tb_block_norm(None, h, w_pre=self.layers[0]["norm"], rotate_out=True)
        for i, w in enumerate(self.layers):
            qkv = tb.tb_ternary_gemm(z, *w["qkv"]).view(-1, c.heads + 2 * c.heads_kv, HEAD_DIM)
            q, k, v = qkv.split([c.heads, c.heads_kv, c.heads_kv], dim=1)
            if self.freq is None:
                tb.tb_paged_append(k, v, w["k"], w["v"], *where, max_q, **w["scales"])
            else:
                q = tb.tb_paged_append_rotary(q, k, v, w["k"], w["v"], *where, max_q, self.freq, turn_in=True, turn_out=True,
                                              **w["scales"])
            o = tb.tb_paged_attention(q, w["k"], w["v"], *where, max_q, max(ends), **w["scales"])
            y = tb.tb_ternary_gemm(o.view(-1, c.heads * HEAD_DIM), *w["out"], out_dtype=torch.float32)
            _, z = tb.tb_block_norm(y, h, w_pre=w["norm2"], rotate_in=True, rotate_out=True, h=h)
            up, gate = tb.tb_ternary_gemm_rotated(z, *w["up"]), tb.tb_ternary_gemm_rotated(z, *w["gate"])
            y = tb.tb_ternary_gemm(tb.tb_fwht128(torch.nn.functional.silu(gate) * up), *w["down"],
                                   out_dtype=torch.float32)
            last = i + 1 == c.layers
            _, z = tb.tb_block_norm(y, h, w_pre=self.last_norm if last else self.layers[i + 1]["norm"],
                                    rotate_in=True, rotate_out=not last, h=h)
        return z.float() @ self.head.t()

    def held(self):
        """Tokens whose keys and values are in the cache: all but the last."""
        return [max(len(t) - 1, 0) for t in self.tokens]

    def probabilities(self, logits):
        return torch.softmax(logits / self.config.temperature, dim=-1)

    def _offsets(self, lists):
        cu = [0]
        for x in lists:
            cu.append(cu[-1] + len(x))
        return cu

    def _verify(self, logits, q, drafts, max_draft, so_far):
        """`so_far`: the sequences' tokens before their drafts."""
        cu = self._offsets(drafts)
        ids, offsets = self._ints([t for d in drafts for t in d]), self._ints(cu)
        mask = {} if self.mask is None else dict(mask=self.mask, mask_row=self._ints([0] * logits.shape[0]))
        p = tb.tb_token_probs(logits, self.params, ids, offsets, max_draft, history=self._ints([t for s in so_far for t in s]),
                              cu_history=self._ints(self._offsets(so_far)), prompt_len=self._ints(self.prompt), **mask)
        u = torch.rand(cu[-1], generator=self.random, device=self.device)
        u_next = torch.rand(len(drafts), generator=self.random, device=self.device)
        return tb.tb_verify_draft(p, q, ids, u, u_next, offsets, max_draft)

    def prefill(self, prompts):
        """Start the batch: the prompts' keys and values, and a first token of
        each.  Returns the logits that it was drawn from [batch, vocab]."""
        logits = self.forward(prompts)
        ends = torch.tensor([len(p) for p in prompts], device=self.device).cumsum(0) - 1
        logits = logits[ends]
        self.prompt = [len(p) for p in prompts]
        _, drawn = self._verify(logits, None, [[] for _ in prompts], 0, prompts)
        self.tokens = [list(p) + t for p, t in zip(prompts, drawn.tolist())]
        return logits

    def draft(self, most):
        """Up to `most` tokens for each sequence, as long as the drafter is sure
        enough (which must not depend on the token drawn: it is verified as a draw
        from all of q), and the probabilities that each was drawn from [all
        drafts, vocab]."""
        last = torch.tensor([t[-1] for t in self.tokens], device=self.device)
        room = [min(most, self.max_tokens - len(t)) for t in self.tokens]
        drafts, rows = [[] for _ in room], [[] for _ in room]
        open_ = [True] * len(room)
        for j in range(most):
            _, z = tb.tb_block_norm(None, self.embedding[last], w_pre=self.last_norm)
            q = self.probabilities(z.float() @ self.head.t())
            last = torch.multinomial(q, 1, generator=self.random).squeeze(1)
            sure = (q.amax(dim=1) >= self.config.sure).tolist()
            for b, t in enumerate(last.tolist()):
                open_[b] = open_[b] and sure[b] and j < room[b]
                if open_[b]:
                    drafts[b].append(t)
                    rows[b].append(q[b])
        rows = [x for r in rows for x in r]
        return drafts, torch.stack(rows) if rows else None

    def step(self, max_draft):
        """A step of every sequence.  Returns (kept drafts of each, the logits
        that each one's last token was drawn from [batch, vocab])."""
        drafts, q = self.draft(max_draft)
        new = [t[-1:] + d for t, d in zip(self.tokens, drafts)]
        logits = self.forward(new)
        kept, out = self._verify(logits, q, drafts, max_draft, self.tokens)
        first = torch.tensor([0] + [len(n) for n in new[:-1]], device=self.device).cumsum(0)
        for t, n, row in zip(self.tokens, kept.tolist(), out.tolist()):
            t += row[:n + 1]
        return kept.tolist(), logits[first + kept]


def prompts_of(batch, longest, vocab, seed=0):
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.randint(1, longest + 1, (batch,), generator=gen).tolist()
    return [torch.randint(0, vocab, (n,), generator=gen).tolist() for n in lengths]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--max-draft", type=int, default=4)
    ap.add_argument("--cache", choices=["bf16", "fp8", "int4"], default="bf16")
    ap.add_argument("--rotary", type=float, default=0.0, help="base of the positions' frequencies (0: no positions)")
    ap.add_argument("--repeats", type=float, default=1.0)
    ap.add_argument("--presence", type=float, default=0.0)
    ap.add_argument("--frequency", type=float, default=0.0)
    args = ap.parse_args()
    config = Config(cache=args.cache, rotary=args.rotary, repeats=args.repeats, presence=args.presence,
                    frequency=args.frequency)
    decoder = Decoder(config, args.batch, args.prompt + 1 + args.steps * (args.max_draft + 1))
    prompts = prompts_of(args.batch, args.prompt, config.vocab)
    decoder.prefill(prompts)
    kept = 0
    for _ in range(args.steps):
        kept += sum(decoder.step(args.max_draft)[0])
    made = sum(len(t) - len(p) for t, p in zip(decoder.tokens, prompts))
    print(f"{made} tokens in {args.steps} steps of {args.batch} sequences, {kept} of them drafts that were kept")
    for p, t in zip(prompts, decoder.tokens):
        print(f"  {len(p)} prompt tokens, then {t[len(p):len(p) + 16]} ...")


if __name__ == "__main__":
    main()
