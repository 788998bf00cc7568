"""A small decoder served from lattice-coded weights and the paged 8-bit or 4-bit cache.

    python -m lattice_vq_weight_gb300.serve_example

Two attention layers with random weights, quantized to E8 codes; every product
of a step is a GEMM from the codes.  Requests of different lengths start with
their prompts and then take speculative steps: a few drafted tokens each, one
pass of the model over them, and the drafts that survive kept.  A step runs

    lq_kv_plan          blocks, slots and positions of the new tokens
    lq_gemm             q, k and v of a layer, from the codes
    lq_qk_norm_rope     head norms and rotation, in place
    lq_kv_append        keys and values into the cache (lq_kv_append_q4 in 4 bits)
    lq_attention_paged  attention over it (lq_attention_paged_q4)
    lq_verify_draft     accepted drafts and the next token
    lq_token_logprobs   the tokens' log probabilities and their most likely alternatives

The weights, cache pools, block tables and lengths are allocated once; what
depends on the number of new tokens (slots, positions, workspace, outputs) comes
from torch's caching allocator step by step, and the free list is made with the
host waiting (`nonzero`), which a server that keeps one would not do.
"""
from __future__ import annotations

import torch

import lattice_vq_weight_gb300 as L

HIDDEN, Q_HEADS, KV_HEADS, DIM, LAYERS, VOCAB = 512, 8, 2, 64, 2, 1000
BLOCK, TILE, MAX_POS = 16, 256, 4096
GROUP, ALTERNATIVES = 32, 5                   # of the 4-bit cache; of the scores


class Server:
    """Weights, cache pools and request state of the example."""

    def __init__(self, batch: int, num_blocks: int = 512, drafts: int = 3, seed: int = 0, device="cuda",
                 cache_bits: int = 8):
        g = torch.Generator(device=device).manual_seed(seed)
        self.batch, self.drafts, self.device, self.gen = batch, drafts, device, g
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

        def weight(rows, cols):
            w = (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).bfloat16()
            return L.quantize(w, lattice="e8", tile=TILE, seed=seed, beta=0.25, dev_status=self.status)

        self.embed = torch.randn((VOCAB, HIDDEN), generator=g, device=device).bfloat16()
        self.qkv = [weight((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN) for _ in range(LAYERS)]
        self.proj = [weight(HIDDEN, Q_HEADS * DIM) for _ in range(LAYERS)]
        self.head = weight(VOCAB, HIDDEN)
        self.norms = [(torch.ones(DIM, device=device), torch.ones(DIM, device=device)) for _ in range(LAYERS)]
        angle = torch.arange(MAX_POS, device=device)[:, None] * 10000.0 ** (
            -torch.arange(0, DIM, 2, device=device) / DIM)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        if cache_bits == 4:
            self.caches = [L.paged_cache_q4(num_blocks, KV_HEADS, BLOCK, DIM, GROUP, device) for _ in range(LAYERS)]
            self.append, self.attention = L.lq_kv_append_q4, L.lq_attention_paged_q4
            self.attention_size = L.lq_attention_paged_q4_workspace_size
        else:
            self.caches = [L.paged_cache(num_blocks, KV_HEADS, BLOCK, DIM, device) for _ in range(LAYERS)]
            self.append, self.attention = L.lq_kv_append, L.lq_attention_paged
            self.attention_size = L.lq_attention_paged_workspace_size

        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
        self.num_blocks = num_blocks
        self.cached, self.kv_lens, self.cu, self.used = ints(batch), ints(batch), ints(batch + 1), ints(1)
        self.table = ints(batch, num_blocks // batch) - 1
        self.last = None                       # the token each request continues from

    def free_blocks(self):
        """Blocks that no request's cached tokens hold, smallest first."""
        held = torch.arange(self.table.shape[1], device=self.device)[None] < (self.cached[:, None] + BLOCK - 1) // BLOCK
        taken = torch.zeros(self.num_blocks, dtype=torch.bool, device=self.device)
        taken[self.table[held].long()] = True
        return torch.nonzero(~taken).flatten().int()

    def product(self, codes, x):
        return L.gemm(*codes, x, lattice="e8", tile=TILE, dev_status=self.status, out_dtype=torch.bfloat16)

    def forward(self, tokens, new_lens):
        """Run the model over the requests' new tokens (one after the other); hidden states of all of them."""
        n, st = tokens.numel(), self.status
        slots = torch.empty((n,), dtype=torch.int64, device=self.device)
        positions = torch.empty((n,), dtype=torch.int32, device=self.device)
        L.lq_kv_plan(self.cached, new_lens, BLOCK, self.free_blocks(), self.table, self.cu, self.kv_lens, slots,
                     positions, self.used, st)
        size = self.attention_size(self.batch, n, Q_HEADS, KV_HEADS, DIM)
        workspace = torch.empty((size,), dtype=torch.uint8, device=self.device)
        x = self.embed[tokens.long()]
        for layer in range(LAYERS):
            heads = self.product(self.qkv[layer], x).unflatten(1, (-1, DIM))
            q, k, v = heads.split((Q_HEADS, KV_HEADS, KV_HEADS), 1)
            L.lq_qk_norm_rope(q, k, *self.norms[layer], 1e-6, positions, self.cos_sin, q, k, dev_status=st)
            self.append(k, v, slots, *self.caches[layer], dev_status=st)
            out = torch.empty((n, Q_HEADS, DIM), dtype=x.dtype, device=self.device)
            self.attention(q, self.cu, self.kv_lens, self.table, *self.caches[layer], out, workspace,
                                 dev_status=st)
            x = x + self.product(self.proj[layer], out.flatten(1))
        self.seen = (q, out)                   # of the last layer
        return x

    def probabilities(self, hidden):
        return torch.softmax(self.product(self.head, hidden).float(), -1)

    def score(self, logits, tokens):
        """Log probabilities, entropies, ranks and alternatives of tokens [b x n] (-1: none) from logits [b n x vocab]."""
        n, f32, i32 = tokens.numel(), torch.float32, torch.int32
        new = lambda dtype, *shape: torch.empty((n, *shape), dtype=dtype, device=self.device)
        out = new(f32), new(f32), new(i32), new(i32, ALTERNATIVES), new(f32, ALTERNATIVES)
        L.lq_token_logprobs(logits, tokens.flatten(), *out, dev_status=self.status)
        return [t.unflatten(0, tokens.shape) for t in out]

    def prompt(self, prompts):
        """Start the requests: one list of tokens each."""
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=self.device)
        tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=self.device)
        hidden = self.forward(tokens, lens)
        logits = self.product(self.head, hidden[(self.cu[1:] - 1).long()])
        p = torch.softmax(logits.float(), -1)
        self.cached.copy_(self.kv_lens)
        # the first token: nothing drafted, so one is drawn from p
        self.last = self.verify(torch.empty((self.batch, 0), dtype=torch.int32, device=self.device), p[:, None], None)[0]
        self.scores = self.score(logits, self.last)
        return self.last

    def verify(self, drafted, target, draft):
        b, k = drafted.shape
        u = torch.rand((b, k + 1), generator=self.gen, device=self.device)
        out = torch.empty((b, k + 1), dtype=torch.int32, device=self.device)
        accepted = torch.empty((b,), dtype=torch.int32, device=self.device)
        L.lq_verify_draft(drafted, None, target, draft, u[:, :k].contiguous(), u[:, k].contiguous(), out, accepted,
                          self.status)
        return out, accepted

    def step(self):
        """One speculative step: drafts from a context-free draft model (the head on the last token's embedding),
        the model over them, and the survivors.  Returns the new tokens [batch x (drafts + 1)], -1 after them."""
        b, k = self.batch, self.drafts
        drafted, dists, token = [], [], self.last[:, -1]
        for _ in range(k):
            dists.append(self.probabilities(self.embed[token.long()]))
            token = torch.multinomial(dists[-1], 1, generator=self.gen)[:, 0].int()
            drafted.append(token)
        drafted = torch.stack(drafted, 1)
        tokens = torch.cat([self.last[:, -1:], drafted], 1)
        new = torch.full((b,), k + 1, dtype=torch.int32, device=self.device)
        hidden = self.forward(tokens.flatten(), new)
        logits = self.product(self.head, hidden)
        target = torch.softmax(logits.float(), -1).view(b, k + 1, VOCAB)
        out, accepted = self.verify(drafted, target, torch.stack(dists, 1))
        self.scores = self.score(logits, out)
        # the cache keeps the last token and the accepted drafts; what the refused
        # ones wrote lies past the length and is written over
        self.cached += 1 + accepted
        self.last = out.gather(1, accepted[:, None].long())
        return out


def main() -> None:
    for bits in (8, 4):
        s = Server(batch=4, cache_bits=bits)
        first = s.prompt([[1, 2, 3], list(range(40)), [7] * 17, list(range(100, 164))])
        print(f"{bits}-bit cache, first tokens:", first[:, 0].tolist())
        for i in range(4):
            out = s.step()
            print(f"step {i}: cached {s.cached.tolist()}, new tokens {[[t for t in r if t >= 0] for r in out.tolist()]}, "
                  f"log probabilities {[round(float(x), 2) for x in s.scores[0][out >= 0]]}")
        assert int(s.status) == 0, int(s.status)


if __name__ == "__main__":
    main()
