"""The serving example runs the paged cache's operators together: its state stays consistent, and its attention equals
attention in 64 bits over what the cache gives back."""
import numpy as np
import pytest

from tests._parity import normwise_rel
from tests.gpu_util import cuda

pytestmark = pytest.mark.gpu


def test_prompts_then_speculative_steps():
    torch, L = cuda()
    from lattice_vq_weight_gb300 import serve_example as E
    prompts = [[5], list(range(33)), [9] * 16]
    s = E.Server(batch=3, num_blocks=96, drafts=3, seed=4)
    first = s.prompt(prompts)
    assert s.cached.tolist() == [1, 33, 16] and bool(((first >= 0) & (first < E.VOCAB)).all())
    for _ in range(6):
        before = s.cached.clone()
        out = s.step()
        kept = (out >= 0).sum(1)
        assert bool(((kept >= 1) & (kept <= 4)).all()) and torch.equal(s.cached, before + kept.int())
        assert bool((out < E.VOCAB).all()) and bool((s.last[:, 0] == out.gather(1, kept[:, None] - 1)[:, 0]).all())
        # no block in two places
        held = [s.table[i, :(int(s.kv_lens[i]) + E.BLOCK - 1) // E.BLOCK].tolist() for i in range(3)]
        flat = [b for r in held for b in r]
        assert len(set(flat)) == len(flat) and min(flat) >= 0 and max(flat) < 96
        # the last layer's attention against the cache's values in 64 bits
        q, got = (t.float().cpu().numpy().astype(np.float64) for t in s.seen)
        cu, lens = s.cu.tolist(), s.kv_lens.tolist()
        for i in range(3):
            pos = torch.arange(lens[i], device="cuda")
            slots = s.table[i].long()[pos // E.BLOCK] * E.BLOCK + pos % E.BLOCK
            k, v = (torch.empty((lens[i], E.KV_HEADS, E.DIM), device="cuda") for _ in range(2))
            L.lq_kv_gather(slots, *s.caches[-1], k, v)
            k, v = (t.cpu().numpy().astype(np.float64) for t in (k, v))
            for r in range(cu[i], cu[i + 1]):
                last = lens[i] - (cu[i + 1] - r)
                for h in range(E.Q_HEADS):
                    g = h * E.KV_HEADS // E.Q_HEADS
                    w = k[:last + 1, g] @ q[r, h] / np.sqrt(E.DIM)
                    w = np.exp(w - w.max())
                    # bf16 outputs: their rounding, and weights of 11 bits
                    assert normwise_rel(got[r, h], w @ v[:last + 1, g] / w.sum()) < 2.0 ** -8
    assert int(s.status) == 0
