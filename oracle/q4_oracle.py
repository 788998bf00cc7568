"""CPU oracle of the paged 4-bit KV cache and of token scoring: plain loops in
float64 (float32 where the format is defined by such steps), sharing no code
with the kernels.  Test infrastructure."""
import math

import numpy as np


def values(codes, scales):
    """float16 values of codes [..., d / 2] with scales [..., groups, 2]: fp16(fma(16 + code, s, b))."""
    codes, scales = np.asarray(codes), np.asarray(scales).astype(np.float64)
    d = 2 * codes.shape[-1]
    group = d // scales.shape[-2]
    out = np.empty((*codes.shape[:-1], d), np.float16)
    for j in range(d):
        c = (codes[..., j // 2] >> (4 * (j % 2))) & 15
        # the sum of an 11-bit product's 16 bits and a base is exact in float64
        out[..., j] = ((16.0 + c) * scales[..., j // group, 0] + scales[..., j // group, 1]).astype(np.float16)
    return out


def quantize(x, group):
    """(codes [..., d / 2], scales [..., groups, 2]) of float32 vectors x [..., d], in the format's float32 steps."""
    f = np.float32
    x = np.array(x, dtype=f)
    x[~np.isfinite(x)] = 0
    x = np.clip(x, f(-16384), f(16384))
    d = x.shape[-1]
    codes = np.zeros((*x.shape[:-1], d // 2), np.uint8)
    scales = np.zeros((*x.shape[:-1], d // group, 2), np.float16)
    for g in range(d // group):
        part = x[..., g * group:(g + 1) * group]
        low, high = part.min(-1), part.max(-1)
        s = ((high - low) / f(15)).astype(np.float16)
        b = (low - f(16) * s.astype(f)).astype(np.float16)
        r = np.where(s > 0, f(1) / np.where(s > 0, s, 1).astype(f), f(0))
        c = np.rint((part - b.astype(f)[..., None]) * r[..., None]) - f(16)
        c = np.clip(c, 0, 15).astype(np.uint8)
        for j in range(group):
            at = g * group + j
            codes[..., at // 2] |= c[..., j] << (4 * (at % 2))
        scales[..., g, 0], scales[..., g, 1] = s, b
    return codes, scales


def append(x, slots, codes, scales):
    """Codes and scales of a cache after rows x [tokens x heads x d] went to `slots` (negative or past it: left out)."""
    codes, scales = np.array(codes), np.array(scales)
    nb, _, bs, _ = codes.shape
    group = 2 * codes.shape[-1] // scales.shape[-2]
    for t, slot in enumerate(slots):
        if 0 <= slot < nb * bs:
            codes[slot // bs, :, slot % bs], scales[slot // bs, :, slot % bs] = quantize(x[t], group)
    return codes, scales


def attention(q, cu_q, kv_lens, table, k_codes, k_scales, v_codes, v_scales, sm_scale):
    """out [total_q x q_heads x d]; a block outside the pool or the table hides its tokens."""
    q = np.asarray(q, dtype=np.float64)
    nb, hk, bs, _ = k_codes.shape
    group = q.shape[1] // hk
    out = np.zeros(q.shape)
    for i in range(len(kv_lens)):
        n = int(cu_q[i + 1]) - int(cu_q[i])
        length = min(int(kv_lens[i]), table.shape[1] * bs)
        pos = [p for p in range(length) if 0 <= table[i][p // bs] < nb]
        if not pos:
            continue
        blk = np.array([table[i][p // bs] for p in pos], dtype=np.int64)
        off = np.array([p % bs for p in pos], dtype=np.int64)
        k = values(k_codes[blk, :, off], k_scales[blk, :, off]).astype(np.float64)
        v = values(v_codes[blk, :, off], v_scales[blk, :, off]).astype(np.float64)
        for j in range(n):
            seen = sum(p <= int(kv_lens[i]) - n + j for p in pos)
            if not seen:
                continue
            for h in range(q.shape[1]):
                s = sm_scale * (k[:seen, h // group] @ q[int(cu_q[i]) + j, h])
                w = np.exp(s - s.max())
                out[int(cu_q[i]) + j, h] = w @ v[:seen, h // group] / w.sum()
    return out


def token_logprobs(logits, tokens, top):
    """(logprobs, entropy, ranks, top_tokens, top_logprobs) of rows of finite or -inf logits; the order is that of
    the float32 differences from the row's largest, then of the tokens."""
    n, vocab = logits.shape
    logprobs, entropy = np.zeros(n), np.zeros(n)
    ranks, top_tokens = np.full(n, -1, np.int64), np.zeros((n, top), np.int64)
    top_logprobs = np.zeros((n, top))
    for i in range(n):
        x = np.asarray(logits[i], dtype=np.float64)
        m = x.max() if x.max() > -math.inf else 0.0
        with np.errstate(over="ignore"):
            d = x.astype(np.float32) - np.float32(m)
        order = sorted(range(vocab), key=lambda v: (-d[v], v))
        x = x - m                          # (a sum with m itself would lose a small logarithm beside a large m)
        total = np.exp(x).sum()
        lse = math.log(total) if total > 0 else 0.0
        p = np.exp(x - lse)
        entropy[i] = -sum(float(a) * float(b - lse) for a, b in zip(p, x) if a > 0)
        top_tokens[i] = order[:top]
        top_logprobs[i] = x[order[:top]] - lse
        t = int(tokens[i])
        if 0 <= t < vocab:
            logprobs[i] = x[t] - lse
            ranks[i] = order.index(t)
    return logprobs, entropy, ranks, top_tokens, top_logprobs
