"""Float64 CPU oracle of the operators that serve requests from a paged 8-bit
KV cache: plain loops over requests, heads and tokens, sharing no code with
the kernels.  Test infrastructure."""
import math

import numpy as np


def plan(cached, new, block_size, free, table, max_tokens):
    """(table, cu, kv_lens, slots, positions, used, in_range) from the lengths; `table` is not changed."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    cached_in, new_in = list(map(int, cached)), list(map(int, new))
    cached, new = [max(0, c) for c in cached_in], [max(0, n) for n in new_in]
    ok = cached == cached_in and new == new_in
    slots, positions = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    cu, kv_lens, used, t = [0], [], 0, 0
    for i, (c, n) in enumerate(zip(cached, new)):
        have, need = -(-c // block_size), -(-(c + n) // block_size)
        ok &= need <= width
        for j in range(have, max(need, width)):
            block = -1
            if j < need:
                block = int(free[used]) if used < len(free) else -1
                used += 1
            if j < width:
                table[i, j] = block
        for p in range(c, c + n):
            if t < max_tokens:
                j = p // block_size
                block = table[i, j] if j < width else -1
                slots[t] = block * block_size + p % block_size if block >= 0 else -1
                positions[t] = p
            t += 1
        cu.append(cu[-1] + n)
        kv_lens.append(c + n)
    ok &= used <= len(free) and t <= max_tokens
    return table, np.array(cu), np.array(kv_lens, dtype=np.int64), slots, positions, used, ok


def norm_rope(x, weight, eps, positions, cos_sin, rot, interleaved):
    """x [tokens x heads x d]: norm (weight None: none), then the rotation of the first `rot` dimensions."""
    y = np.array(x, dtype=np.float64)
    half = rot // 2
    for t in range(y.shape[0]):
        row = np.asarray(cos_sin[positions[t]], dtype=np.float64)
        for h in range(y.shape[1]):
            v = y[t, h]
            if weight is not None:
                v = v / math.sqrt(float(np.mean(v * v)) + eps) * np.asarray(weight, dtype=np.float64)
            out = v.copy()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                c, s = row[i], row[half + i]
                out[a], out[b] = v[a] * c - v[b] * s, v[b] * c + v[a] * s
            y[t, h] = out
    return y


def append(x, slots, codes, scales):
    """Real-valued codes and scales after rows x [tokens x heads x d] went to `slots`: the codes before
    rounding (a rounded code is within 1/2 of them), untouched blocks as they were."""
    codes, scales = np.array(codes, dtype=np.float64), np.array(scales, dtype=np.float64)
    bs = codes.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        e = t + 1
        while e < len(slots) and slots[e] == slots[e - 1] + 1 and slots[e] % bs:
            e += 1
        b, off = int(slots[t]) // bs, int(slots[t]) % bs
        rows = np.array(x[t:e], dtype=np.float64)
        rows[~np.isfinite(rows)] = 0.0
        for h in range(codes.shape[1]):
            old = scales[b, h] if off else 0.0
            s = max(old, np.abs(rows[:, h]).max() / 127)
            if off and s > old:
                codes[b, h, :off] *= old / s
            codes[b, h, off:off + e - t] = rows[:, h] / s if s > 0 else 0.0
            scales[b, h] = s
        t = e
    return codes, scales


def attention(q, cu_q, kv_lens, table, k_codes, k_scales, v_codes, v_scales, sm_scale):
    """out [total_q x q_heads x d]; a block outside the pool or the table hides its tokens."""
    q = np.asarray(q, dtype=np.float64)
    nb, hk, bs, d = k_codes.shape
    group = q.shape[1] // hk
    out = np.zeros(q.shape)
    for i in range(len(kv_lens)):
        n = int(cu_q[i + 1]) - int(cu_q[i])
        length = min(int(kv_lens[i]), table.shape[1] * bs)
        pos = [p for p in range(length) if 0 <= table[i][p // bs] < nb]
        blk = np.array([table[i][p // bs] for p in pos], dtype=np.int64)
        off = np.array([p % bs for p in pos], dtype=np.int64)
        for j in range(n):
            last = int(kv_lens[i]) - n + j
            keep = np.array([p <= last for p in pos], dtype=bool)
            if not keep.any():
                continue
            for h in range(q.shape[1]):
                g, b, o = h // group, blk[keep], off[keep]
                k = k_codes[b, g, o].astype(np.float64) * k_scales[b, g].astype(np.float64)[:, None]
                v = v_codes[b, g, o].astype(np.float64) * v_scales[b, g].astype(np.float64)[:, None]
                s = sm_scale * (k @ q[int(cu_q[i]) + j, h])
                w = np.exp(s - s.max())
                out[int(cu_q[i]) + j, h] = w @ v / w.sum()
    return out


def verify(tokens, lens, target, draft, u_accept, u_sample):
    """(out_tokens, accepted): float32 comparisons and differences, whole-number weights."""
    b, k = tokens.shape
    vocab = target.shape[2]
    out, accepted = np.full((b, k + 1), -1, np.int64), np.zeros(b, np.int64)
    f = np.float32
    for r in range(b):
        n = k if lens is None else min(max(int(lens[r]), 0), k)
        a = 0
        while a < n:
            x = int(tokens[r, a])
            if not 0 <= x < vocab:
                break
            q = f(1) if draft is None else f(draft[r, a, x])
            if not f(u_accept[r, a]) * q < f(target[r, a, x]):
                break
            a += 1
        row = np.asarray(target[r, a], dtype=np.float32)
        rest = row.copy()
        if a < n:
            if draft is not None:
                rest = row - np.asarray(draft[r, a], dtype=np.float32)
            elif 0 <= int(tokens[r, a]) < vocab:
                rest[int(tokens[r, a])] = 0
        drawn = -1
        for w in (rest, row):
            whole = [int(math.floor(min(float(v), 4.0) * 2.0 ** 36)) if v > 0 else 0 for v in w]
            total = sum(whole)
            if total:
                goal = (int(float(f(u_sample[r])) * 2 ** 24) * total) >> 24
                run = 0
                for v, c in enumerate(whole):
                    run += c
                    if run > goal:
                        drawn = v
                        break
                break
        out[r, :a] = tokens[r, :a]
        out[r, a] = drawn
        accepted[r] = a
    return out, accepted
