"""Cases for the operators that serve requests from a paged 8-bit KV cache.

Five operators, in the order in which a serving step runs them:

  plan     block tables and slot maps from the requests' lengths
  rope     RMS norm of every query and key head and the position rotation, one pass
  append   new keys and values written into the 8-bit cache (one scale per block of
           tokens and head), and read back as the values that the cache stands for
  attend   attention of one or more query tokens per request over that cache
  verify   drafted tokens accepted or replaced from given random numbers

`run` computes a case in elementary torch operations, or, where `own` is true,
with the package's own calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of a few requests that are being decoded
        dict(name="plan decode b16", op="plan", batch=16, block=64, lo=1, hi=8192, new_lo=1, new_hi=1, width=256, lens=1),
        # a full batch, prompts and continued requests together, small blocks
        dict(name="plan mixed b512", op="plan", batch=512, block=16, lo=0, hi=4096, new_lo=1, new_hi=2048, width=512,
             lens=2),
        # decode step of a batch: 32 query and 8 key heads of 128
        dict(name="rope decode t16", op="rope", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128, inter=0, norm=1,
             dtype="bf16"),
        # a prompt chunk: 64 query and 8 key heads of 128
        dict(name="rope prompt t8191", op="rope", tokens=8191, q_heads=64, kv_heads=8, dim=128, rot=128, inter=0, norm=1,
             dtype="bf16"),
        # one new token per request, somewhere inside its last block
        dict(name="append decode b64", op="append", batch=64, block=16, kv_heads=8, dim=128, lo=1, hi=4096, new_lo=1,
             new_hi=1, dtype="bf16", lens=3),
        # prompts of seven requests written at once
        dict(name="append prompt b7", op="append", batch=7, block=64, kv_heads=8, dim=128, lo=0, hi=300, new_lo=300,
             new_hi=4000, dtype="bf16", lens=4),
        # a single long request: 8 key heads, 4 query heads each, 32768 tokens
        dict(name="attend one 32k", op="attend", batch=1, block=64, q_heads=32, kv_heads=8, dim=128, lo=32768, hi=32768,
             q_lo=1, q_hi=1, dtype="bf16", lens=5),
        # a ragged decode batch, 8 query heads per key head, small blocks
        dict(name="attend ragged b64", op="attend", batch=64, block=16, q_heads=64, kv_heads=8, dim=128, lo=100, hi=16000,
             q_lo=1, q_hi=1, dtype="bf16", lens=6),
        # drafted tokens checked in one pass, an odd number of heads of 64, 32-bit queries and outputs
        dict(name="attend drafts f32 b16", op="attend", batch=16, block=32, q_heads=14, kv_heads=2, dim=64, lo=20, hi=6000,
             q_lo=2, q_hi=6, dtype="f32", lens=7),
        # a prompt in chunks: about 2000 query tokens over what is already cached
        dict(name="attend prompt b3", op="attend", batch=3, block=64, q_heads=32, kv_heads=8, dim=128, lo=2048, hi=8000,
             q_lo=1500, q_hi=2047, dtype="bf16", lens=8),
        # one request with three drafted tokens
        dict(name="verify b1", op="verify", batch=1, draft=3, vocab=32000, dtype="f32", onehot=0),
        # a large batch with five drafted tokens each and a large vocabulary
        dict(name="verify b96", op="verify", batch=96, draft=5, vocab=128256, dtype="f32", onehot=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attend", "attend", "verify"])
    lens = rng.randrange(1 << 20)
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "plan":
        hi = _log(rng, 16, 8192)
        new_hi = rng.choice([1, 6, _log(rng, 16, 2048)])
        return dict(op=op, batch=_log(rng, 1, 512), block=block, lo=0, hi=hi, new_lo=min(1, new_hi), new_hi=new_hi,
                    width=(hi + new_hi + block - 1) // block + rng.randrange(40), lens=lens)
    if op == "rope":
        kv_heads = rng.choice([1, 2, 3, 8])
        dim = rng.choice([64, 80, 96, 128, 256])
        q_heads = kv_heads * rng.choice([1, 4, 5, 7, 8])
        most = min(8191, (60000000 if dtype == "bf16" else 30000000) // ((q_heads + kv_heads) * dim))
        return dict(op=op, tokens=_log(rng, 1, most), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, 32]), inter=rng.randrange(2), norm=rng.randrange(2), dtype=dtype)
    if op == "append":
        new_hi = rng.choice([1, 5, _log(rng, 10, 2000)])
        return dict(op=op, batch=_log(rng, 1, 256 if new_hi < 10 else 8), block=block, kv_heads=rng.choice([1, 2, 5, 8]),
                    dim=rng.choice([64, 80, 128, 256]), lo=0, hi=_log(rng, 16, 2000), new_lo=1, new_hi=new_hi, dtype=dtype,
                    lens=lens)
    if op == "attend":
        kv_heads, group = rng.choice([(8, 4), (8, 8), (1, 16), (2, 7), (4, 1), (5, 3)])
        dim = rng.choice([64, 128, 128, 256])
        if rng.randrange(4) == 0:      # a prompt chunk
            batch, q_hi = rng.randrange(1, 4), _log(rng, 40, 1500)
            most = int(5e10 / (batch * q_hi * kv_heads * group * dim))        # of the pairs that the largest listed case has
            return dict(op=op, batch=batch, block=block, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, lo=q_hi,
                        hi=_log(rng, q_hi, max(q_hi, min(6000, most))), q_lo=max(1, q_hi // 2), q_hi=q_hi, dtype=dtype,
                        lens=lens)
        batch = _log(rng, 1, 128)
        q_hi = rng.choice([1, 1, rng.randrange(2, 9)])
        hi = _log(rng, 16, min(60000, 500000 // batch))
        return dict(op=op, batch=batch, block=block, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, lo=min(q_hi, hi),
                    hi=hi, q_lo=1, q_hi=q_hi, dtype=dtype, lens=lens)
    return dict(op=op, batch=_log(rng, 1, 96), draft=rng.randrange(1, 8), vocab=_log(rng, 1000, 128256) | 1, dtype=dtype,
                onehot=int(rng.randrange(4) == 0))


def _lengths(case):
    """The requests' (cached, new) lengths: part of the case, the same for every seed."""
    r = random.Random(case["lens"])
    b = case["batch"]
    if case["op"] == "attend":
        new = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(b)]
        total = [max(n, _log(r, max(1, case["lo"]), case["hi"])) for n in new]
        return [t - n for t, n in zip(total, new)], new
    cached = [r.randint(case["lo"], case["hi"]) for _ in range(b)]
    if case["op"] == "plan":
        cached = [0 if r.randrange(3) == 0 and case["lo"] == 0 else c for c in cached]
    return cached, [r.randint(case["new_lo"], case["new_hi"]) for _ in range(b)]


def _blocks(tokens, block):
    return -(-tokens // block)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device=dev)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "rope":
        t, dt = case["tokens"], DTYPES[case["dtype"]]
        hq, hk, d, rot = case["q_heads"], case["kv_heads"], case["dim"], case["rot"]
        # q, k and v lie side by side in one projection's output, as a fused product writes them
        s["qkv"] = randn(t, (hq + 2 * hk) * d).mul_(0.5).to(dt)
        s["q"] = s["qkv"][:, :hq * d].unflatten(1, (hq, d))
        s["k"] = s["qkv"][:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["qw"] = (1 + 0.1 * randn(d)) if case["norm"] else None
        s["kw"] = (1 + 0.1 * randn(d)) if case["norm"] else None
        s["eps"] = 1e-6
        max_pos = 32768
        s["pos"] = torch.randint(0, max_pos, (t,), generator=g, device=dev, dtype=torch.int32)
        ang = torch.arange(max_pos, device=dev, dtype=torch.float64)[:, None] * (
            500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot))
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_out"], s["k_out"] = torch.empty((t, hq, d), dtype=dt, device=dev), torch.empty((t, hk, d), dtype=dt, device=dev)
        return s
    if case["op"] == "verify":
        b, k, v, dt = case["batch"], case["draft"], case["vocab"], DTYPES[case["dtype"]]
        logits = randn(b, k + 1, v).mul_(3.0)
        s["target"] = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(logits[:, :k] + 0.7 * randn(b, k, v), -1)
        # the draft model's own samples (the largest of p / exponential noise)
        s["tokens"] = (draft / rand(b, k, v).clamp_(1e-12, 1).log().neg_().clamp_(min=1e-12)).argmax(-1).int()
        s["draft"] = None if case["onehot"] else draft.to(dt)
        s["draft_lens"] = torch.randint(max(0, k - 2), k + 1, (b,), generator=g, device=dev, dtype=torch.int32)
        s["u_accept"], s["u_sample"] = rand(b, k), rand(b)
        s["out"] = torch.empty((b, k + 1), dtype=torch.int32, device=dev)
        s["accepted"] = torch.empty((b,), dtype=torch.int32, device=dev)
        return s

    cached, new = _lengths(case)
    b, bs = case["batch"], case["block"]
    need = [_blocks(c + n, bs) for c, n in zip(cached, new)]
    have = [_blocks(c, bs) for c in cached]
    pool = sum(need) + 8
    order = torch.randperm(pool, generator=g, device=dev, dtype=torch.int32)
    n_new = sum(new)
    s["cached"], s["new"], s["n_new"], s["block"] = ints(cached), ints(new), n_new, bs
    if case["op"] == "plan":
        width = max(case["width"], max(need))
        table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
        held = torch.arange(width, device=dev)[None, :] < ints(have)[:, None]
        table[held] = order[:sum(have)]
        s["table"], s["free"] = table, order[sum(have):].contiguous()
        s["slots"] = torch.empty((n_new,), dtype=torch.int64, device=dev)
        s["pos"] = torch.empty((n_new,), dtype=torch.int32, device=dev)
        s["cu"], s["kv_lens"] = torch.empty((b + 1,), dtype=torch.int32, device=dev), torch.empty_like(s["cached"])
        s["used"] = torch.empty((1,), dtype=torch.int32, device=dev)
        return s

    # the cache: codes of roughly normal values, one scale per block and head
    hk, d = case["kv_heads"], case["dim"]
    for n in ("k", "v"):
        codes = torch.empty((pool, hk, bs, d), dtype=torch.int8, device=dev)
        step = max(1, (1 << 26) // (hk * bs * d))
        for at in range(0, pool, step):
            part = codes[at:at + step]
            part.copy_(randn(*part.shape).mul_(36).round_().clamp_(-127, 127))
        s[n + "_cache"] = codes
        s[n + "_scales"] = (0.02 + 0.02 * rand(pool, hk)) * (1.0 if n == "k" else 0.5)
    width = max(need)
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev)[None, :] < ints(need)[:, None]] = order[:sum(need)]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        s["k"], s["v"] = randn(n_new, hk, d).to(dt), randn(n_new, hk, d).mul_(0.5).to(dt)
        req = torch.repeat_interleave(torch.arange(b, device=dev), s["new"].long(), output_size=n_new)
        first = s["new"].cumsum(0) - s["new"]
        pos = torch.arange(n_new, device=dev) - first[req] + s["cached"][req]
        s["slots"] = table[req, pos // bs].long() * bs + pos % bs
        # the blocks that new tokens fall into, every slot of them up to the last written one
        touched = ints([i * width + j for i in range(b) for j in range(cached[i] // bs, need[i])], torch.int64)
        base = table.flatten()[touched].long() * bs
        s["touched"] = table.flatten()[touched].long()
        filled = ints([min(bs, cached[i] + new[i] - j * bs) for i in range(b) for j in range(cached[i] // bs, need[i])])
        inside = torch.arange(bs, device=dev)[None, :]
        s["read"] = (base[:, None] + inside)[inside < filled[:, None]].contiguous()
        s["k_back"] = torch.empty((s["read"].numel(), hk, d), dtype=torch.float32, device=dev)
        s["v_back"] = torch.empty_like(s["k_back"])
        return s
    s["table"], s["kv_lens"] = table, s["cached"] + s["new"]
    s["cu"] = torch.cat([torch.zeros(1, device=dev), s["new"].cumsum(0)]).int()
    s["max_q"], s["max_kv"] = max(new), max(c + n for c, n in zip(cached, new))
    s["q"] = randn(n_new, case["q_heads"], d).to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_plan(s):
    bs, table, b = s["block"], s["table"], s["table"].shape[0]
    cached, new = s["cached"], s["new"]
    have, need = (cached + bs - 1) // bs, (cached + new + bs - 1) // bs
    add = need - have
    end = add.cumsum(0)
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    take = (end - add)[:, None] + j - have[:, None]
    fresh = s["free"][take.clamp(0, s["free"].numel() - 1)]
    table = torch.where(j < have[:, None], table, torch.where(j < need[:, None], fresh, -1))
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    req = torch.repeat_interleave(torch.arange(b, device=table.device), new.long(), output_size=s["n_new"])
    pos = torch.arange(s["n_new"], device=table.device) - cu[req] + cached[req]
    slots = table[req, pos // bs].long() * bs + pos % bs
    return {"table": table, "slots": slots, "positions": pos.int(), "cu": cu.int(), "kv_lens": cached + new,
            "used": end[-1:].int()}


def _rotate(x, w, eps, cos, sin, rot, inter, norm):
    y = x.float()
    if norm:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w
    r = y[..., :rot]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    rows = s["cos_sin"][s["pos"].long()][:, None, :]
    cos, sin = rows[..., :c["rot"] // 2], rows[..., c["rot"] // 2:]
    return {n: _rotate(s[n], s[n + "w"], s["eps"], cos, sin, c["rot"], c["inter"], c["norm"]) for n in ("q", "k")}


def _write(x, codes, scales, slots, touched):
    """The codes and scales of the cache after rows x were written to its slots."""
    nb, hk, bs, d = codes.shape
    block, off = slots // bs, slots % bs
    x = x.float()
    amax = x.abs().amax(-1)
    top = torch.zeros((nb, hk), device=x.device).scatter_reduce_(0, block[:, None].expand(-1, hk), amax, "amax")
    first = torch.full((nb,), bs, device=x.device).scatter_reduce_(0, block, off, "amin")[touched]
    old = torch.where(first[:, None] > 0, scales[touched], 0.0)
    new = torch.maximum(old, top[touched] / torch.full_like(top[touched], 127.0))
    kept = codes[touched].float()
    grown = (new > old) & (first[:, None] > 0)
    again = (kept * old[..., None, None] / torch.where(new > 0, new, 1.0)[..., None, None]).round()
    codes, scales = codes.clone(), scales.clone()
    codes[touched] = torch.where(grown[..., None, None], again, kept).to(torch.int8)
    scales[touched] = new
    s = scales[block]
    codes[block, :, off] = (x / torch.where(s > 0, s, 1.0)[..., None]).round().clamp(-127, 127).to(torch.int8)
    return codes, scales


def _plain_append(s):
    out = {}
    bs = s["block"]
    block, off = s["read"] // bs, s["read"] % bs
    for n in ("k", "v"):
        codes, scales = _write(s[n], s[n + "_cache"], s[n + "_scales"], s["slots"], s["touched"])
        out[n] = codes[block, :, off].float() * scales[block][..., None]
        out[n + "_scales"] = scales
    return out


def _plain_attend(s):
    c, bs, dev = s["case"], s["block"], s["q"].device
    b, hq, hk, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    lq, lk = s["max_q"], s["max_kv"]
    t = torch.arange(lk, device=dev)
    block = s["table"][:, t // bs].clamp(min=0).long()                                   # [b, lk]

    def rows(n):
        x = s[n + "_cache"][block, :, t % bs].float()                                    # [b, lk, hk, d]
        return (x * s[n + "_scales"][block][..., None]).permute(0, 2, 1, 3)

    i = torch.arange(lq, device=dev)
    n_q = s["new"][:, None]
    at = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][at].float().view(b, lq, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    x = (q @ rows("k").transpose(2, 3)).view(b, hk, hq // hk, lq, lk) * (d ** -0.5)
    see = t[None, None, :] <= (s["kv_lens"][:, None] - n_q + i)[:, :, None]              # [b, lq, lk]
    x = x.masked_fill(~see[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    x = x / x.sum(-1, keepdim=True)
    o = (x.view(b, hk, -1, lk) @ rows("v")).view(b, hk, hq // hk, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d)
    req = torch.repeat_interleave(torch.arange(b, device=dev), s["new"].long(), output_size=s["n_new"])
    return o[req, torch.arange(s["n_new"], device=dev) - s["cu"][req]].to(s["q"].dtype)


def _plain_verify(s):
    b, k = s["tokens"].shape
    dev = s["tokens"].device
    n, i = s["draft_lens"].long(), torch.arange(k, device=dev)
    x = s["tokens"].long()[..., None]
    p = s["target"][:, :k].gather(2, x)[..., 0].float()
    q = 1.0 if s["draft"] is None else s["draft"].gather(2, x)[..., 0].float()
    ok = (s["u_accept"] * q < p) & (i < n[:, None])
    acc = ok.int().cumprod(1).sum(1)
    r = torch.arange(b, device=dev)
    row = s["target"][r, acc].float()
    last = acc.clamp(max=k - 1)
    if s["draft"] is None:
        other = torch.zeros_like(row).scatter_(1, x[r, last], 2.0)
    else:
        other = s["draft"][r, last].float()
    rest = torch.where((acc < n)[:, None], (row - other).clamp(min=0), row)
    w = (rest * 2.0 ** 36).floor().long()
    w = torch.where(w.sum(1, keepdim=True) > 0, w, (row * 2.0 ** 36).floor().long())
    c = w.cumsum(1)
    goal = ((s["u_sample"] * 2.0 ** 24).long() * c[:, -1]) >> 24
    token = (c <= goal[:, None]).sum(1)
    j = torch.arange(k + 1, device=dev)
    drafted = torch.cat([s["tokens"], s["tokens"][:, :1]], 1)
    out = torch.where(j < acc[:, None], drafted, torch.where(j == acc[:, None], token.int()[:, None], -1))
    return {"tokens": out, "accepted": acc.int()}


def _own_plan(s):
    import lattice_vq_weight_gb300 as L
    L.lq_kv_plan(s["cached"], s["new"], s["block"], s["free"], s["table"], s["cu"], s["kv_lens"], s["slots"], s["pos"],
                 s["used"])
    return {"table": s["table"], "slots": s["slots"], "positions": s["pos"], "cu": s["cu"], "kv_lens": s["kv_lens"],
            "used": s["used"]}


def _own_rope(s):
    import lattice_vq_weight_gb300 as L
    L.lq_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["pos"], s["cos_sin"], s["q_out"], s["k_out"],
                      interleaved=bool(s["case"]["inter"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s):
    import lattice_vq_weight_gb300 as L
    cache = (s["k_cache"], s["k_scales"], s["v_cache"], s["v_scales"])
    L.lq_kv_append(s["k"], s["v"], s["slots"], *cache)
    L.lq_kv_gather(s["read"], *cache, s["k_back"], s["v_back"])
    return {"k": s["k_back"], "k_scales": s["k_scales"], "v": s["v_back"], "v_scales": s["v_scales"]}


def _own_attend(s):
    import lattice_vq_weight_gb300 as L
    if "workspace" not in s:       # kept by the program from step to step
        c = s["case"]
        size = L.lq_attention_paged_workspace_size(c["batch"], s["q"].shape[0], c["q_heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.empty((size,), dtype=torch.uint8, device=s["q"].device)
    L.lq_attention_paged(s["q"], s["cu"], s["kv_lens"], s["table"], s["k_cache"], s["k_scales"], s["v_cache"],
                         s["v_scales"], s["out"], s["workspace"])
    return s["out"]


def _own_verify(s):
    import lattice_vq_weight_gb300 as L
    L.lq_verify_draft(s["tokens"], s["draft_lens"], s["target"], s["draft"], s["u_accept"], s["u_sample"], s["out"],
                      s["accepted"])
    return {"tokens": s["out"], "accepted": s["accepted"]}


_plain = {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend,
          "verify": _plain_verify}
_own = {"plan": _own_plan, "rope": _own_rope, "append": _own_append, "attend": _own_attend, "verify": _own_verify}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * n * e + case["tokens"] * (4 + 4 * case["rot"]), "flops": 8 * n}
    if case["op"] == "verify":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = 1 if case["onehot"] else 2
        return {"bytes": case["batch"] * (rows * case["vocab"] * e + 16 * case["draft"]),
                "flops": 3 * case["batch"] * case["vocab"]}
    cached, new = _lengths(case)
    bs, n = case["block"], sum(new)
    need = [_blocks(c + m, bs) for c, m in zip(cached, new)]
    if case["op"] == "plan":
        have = [_blocks(c, bs) for c in cached]
        add, width = sum(need) - sum(have), max(case["width"], max(need))
        return {"bytes": 16 * case["batch"] + 4 * add + 4 * (case["batch"] * width - sum(have)) + 12 * n, "flops": 4 * n}
    hk, d = case["kv_heads"], case["dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        touched = sum(m - c // bs for m, c in zip(need, cached))
        back = sum(c + m - c // bs * bs for c, m in zip(cached, new))      # slots that are read back
        return {"bytes": 2 * hk * (n * d * (e + 1) + 8 * touched + back * d * 5) + 8 * n + 8 * back,
                "flops": 2 * hk * d * (3 * n + back)}
    total = sum(c + m for c, m in zip(cached, new))
    pairs = sum(m * c + m * (m + 1) // 2 for c, m in zip(cached, new))
    return {"bytes": 2 * hk * (total * d + 4 * sum(need)) + 4 * sum(need) + 2 * n * case["q_heads"] * d * e,
            "flops": 4 * d * case["q_heads"] * pairs}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    if case["op"] in ("plan", "verify"):
        return None                                            # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        half, out = case["rot"] // 2, {}
        first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
        second = first + (1 if case["inter"] else half)
        table = s["cos_sin"].double().index_select(0, s["pos"].long())
        turn = torch.complex(table[:, :half], table[:, half:]).unsqueeze(1)
        for n in ("q", "k"):
            y = s[n].double()
            if case["norm"]:
                y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / case["dim"] + s["eps"]).sqrt()
                y = y * s[n + "w"].double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            out[n] = y
        return out
    bs = case["block"]
    if case["op"] == "append":
        out = {}
        for n in ("k", "v"):
            codes, scales = s[n + "_cache"].double(), s[n + "_scales"].double()
            block = s["slots"] // bs
            edge = torch.nonzero(torch.diff(block, prepend=block[:1] - 1)).flatten().tolist() + [block.numel()]
            slot = s["slots"].tolist()
            for a, z in zip(edge[:-1], edge[1:]):              # one block at a time
                at, off = slot[a] // bs, slot[a] % bs
                x = s[n][a:z].double().transpose(0, 1)         # [heads, tokens, d]
                size = x.abs().amax((1, 2)) / 127
                if off:
                    grown = torch.maximum(size, scales[at])
                    ratio = torch.where(grown > scales[at], scales[at] / grown, 1.0)
                    codes[at] = torch.round(codes[at] * ratio[:, None, None])
                    size = grown
                scales[at] = size
                codes[at, :, off:off + z - a] = torch.round(x / size.clamp(min=1e-300)[:, None, None]).clamp(-127, 127)
            values = codes * scales[:, :, None, None]
            out[n] = values[s["read"] // bs, :, s["read"] % bs]
            out[n + "_scales"] = scales
        return out
    cached, new = _lengths(case)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if sum(m * (c + m) for c, m in zip(cached, new)) * hq * d > 2e12:
        return None
    outs, at = [], 0
    for i, (c, m) in enumerate(zip(cached, new)):              # one request at a time
        ids = s["table"][i, :_blocks(c + m, bs)].long()
        kv = [(s[n + "_cache"][ids].double() * s[n + "_scales"][ids].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)
              [:, :c + m] for n in ("k", "v")]
        q = s["q"][at:at + m].double()
        hide = torch.ones((m, c + m), dtype=torch.bool, device="cuda").triu(c + 1)
        heads = []
        for h in range(hq):
            x = (q[:, h] @ kv[0][h * hk // hq].T) / math.sqrt(d)
            x[hide] = -math.inf
            heads.append(torch.softmax(x, -1) @ kv[1][h * hk // hq])
        outs.append(torch.stack(heads, 1))
        at += m
    return torch.cat(outs)
