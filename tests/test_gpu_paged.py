"""The paged cache's operators but the attention, on the GPU against the float64 oracle: block tables
and slots, head norms with rotation, cache writes and reads, draft verification."""
import numpy as np
import pytest

import oracle.paged_oracle as P
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu


def i32(torch, a):
    return to_dev(torch, np.asarray(a, dtype=np.int32))


def status_word(torch):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan
def run_plan(cached, new, bs, free, table, max_tokens, stride=None):
    torch, L = cuda()
    b, width = table.shape
    full = torch.full((b, stride or width), 12345, dtype=torch.int32, device="cuda")
    full[:, :width] = i32(torch, table)
    dt = full[:, :width]
    cu, lens = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (b + 1, b))
    slots = torch.full((max_tokens,), -7, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens,), -7, dtype=torch.int32, device="cuda")
    used, st = torch.full((1,), -7, dtype=torch.int32, device="cuda"), status_word(torch)
    for _ in range(2):      # a second call with the same inputs changes nothing
        L.lq_kv_plan(i32(torch, cached), i32(torch, new), bs, i32(torch, free), dt, cu, lens, slots, pos, used, st)
    torch.cuda.synchronize()
    assert bool((full[:, width:] == 12345).all())
    return [x.cpu().numpy() for x in (dt, cu, lens, slots, pos)] + [int(used), int(st)]


def check_plan(cached, new, bs, free, table, max_tokens, stride=None):
    torch, L = cuda()
    got = run_plan(cached, new, bs, free, table, max_tokens, stride)
    t, cu, lens, slots, pos, used, ok = P.plan(cached, new, bs, free, table, max_tokens)
    for g, want in zip(got, (t, cu, lens, slots, pos, used)):
        assert np.array_equal(g, want)
    assert got[-1] == (0 if ok else L.LQ_DEV_RANGE)


@pytest.mark.parametrize("batch,bs,hi,new_hi", [(1, 16, 0, 1), (1, 64, 500, 1), (3, 16, 40, 40), (33, 128, 1000, 300),
                                                (257, 32, 200, 1), (1000, 16, 60, 9), (5, 64, 0, 5000), (8192, 16, 30, 2)])
def test_plan(batch, bs, hi, new_hi):
    rng = np.random.default_rng(batch + bs)
    cached, new = rng.integers(0, hi + 1, batch), rng.integers(0, new_hi + 1, batch)
    new[rng.integers(0, batch)] = new_hi
    have = -(-cached // bs)
    need = -(-(cached + new) // bs)
    width = int(need.max()) + 3
    ids = rng.permutation(int(need.sum()) + 5)
    table = np.full((batch, width), -1)
    at = 0
    for i in range(batch):
        table[i, :have[i]] = ids[at:at + have[i]]
        at += have[i]
    check_plan(cached, new, bs, ids[at:], table, int(new.sum()) + 7, stride=width + 5)


@pytest.mark.parametrize("case", ["pool", "pool empty", "table", "tokens", "negative", "zero width"])
def test_plan_that_does_not_fit(case):
    cached, new, free, width, tokens = [16, 5, 0], [20, 30, 17], list(range(10, 20)), 4, 80
    if case == "pool":
        free = free[:3]
    elif case == "pool empty":
        free = []
    elif case == "table":
        width = 2
    elif case == "tokens":
        tokens = 40
    elif case == "negative":
        cached, new = [16, -5, 0], [20, 30, -17]
    elif case == "zero width":
        cached, width = [0, 0, 0], 0
    table = np.full((3, width), -1)
    if width:
        table[0, 0], table[1, 0] = 3, 4
    check_plan(cached, new, 16, free, table, tokens)


# ------------------------------------------------------------------ norm and rotation
ROPE = [(1, 1, 1, 64, 64, False, True), (7, 4, 2, 128, 128, False, True), (5, 3, 1, 80, 80, False, True),
        (3, 5, 5, 96, 32, True, True), (9, 14, 2, 64, 64, True, False), (2, 2, 1, 256, 256, False, True),
        (4, 7, 1, 8, 0, False, True), (300, 32, 8, 128, 64, False, True), (2, 1, 0, 16, 16, True, True),
        (700, 17, 4, 136, 48, False, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,norm", ROPE)
def test_norm_rope(dtype, tokens, hq, hk, d, rot, inter, norm):
    torch, L = cuda()
    rng = np.random.default_rng(d + tokens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    qkv = to_dev(torch, rng.standard_normal((tokens, (hq + 2 * hk) * d)).astype(np.float32) * 3).to(dt)
    q, k = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    w = [to_dev(torch, rng.uniform(0.5, 2, d).astype(np.float32)) if norm else None for _ in range(2)]
    if tokens == 300:
        w[1] = None                                    # queries normed, keys not
    pos = rng.integers(0, 50, tokens).astype(np.int32)
    ang = rng.uniform(-4, 4, (50, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    qo, ko, st = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous()), status_word(torch)
    args = (w[0], w[1], 1e-5, to_dev(torch, pos), to_dev(torch, table))
    L.lq_qk_norm_rope(q, k, *args, qo, ko, interleaved=inter, dev_status=st)
    want = [P.norm_rope(x.float().cpu().numpy(), None if y is None else y.cpu().numpy(), 1e-5, pos, table, rot, inter)
            for x, y in zip((q, k), w)]
    L.lq_qk_norm_rope(q, k, *args, q, k, interleaved=inter, dev_status=st)     # in place, in the strided input
    torch.cuda.synchronize()
    assert int(st) == 0
    for got, place, ref in zip((qo, ko), (q, k), want):
        assert torch.equal(got, place)
        # fp32 steps: about ten roundings of values no larger than the head's largest; then one bf16 rounding
        big = np.abs(ref).max(axis=-1, keepdims=True) if ref.size else 0.0
        tol = 16 * 2.0 ** -24 * big * np.sqrt(2) + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
        assert (np.abs(got.float().cpu().numpy() - ref) <= tol).all()


def test_norm_rope_position_outside_the_table():
    torch, L = cuda()
    x = to_dev(torch, np.random.default_rng(3).standard_normal((3, 2, 64)).astype(np.float32))
    table = torch.zeros((4, 64), device="cuda")
    out, ko, st = torch.empty_like(x), torch.empty_like(x[:, :1]).contiguous(), status_word(torch)
    k = x[:, :1].contiguous()
    L.lq_qk_norm_rope(x, k, None, None, 0.0, i32(torch, [4, 1, -1]), table, out, ko, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == L.LQ_DEV_RANGE
    assert torch.equal(out[0], x[0]) and torch.equal(out[2], x[2]) and not out[1].any()


# ------------------------------------------------------------------ cache writes and reads
def make_cache(torch, rng, nb, hk, bs, d):
    codes = [rng.integers(-127, 128, (nb, hk, bs, d)).astype(np.int8) for _ in range(2)]
    scales = [rng.uniform(0.005, 0.03, (nb, hk)).astype(np.float32) for _ in range(2)]
    return codes, scales, [to_dev(torch, codes[0]), to_dev(torch, scales[0]), to_dev(torch, codes[1]),
                           to_dev(torch, scales[1])]


def check_append(x, slots, codes, scales, cache, bs):
    """Codes within rounding of the oracle's real-valued ones: half a code plus 127 times the quotient's
    error (two fp32 roundings of the scale and the quotient, a third of the rescaled code's product)."""
    for n in range(2):
        want, s = P.append(x[n], slots, codes[n], scales[n])
        got, gs = cache[2 * n].cpu().numpy().astype(np.float64), cache[2 * n + 1].cpu().numpy()
        assert np.allclose(gs, s, rtol=2.0 ** -23, atol=0)
        written = np.zeros(want.shape[:3], bool)
        for slot in slots[slots >= 0]:
            written[slot // bs, :, slot % bs] = True
        changed = (want != codes[n])
        assert np.array_equal(got[~changed], codes[n][~changed].astype(np.float64)) or \
            (np.abs(got - want)[~changed] <= 0.5 + 127 * 2.0 ** -22).all()
        assert (np.abs(got - want) <= 0.5 + 127 * 2.0 ** -22).all()
        assert np.array_equal(got[~written & ~changed.any(-1)],
                              codes[n][~written & ~changed.any(-1)].astype(np.float64))


APPEND = [(16, 64, 1, [(0, 1)]), (16, 128, 3, [(5, 1), (15, 1), (16, 1), (31, 2)]), (32, 80, 2, [(0, 100), (33, 1), (7, 60)]),
          (64, 128, 8, [(63, 2), (0, 64), (100, 200)]), (128, 256, 1, [(1, 127), (3, 400)]), (128, 16, 5, [(127, 1), (0, 129)]),
          (64, 64, 2, [(i % 70, 1) for i in range(700)])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,d,hk,reqs", APPEND)
def test_append_and_gather(dtype, bs, d, hk, reqs):
    torch, L = cuda()
    rng = np.random.default_rng(bs + d)
    counts = [-(-(c + n) // bs) for c, n in reqs]
    nb = sum(counts) + 2
    ids = rng.permutation(nb)
    slots, at = [], 0
    for (c, n), m in zip(reqs, counts):
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(c, c + n)] + [-1]
        at += m
    slots = np.array(slots, dtype=np.int64)
    codes, scales, cache = make_cache(torch, rng, nb, hk, bs, d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wide = to_dev(torch, (rng.standard_normal((len(slots), 3 * hk * d)) *
                          rng.choice([0.1, 1, 4], (len(slots), 1))).astype(np.float32)).to(dt)
    k, v = (wide[:, n * hk * d:(n + 1) * hk * d].unflatten(1, (hk, d)) for n in (1, 2))
    st = status_word(torch)
    L.lq_kv_append(k, v, to_dev(torch, slots), *cache, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    x = [t.float().cpu().numpy() for t in (k, v)]
    check_append(x, slots, codes, scales, cache, bs)
    first = [t.clone() for t in cache]
    L.lq_kv_append(k, v, to_dev(torch, slots), *cache, dev_status=st)     # the same rows again change nothing
    torch.cuda.synchronize()
    for a, b in zip(first, cache):
        assert torch.equal(a, b)
    for out_dt in (torch.float32, torch.bfloat16):
        ko, vo = (torch.empty((len(slots), hk, d), dtype=out_dt, device="cuda") for _ in range(2))
        L.lq_kv_gather(to_dev(torch, slots), *cache, ko, vo, dev_status=st)
        torch.cuda.synchronize()
        for n, out in ((0, ko), (1, vo)):
            b, o = slots // bs, slots % bs
            val = cache[2 * n].cpu()[b, :, o].float() * cache[2 * n + 1].cpu()[b][..., None]
            val[slots < 0] = 0
            assert torch.equal(out.cpu(), val.to(out_dt))
    assert int(st) == 0


def test_append_zeros_nonfinite_and_slots_past_the_cache():
    torch, L = cuda()
    rng = np.random.default_rng(9)
    codes, scales, cache = make_cache(torch, rng, 3, 2, 16, 64)
    x = rng.standard_normal((5, 2, 64)).astype(np.float32)
    x[0] = 0                                     # a block that starts with zeros
    x[2, 1, 5], x[2, 0, 7] = np.nan, np.inf
    x[4] = -np.inf                               # a block of nothing finite
    slots = np.array([0, 1, 17, 48, 32], dtype=np.int64)
    st = status_word(torch)
    L.lq_kv_append(to_dev(torch, x), to_dev(torch, x), to_dev(torch, slots), *cache, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == L.LQ_DEV_RANGE | L.LQ_DEV_NONFINITE
    keep = np.array([0, 1, 2, 4])
    check_append([x[keep]] * 2, slots[keep], codes, scales, cache, 16)
    assert not cache[0][0, :, 0].any() and not cache[0][2, :, 0].any() and not cache[1][2].any()
    ko, vo = (torch.empty((2, 2, 64), device="cuda") for _ in range(2))
    st.zero_()
    L.lq_kv_gather(to_dev(torch, np.array([-1, 48], dtype=np.int64)), *cache, ko, vo, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == L.LQ_DEV_RANGE and not ko.any() and not vo.any()


def test_append_rounds_halves_to_even_and_clips_nothing():
    """Values whose quotients are exactly k + 1/2 (scale a power of two), both signs."""
    torch, L = cuda()
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :8] = [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5]
    _, _, cache = make_cache(torch, np.random.default_rng(0), 1, 1, 16, 64)
    L.lq_kv_append(to_dev(torch, x), to_dev(torch, x), to_dev(torch, np.zeros(1, np.int64)), *cache)
    torch.cuda.synchronize()
    assert cache[0][0, 0, 0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 64] and float(cache[1][0, 0]) == 1.0


# ------------------------------------------------------------------ verification
def probs(rng, shape, sharp):
    z = rng.standard_normal(shape) * sharp
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,k,vocab,onehot,lens", [(1, 3, 1000, False, False), (5, 1, 77, True, False),
                                                       (9, 4, 5001, False, True), (3, 7, 32000, True, True),
                                                       (2, 0, 333, False, False), (64, 2, 1, False, True),
                                                       (4, 40, 260, False, True), (2, 2, 128256, False, False)])
def test_verify(dtype, batch, k, vocab, onehot, lens):
    torch, L = cuda()
    rng = np.random.default_rng(vocab + k)
    p = probs(rng, (batch, k + 1, vocab), 2.0)
    q = probs(rng, (batch, k, vocab), 2.0)
    if k:
        q[:, ::2] = (p[:, :k] * rng.uniform(0.5, 1.1, p[:, :k].shape).astype(np.float32))[:, ::2]    # near the target
    x = np.minimum((rng.random((batch, k)) * 50).astype(np.int32), vocab - 1)
    n = rng.integers(0, k + 1, batch).astype(np.int32) if lens else None
    ua, us = rng.random((batch, k), np.float32), rng.random(batch, np.float32)
    us[0] = 0.0
    if batch > 1:
        us[1] = np.float32(1 - 2.0 ** -24)
    if dtype == "bf16":
        p, q = (torch.from_numpy(a).bfloat16().float().numpy() for a in (p, q))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    padded = torch.full((batch, k + 1, vocab + 3), 9.0, dtype=dt, device="cuda")     # rows further apart than they are long
    padded[:, :, :vocab] = to_dev(torch, p).to(dt)
    out = torch.full((batch, k + 1), -9, dtype=torch.int32, device="cuda")
    acc, st = torch.full((batch,), -9, dtype=torch.int32, device="cuda"), status_word(torch)
    L.lq_verify_draft(to_dev(torch, x), None if n is None else to_dev(torch, n), padded[:, :, :vocab],
                      None if onehot else to_dev(torch, q).to(dt), to_dev(torch, ua), to_dev(torch, us), out, acc, st)
    torch.cuda.synchronize()
    want, wacc = P.verify(x, n, p, None if onehot else q, ua, us)
    assert np.array_equal(acc.cpu().numpy(), wacc) and np.array_equal(out.cpu().numpy(), want)
    assert int(st) == 0


def test_verify_edges():
    """Equal distributions (nothing left of p - q), tokens and lengths out of range, rows without weight,
    NaN and infinity in the row drawn from and in rows that are not."""
    torch, L = cuda()
    rng = np.random.default_rng(4)
    b, k, v = 7, 2, 300
    p = probs(rng, (b, k + 1, v), 1.0)
    q = p[:, :k].copy()
    x = np.tile(np.array([[3, 5]], np.int32), (b, 1))
    ua, us = np.full((b, k), 0.5, np.float32), rng.random(b, np.float32)
    lens = np.full(b, k, np.int32)
    q[0, 0] = p[0, 0] * 1.5                     # refused at 0 with p - q nowhere positive: drawn from p
    ua[0, 0] = 0.9
    x[1, 1] = v                                 # token out of range
    x[2, 0] = -1
    lens[3] = 99                                # length out of range
    lens[4] = -1
    p[5, 2] = 0                                 # no weight in the row drawn from
    p[6, 2, 7], p[6, 2, 8] = np.nan, np.inf     # counted as zero and as 4
    p[0, 2], q[2, 1] = np.nan, np.nan           # rows that are not looked at
    out = torch.full((b, k + 1), -9, dtype=torch.int32, device="cuda")
    acc, st = torch.full((b,), -9, dtype=torch.int32, device="cuda"), status_word(torch)
    L.lq_verify_draft(to_dev(torch, x), to_dev(torch, lens), to_dev(torch, p), to_dev(torch, q), to_dev(torch, ua),
                      to_dev(torch, us), out, acc, st)
    torch.cuda.synchronize()
    want, wacc = P.verify(x, lens, p, q, ua, us)
    assert np.array_equal(acc.cpu().numpy(), wacc) and np.array_equal(out.cpu().numpy(), want)
    assert want[5, 2] == -1 and wacc[0] == 0 and want[0, 0] >= 0
    assert int(st) == L.LQ_DEV_RANGE | L.LQ_DEV_NONFINITE


def test_calls_follow_the_stream_they_are_given():
    """Inputs produced on a side stream and used there; a second stream waits for the result."""
    torch, L = cuda()
    s = torch.cuda.Stream()
    x = torch.zeros((64, 4, 128), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            x += 0.5
        ko, vo = torch.empty_like(x), torch.empty_like(x)
        cache = L.paged_cache(4, 4, 16, 128, "cuda")
        slots = torch.arange(64, device="cuda")
        L.lq_kv_append(x, x, slots, *cache)
        L.lq_kv_gather(slots, *cache, ko, vo)
    torch.cuda.current_stream().wait_stream(s)
    assert bool((ko == 10).all()) and bool((vo == 10).all())
