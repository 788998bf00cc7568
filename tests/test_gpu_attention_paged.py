"""lq_attention_paged on the GPU against the float64 oracle."""
import numpy as np
import pytest

import oracle.paged_oracle as P
from tests._parity import normwise_rel
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu

# Per query token and head (normwise over head_dim).  bf16: the output's rounding (2^-9) plus weights rounded to
# 11 bits or better (2^-12 each, of random sign), with a factor of two for values that cancel.  f32: some tens of
# fp32 roundings in a score of size about 30, in the exponent and in the sums: 1e-5.
TOL = {"bf16": 2.0 ** -8, "f32": 1e-5}


def build(torch, rng, reqs, hq, hk, bs, d, dtype, spare=3, v_scale=(0.005, 0.03), q_size=1.0, pad=0):
    counts = [-(-max(0, n) // bs) for n, _ in reqs]
    nb = sum(counts) + spare
    ids = rng.permutation(nb)
    width = max(counts + [1]) + 1
    table = np.full((len(reqs), width), -1, dtype=np.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = ids[at:at + c]
        at += c
    kc, vc = (np.clip(np.rint(rng.standard_normal((nb, hk, bs, d)) * 36), -127, 127).astype(np.int8) for _ in range(2))
    ks = rng.uniform(0.02, 0.04, (nb, hk)).astype(np.float32)
    vs = rng.uniform(*v_scale, (nb, hk)).astype(np.float32)
    cu = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = to_dev(torch, (q_size * rng.standard_normal((int(cu[-1]), hq * d + pad))).astype(np.float32)).to(dt)
    q = q[:, :hq * d].unflatten(1, (hq, d))
    lens = np.array([n for n, _ in reqs], dtype=np.int32)
    return dict(q=q, cu=cu, lens=lens, table=table, kc=kc, ks=ks, vc=vc, vs=vs)


def run(torch, L, s, status=None, sm_scale=None, out=None, stream_table=None):
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", "kc", "ks", "vc", "vs")}
    if stream_table is not None:
        dev["table"] = stream_table
    hq, d = s["q"].shape[1:]
    hk = s["kc"].shape[1]
    ws = torch.empty(L.lq_attention_paged_workspace_size(len(s["lens"]), s["q"].shape[0], hq, hk, d), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)
    if out is None:
        out = torch.full(tuple(s["q"].shape), float("nan"), dtype=s["q"].dtype, device="cuda")
    args = (s["q"], dev["cu"], dev["lens"], dev["table"], dev["kc"], dev["ks"], dev["vc"], dev["vs"], out, ws)
    L.lq_attention_paged(*args, sm_scale=sm_scale, dev_status=status)
    torch.cuda.synchronize()
    return out


def reference(s, sm_scale=None):
    d = s["q"].shape[2]
    return P.attention(s["q"].float().cpu().numpy(), s["cu"], s["lens"], s["table"], s["kc"], s["ks"], s["vc"], s["vs"],
                       d ** -0.5 if sm_scale is None else sm_scale)


def check(got, ref, dtype, rows=None):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g if rows is None else g[rows]).all()
    for t in (range(ref.shape[0]) if rows is None else rows):
        for h in range(ref.shape[1]):
            if not ref[t, h].any():
                assert not g[t, h].any()
            else:
                assert normwise_rel(g[t, h], ref[t, h]) < TOL[dtype], (t, h)


CASES = [
    # (kv_len, q_len) per request, q_heads, kv_heads, block, head_dim
    ([(1, 1)], 1, 1, 16, 128),
    ([(17, 1), (16, 1), (15, 1), (33, 1)], 4, 2, 16, 128),
    ([(300, 1), (1, 1), (64, 1), (65, 1)], 32, 8, 64, 128),
    ([(5000, 1)], 8, 1, 128, 128),
    ([(700, 1), (130, 1)], 7, 1, 32, 64),
    ([(257, 3), (40, 5), (9, 9), (128, 1)], 14, 2, 32, 64),
    ([(333, 2), (50, 50)], 3, 3, 16, 256),
    ([(400, 130)], 8, 2, 64, 128),
    ([(200, 200), (1000, 17), (64, 1)], 10, 2, 128, 128),
    ([(150, 70)], 16, 1, 16, 64),
    ([(900, 300)], 4, 4, 32, 128),
    ([(i * 7 % 90 + 1, 1) for i in range(150)], 2, 1, 16, 128),
    # many rows for few heads over long caches: the positions are split
    ([(5000, 40)], 4, 2, 16, 128),
    ([(3000, 70), (100, 66)], 4, 1, 64, 256),
    ([(2600, 300), (700, 5)], 2, 1, 32, 64),
    ([(3, 200), (4000, 90)], 2, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reqs,hq,hk,bs,d", CASES)
def test_attention(dtype, reqs, hq, hk, bs, d):
    torch, L = cuda()
    s = build(torch, np.random.default_rng(sum(n for n, _ in reqs) + d), reqs, hq, hk, bs, d, dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, reference(s), dtype)
    assert torch.equal(got, run(torch, L, s, st))          # equal calls, equal bits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing_and_requests_without_rows(dtype):
    """No cached tokens, more query tokens than tokens, requests with no query tokens: zeros or nothing."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(5), [(0, 2), (3, 8), (50, 0), (70, 1), (0, 0), (20, 40)], 6, 2, 16, 128, dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    ref = reference(s)
    assert int(st) == 0 and not ref[:7].any() and ref[7:11].any()
    check(got, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 70])
@pytest.mark.parametrize("exponent", [-105, -40, 105])
def test_queries_near_the_ends_of_their_range(dtype, q_len, exponent):
    """Queries times a power of two and the scale, here below 0, times its inverse: the result does not move."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(16), [(300, q_len), (90, 3)], 8, 2, 32, 128, dtype, q_size=2.0 ** exponent)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = -0.088 * 2.0 ** -exponent
    got = run(torch, L, s, st, sm_scale=scale)
    assert int(st) == 0
    check(got, reference(s, scale), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 5, 200])
def test_strides_scale_and_peaked_scores(dtype, q_len):
    """Queries and outputs as columns of wider rows, a table wider than its columns, sm_scale given, scores in
    the hundreds (the softmax is nearly one-hot)."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(6), [(500, q_len), (260, 1)], 8, 2, 32, 128, dtype, pad=64, q_size=4.0)
    wide = to_dev(torch, np.concatenate([s["table"], np.full((2, 9), 77, np.int32)], 1))
    rows = torch.full((s["q"].shape[0], 8 * 128 + 40), 3.0, dtype=s["q"].dtype, device="cuda")
    out = rows[:, :1024].unflatten(1, (8, 128))
    got = run(torch, L, s, None, sm_scale=0.2, out=out, stream_table=wide[:, :s["table"].shape[1]])
    check(got, reference(s, 0.2), dtype)
    assert bool((rows[:, 1024:] == 3.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("span", [(1e-30, 1e-28), (1e25, 1e27), (1e-9, 1e3)])
def test_value_scales_of_any_size(dtype, span):
    """Value scales far from one, and scales that differ by powers of ten between blocks."""
    torch, L = cuda()
    rng = np.random.default_rng(7)
    s = build(torch, rng, [(400, 2)], 4, 2, 16, 128, dtype)
    s["vs"] = np.exp(rng.uniform(np.log(span[0]), np.log(span[1]), s["vs"].shape)).astype(np.float32)
    check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_scales(dtype):
    """Blocks of zeros among others; all values zero; all keys zero (a plain mean)."""
    torch, L = cuda()
    rng = np.random.default_rng(8)
    s = build(torch, rng, [(90, 3)], 4, 2, 16, 128, dtype)
    s["vs"][::2] = 0
    check(run(torch, L, s), reference(s), dtype)
    s["ks"][:] = 0
    check(run(torch, L, s), reference(s), dtype)
    s["vs"][:] = 0
    assert float(run(torch, L, s).abs().max()) < 1e-30


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("q_len", [2, 40, 200])
def test_scales_a_row_does_not_see(dtype, bad, q_len):
    """A block that only later query tokens see holds non-finite or enormous scales: earlier ones are not touched by
    it; nor by blocks past the length or in the pool."""
    torch, L = cuda()
    rng = np.random.default_rng(9)
    s = build(torch, rng, [(15 * 16 + 1, q_len)], 4, 2, 16, 128, dtype)
    last = s["table"][0, 15]
    used = s["table"][0, :16]
    for n in ("ks", "vs"):
        s[n][last] = bad
        s[n][[b for b in range(s[n].shape[0]) if b not in used]] = bad
    ref = reference({**s, "lens": np.array([15 * 16], np.int32), "cu": np.array([0, q_len - 1], np.int32)})
    got = run(torch, L, s)
    # the last query token alone sees position 240, the bad block's only token in use
    check(got, ref, dtype, rows=range(q_len - 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_queries_stay_in_their_row(dtype, bad):
    torch, L = cuda()
    s = build(torch, np.random.default_rng(10), [(100, 3), (50, 1)], 4, 2, 16, 128, dtype)
    ref = reference(s)
    s["q"][1, 2, 5] = bad
    got = run(torch, L, s)
    assert not bool(torch.isfinite(got[1, 2]).any())
    ref[1, 2] = 0
    got[1, 2] = 0
    check(got, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_blocks_outside_the_pool_and_lengths_past_the_table(dtype):
    torch, L = cuda()
    rng = np.random.default_rng(11)
    for entry in (-1, 1 << 30):
        s = build(torch, rng, [(100, 2), (64, 1)], 4, 2, 16, 128, dtype)
        s["table"][0, 2] = entry
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(torch, L, s, st)
        assert int(st) == L.LQ_DEV_RANGE
        check(got, reference(s), dtype)
    s = build(torch, rng, [(100, 2), (64, 1)], 4, 2, 16, 128, dtype)
    s["table"] = np.ascontiguousarray(s["table"][:, :5])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    check(got, reference(s), dtype)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes whose used blocks lie at its end."""
    torch, L = cuda()
    nb, hk, bs, d = 70000, 4, 128, 128          # 4.6 GB of codes each for K and V
    rng = np.random.default_rng(12)
    s = build(torch, rng, [(600, 2), (100, 1)], 8, hk, bs, d, "bf16", spare=0)
    n = s["kc"].shape[0]
    cache = L.paged_cache(nb, hk, bs, d, "cuda")
    for dst, src in zip(cache, ("kc", "ks", "vc", "vs")):
        dst[nb - n:] = to_dev(torch, s[src])
    table = np.where(s["table"] >= 0, s["table"] + nb - n, -1).astype(np.int32)
    ws = torch.empty(L.lq_attention_paged_workspace_size(2, 3, 8, hk, d), dtype=torch.uint8, device="cuda")
    out, st = torch.empty_like(s["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_attention_paged(s["q"], to_dev(torch, s["cu"]), to_dev(torch, s["lens"]), to_dev(torch, table), *cache, out, ws,
                         dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    check(out, reference(s), "bf16")
    # and writes and reads at that end
    slots = torch.arange(nb * bs - 5, nb * bs, device="cuda")
    x = torch.randn((5, hk, d), device="cuda")
    L.lq_kv_append(x, x, slots, *cache)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    L.lq_kv_gather(slots, *cache, ko, vo)
    torch.cuda.synchronize()
    step = cache[1][nb - 1].view(1, hk, 1)
    assert bool(((ko - x).abs() <= 0.5001 * step).all()) and bool((vo == ko).sum() > 0)
    del cache


def test_tokens_of_a_graph_replay():
    """The call captures into a CUDA graph and follows lengths that change between replays."""
    torch, L = cuda()
    rng = np.random.default_rng(13)
    s = build(torch, rng, [(300, 1), (200, 1)], 8, 2, 16, 128, "bf16")
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", "kc", "ks", "vc", "vs")}
    ws = torch.empty(L.lq_attention_paged_workspace_size(2, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(s["q"])
    call = lambda: L.lq_attention_paged(s["q"], dev["cu"], dev["lens"], dev["table"], dev["kc"], dev["ks"], dev["vc"],
                                        dev["vs"], out, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([300, 200], [1, 150], [37, 0]):
        s["lens"] = np.array(lens, np.int32)
        dev["lens"].copy_(to_dev(torch, s["lens"]))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(out, reference(s), "bf16")
