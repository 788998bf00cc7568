"""lq_attention_paged_q4 on the GPU against the oracle."""
import numpy as np
import pytest

import oracle.q4_oracle as Q
from tests._parity import normwise_rel
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu

# Per query token and head (normwise over head_dim).  bf16: the output's rounding (2^-9) plus weights rounded to
# 11 bits or better (2^-12 each, of random sign), with a factor of two for values that cancel.  f32: some tens of
# fp32 roundings in a score of size about 30, in the exponent and in the sums: 1e-5.
TOL = {"bf16": 2.0 ** -8, "f32": 1e-5}
CACHE = ("kc", "ks", "vc", "vs")


def build(torch, rng, reqs, hq, hk, bs, d, group, dtype, spare=3, q_size=1.0, pad=0):
    counts = [-(-max(0, n) // bs) for n, _ in reqs]
    nb = sum(counts) + spare
    ids = rng.permutation(nb)
    table = np.full((len(reqs), max(counts + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = ids[at:at + c]
        at += c
    s = {"table": table, "lens": np.array([n for n, _ in reqs], np.int32),
         "cu": np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)}
    for n, size in (("k", 1.0), ("v", 0.5)):
        c = np.clip(np.rint(rng.standard_normal((nb, hk, bs, d)) * 2.7 + 7.5), 0, 15).astype(np.uint8)
        s[n + "c"] = c[..., ::2] | c[..., 1::2] << 4
        scale = rng.uniform(0.2, 0.4, (nb, hk, bs, d // group)) * size
        s[n + "s"] = np.stack([scale, scale * (-23.5 + 0.5 * rng.standard_normal(scale.shape))], -1).astype(np.float16)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = to_dev(torch, (q_size * rng.standard_normal((int(s["cu"][-1]), hq * d + pad))).astype(np.float32)).to(dt)
    s["q"] = q[:, :hq * d].unflatten(1, (hq, d))
    return s


def workspace(torch, L, s):
    hq, d = s["q"].shape[1:]
    size = L.lq_attention_paged_q4_workspace_size(len(s["lens"]), s["q"].shape[0], hq, s["kc"].shape[1], d)
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")


def run(torch, L, s, status=None, sm_scale=None, out=None, table=None):
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", *CACHE)}
    if out is None:
        out = torch.full(tuple(s["q"].shape), float("nan"), dtype=s["q"].dtype, device="cuda")
    L.lq_attention_paged_q4(s["q"], dev["cu"], dev["lens"], dev["table"] if table is None else table,
                            *(dev[n] for n in CACHE), out, workspace(torch, L, s), sm_scale=sm_scale, dev_status=status)
    torch.cuda.synchronize()
    return out


def reference(s, sm_scale=None):
    return Q.attention(s["q"].float().cpu().numpy(), s["cu"], s["lens"], s["table"], *(s[n] for n in CACHE),
                       s["q"].shape[2] ** -0.5 if sm_scale is None else sm_scale)


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
    # (kv_len, q_len) per request, q_heads, kv_heads, block, head_dim, group
    ([(1, 1)], 1, 1, 16, 128, 128),
    ([(17, 1), (16, 1), (15, 1), (33, 1)], 4, 2, 16, 128, 64),
    ([(300, 1), (1, 1), (64, 1), (65, 1)], 32, 8, 64, 128, 32),
    ([(5000, 1)], 8, 1, 128, 128, 64),
    ([(700, 1), (130, 1)], 7, 1, 32, 64, 64),
    ([(257, 3), (40, 5), (9, 9), (128, 1)], 14, 2, 32, 64, 32),
    ([(333, 2), (50, 50)], 3, 3, 16, 256, 128),
    ([(150, 1), (31, 1)], 8, 2, 64, 256, 32),
    ([(400, 130)], 8, 2, 64, 128, 128),
    ([(200, 200), (1000, 17), (64, 1)], 10, 2, 128, 128, 32),
    ([(150, 70)], 16, 1, 16, 64, 32),
    ([(900, 300)], 4, 4, 32, 128, 64),
    ([(i * 7 % 90 + 1, 1) for i in range(150)], 2, 1, 16, 128, 64),
    # many rows for few heads over long caches: the positions are split
    ([(5000, 40)], 4, 2, 16, 128, 64),
    ([(3001, 70), (100, 66)], 4, 1, 64, 256, 64),
    ([(2600, 300), (700, 5)], 2, 1, 32, 64, 32),
    ([(3, 200), (4000, 90)], 2, 2, 128, 128, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reqs,hq,hk,bs,d,group", CASES)
def test_attention(dtype, reqs, hq, hk, bs, d, group):
    torch, L = cuda()
    s = build(torch, np.random.default_rng(sum(n for n, _ in reqs) + d), reqs, hq, hk, bs, d, group, dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, reference(s), dtype)
    assert torch.equal(got, run(torch, L, s, st))          # equal calls, equal bits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 129])
def test_every_number_of_rows(dtype, d, rows):
    """Query rows of a kv head around the kernels' tile sizes, the request's last tokens inside a tile and a block."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(rows), [(rows + 75, rows), (rows, rows)], 3, 3, 16, d, 32, dtype)
    check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("q_len", [1, 40])
def test_lengths_around_tiles(dtype, length, q_len):
    torch, L = cuda()
    for bs in (16, 128):
        s = build(torch, np.random.default_rng(length), [(length, q_len)], 2, 1, bs, 128, 64, dtype)
        check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing_and_requests_without_rows(dtype):
    """No cached tokens, more query tokens than tokens, requests with no query tokens: zeros or nothing."""
    torch, L = cuda()
    for reqs in ([(0, 2), (3, 8), (50, 0), (70, 1), (0, 0), (20, 40)], [(0, 1), (9, 1), (0, 1)], [(0, 300), (10, 290)]):
        s = build(torch, np.random.default_rng(5), reqs, 6, 2, 16, 128, 64, dtype)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(torch, L, s, st)
        assert int(st) == 0
        check(got, reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 70])
def test_tokens_that_no_request_owns(dtype, q_len):
    torch, L = cuda()
    s = build(torch, np.random.default_rng(15), [(90, q_len), (40, 2)], 4, 2, 16, 128, 64, dtype)
    s["cu"] = np.array([0, q_len - 1, q_len], np.int32)        # the last tokens are nobody's
    check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 70])
@pytest.mark.parametrize("exponent", [-105, -40, 105])
def test_queries_near_the_ends_of_their_range(dtype, q_len, exponent):
    """Queries times a power of two and the scale, here below 0, times its inverse: the result does not move."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(16), [(300, q_len), (90, 3)], 8, 2, 32, 128, 32, dtype, q_size=2.0 ** exponent)
    scale = -0.088 * 2.0 ** -exponent
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st, sm_scale=scale)
    assert int(st) == 0
    check(got, reference(s, scale), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 5, 200])
def test_strides_scale_and_peaked_scores(dtype, q_len):
    """Queries and outputs as columns of wider rows, a table wider than its columns, sm_scale given, scores in
    the hundreds (the softmax is nearly one-hot)."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(6), [(500, q_len), (260, 1)], 8, 2, 32, 128, 64, dtype, pad=64, q_size=4.0)
    wide = to_dev(torch, np.concatenate([s["table"], np.full((2, 9), 77, np.int32)], 1))
    rows = torch.full((s["q"].shape[0], 8 * 128 + 40), 3.0, dtype=s["q"].dtype, device="cuda")
    got = run(torch, L, s, None, sm_scale=0.2, out=rows[:, :1024].unflatten(1, (8, 128)),
              table=wide[:, :s["table"].shape[1]])
    check(got, reference(s, 0.2), dtype)
    assert bool((rows[:, 1024:] == 3.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 60])
@pytest.mark.parametrize("size", [2.0 ** -13, 2.0 ** 10, None])
def test_cached_values_of_any_size(dtype, q_len, size):
    """Values near the ends of fp16's range, and of sizes that differ by powers of ten between tokens and groups."""
    torch, L = cuda()
    rng = np.random.default_rng(7)
    s = build(torch, rng, [(400, q_len)], 4, 2, 16, 128, 32, dtype)
    f = size if size is not None else np.exp(rng.uniform(np.log(1e-3), np.log(1e3), s["vs"].shape[:-1]))[..., None]
    s["vs"] = (s["vs"].astype(np.float64) * f).astype(np.float16)
    check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 60])
def test_equal_keys_and_zero_values(dtype, q_len):
    """All keys alike (a plain mean); all values zero."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(8), [(90, q_len)], 4, 2, 16, 128, 64, dtype)
    s["ks"][:] = 0
    check(run(torch, L, s), reference(s), dtype)
    s["vs"][:] = 0
    assert not run(torch, L, s).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 3, 40, 200])
@pytest.mark.parametrize("bs", [16, 128])
def test_slots_without_tokens_may_hold_anything(dtype, q_len, bs):
    """NaN and infinite scales behind the last token of a block and in blocks that no request has."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(9), [(245, q_len), (1, 1), (130, 1)], 4, 2, bs, 128, 32, dtype)
    ref = reference(s)
    held = np.zeros((s["kc"].shape[0], bs), bool)
    for i, n in enumerate(s["lens"]):
        for p in range(n):
            held[s["table"][i, p // bs], p % bs] = True
    for n in ("ks", "vs"):
        for value, part in ((np.nan, slice(0, 3)), (np.inf, slice(3, 9)), (-np.inf, slice(9, None))):
            empty = ~held
            keep = np.zeros_like(empty)
            keep[:, part] = True
            s[n].transpose(0, 2, 1, 3, 4)[empty & keep] = value
    s["kc"].transpose(0, 2, 1, 3)[~held] = 255
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [3, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_queries_stay_in_their_row(dtype, q_len, bad):
    torch, L = cuda()
    s = build(torch, np.random.default_rng(10), [(100, q_len), (50, 1)], 4, 2, 16, 128, 64, dtype)
    ref = reference(s)
    s["q"][1, 2, 5] = bad
    got = run(torch, L, s)
    assert not bool(torch.isfinite(got[1, 2]).any())
    ref[1, 2] = 0
    got[1, 2] = 0
    check(got, ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 50])
@pytest.mark.parametrize("bs", [16, 64])
def test_blocks_outside_the_pool_and_lengths_past_the_table(dtype, q_len, bs):
    torch, L = cuda()
    rng = np.random.default_rng(11)
    for entry in (-1, 1 << 30):
        s = build(torch, rng, [(300, q_len), (64, 1)], 4, 2, bs, 128, 64, dtype)
        s["table"][0, 2] = entry
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(torch, L, s, st)
        assert int(st) == L.LQ_DEV_RANGE
        check(got, reference(s), dtype)
    s = build(torch, rng, [(300, q_len), (64, 1)], 4, 2, bs, 128, 64, dtype)
    s["table"] = np.ascontiguousarray(s["table"][:, :-2])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    check(got, reference(s), dtype)
    s["table"][:] = -1                                         # nothing is there
    st.zero_()
    assert not run(torch, L, s, st).any() and int(st) == L.LQ_DEV_RANGE


@pytest.mark.parametrize("q_len", [1, 60])
def test_offsets_past_32_bits(q_len):
    """A pool of more than 2^32 bytes of codes whose used blocks lie at its end."""
    torch, L = cuda()
    nb, hk, bs, d, group = 140000, 4, 128, 128, 128            # 4.6 GB of codes each for K and V
    s = build(torch, np.random.default_rng(12), [(600, q_len), (100, 1)], 8, hk, bs, d, group, "bf16", spare=0)
    n = s["kc"].shape[0]
    cache = L.paged_cache_q4(nb, hk, bs, d, group, "cuda")
    for dst, src in zip(cache, CACHE):
        dst[nb - n:] = to_dev(torch, s[src])
    table = np.where(s["table"] >= 0, s["table"] + nb - n, -1).astype(np.int32)
    out, st = torch.empty_like(s["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_attention_paged_q4(s["q"], to_dev(torch, s["cu"]), to_dev(torch, s["lens"]), to_dev(torch, table), *cache, out,
                            workspace(torch, L, s), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    check(out, reference(s), "bf16")
    # and writes and reads at that end
    slots = torch.arange(nb * bs - 5, nb * bs, device="cuda")
    x = torch.randn((5, hk, d), device="cuda")
    L.lq_kv_append_q4(x, x, slots, *cache)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    L.lq_kv_gather_q4(slots, *cache, ko, vo)
    want = Q.values(*Q.quantize(x.cpu().numpy(), group)).astype(np.float32)
    assert np.array_equal(ko.cpu().numpy(), want) and torch.equal(ko, vo)
    del cache


@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("f32", 1), ("bf16", 40)])
def test_replayed_graphs(dtype, q_len):
    """Two captured calls that share a workspace on one stream, each following lengths that change between replays."""
    torch, L = cuda()
    cases, graphs = [], []
    for seed in (13, 14):
        s = build(torch, np.random.default_rng(seed), [(300, q_len), (200, q_len)], 8, 2, 16, 128, 64, dtype)
        cases.append((s, {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", *CACHE)}, torch.empty_like(s["q"])))
    ws = workspace(torch, L, cases[0][0])

    def call(s, dev, out):
        L.lq_attention_paged_q4(s["q"], dev["cu"], dev["lens"], dev["table"], *(dev[n] for n in CACHE), out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*cases[0])
    torch.cuda.synchronize()
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(*c)
    for lens in ([300, 200], [1, 150], [37, 0]):
        for s, dev, out in cases:
            s["lens"] = np.array(lens, np.int32)
            dev["lens"].copy_(to_dev(torch, s["lens"]))
            out.fill_(7.0)
        for g in (*graphs, *graphs):
            g.replay()
        torch.cuda.synchronize()
        for s, _, out in cases:
            check(out, reference(s), dtype)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(8, 2), (4, 4)])
def test_requests_of_very_different_lengths(d, hq, hk):
    """Long requests beside short and empty ones, enough query rows for the tensor-core kernel: how many CTAs share a
    request follows from the lengths, which change under a captured graph.  Bytes around the workspace stay."""
    torch, L = cuda()
    reqs = [(9000, 37), (0, 3), (1, 150), (64, 17), (0, 0), (700, 300), (129, 1), (2500, 90), (65, 65)]
    s = build(torch, np.random.default_rng(d + hq), reqs, hq, hk, 16, d, 32, "bf16")
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", *CACHE)}
    out = torch.full(tuple(s["q"].shape), float("nan"), dtype=s["q"].dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = L.lq_attention_paged_q4_workspace_size(len(reqs), s["q"].shape[0], hq, hk, d)
    guarded = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    work = guarded[4096:4096 + size]
    work.fill_(0xFF)

    def call():
        L.lq_attention_paged_q4(s["q"], dev["cu"], dev["lens"], dev["table"], *(dev[n] for n in CACHE), out, work,
                                dev_status=st)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([n for n, _ in reqs], [40, 0, 1, 30, 0, 333, 129, 2400, 64], [8, 0, 1, 0, 0, 7, 2, 5, 1]):
        s["lens"] = np.array(lens, np.int32)
        dev["lens"].copy_(to_dev(torch, s["lens"]))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(out, reference(s), "bf16")
    assert int(st) == 0
    assert bool((guarded[:4096] == 0xA5).all()) and bool((guarded[4096 + size:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [2, 70])
def test_maxima_that_rise(dtype, d, q_len):
    """Keys that grow with their position: the running maximum moves again and again."""
    torch, L = cuda()
    reqs = [(3001, q_len), (700, q_len)]
    s = build(torch, np.random.default_rng(31), reqs, 4, 2, 16, d, 64, dtype, q_size=8.0)
    for i, (n, _) in enumerate(reqs):
        size = np.linspace(0.02, 1.0, n) ** 2
        for p in range(n):
            s["ks"][s["table"][i, p // 16], :, p % 16] = (s["ks"][s["table"][i, p // 16], :, p % 16].astype(np.float64)
                                                           * size[p]).astype(np.float16)
    check(run(torch, L, s), reference(s), dtype)


@pytest.mark.parametrize("d,q_len", [(64, 14), (128, 10), (256, 5)])
@pytest.mark.parametrize("length", [40, 750])
def test_many_requests_with_some_rows(d, q_len, length):
    """More requests than CTAs can share, rows between the two kernels' ranges, short contexts and longer ones."""
    torch, L = cuda()
    rng = np.random.default_rng(d + length)
    reqs = [(int(n), q_len) for n in rng.integers(1, length, 170)]
    s = build(torch, rng, reqs, 16, 4, 16, d, 64, "bf16")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == 0
    seen = [i for i in range(0, len(reqs) * q_len, 37)]
    check(got, reference(s), "bf16", seen)
