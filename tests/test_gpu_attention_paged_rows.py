"""lq_attention_paged's special cases at every number of query rows: a few (the split kernel), some dozens and prompts (the
tensor-core kernel), and few row tiles over long caches, whose positions several CTAs share."""
import numpy as np
import pytest

from tests.gpu_util import cuda, to_dev
from tests.test_gpu_attention_paged import build, check, reference, run

pytestmark = pytest.mark.gpu

# (kv_len, q_len) per request, q_heads, kv_heads, block, head_dim
SHAPES = [([(100, 2), (64, 1)], 4, 2, 16, 128), ([(130, 40), (64, 25)], 4, 2, 16, 128), ([(420, 200), (300, 130)], 4, 2, 32, 64),
          ([(260, 70), (200, 66)], 3, 1, 64, 256), ([(5000, 40)], 4, 2, 16, 128), ([(3000, 70)], 4, 1, 64, 256),
          ([(2600, 300)], 2, 1, 128, 64)]
both = pytest.mark.parametrize("dtype", ["bf16", "f32"])
every = pytest.mark.parametrize("shape", range(len(SHAPES)))


def made(torch, shape, dtype, seed=41, **kw):
    return build(torch, np.random.default_rng(seed + shape), *SHAPES[shape], dtype, **kw)


def status(torch):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@both
@every
def test_zero_scales(dtype, shape):
    torch, L = cuda()
    s = made(torch, shape, dtype)
    s["vs"][::2] = 0
    check(run(torch, L, s), reference(s), dtype)
    s["ks"][:] = 0                               # a plain mean
    check(run(torch, L, s), reference(s), dtype)
    s["vs"][:] = 0
    assert not run(torch, L, s).any()


@both
@every
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_queries(dtype, shape, bad):
    """They stay in their own row."""
    torch, L = cuda()
    s = made(torch, shape, dtype)
    ref = reference(s)
    n, hq, d = s["q"].shape
    rows = [(0, 1, 5), (n // 2, 0, 0), (n - 1, hq - 1, d - 1)]
    for t, h, c in rows:
        s["q"][t, h, c] = bad
    got = run(torch, L, s)
    for t, h, _ in rows:
        assert not bool(torch.isfinite(got[t, h]).any())
        ref[t, h] = 0
        got[t, h] = 0
    check(got, ref, dtype)


@both
@every
@pytest.mark.parametrize("entry", [-1, 1 << 30, -(1 << 31)])
def test_blocks_outside_the_pool(dtype, shape, entry):
    torch, L = cuda()
    s = made(torch, shape, dtype)
    s["table"][0, 1] = entry
    s["table"][0, (s["lens"][0] - 1) // s["kc"].shape[2] // 2] = entry
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    check(got, reference(s), dtype)


@both
@every
def test_a_request_without_any_block(dtype, shape):
    torch, L = cuda()
    s = made(torch, shape, dtype)
    s["table"][0, :] = -1
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    ref = reference(s)
    assert not ref[:s["cu"][1]].any()
    check(got, ref, dtype)


@both
@every
def test_lengths_past_the_table(dtype, shape):
    """Cut at the table's end: the first query tokens see what is left, as by their positions."""
    torch, L = cuda()
    s = made(torch, shape, dtype)
    s["table"] = np.ascontiguousarray(s["table"][:, :max(1, (s["table"].shape[1] - 1) * 2 // 3)])
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    check(got, reference(s), dtype)


@both
@every
def test_zero_scales_of_missing_and_far_blocks_together(dtype, shape):
    """Zeros, a missing block and values far apart in one request."""
    torch, L = cuda()
    s = made(torch, shape, dtype)
    used = [b for b in s["table"][0] if b >= 0]
    s["vs"][used[::3]] = 0
    s["vs"][used[1::3]] *= 2.0 ** 90
    s["table"][0, len(used) // 2] = -1
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == L.LQ_DEV_RANGE
    check(got, reference(s), dtype)


@both
@every
def test_more_query_tokens_than_tokens_and_empty_requests(dtype, shape):
    """Rows that see nothing, among requests of no rows or no tokens."""
    torch, L = cuda()
    reqs, hq, hk, bs, d = SHAPES[shape]
    q = reqs[0][1]
    reqs = [(0, 0), (q // 2, q), (0, q), reqs[0], (40, 0), (1, q)]
    s = build(torch, np.random.default_rng(50 + shape), reqs, hq, hk, bs, d, dtype)
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, reference(s), dtype)


@both
@pytest.mark.parametrize("rows_past", [0, 3])
@every
def test_rows_that_no_request_owns(dtype, shape, rows_past):
    torch, L = cuda()
    s = made(torch, shape, dtype)
    n = int(s["cu"][-1])
    s["q"] = torch.cat([s["q"], s["q"][:rows_past]]) if rows_past else s["q"]
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == 0 and not got[n:].any()
    check(got[:n], reference(s)[:n], dtype)


def test_offsets_past_32_bits_in_prompts():
    """A pool of more than 2^32 bytes of codes whose used blocks lie at its end, read by the tensor-core kernel."""
    torch, L = cuda()
    nb, hk, bs, d = 70000, 4, 128, 128
    s = build(torch, np.random.default_rng(61), [(600, 200), (300, 70)], 8, hk, bs, d, "bf16", spare=0)
    n = s["kc"].shape[0]
    cache = L.paged_cache(nb, hk, bs, d, "cuda")
    for dst, src in zip(cache, ("kc", "ks", "vc", "vs")):
        dst[nb - n:] = to_dev(torch, s[src])
    table = np.where(s["table"] >= 0, s["table"] + nb - n, -1).astype(np.int32)
    ws = torch.empty(L.lq_attention_paged_workspace_size(2, 270, 8, hk, d), dtype=torch.uint8, device="cuda")
    out, st = torch.empty_like(s["q"]), status(torch)
    L.lq_attention_paged(s["q"], to_dev(torch, s["cu"]), to_dev(torch, s["lens"]), to_dev(torch, table), *cache, out, ws,
                         dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    check(out, reference(s), "bf16")
    del cache


@pytest.mark.parametrize("q_len", [40, 200])
def test_a_graph_of_prompts(q_len):
    """Captured once, replayed with other lengths and other splits of the rows between the requests."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(62), [(700, q_len), (500, q_len)], 8, 2, 16, 128, "bf16")
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", "kc", "ks", "vc", "vs")}
    ws = torch.empty(L.lq_attention_paged_workspace_size(2, 2 * q_len, 8, 2, 128), dtype=torch.uint8, device="cuda")
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
    for lens, cut in (([700, 500], q_len), ([q_len, 30], q_len + 10), ([300, 499], 3), ([5, 0], 2 * q_len)):
        s["lens"], s["cu"] = np.array(lens, np.int32), np.array([0, cut, 2 * q_len], np.int32)
        dev["lens"].copy_(to_dev(torch, s["lens"]))
        dev["cu"].copy_(to_dev(torch, s["cu"]))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(out, reference(s), "bf16")


@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("f32", 1), ("bf16", 70), ("bf16", 4)])
def test_thirty_thousand_positions(dtype, q_len):
    """Sums over a long cache stay within the same tolerances (a truncating accumulator's bias would show)."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(63), [(30000, q_len)], 4, 1, 128, 128, dtype)
    # values that do not cancel
    s["vc"] = np.abs(s["vc"])
    st = status(torch)
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, reference(s), dtype)
