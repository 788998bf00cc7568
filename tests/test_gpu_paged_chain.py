"""Plan, norms with rotation, cache writes, attention and read-back called back to back, each on what the call before has
just written, give the bits of the same calls with a synchronisation after each."""
import numpy as np
import pytest

from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu

STEPS = 30


def serve(torch, L, reqs, hq, hk, bs, d, dt, q_len, synced):
    rng = np.random.default_rng(21)
    sync = torch.cuda.synchronize if synced else (lambda: None)
    b, n = len(reqs), len(reqs) * q_len
    held = [-(-c // bs) for c in reqs]
    need = [-(-(c + STEPS * q_len) // bs) for c in reqs]
    nb, width = sum(need), max(need)
    ids = rng.permutation(nb).astype(np.int32)
    rows = np.full((b, width), -1, np.int32)
    at = 0
    for i, c in enumerate(held):
        rows[i, :c] = ids[at:at + c]
        at += c
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
    table, free = to_dev(torch, rows), to_dev(torch, ids)
    cache = L.paged_cache(nb, hk, bs, d, "cuda")
    codes = rng.integers(-127, 128, (2, nb, hk, bs, d)).astype(np.int8)
    for c, x in zip((cache[0], cache[2]), codes):
        c.copy_(to_dev(torch, x))
    for s in (cache[1], cache[3]):
        s.copy_(to_dev(torch, rng.uniform(0.001, 0.002, (nb, hk)).astype(np.float32)))
    # later rows are larger: almost every write makes its block's scales grow
    grow = np.linspace(0.2, 3.0, STEPS)[:, None, None, None]
    x = [to_dev(torch, (rng.standard_normal((STEPS, n, h, d)) * grow).astype(np.float32)).to(dt) for h in (hq, hk, hk)]
    w = to_dev(torch, rng.uniform(0.5, 2, d).astype(np.float32))
    angles = to_dev(torch, rng.uniform(-1, 1, (max(reqs) + STEPS * q_len, d)).astype(np.float32))
    lens = [to_dev(torch, np.array(reqs, np.int32))] + [i32(b) for _ in range(STEPS)]
    new, cu, used, st = to_dev(torch, np.full(b, q_len, np.int32)), i32(b + 1), i32(1), i32(1)
    slots, pos = torch.zeros(n, dtype=torch.int64, device="cuda"), i32(n)
    ws = torch.empty(L.lq_attention_paged_workspace_size(b, n, hq, hk, d), dtype=torch.uint8, device="cuda")
    out = torch.zeros((STEPS, n, hq, d), dtype=dt, device="cuda")
    back = torch.zeros((STEPS, 2, n, hk, d), dtype=dt, device="cuda")
    torch.cuda.synchronize()
    for s in range(STEPS):
        q, k, v = (t[s] for t in x)
        L.lq_kv_plan(lens[s], new, bs, free[at:], table, cu, lens[s + 1], slots, pos, used, st)
        sync()
        L.lq_qk_norm_rope(q, k, w, None, 1e-6, pos, angles, q, k, dev_status=st)
        sync()
        L.lq_kv_append(k, v, slots, *cache, dev_status=st)
        sync()
        L.lq_attention_paged(q, cu, lens[s + 1], table, *cache, out[s], ws, dev_status=st)
        sync()
        L.lq_kv_gather(slots, *cache, back[s, 0], back[s, 1], dev_status=st)
        sync()
        at += sum(-(-(c + (s + 1) * q_len) // bs) + -(c + s * q_len) // bs for c in reqs)
    torch.cuda.synchronize()
    assert int(st) == 0
    return [out, back, table, lens[-1], *cache]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("reqs,hq,hk,bs,d,q_len", [([5, 40, 0, 300], 16, 8, 16, 64, 1), ([100, 33], 8, 8, 32, 128, 5),
                                                   ([700, 0, 90], 16, 8, 16, 128, 40)])
def test_calls_back_to_back(dtype, reqs, hq, hk, bs, d, q_len):
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    want = serve(torch, L, reqs, hq, hk, bs, d, dt, q_len, True)
    for _ in range(5):
        for got, ref in zip(serve(torch, L, reqs, hq, hk, bs, d, dt, q_len, False), want):
            assert torch.equal(got, ref)
