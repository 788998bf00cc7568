"""Guard bytes around every output, cache and workspace of the paged cache's calls."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,bs,hq,hk,reqs", [(128, 16, 4, 2, [(3, 1), (17, 5), (0, 40)]), (64, 32, 7, 1, [(200, 1)]),
                                             (256, 64, 2, 2, [(63, 2), (0, 130)]), (128, 128, 8, 1, [(3000, 70)])])
def test_paged_calls_stay_in_bounds(dtype, d, bs, hq, hk, reqs):
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    G = lambda *a: Guarded(torch, *a)
    b, n = len(reqs), sum(m for _, m in reqs)
    need = [-(-(c + m) // bs) for c, m in reqs]
    nb, width = sum(need), max(need)
    cached, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*reqs))
    table, cu, lens = G((b, width), torch.int32), G((b + 1,), torch.int32), G((b,), torch.int32)
    slots, pos, used = G((n,), torch.int64), G((n,), torch.int32), G((1,), torch.int32)
    table.t.fill_(-1)
    at = 0
    for i, (c, _) in enumerate(reqs):
        held = -(-c // bs)
        table.t[i, :held] = torch.arange(at, at + held, dtype=torch.int32, device="cuda")
        at += held
    free = torch.arange(at, nb, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_kv_plan(cached, new, bs, free, table.t, cu.t, lens.t, slots.t, pos.t, used.t, st)
    q, k, v = (torch.randn((n, h, d), device="cuda").to(dt) for h in (hq, hk, hk))
    w = torch.ones(d, device="cuda")
    table_cs = torch.rand((4000, d), device="cuda")
    qo, ko = G((n, hq, d), dt), G((n, hk, d), dt)
    L.lq_qk_norm_rope(q, k, w, w, 1e-6, pos.t, table_cs, qo.t, ko.t, dev_status=st)
    cache = [G((nb, hk, bs, d), torch.int8), G((nb, hk), torch.float32), G((nb, hk, bs, d), torch.int8),
             G((nb, hk), torch.float32)]
    for c in cache:
        c.t.zero_()
    pool = [c.t for c in cache]
    L.lq_kv_append(ko.t, v, slots.t, *pool, dev_status=st)
    kb, vb = G((n, hk, d), dt), G((n, hk, d), dt)
    L.lq_kv_gather(slots.t, *pool, kb.t, vb.t, dev_status=st)
    out = G((n, hq, d), dt)
    ws = G((L.lq_attention_paged_workspace_size(b, n, hq, hk, d),), torch.uint8)
    L.lq_attention_paged(qo.t, cu.t, lens.t, table.t, *pool, out.t, ws.t, dev_status=st)
    p = torch.softmax(torch.randn((b, 4, 333), device="cuda"), -1).to(dt)
    u = torch.rand((b, 3), device="cuda")
    toks, acc = G((b, 4), torch.int32), G((b,), torch.int32)
    L.lq_verify_draft(torch.zeros((b, 3), dtype=torch.int32, device="cuda"), None, p, p[:, :3].contiguous(), u,
                      u[:, 0].contiguous(), toks.t, acc.t, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(used.t) == free.numel()
    for g in [table, cu, lens, slots, pos, used, qo, ko, *cache, kb, vb, out, ws, toks, acc]:
        assert g.intact()
    assert np.isfinite(out.t.float().cpu().numpy()).all()
