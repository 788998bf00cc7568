"""lq_qk_norm_rope: an infinity or NaN in a value that is not rotated stays in that value."""
import numpy as np
import pytest

import oracle.paged_oracle as P
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("d,rot,at", [(64, 32, 33), (128, 64, 71), (256, 16, 250), (80, 48, 48), (64, 0, 5)])
def test_beside_the_rotation(dtype, inter, bad, d, rot, at):
    torch, L = cuda()
    rng = np.random.default_rng(d + at)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = to_dev(torch, rng.standard_normal((3, 2, d)).astype(np.float32)).to(dt)
    q[1, 1, at] = bad
    k = q[:, :1].contiguous()
    ang = rng.uniform(-4, 4, (9, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = np.array([3, 8, 0], np.int32)
    qo, ko, st = torch.empty_like(q), torch.empty_like(k), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_qk_norm_rope(q, k, None, None, 0.0, to_dev(torch, pos), to_dev(torch, table), qo, ko, interleaved=inter,
                      dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert torch.equal(qo[..., rot:].nan_to_num(7.0, 8.0, 9.0), q[..., rot:].nan_to_num(7.0, 8.0, 9.0))   # as they were
    clean = q.clone()
    clean[1, 1, at] = 0.0
    want = P.norm_rope(clean.float().cpu().numpy(), None, 0.0, pos, table, rot, inter)[..., :rot]
    got = qo[..., :rot].float().cpu().numpy()
    # fp32 steps on values of at most the pair's size, one bf16 rounding
    assert np.isfinite(got).all()
    tol = 4 * 2.0 ** -24 * np.abs(want).max(initial=0.0) + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_position_outside_the_table(dtype, inter, bad):
    """Such a token is not rotated: every value passes through as it is."""
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = to_dev(torch, np.random.default_rng(3).standard_normal((2, 3, 64)).astype(np.float32)).to(dt)
    q[0, 1, 9] = bad
    k = q[:, :1].contiguous()
    qo, ko, st = torch.empty_like(q), torch.empty_like(k), torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = to_dev(torch, np.array([40, -2], np.int32))
    L.lq_qk_norm_rope(q, k, None, None, 0.0, pos, torch.ones((4, 64), device="cuda"), qo, ko, interleaved=inter,
                      dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == L.LQ_DEV_RANGE
    assert torch.equal(qo.nan_to_num(7.0, 8.0), q.nan_to_num(7.0, 8.0)) and torch.equal(ko, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_an_infinity_under_the_norm(dtype, inter):
    """The norm of a head with an infinity is infinite: its other unrotated values become 0, not NaN."""
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = to_dev(torch, np.random.default_rng(4).standard_normal((1, 1, 128)).astype(np.float32)).to(dt)
    q[0, 0, 100] = float("inf")
    k = q.clone()
    w = torch.ones(128, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    L.lq_qk_norm_rope(q, k, w, w, 1e-6, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones((1, 64), device="cuda"),
                      qo, ko, interleaved=inter)
    torch.cuda.synchronize()
    for o in (qo, ko):
        assert bool(o[0, 0, 100].isnan()) and not bool(o[0, 0, :100].any()) and not bool(o[0, 0, 101:].any())
