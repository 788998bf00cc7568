"""lq_attention_paged where the value scales that a row sees are far apart: blocks of zeros beside large values, scales
a hundred powers of two apart in either order, scales near the ends of fp32.  What a position weighs does not depend on
the size of its values."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_attention_paged import TOL, build, check, reference, run

pytestmark = pytest.mark.gpu

# requests (kv_len, q_len): few rows; some dozens; a prompt; positions split between CTAs
SHAPES = [([(400, 2)], 4, 2, 16, 128), ([(300, 40)], 4, 2, 16, 128), ([(500, 200)], 4, 2, 32, 64),
          ([(260, 90)], 3, 1, 64, 256), ([(3000, 70)], 4, 1, 64, 128), ([(9000, 1)], 8, 1, 128, 128),
          ([(2600, 80)], 2, 1, 16, 256), ([(70, 6), (1, 1), (900, 3)], 6, 2, 16, 64)]


def scales(kind, rng, shape):
    v = rng.uniform(0.005, 0.03, shape)
    n = shape[0]
    some = rng.random(shape) < 0.5
    if kind == "zeros beside 2^35":
        v = np.where(some, 0.0, 2.0 ** 35)
    elif kind == "zeros beside 2^100":
        v = np.where(some, 0.0, v * 2.0 ** 100)
    elif kind == "zeros beside ordinary":
        v = np.where(some, 0.0, v)
    elif kind == "2^70 beside 2^-70":
        v = np.where(some, v * 2.0 ** 70, v * 2.0 ** -70)
    elif kind == "growing":
        v = v * 2.0 ** np.linspace(-120, 115, n)[:, None]
    elif kind == "shrinking":
        v = v * 2.0 ** np.linspace(115, -120, n)[:, None]
    elif kind == "any":
        v = v * 2.0 ** rng.uniform(-125, 115, shape)
    elif kind == "tiny":
        v = v * 2.0 ** -112
    return v.astype(np.float32)


KINDS = ["zeros beside 2^35", "zeros beside 2^100", "zeros beside ordinary", "2^70 beside 2^-70", "growing", "shrinking",
         "any", "tiny"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_value_scales_far_apart(dtype, kind, shape):
    torch, L = cuda()
    rng = np.random.default_rng(31 + shape)
    s = build(torch, rng, *SHAPES[shape], dtype)
    used = [b for row in s["table"] for b in row if b >= 0]
    s["vs"][used] = scales(kind, rng, s["vs"][used].shape)       # in the order of the positions
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st)
    assert int(st) == 0
    check(got, reference(s), dtype)
    assert torch.equal(got, run(torch, L, s, st))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [-60.0, -10.0, 10.0, 60.0, 150.0])
@pytest.mark.parametrize("big", [1.0, 2.0 ** 40, 2.0 ** 110])
@pytest.mark.parametrize("q_len", [1, 40, 200])
def test_scores_against_scales(dtype, gap, big, q_len):
    """Positions of zeros whose scores are above (or below) those of the values: they take their share of the weights
    whatever the values' scale, and a row whose values are nothing beside the weights of zeros stays exact."""
    torch, L = cuda()
    rng = np.random.default_rng(32)
    hk, bs, d = 2, 16, 128
    s = build(torch, rng, [(20 * bs, q_len)], 4, hk, bs, d, dtype)
    s["kc"][:] = 0
    s["kc"][..., 0] = 64
    s["q"][..., 0] = 1.0
    # a block's score in nats, by its key scale (sm_scale 1): zeros `gap` above the others
    zero = np.arange(20) % 3 != 1
    used = s["table"][0, :20]
    s["ks"][used] = np.where(zero, gap / 64, 0.0)[:, None].astype(np.float32) + np.float32(0.001)
    s["vs"][used] = (np.where(zero, 0.0, big)[:, None] * rng.uniform(0.5, 1, (20, hk))).astype(np.float32)
    ref = reference(s, 1.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(torch, L, s, st, sm_scale=1.0)
    assert int(st) == 0
    g = got.float().cpu().numpy().astype(np.float64)
    for t in range(q_len):
        for h in range(4):
            # (an output below fp32's normal numbers may be 0)
            err = np.linalg.norm(g[t, h] - ref[t, h])
            assert err <= TOL[dtype] * np.linalg.norm(ref[t, h]) + 2.0 ** -126 * np.sqrt(d), (t, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [2, 200])
def test_a_block_of_zeros_takes_half_of_the_weight(dtype, q_len):
    """By hand: all scores equal, one of two blocks zero, the other 127 codes times 2^35 (and times 2^-110)."""
    torch, L = cuda()
    s = build(torch, np.random.default_rng(33), [(32 + q_len, q_len)], 2, 1, 16, 128, dtype)
    s["kc"][:] = 0
    s["vc"][:] = 127
    blocks = s["table"][0, :2]
    for value in (2.0 ** 35, 2.0 ** -110):
        s["vs"][:] = 0
        s["vs"][blocks[1]] = value
        got = run(torch, L, s)
        seen = np.arange(q_len) + 33
        want = 127 * value * 16 / seen
        assert np.allclose(got.float().cpu().numpy(), want[:, None, None], rtol=TOL[dtype], atol=0)
