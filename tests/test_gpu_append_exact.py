"""lq_kv_append bit for bit: scales and codes are IEEE fp32 quotients, half to even, whatever the size of the values."""
import numpy as np
import pytest

from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu

F = np.float32


def append(x, slots, codes, scales):
    """The same in numpy's fp32: x [tokens x heads x d], codes [blocks x heads x bs x d] int8 and scales changed in place."""
    bs = codes.shape[2]
    t = 0
    while t < len(slots):
        e = t + 1
        while e < len(slots) and slots[e] == slots[e - 1] + 1 and slots[e] % bs:
            e += 1
        b, off = int(slots[t]) // bs, int(slots[t]) % bs
        for h in range(codes.shape[1]):
            rows = x[t:e, h]
            old = scales[b, h] if off else F(0)
            s = max(old, F(np.abs(rows).max() / F(127)))
            div = s if s > 0 else F(1)
            if off and s > old:
                codes[b, h, :off] = np.clip(np.rint(codes[b, h, :off].astype(F) * old / div), -127, 127).astype(np.int8)
            codes[b, h, off:off + e - t] = np.clip(np.rint(rows / div), -127, 127).astype(np.int8)
            scales[b, h] = s
        t = e


def values(kind, rng, shape):
    x = rng.standard_normal(shape).astype(F)
    if kind == "halves":               # the block's largest is 127 steps: multiples of half a step, and one ulp beside them
        step = F(2.0) ** rng.integers(-20, 20)
        x = rng.integers(-254, 255, shape).astype(F) * F(0.5) * step
        near = rng.random(shape)
        x = np.where(near < 0.3, np.nextafter(x, F(np.inf)), np.where(near < 0.6, np.nextafter(x, F(-np.inf)), x))
    elif kind == "halves of any scale":
        top = F(rng.uniform(0.5, 2))
        s = F(top / F(127))
        x = ((rng.integers(-127, 127, shape).astype(F) + F(0.5)) * s).astype(F)
        near = rng.random(shape)
        x = np.where(near < 0.3, np.nextafter(x, F(np.inf)), np.where(near < 0.6, np.nextafter(x, F(-np.inf)), x))
        x.reshape(-1)[::97] = top
    elif kind == "large":
        x *= F(2.0) ** 120
    elif kind == "tiny":
        x *= F(2.0) ** -118
    elif kind == "subnormal":
        x *= F(2.0) ** -133
    elif kind == "of all sizes":
        x *= F(2.0) ** rng.integers(-60, 60, shape).astype(F)
    return x.astype(F)


KINDS = ["normal", "halves", "halves of any scale", "large", "tiny", "subnormal", "of all sizes"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs,d,hk,runs", [(16, 64, 3, 1), (64, 128, 2, 7), (128, 256, 1, 50), (32, 80, 2, 33)])
def test_codes_and_scales(dtype, kind, bs, d, hk, runs):
    """A block filled by calls of a few rows each, so that its rows are coded again and again, and prompts beside it."""
    torch, L = cuda()
    rng = np.random.default_rng(len(kind) + bs + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    nb = 6
    codes = [rng.integers(-127, 128, (nb, hk, bs, d)).astype(np.int8) for _ in range(2)]
    scales = [(rng.uniform(0.5, 2, (nb, hk)) * 2.0 ** -126).astype(F) for _ in range(2)]
    cache = [to_dev(torch, a) for n in range(2) for a in (codes[n], scales[n])]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = 0
    while at < bs:
        n = int(min(bs - at, rng.integers(1, runs + 1)))
        # rows of block 4, and a run that goes over from block 1 to block 2
        slots = np.array([4 * bs + at + i for i in range(n)] + [2 * bs - 1 - at + i for i in range(at + 2)], dtype=np.int64)
        grow = F(2.0) ** rng.integers(0, 3)
        x = [to_dev(torch, values(kind, rng, (len(slots), hk, d)) * grow).to(dt) for _ in range(2)]
        L.lq_kv_append(x[0], x[1], to_dev(torch, slots), *cache, dev_status=st)
        torch.cuda.synchronize()
        for i in range(2):
            append(x[i].float().cpu().numpy(), slots, codes[i], scales[i])
            assert np.array_equal(cache[2 * i + 1].cpu().numpy(), scales[i])
            assert np.array_equal(cache[2 * i].cpu().numpy(), codes[i])
        at += n
    assert int(st) == 0
