"""lq_kv_append_q4 and lq_kv_gather_q4 on the GPU against the oracle, bit for bit (the format is defined by IEEE steps)."""
import numpy as np
import pytest

import oracle.q4_oracle as Q
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu


def pool(torch, rng, nb, hk, bs, d, group):
    """A cache of arbitrary contents, as numpy arrays and on the device."""
    host = []
    for _ in range(2):
        host.append(rng.integers(0, 256, (nb, hk, bs, d // 2), dtype=np.uint8))
        host.append(rng.standard_normal((nb, hk, bs, d // group, 2)).astype(np.float16))
    return host, [to_dev(torch, x) for x in host]


def rows(torch, rng, shape, dtype, size=1.0):
    """Device rows of the dtype and the same numbers as float32 on the host."""
    x = to_dev(torch, (size * rng.standard_normal(shape)).astype(np.float32))
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return x, x.float().cpu().numpy()


def same(dev, host):
    got = dev.cpu().numpy()
    return np.array_equal(got.view(np.uint16) if got.dtype == np.float16 else got,
                          host.view(np.uint16) if host.dtype == np.float16 else host)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("tokens,hk,bs", [(1, 1, 16), (37, 3, 32), (130, 2, 64), (9, 5, 128)])
def test_append_and_gather(dtype, d, group, tokens, hk, bs):
    torch, L = cuda()
    rng = np.random.default_rng(tokens * d + group)
    nb = -(-tokens // bs) + 2
    host, dev = pool(torch, rng, nb, hk, bs, d, group)
    slots = rng.permutation(nb * bs)[:tokens].astype(np.int64)
    (k, kh), (v, vh) = (rows(torch, rng, (tokens, hk, d), dtype, s) for s in (1.0, 30.0))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_kv_append_q4(k, v, to_dev(torch, slots), *dev, dev_status=st)
    want = [*Q.append(kh, slots, *host[:2]), *Q.append(vh, slots, *host[2:])]
    assert int(st) == 0 and all(same(g, w) for g, w in zip(dev, want))
    # every slot back, a few of them left out or past the cache
    read = rng.permutation(nb * bs).astype(np.int64)
    read[::7] = -3
    values = [Q.values(want[i], want[i + 1]).transpose(0, 2, 1, 3).reshape(nb * bs, hk, d) for i in (0, 2)]
    for out_dtype in (torch.float32, torch.bfloat16):
        out = [torch.full((len(read), hk, d), 9.0, dtype=out_dtype, device="cuda") for _ in range(2)]
        L.lq_kv_gather_q4(to_dev(torch, read), *dev, *out, dev_status=st)
        for o, w in zip(out, values):
            w = np.where(read[:, None, None] >= 0, w[read].astype(np.float32), np.float32(0))
            assert torch.equal(o, to_dev(torch, w).to(out_dtype))
    assert int(st) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_between_two_codes_and_narrow_groups(dtype):
    """Groups on a grid of half steps (ties to the even code), constant groups, groups narrower than fp16's least
    number, and far from zero for their width."""
    torch, L = cuda()
    rng = np.random.default_rng(1)
    n, hk, d, group, bs = 64, 2, 128, 32, 16
    x = rng.integers(0, 31, (n, hk, d)).astype(np.float32) / 2
    x[..., ::32], x[..., 1::32] = 0, 15
    x *= 2.0 ** rng.integers(-20, 8, (n, 1, 1)).astype(np.float32)
    x[:8] = 0.375
    x[8:16] *= 1e-9
    x[16:24] += 100
    x[24:32] = 0
    x[32:40] = -x[32:40]
    xd = to_dev(torch, x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    host, dev = pool(torch, rng, 4, hk, bs, d, group)
    slots = np.arange(n, dtype=np.int64)
    L.lq_kv_append_q4(xd, -xd, to_dev(torch, slots), *dev)
    xh = xd.float().cpu().numpy()
    want = [*Q.append(xh, slots, *host[:2]), *Q.append(-xh, slots, *host[2:])]
    assert all(same(g, w) for g, w in zip(dev, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_status_and_rows_left_out(dtype):
    torch, L = cuda()
    rng = np.random.default_rng(2)
    hk, d, group, bs = 2, 64, 64, 16
    host, dev = pool(torch, rng, 2, hk, bs, d, group)
    (k, kh), (v, vh) = (rows(torch, rng, (4, hk, d), dtype) for _ in range(2))
    slots = np.array([3, -1, 31, -(1 << 40)], np.int64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        st.zero_()
        L.lq_kv_append_q4(k, v, to_dev(torch, slots), *dev, dev_status=st)
        want = [*Q.append(kh, slots, *host[:2]), *Q.append(vh, slots, *host[2:])]
        assert all(same(g, w) for g, w in zip(dev, want))
        return int(st)

    assert call() == 0
    slots[1] = 32                                              # one past the cache
    assert call() == L.LQ_DEV_RANGE
    slots[1] = 1 << 50
    assert call() == L.LQ_DEV_RANGE
    slots[1] = -1
    for bad in (np.nan, np.inf, -np.inf):
        kh[0, 1, 5] = bad
        k[0, 1, 5] = float(bad)
        assert call() == L.LQ_DEV_NONFINITE
    kh[0, 1, 5], vh[2, 0, 63] = 1.0, -65536.0 if dtype == "bf16" else -3e38
    k[0, 1, 5], v[2, 0, 63] = 1.0, float(vh[2, 0, 63])
    assert call() == L.LQ_DEV_RANGE
    out = [torch.empty((2, hk, d), device="cuda") for _ in range(2)]
    st.zero_()
    L.lq_kv_gather_q4(torch.tensor([32, -1], device="cuda"), *dev, *out, dev_status=st)
    assert int(st) == L.LQ_DEV_RANGE and not any(o.any() for o in out)
    L.lq_kv_append_q4(k[:0], v[:0], torch.empty(0, dtype=torch.int64, device="cuda"), *dev)
    L.lq_kv_gather_q4(torch.empty(0, dtype=torch.int64, device="cuda"), *dev, *[o[:0] for o in out])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows_and_another_stream(dtype):
    """k and v as columns of one projection's output, on a stream of the caller's, captured and replayed."""
    torch, L = cuda()
    rng = np.random.default_rng(3)
    n, hk, d, group, bs = 33, 2, 128, 64, 32
    host, dev = pool(torch, rng, 3, hk, bs, d, group)
    qkv, qkvh = rows(torch, rng, (n, 5 * hk * d), dtype)
    k, v = (qkv[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in (2, 4))
    slots = rng.permutation(96)[:n].astype(np.int64)
    sd = to_dev(torch, slots)
    out = [torch.empty((n, hk, d), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lq_kv_append_q4(k, v, sd, *dev)
        L.lq_kv_gather_q4(sd, *dev, *out)
    for _ in range(2):
        qkv.copy_(torch.randn_like(qkv.float()))
        xh = qkv.float().cpu().numpy()
        kh, vh = (xh[:, i * hk * d:(i + 1) * hk * d].reshape(n, hk, d) for i in (2, 4))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.synchronize()
        want = [*Q.append(kh, slots, *host[:2]), *Q.append(vh, slots, *host[2:])]
        assert all(same(x, w) for x, w in zip(dev, want))
        for o, i in zip(out, (0, 2)):
            w = Q.values(want[i], want[i + 1]).transpose(0, 2, 1, 3).reshape(96, hk, d)[slots]
            assert np.array_equal(o.cpu().numpy(), w.astype(np.float32))
