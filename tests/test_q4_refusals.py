"""What the calls on the 4-bit cache and lq_token_logprobs refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import lattice_vq_weight_gb300 as L
from tests.test_paged_devices import Elsewhere

P = ctypes.c_void_p
GOOD, ODD, EIGHT, NUL = P(0x10000), P(0x10001), P(0x10008), P(0)


@pytest.fixture(scope="module")
def lib():
    from lattice_vq_weight_gb300 import build
    build.build()
    return L.lib


def test_append_and_gather(lib):
    def app(k=GOOD, ldk=256, dt=L.LQ_BF16, tokens=3, slots=GOOD, cache=GOOD, scales=GOOD, nb=4, bs=16, hk=2, d=128, g=64,
            st=NUL):
        return lib.lq_kv_append_q4(k, ldk, GOOD, 256, dt, tokens, slots, cache, scales, GOOD, GOOD, nb, bs, hk, d, g, st,
                                   NUL)
    assert app(dt=7) == L.LQ_ERR_DTYPE
    assert app(bs=20) == app(bs=8) == app(d=96) == app(d=512) == app(d=0) == L.LQ_ERR_UNSUPPORTED
    assert app(g=16) == app(g=256) == app(g=0) == app(g=48) == app(d=64, g=128) == L.LQ_ERR_UNSUPPORTED
    assert app(ldk=255) == app(ldk=257) == app(nb=-1) == app(nb=1 << 31) == app(hk=0) == app(hk=1025) == L.LQ_ERR_SHAPE
    assert app(tokens=-1) == app(tokens=1 << 31) == L.LQ_ERR_SHAPE
    for bad in (dict(k=NUL), dict(slots=NUL), dict(cache=NUL), dict(scales=NUL), dict(k=EIGHT), dict(cache=EIGHT),
                dict(scales=EIGHT), dict(slots=P(0x10004)), dict(st=ODD)):
        assert app(**bad) == L.LQ_ERR_ARG
    assert app(tokens=0) == L.LQ_OK

    def gat(slots=GOOD, n=3, cache=GOOD, scales=GOOD, bs=16, d=128, g=32, out=GOOD, dt=L.LQ_F32):
        return lib.lq_kv_gather_q4(slots, n, cache, scales, GOOD, GOOD, 4, bs, 2, d, g, out, GOOD, dt, NUL, NUL)
    assert gat(dt=5) == L.LQ_ERR_DTYPE and gat(bs=1) == gat(d=8) == gat(g=24) == L.LQ_ERR_UNSUPPORTED
    assert gat(n=-1) == gat(n=1 << 60) == L.LQ_ERR_SHAPE
    assert gat(slots=NUL) == gat(cache=NUL) == gat(scales=EIGHT) == gat(out=NUL) == gat(out=EIGHT) == L.LQ_ERR_ARG
    assert gat(n=0) == L.LQ_OK


def test_attention(lib):
    def call(q=GOOD, ldq=1024, dt=L.LQ_BF16, total=4, cu=GOOD, batch=2, table=GOOD, stride=8, width=8, cache=GOOD,
             scales=GOOD, nb=4, bs=16, hq=8, hk=2, d=128, g=64, scale=0.1, out=GOOD, ldo=1024, ws=GOOD, nbytes=1 << 30):
        return lib.lq_attention_paged_q4(q, ldq, dt, total, cu, GOOD, batch, table, stride, width, cache, scales, GOOD,
                                         GOOD, nb, bs, hq, hk, d, g, scale, out, ldo, ws, ctypes.c_size_t(nbytes), NUL, NUL)
    assert call(dt=3) == L.LQ_ERR_DTYPE
    assert call(bs=8) == call(d=96) == call(g=16) == call(d=64, g=128, ldq=512) == L.LQ_ERR_UNSUPPORTED
    assert call(hq=7) == call(hq=0) == call(hk=0) == call(ldq=1023) == call(ldq=1028) == call(ldo=512) == L.LQ_ERR_SHAPE
    assert call(batch=0) == call(batch=L.LQ_MAX_REQUESTS + 1) == call(total=-1) == call(stride=7) == L.LQ_ERR_SHAPE
    assert call(nb=1 << 31) == call(nb=(1 << 31) - 1, hk=8, bs=128) == call(nbytes=0) == L.LQ_ERR_SHAPE
    for bad in (dict(q=NUL), dict(cu=NUL), dict(table=NUL), dict(cache=NUL), dict(scales=NUL), dict(out=NUL), dict(ws=NUL),
                dict(q=EIGHT), dict(out=EIGHT), dict(cache=EIGHT), dict(scales=EIGHT), dict(ws=EIGHT),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == L.LQ_ERR_ARG
    assert call(total=0) == L.LQ_OK
    size = L.lq_attention_paged_q4_workspace_size
    assert size(2, 4, 8, 2, 128) > 0
    assert size(2, 4, 7, 2, 128) == size(2, 4, 8, 2, 96) == size(-1, 4, 8, 2, 128) == 0


def test_token_logprobs(lib):
    def call(x=GOOD, ld=100, dt=L.LQ_F32, rows=2, vocab=100, tok=GOOD, lp=GOOD, ent=NUL, rank=NUL, top=3, tt=GOOD, tl=GOOD):
        return lib.lq_token_logprobs(x, ld, dt, rows, vocab, tok, lp, ent, rank, top, tt, tl, NUL, NUL)
    assert call(dt=9) == L.LQ_ERR_DTYPE
    assert call(ld=99) == call(rows=-1) == call(rows=(1 << 24) + 1) == call(vocab=0) == L.LQ_ERR_SHAPE
    assert call(vocab=(1 << 24) + 1, ld=1 << 25) == call(top=-1) == call(top=33) == call(vocab=2, top=3) == L.LQ_ERR_SHAPE
    for bad in (dict(x=NUL), dict(x=ODD), dict(x=P(0x10002)), dict(tok=NUL), dict(lp=NUL), dict(lp=ODD), dict(ent=ODD),
                dict(rank=ODD), dict(tt=NUL), dict(tl=NUL), dict(tt=ODD)):
        assert call(**bad) == L.LQ_ERR_ARG
    assert call(dt=L.LQ_BF16, x=ODD) == L.LQ_ERR_ARG
    assert call(rows=0) == L.LQ_OK
    assert L.LQ_MAX_ALTERNATIVES == 32


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def calls():
    cache = L.paged_cache_q4(4, 2, 16, 64, 32, "cpu")
    k, q = torch.zeros((3, 2, 64)), torch.zeros((3, 4, 64))
    slots = torch.zeros(3, dtype=torch.int64)
    return {
        "lq_kv_append_q4": (k, k, slots, *cache),
        "lq_kv_gather_q4": (slots, *cache, k, k.clone()),
        "lq_attention_paged_q4": (q, i32(3), i32(2), i32(2, 4), *cache, torch.zeros_like(q),
                                  torch.zeros(1 << 20, dtype=torch.uint8)),
        "lq_token_logprobs": (torch.zeros((3, 50)), i32(3), torch.zeros(3), torch.zeros(3), i32(3), i32(3, 4),
                              torch.zeros((3, 4))),
    }


def test_the_binding_refuses_tensors_that_do_not_fit():
    c = calls()

    def refused(name, i, t):
        args = list(c[name])
        args[i] = t
        with pytest.raises((ValueError, TypeError)):
            getattr(L, name)(*args)

    k, _, slots, kc, ks, vc, vs = c["lq_kv_append_q4"]
    for i, t in ((0, k[:, :1]), (1, k.bfloat16()), (2, slots.int()), (2, slots[:2]), (3, kc.to(torch.int8)), (3, kc[0]),
                 (4, ks.float()), (4, ks[..., :1]), (4, ks.flatten(3)), (4, ks[:, :1]), (5, vc[:3]), (5, vc.transpose(1, 2)),
                 (6, vs[:, :, :, :1]), (0, k.transpose(1, 2).contiguous().transpose(1, 2)), (0, k.double())):
        refused("lq_kv_append_q4", i, t)
    refused("lq_kv_gather_q4", 5, k[:2])
    refused("lq_kv_gather_q4", 5, k.bfloat16())
    for i, t in ((0, torch.zeros((3, 4, 128))), (1, i32(2)), (3, i32(1, 4)), (3, i32(4, 2).t()), (8, torch.zeros((3, 4, 64)).bfloat16()),
                 (9, torch.zeros((1 << 10, 1 << 10), dtype=torch.uint8).t()[:, ::2])):
        refused("lq_attention_paged_q4", i, t)
    x = c["lq_token_logprobs"][0]
    for i, t in ((0, x[None]), (0, torch.zeros((50, 3)).t()), (0, x.half()), (1, i32(3).long()), (1, i32(2)), (2, x[:, 0]),
                 (3, torch.zeros(3).double()), (4, torch.zeros(3)), (5, i32(3, 5)), (5, None), (6, None)):
        refused("lq_token_logprobs", i, t)
    with pytest.raises(ValueError):
        L.paged_cache_q4(4, 2, 16, 64, 48, "cpu")


@pytest.mark.parametrize("name", sorted(calls()))
def test_host_tensors_and_several_devices(name, monkeypatch):
    """Every tensor is looked at, and the kernels are launched on the tensors' device, whatever the current one is."""
    with pytest.raises(ValueError, match="device"):
        getattr(L, name)(*calls()[name], stream=0)
    called, current = [], [0]

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: called.append((fn, current[0])) or 0

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *_):
            current[0] = self.old

    monkeypatch.setattr(L, "_LIB", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    args = calls()[name]
    put = lambda i, dev, rest=0: [Elsewhere(a, dev if j == i else rest) if isinstance(a, torch.Tensor) else a
                                  for j, a in enumerate(args)]
    getattr(L, name)(*put(-1, 0), dev_status=Elsewhere(i32(1), 0), stream=0)
    getattr(L, name)(*put(-1, 0, rest=1), stream=0)
    assert called == [(name, 0), (name, 1)] and current == [0]
    for i, a in enumerate(args):
        if isinstance(a, torch.Tensor):
            for dev in (-1, 1):
                with pytest.raises(ValueError, match="device"):
                    getattr(L, name)(*put(i, dev), stream=0)
    with pytest.raises(ValueError, match="device"):
        getattr(L, name)(*put(-1, 0), dev_status=Elsewhere(i32(1), -1), stream=0)
    assert len(called) == 2
