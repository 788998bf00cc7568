"""What the paged cache's calls refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest

import lattice_vq_weight_gb300 as L

P = ctypes.c_void_p
GOOD, ODD, EIGHT, NUL = P(0x10000), P(0x10002), P(0x10008), P(0)


@pytest.fixture(scope="module")
def lib():
    from lattice_vq_weight_gb300 import build
    build.build()
    return L.lib


def test_plan(lib):
    def call(batch=2, bs=16, free=GOOD, nfree=8, table=GOOD, stride=4, width=4, cu=GOOD, slots=GOOD, tokens=8, lens=GOOD):
        return lib.lq_kv_plan(lens, GOOD, batch, bs, free, nfree, table, stride, width, cu, GOOD, slots, GOOD, tokens,
                              GOOD, NUL, NUL)
    assert call(bs=8) == call(bs=48) == call(bs=256) == L.LQ_ERR_UNSUPPORTED
    assert call(batch=-1) == call(batch=L.LQ_MAX_REQUESTS + 1) == L.LQ_ERR_SHAPE
    assert call(stride=3) == call(width=-1) == call(nfree=-1) == call(tokens=-1) == call(tokens=1 << 31) == L.LQ_ERR_SHAPE
    assert call(cu=NUL) == call(lens=NUL) == call(table=NUL) == call(free=NUL) == call(slots=NUL) == L.LQ_ERR_ARG
    assert call(slots=P(0x10004)) == call(table=ODD) == L.LQ_ERR_ARG


def test_norm_rope(lib):
    def call(q=GOOD, ldq=512, hq=4, ldk=128, hk=1, dt=L.LQ_BF16, tokens=3, d=128, qw=GOOD, eps=1e-6, pos=GOOD, cs=GOOD,
             rot=128, out=GOOD):
        return lib.lq_qk_norm_rope(q, ldq, hq, GOOD, ldk, hk, dt, tokens, d, qw, GOOD, eps, pos, cs, 100, rot, 0, out, 512,
                                   GOOD, 128, NUL, NUL)
    assert call(dt=2) == L.LQ_ERR_DTYPE
    assert call(d=264) == call(d=12) == call(d=0) == call(rot=24) == L.LQ_ERR_UNSUPPORTED
    assert call(rot=144) == call(ldq=511) == call(ldq=513) == call(ldk=64) == call(tokens=-1) == L.LQ_ERR_SHAPE
    assert call(q=NUL) == call(out=NUL) == call(pos=NUL) == call(cs=NUL) == call(q=EIGHT) == call(qw=EIGHT) == L.LQ_ERR_ARG
    assert call(eps=-1.0) == call(eps=float("nan")) == L.LQ_ERR_ARG
    assert call(tokens=0) == L.LQ_OK


def test_append_and_gather(lib):
    def app(k=GOOD, ldk=256, dt=L.LQ_BF16, tokens=3, slots=GOOD, cache=GOOD, nb=4, bs=16, hk=2, d=128):
        return lib.lq_kv_append(k, ldk, GOOD, 256, dt, tokens, slots, cache, GOOD, GOOD, GOOD, nb, bs, hk, d, NUL, NUL)
    assert app(dt=7) == L.LQ_ERR_DTYPE
    assert app(bs=20) == app(d=72) == app(d=272) == L.LQ_ERR_UNSUPPORTED
    assert app(ldk=255) == app(ldk=257) == app(nb=-1) == app(hk=0) == app(tokens=-1) == L.LQ_ERR_SHAPE
    assert app(k=NUL) == app(slots=NUL) == app(cache=NUL) == app(k=EIGHT) == app(cache=EIGHT) == L.LQ_ERR_ARG
    assert app(tokens=0) == L.LQ_OK

    def gat(slots=GOOD, n=3, cache=GOOD, bs=16, d=128, out=GOOD, dt=L.LQ_F32):
        return lib.lq_kv_gather(slots, n, cache, GOOD, GOOD, GOOD, 4, bs, 2, d, out, GOOD, dt, NUL, NUL)
    assert gat(dt=5) == L.LQ_ERR_DTYPE and gat(bs=1) == gat(d=8) == L.LQ_ERR_UNSUPPORTED
    assert gat(n=-1) == gat(n=1 << 60) == L.LQ_ERR_SHAPE
    assert gat(slots=NUL) == gat(cache=NUL) == gat(out=NUL) == gat(out=EIGHT) == L.LQ_ERR_ARG
    assert gat(n=0) == L.LQ_OK


def test_attention(lib):
    def call(q=GOOD, ldq=1024, dt=L.LQ_BF16, total=4, cu=GOOD, batch=2, table=GOOD, stride=8, width=8, cache=GOOD, nb=4,
             bs=16, hq=8, hk=2, d=128, scale=0.1, out=GOOD, ldo=1024, ws=GOOD, nbytes=1 << 30):
        return lib.lq_attention_paged(q, ldq, dt, total, cu, GOOD, batch, table, stride, width, cache, GOOD, GOOD, GOOD, nb,
                                      bs, hq, hk, d, scale, out, ldo, ws, ctypes.c_size_t(nbytes), NUL, NUL)
    assert call(dt=3) == L.LQ_ERR_DTYPE
    assert call(bs=8) == call(d=96, ldq=1024) == L.LQ_ERR_UNSUPPORTED
    assert call(hq=7) == call(hq=0) == call(hk=0) == call(ldq=1023) == call(ldq=1028) == call(ldo=512) == L.LQ_ERR_SHAPE
    assert call(batch=0) == call(batch=L.LQ_MAX_REQUESTS + 1) == call(total=-1) == call(stride=7) == L.LQ_ERR_SHAPE
    assert call(nbytes=0) == L.LQ_ERR_SHAPE
    assert call(q=NUL) == call(cu=NUL) == call(table=NUL) == call(cache=NUL) == call(out=NUL) == call(ws=NUL) == L.LQ_ERR_ARG
    assert call(q=EIGHT) == call(out=EIGHT) == call(cache=EIGHT) == call(ws=EIGHT) == L.LQ_ERR_ARG
    assert call(scale=float("nan")) == call(scale=float("inf")) == L.LQ_ERR_ARG
    assert call(total=0) == L.LQ_OK
    size = L.lq_attention_paged_workspace_size
    assert size(2, 4, 8, 2, 128) > 0
    assert size(2, 4, 7, 2, 128) == size(2, 4, 8, 2, 96) == size(-1, 4, 8, 2, 128) == 0


def test_verify(lib):
    def call(batch=2, k=3, vocab=100, p=GOOD, prow=100, q=GOOD, qrow=100, dt=L.LQ_F32, ua=GOOD, us=GOOD, out=GOOD,
             tok=GOOD):
        return lib.lq_verify_draft(tok, NUL, batch, k, vocab, p, 400, prow, q, 300, qrow, dt, ua, us, out, GOOD, NUL, NUL)
    assert call(dt=9) == L.LQ_ERR_DTYPE
    assert call(batch=-1) == call(k=-1) == call(k=1025) == call(vocab=0) == call(vocab=(1 << 24) + 1) == L.LQ_ERR_SHAPE
    assert call(prow=99) == call(qrow=99) == L.LQ_ERR_SHAPE
    assert call(p=NUL) == call(p=ODD) == call(q=ODD) == call(ua=NUL) == call(us=NUL) == call(out=NUL) == call(tok=NUL)
    assert call(p=NUL) == L.LQ_ERR_ARG and call(batch=0) == L.LQ_OK


def test_the_binding_refuses_tensors_that_do_not_fit():
    """Shapes, dtypes and strides the kernels would misread raise before the library is called."""
    import torch
    cache = L.paged_cache(4, 2, 16, 64, "cpu")
    k = torch.zeros((3, 2, 64))
    slots = torch.zeros(3, dtype=torch.int64)
    bad = [(k[:, :1], k[:, :1], slots, *cache), (k, k.bfloat16(), slots, *cache), (k, k, slots.int(), *cache),
           (k, k, slots[:2], *cache), (k, k, slots, cache[0].float(), *cache[1:]), (k, k, slots, cache[0], cache[1].t(), *cache[2:]),
           (k.transpose(1, 2).contiguous().transpose(1, 2), k, slots, *cache)]
    for args in bad:
        with pytest.raises(ValueError):
            L.lq_kv_append(*args)
    i = lambda *n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.lq_kv_plan(i(2), i(3), 16, i(4), i(2, 4), i(3), i(2), slots, i(3), i(1))
    with pytest.raises(ValueError):
        L.lq_kv_plan(i(2), i(2), 16, i(4), i(4, 2).t(), i(3), i(2), slots, i(3), i(1))
    with pytest.raises(TypeError):
        L.lq_qk_norm_rope(k, k.bfloat16(), None, None, 0.0, i(3), torch.zeros(9, 64), k, k)
    with pytest.raises(ValueError):
        L.lq_qk_norm_rope(k, k, torch.zeros(32), None, 0.0, i(3), torch.zeros(9, 64), k, k)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.lq_attention_paged(k, i(2), i(2), i(2, 4), *cache, k, ws)
    with pytest.raises(ValueError):
        L.lq_attention_paged(k, i(3), i(2), i(1, 4), *cache, k, ws)
    p = torch.zeros((2, 3, 50))
    u = torch.zeros((2, 2))
    with pytest.raises(ValueError):
        L.lq_verify_draft(i(2, 2), None, p[:, :2], None, u, u[:, 0].contiguous(), i(2, 3), i(2))
    with pytest.raises(ValueError):
        L.lq_verify_draft(i(2, 2), None, p, p[:, :2, ::2], u, u[:, 0].contiguous(), i(2, 3), i(2))
