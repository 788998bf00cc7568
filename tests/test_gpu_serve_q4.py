"""The operators of the 4-bit cache and the scoring of tokens as they are used together: in the serving example, back to
back on one another's outputs, in one captured graph, on two streams at once, and within guard bytes."""
import numpy as np
import pytest

import oracle.q4_oracle as Q
from tests._parity import normwise_rel
from tests.gpu_util import cuda, to_dev
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu


def test_the_serving_example_on_the_4_bit_cache():
    torch, L = cuda()
    from lattice_vq_weight_gb300 import serve_example as E
    s = E.Server(batch=3, num_blocks=96, drafts=3, seed=4, cache_bits=4)
    s.prompt([[5], list(range(33)), [9] * 16])
    for _ in range(5):
        before = s.cached.clone()
        out = s.step()
        kept = (out >= 0).sum(1)
        assert torch.equal(s.cached, before + kept.int()) and bool((out < E.VOCAB).all())
        # the last layer's attention against the cache's values in 64 bits
        q, got = (t.float().cpu().numpy().astype(np.float64) for t in s.seen)
        ref = Q.attention(q, s.cu.tolist(), s.kv_lens.tolist(), s.table.cpu().numpy(),
                          *(t.cpu().numpy() for t in s.caches[-1]), E.DIM ** -0.5)
        for r in range(len(q)):
            for h in range(E.Q_HEADS):
                # bf16 outputs: their rounding, and weights of 11 bits
                assert normwise_rel(got[r, h], ref[r, h]) < 2.0 ** -8
        # the scores: probabilities of the tokens that came out, none where there is none
        logp, entropy, ranks, top, top_logp = s.scores
        assert bool((logp[out >= 0] <= 0).all()) and not bool(logp[out < 0].any()) and bool((ranks[out < 0] == -1).all())
        assert bool((entropy >= 0).all()) and bool((top_logp[..., :1] >= top_logp).all())
        first = ranks == 0
        assert torch.equal(top[..., 0][first], out[first])
    assert int(s.status) == 0


def chain(torch, L, seed, reqs, hq, hk, bs, d, group, dt, q_len, vocab, stream=None):
    """Inputs and buffers of a serving step, and the step: write, attention, logits, scores, read back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    b, n = len(reqs), len(reqs) * q_len
    need = [-(-c // bs) for c in reqs]
    table = torch.full((b, max(need)), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = torch.arange(at, at + c)
        at += c
    pos = [c - q_len + j for c in reqs for j in range(q_len)]
    row = [i for i in range(b) for _ in range(q_len)]
    slots = torch.tensor([int(table[i, p // bs]) * bs + p % bs for i, p in zip(row, pos)], device="cuda")
    cache = L.paged_cache_q4(sum(need), hk, bs, d, group, "cuda")
    k0, v0 = rand(sum(need) * bs, hk, d).to(dt), rand(sum(need) * bs, hk, d).to(dt)
    L.lq_kv_append_q4(k0, v0, torch.arange(sum(need) * bs, device="cuda"), *cache)
    s = dict(q=rand(n, hq, d).to(dt), k=rand(n, hk, d).to(dt), v=rand(n, hk, d).to(dt), head=rand(hq * d, vocab).to(dt),
             lens=torch.tensor(reqs, dtype=torch.int32, device="cuda"), table=table.cuda(), slots=slots, cache=cache,
             cu=torch.arange(0, n + 1, q_len, dtype=torch.int32, device="cuda"),
             tokens=torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32),
             out=torch.zeros((n, hq, d), dtype=dt, device="cuda"), logits=torch.zeros((n, vocab), dtype=dt, device="cuda"),
             back=[torch.zeros((n, hk, d), device="cuda") for _ in range(2)],
             ws=torch.empty(L.lq_attention_paged_q4_workspace_size(b, n, hq, hk, d), dtype=torch.uint8, device="cuda"),
             scores=[torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),
                     torch.zeros(n, dtype=torch.int32, device="cuda"),
                     torch.zeros((n, 4), dtype=torch.int32, device="cuda"), torch.zeros((n, 4), device="cuda")])

    def step(sync=lambda: None):
        L.lq_kv_append_q4(s["k"], s["v"], s["slots"], *cache)
        sync()
        L.lq_attention_paged_q4(s["q"], s["cu"], s["lens"], s["table"], *cache, s["out"], s["ws"])
        sync()
        torch.mm(s["out"].flatten(1), s["head"], out=s["logits"])
        sync()
        L.lq_token_logprobs(s["logits"], s["tokens"], *s["scores"])
        sync()
        L.lq_kv_gather_q4(s["slots"], *cache, *s["back"])
        sync()
        return [s["out"], *s["scores"], *s["back"], *cache]

    return s, step


CASES = [([5, 40, 1, 300], 16, 8, 16, 64, 32, 1, 1000), ([100, 33], 8, 8, 32, 128, 64, 5, 5001),
         ([700, 60, 90], 16, 8, 16, 128, 128, 40, 777), ([400, 64], 8, 2, 64, 256, 128, 50, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_calls_back_to_back(dtype, case):
    """Without a synchronisation, and replayed from one graph, the calls give the bits of the same calls with one after
    each."""
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    reqs, hq, hk, bs, d, group, q_len, vocab = case
    s, step = chain(torch, L, 3, reqs, hq, hk, bs, d, group, dt, q_len, vocab)
    x = {n: [torch.randn_like(s[n].float()).to(dt) for _ in range(6)] for n in ("q", "k", "v")}
    want = []
    for i in range(6):
        for n in x:
            s[n].copy_(x[n][i])
        torch.cuda.synchronize()
        want.append([t.clone() for t in step(torch.cuda.synchronize)])
    got = []
    for i in range(6):
        for n in x:
            s[n].copy_(x[n][i])
        got.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = step()
    for i in range(6):
        for n in x:
            s[n].copy_(x[n][i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], results))


def test_two_streams_at_once():
    """Two servers, each on a stream of its own with its own buffers, give what each gives alone."""
    torch, L = cuda()
    runs = [chain(torch, L, seed, *CASES[c][:6], torch.bfloat16, *CASES[c][6:]) for seed, c in ((5, 1), (6, 2))]
    want = []
    for _, step in runs:
        want.append([t.clone() for t in step(torch.cuda.synchronize)])
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for (_, step), stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,group,bs,hq,hk,reqs", [(128, 64, 16, 4, 2, [(4, 1), (22, 5), (40, 40)]), (64, 32, 32, 7, 1, [(201, 1)]),
                                                   (256, 128, 64, 2, 2, [(65, 2), (130, 130)]), (128, 128, 128, 8, 1, [(3070, 70)])])
def test_calls_stay_in_bounds(dtype, d, group, bs, hq, hk, reqs):
    torch, L = cuda()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    G = lambda *a: Guarded(torch, *a)
    b, n = len(reqs), sum(m for _, m in reqs)
    need = [-(-c // bs) for c, _ in reqs]
    nb = sum(need)
    table = np.full((b, max(need)), -1, np.int32)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = range(at, at + c)
        at += c
    cache = [G((nb, hk, bs, d // 2), torch.uint8), G((nb, hk, bs, d // group, 2), torch.float16),
             G((nb, hk, bs, d // 2), torch.uint8), G((nb, hk, bs, d // group, 2), torch.float16)]
    pool = [c.t for c in cache]
    k, v = (torch.randn((nb * bs, hk, d), device="cuda").to(dt) for _ in range(2))
    slots = torch.arange(nb * bs, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_kv_append_q4(k, v, slots, *pool, dev_status=st)
    kb, vb = G((nb * bs, hk, d), dt), G((nb * bs, hk, d), dt)
    L.lq_kv_gather_q4(slots, *pool, kb.t, vb.t, dev_status=st)
    out, ws = G((n, hq, d), dt), G((L.lq_attention_paged_q4_workspace_size(b, n, hq, hk, d),), torch.uint8)
    cu = to_dev(torch, np.concatenate([[0], np.cumsum([m for _, m in reqs])]).astype(np.int32))
    q = torch.randn((n, hq, d), device="cuda").to(dt)
    L.lq_attention_paged_q4(q, cu, to_dev(torch, np.array([c for c, _ in reqs], np.int32)), to_dev(torch, table), *pool, out.t,
                            ws.t, dev_status=st)
    logits, vocab = torch.randn((n, 3001), device="cuda").to(dt), 3001
    score = [G((n,), torch.float32), G((n,), torch.float32), G((n,), torch.int32), G((n, 20), torch.int32),
             G((n, 20), torch.float32)]
    L.lq_token_logprobs(logits, torch.randint(0, vocab, (n,), device="cuda", dtype=torch.int32), *(g.t for g in score),
                        dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for g in [*cache, kb, vb, out, ws, *score]:
        assert g.intact()
    assert np.isfinite(out.t.float().cpu().numpy()).all()
