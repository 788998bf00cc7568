"""lq_token_logprobs on the GPU against the float64 oracle."""
import numpy as np
import pytest

import oracle.q4_oracle as Q
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu

# The sum of exponentials: an error of 2^-22 for each plus n 2^-24 for n additions in line, n up to 64 in a thread
# and a few tens after that; its logarithm is off by as much absolutely.  The difference of two logits and the
# result are rounded once each, relative to their size.
TOL = 2.0 ** -17


def call(torch, L, x, tokens, top, extra=True):
    """Outputs as numpy arrays (logprobs, entropy, ranks, top_tokens, top_logprobs) and the status."""
    n = x.shape[0]
    f = lambda *shape: torch.full(shape, 77.0, device="cuda")
    i = lambda *shape: torch.full(shape, 77, dtype=torch.int32, device="cuda")
    out = [f(n), f(n) if extra else None, i(n) if extra else None, i(n, top) if top else None, f(n, top) if top else None]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_token_logprobs(x, to_dev(torch, np.asarray(tokens, np.int32)), *out, dev_status=st)
    return [None if o is None else o.cpu().numpy() for o in out], int(st)


def check(got, x, tokens, top):
    want = Q.token_logprobs(x, tokens, top)
    for g, w, whole in zip(got, want, (False, False, True, True, False)):
        if g is None:
            continue
        if whole:
            assert np.array_equal(g, w)
        else:
            fine = np.isfinite(w)
            assert np.array_equal(g[~fine], w[~fine].astype(np.float32))
            assert (np.abs(g[fine] - w[fine]) <= TOL * (1 + np.abs(w[fine]))).all()


def rows(torch, rng, n, vocab, dtype, size=3.0):
    x = to_dev(torch, (size * rng.standard_normal((n, vocab))).astype(np.float32))
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4097, 16385, 32000, 50001, 128256, 300001])
def test_sizes(dtype, vocab):
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    for n, top in ((1, min(5, vocab)), (3, min(32, vocab)), (2, 0)):
        x = rows(torch, rng, n, vocab, dtype)
        tokens = rng.integers(0, vocab, n)
        got, st = call(torch, L, x, tokens, top)
        assert st == 0
        check(got, x.float().cpu().numpy(), tokens, top)
        again, _ = call(torch, L, x, tokens, top)
        assert all(a is b is None or a.tobytes() == b.tobytes() for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab", [(150, 515), (1000, 515), (900, 4001), (400, 9999)])
def test_many_rows(dtype, n, vocab):
    """More rows than fit the GPU at once, at odd addresses."""
    torch, L = cuda()
    rng = np.random.default_rng(n)
    x, tokens = rows(torch, rng, n, vocab, dtype), rng.integers(-1, vocab, n)
    got, st = call(torch, L, x, tokens, 4)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 4)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 786433), ("bf16", 1000003), ("f32", 393217), ("f32", 900001)])
def test_rows_longer_than_shared_memory(dtype, vocab):
    """Shares in two or three segments, the last of them one token or more; all equal, and the largest in the last."""
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    x = rows(torch, rng, 3, vocab, dtype)
    x[1] = 1.5
    x[2, vocab - 9:] = 30.0
    tokens = [vocab // 3, vocab - 1, vocab - 5]
    got, st = call(torch, L, x, tokens, 7)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", range(8))
def test_rows_that_start_anywhere(dtype, shift):
    """Rows at every offset from a 16-byte boundary, in wider rows whose other columns are larger."""
    torch, L = cuda()
    rng = np.random.default_rng(shift)
    vocab = 5000 + 3 * shift
    wide = torch.full((3, vocab + 21 + shift), 100.0, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                      device="cuda")
    wide[:, shift:shift + vocab] = rows(torch, rng, 3, vocab, dtype)
    x = wide[:, shift:shift + vocab]
    tokens = rng.integers(0, vocab, 3)
    got, st = call(torch, L, x, tokens, 9)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 9)


def patterns(vocab, rng):
    v = np.arange(vocab)
    yield "all equal", np.zeros(vocab)
    yield "rising", v / 1000
    yield "falling", -v / 1000
    yield "few values", rng.integers(0, 4, vocab).astype(float)
    for period in (8, 32, 128, 256, 512, 2048, 4096):
        yield f"one in {period} high", np.where(v % period == 3, 5.0, 0.0) + 0.001 * rng.standard_normal(vocab)
        yield f"eight in {period} high", np.where(v % period < 8, 5.0, 0.0)
    yield "high at the end", np.where(v >= vocab - 40, 4.0, 0.0)
    yield "a high run", np.where((v >= 1000) & (v < 1700), 4.0, 0.0) + 1e-3 * rng.standard_normal(vocab)
    yield "one token for certain", np.where(v == vocab - 1, 60.0, 0.0)
    yield "zeros of both signs", np.where(v % 2 == 0, -0.0, 0.0)
    yield "far from zero", 1e4 + rng.standard_normal(vocab)
    yield "a wide span", 300 * rng.standard_normal(vocab)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [4096, 33001])
@pytest.mark.parametrize("top", [1, 5, 32])
def test_patterns(dtype, vocab, top):
    """Ties (the lowest token first) and large logits bunched together in every period of the work's division."""
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    names, x = zip(*patterns(vocab, rng))
    x = to_dev(torch, np.stack(x).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    tokens = rng.integers(0, vocab, len(names))
    got, st = call(torch, L, x, tokens, top)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [100, 20001])
def test_masked_tokens(dtype, vocab):
    """Logits of -inf: most of them, all but a few (fewer than the alternatives), all."""
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    x = rows(torch, rng, 4, vocab, dtype)
    x[0, to_dev(torch, rng.random(vocab) < 0.9)] = -float("inf")
    x[1, 3:] = -float("inf")
    x[2, :vocab - 1] = -float("inf")
    tokens = [5, 7, vocab - 1, 0]
    got, st = call(torch, L, x, tokens, 6)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 6)
    x[3] = -float("inf")
    got, st = call(torch, L, x, tokens, 6)
    assert st == L.LQ_DEV_RANGE
    check(got, x.float().cpu().numpy(), tokens, 6)
    assert got[0][3] == -np.inf and got[1][3] == 0 and got[3][3].tolist() == list(range(6))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [90, 30001])
def test_ranks_at_the_ends_of_the_range(dtype, vocab):
    """Masks of the type's lowest value beside -inf, logits all within 2^-100 of one another, a largest logit of 0."""
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    x = rows(torch, rng, 5, vocab, dtype)
    low = torch.finfo(x.dtype).min
    x[0, ::2], x[0, 1::3] = -float("inf"), low
    x[1, 1:] = low
    x[2] *= 2.0 ** -104
    x[3] = -x[3].abs()
    x[3, 7] = 0
    x[4, :] = low
    x[4, 5] = -float("inf")
    for tokens in ([4, 3, 8, 7, 5], [7, 9, 50, 60, 6], [1, 0, 11, 12, 0]):
        got, st = call(torch, L, x, tokens, 3)
        assert st == 0
        check(got, x.float().cpu().numpy(), tokens, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", [0, 777, 20000])
def test_non_finite_logits_stay_in_their_row(dtype, bad, where):
    torch, L = cuda()
    rng = np.random.default_rng(4)
    x = rows(torch, rng, 3, 20001, dtype)
    keep = x.float().cpu().numpy()
    x[1, where] = bad
    tokens = [1, 2, 3]
    got, st = call(torch, L, x, tokens, 5)
    assert st == L.LQ_DEV_NONFINITE
    assert np.isnan(got[0][1]) and np.isnan(got[1][1]) and got[2][1] == -1
    assert (got[3][1] == -1).all() and np.isnan(got[4][1]).all()
    check([g[[0, 2]] for g in got], keep[[0, 2]], [1, 3], 5)


def test_tokens_not_given_or_past_the_vocabulary():
    torch, L = cuda()
    x = rows(torch, np.random.default_rng(5), 4, 300, "f32")
    for tokens, flag in (([-1, 5, -100, 299], 0), ([0, 300, 5, -1], L.LQ_DEV_RANGE), ([0, 1 << 30, 5, -1], L.LQ_DEV_RANGE)):
        got, st = call(torch, L, x, tokens, 3)
        assert st == flag
        check(got, x.cpu().numpy(), tokens, 3)
    got, st = call(torch, L, x, [1, 2, 3, 4], 0, extra=False)  # log probabilities alone
    assert st == 0
    check(got, x.cpu().numpy(), [1, 2, 3, 4], 0)
    call(torch, L, x[:0], [], 3)


def test_a_replayed_graph_and_two_streams():
    """Captured, replayed on new logits, and two calls at once on streams of their own."""
    torch, L = cuda()
    rng = np.random.default_rng(6)
    xs = [rows(torch, rng, 2, 40001, d) for d in ("f32", "bf16")]
    tokens = to_dev(torch, np.array([4, 40000], np.int32))
    outs = [[torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
             torch.empty((2, 7), dtype=torch.int32, device="cuda"), torch.empty((2, 7), device="cuda")] for _ in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for x, o, s in zip(xs, outs, streams):
        L.lq_token_logprobs(x, tokens, *o, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        check([t.cpu().numpy() for t in o], x.float().cpu().numpy(), [4, 40000], 7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, o in zip(xs, outs):
            L.lq_token_logprobs(x, tokens, *o)
    for _ in range(2):
        for x in xs:
            x.copy_(torch.randn_like(x.float()))
        g.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            check([t.cpu().numpy() for t in o], x.float().cpu().numpy(), [4, 40000], 7)
