"""lq_token_logprobs on the GPU where the way in which rows are divided changes, and far into a matrix."""
import numpy as np
import pytest

from tests.gpu_util import cuda
from tests.test_gpu_logprobs import call, check, rows

pytestmark = pytest.mark.gpu

MOST = 208 * 1024 - 32                         # bytes of a share in shared memory at once


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctas", [1, 2, 4, 8])
@pytest.mark.parametrize("more", [0, 1, 8, 9])
def test_rows_that_just_fill_the_shared_memory(dtype, ctas, more):
    """As long as the shared memory of so many CTAs, and a little longer."""
    torch, L = cuda()
    vocab = ctas * (MOST // (2 if dtype == "bf16" else 4)) + more
    rng = np.random.default_rng(vocab)
    x = rows(torch, rng, 3, vocab, dtype)
    x[1, vocab - 1] = 40.0
    tokens = [0, vocab - 1, vocab // 2]
    got, st = call(torch, L, x, tokens, 5)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 5)


def test_rows_far_into_a_matrix():
    """Rows whose elements and bytes lie past 2^32, as columns of a wide buffer."""
    torch, L = cuda()
    vocab, ld = 5001, (1 << 30) + 3
    rng = np.random.default_rng(8)
    buf = torch.empty((4 * ld + vocab,), dtype=torch.bfloat16, device="cuda")      # 8.6 GB
    x = buf.as_strided((5, vocab), (ld, 1))
    x.copy_(rows(torch, rng, 5, vocab, "bf16"))
    tokens = rng.integers(0, vocab, 5)
    got, st = call(torch, L, x, tokens, 6)
    assert st == 0
    check(got, x.float().cpu().numpy(), tokens, 6)
