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
