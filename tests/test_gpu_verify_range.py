"""lq_verify_draft with target weights that are not probabilities: up to 4 they are drawn from as they are, above that they
count as 4 and the status says so."""
import numpy as np
import pytest

import oracle.paged_oracle as P
from tests.gpu_util import cuda, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 33001])
@pytest.mark.parametrize("top", [0.25, 4.0, 4.125, 30.0])
def test_weights_of_any_size(dtype, vocab, top):
    torch, L = cuda()
    rng = np.random.default_rng(vocab)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = (rng.integers(0, 65, (3, 2, vocab)) / 256).astype(np.float32) * (1.0 if top > 0.25 else 0.5)
    p[1, 0, vocab // 2] = top
    p[1, 1, vocab // 3] = top
    p[0, 1, 5] = 60.0                            # in a row that is not drawn from
    x = np.array([[1], [2], [3]], np.int32)
    ua, us = np.array([[0.999], [0.0], [0.0]], np.float32), rng.random(3, np.float32)
    p[0, 0, 1] = 0.0                             # refused
    p[1:, 0, 2:4] = 0.25                         # accepted
    out = torch.full((3, 2), -9, dtype=torch.int32, device="cuda")
    acc, st = torch.full((3,), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lq_verify_draft(to_dev(torch, x), None, to_dev(torch, p).to(dt), None, to_dev(torch, ua), to_dev(torch, us), out, acc,
                      st)
    torch.cuda.synchronize()
    want, wacc = P.verify(x, None, p, None, ua, us)
    assert np.array_equal(acc.cpu().numpy(), wacc) and np.array_equal(out.cpu().numpy(), want)
    assert wacc.tolist() == [0, 1, 1]
    assert int(st) == (L.LQ_DEV_RANGE if top > 4 else 0)
