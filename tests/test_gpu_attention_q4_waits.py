"""The 4-bit attention's tensor-core kernel at every small number of tiles (no wait gives up, whoever is first) and in a
batch of many requests."""
import numpy as np
import pytest

from tests.gpu_util import cuda, to_dev
from tests.test_gpu_attention_q4 import CACHE, build, check, reference, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 8])
def test_no_wait_gives_up(d, tiles):
    """Contexts of so many tiles (64 tokens at head_dim 256, else 128), the last one full or of one token, called again
    and again: the status stays 0 and the bits are the first call's."""
    torch, L = cuda()
    step, rows = (64, 24) if d == 256 else (128, 40)
    lens = [tiles * step, (tiles - 1) * step + 1]
    reqs = [(max(n, rows), rows) for n in lens] * 20
    s = build(torch, np.random.default_rng(tiles), reqs, 4, 2, 16, d, 64, "bf16")
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", *CACHE)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, first = workspace(torch, L, s), None
    out = torch.empty_like(s["q"])
    for _ in range(200):
        out.fill_(float("nan"))
        L.lq_attention_paged_q4(s["q"], dev["cu"], dev["lens"], dev["table"], *(dev[n] for n in CACHE), out, ws, dev_status=st)
        if first is None:
            first = out.clone()
        assert torch.equal(out, first)
    assert int(st) == 0
    check(first, reference(s), "bf16", range(2 * rows))


@pytest.mark.parametrize("d,q_len", [(128, 10), (256, 5)])
def test_every_row_of_many_requests(d, q_len):
    """More requests than CTAs can share, one of them long: every row of every request."""
    torch, L = cuda()
    rng = np.random.default_rng(d)
    reqs = [(int(n), q_len) for n in rng.integers(1, 400, 90)] + [(6000, q_len)]
    s = build(torch, rng, reqs, 16, 4, 16, d, 64, "bf16")
    dev = {n: to_dev(torch, s[n]) for n in ("cu", "lens", "table", *CACHE)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(s["q"], float("nan"))
    L.lq_attention_paged_q4(s["q"], dev["cu"], dev["lens"], dev["table"], *(dev[n] for n in CACHE), out,
                            workspace(torch, L, s), dev_status=st)
    assert int(st) == 0
    check(out, reference(s), "bf16")
