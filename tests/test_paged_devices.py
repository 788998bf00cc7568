"""The binding of the paged cache's calls refuses tensors in host memory, whose addresses a kernel must not get (no GPU
needed: nothing is launched)."""
import pytest
import torch

import lattice_vq_weight_gb300 as L


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def calls():
    cache = L.paged_cache(4, 2, 16, 64, "cpu")
    k, q = torch.zeros((3, 2, 64)), torch.zeros((3, 4, 64))
    slots = torch.zeros(3, dtype=torch.int64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    p, u = torch.zeros((2, 3, 50)), torch.zeros((2, 2))
    return {
        "lq_kv_plan": (i32(2), i32(2), 16, i32(4), i32(2, 4), i32(3), i32(2), slots, i32(3), i32(1)),
        "lq_qk_norm_rope": (q, k, torch.ones(64), torch.ones(64), 1e-6, i32(3), torch.ones(9, 64), q, k),
        "lq_kv_append": (k, k, slots, *cache),
        "lq_kv_gather": (slots, *cache, k, k.clone()),
        "lq_attention_paged": (q, i32(3), i32(2), i32(2, 4), *cache, torch.zeros_like(q), ws),
        "lq_verify_draft": (i32(2, 2), None, p, p[:, :2].contiguous(), u, u[:, 0].contiguous(), i32(2, 3), i32(2)),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_host_tensors(name):
    with pytest.raises(ValueError, match="device"):
        getattr(L, name)(*calls()[name], stream=0)


class Elsewhere:
    """Stands for a tensor on a device by its index; everything else is the tensor's own."""

    def __init__(self, t, device):
        self.t, self.device_index = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.t.is_contiguous()


@pytest.mark.parametrize("name", sorted(calls()))
def test_every_tensor_is_looked_at(name, monkeypatch):
    """One tensor after the other in host memory or on a second device, the rest on the first one."""
    called = []

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: called.append(fn) or 0

    monkeypatch.setattr(L, "_LIB", Lib())
    args = calls()[name]
    put = lambda i, dev: [Elsewhere(a, dev if j == i else 0) if isinstance(a, torch.Tensor) else a
                          for j, a in enumerate(args)]
    status = Elsewhere(i32(1), 0)
    getattr(L, name)(*put(-1, 0), dev_status=status, stream=0)
    assert called == [name]
    for i, a in enumerate(args):
        if isinstance(a, torch.Tensor):
            for dev in (-1, 1):
                with pytest.raises(ValueError, match="device"):
                    getattr(L, name)(*put(i, dev), dev_status=status, stream=0)
    with pytest.raises(ValueError, match="device"):
        getattr(L, name)(*put(-1, 0), dev_status=Elsewhere(i32(1), -1), stream=0)
    assert called == [name]
