"""Tree calls refuse tensors on different GPUs before they reach the library (stand-ins for tensors: no GPU needed)."""

import pytest
import torch

from invariant_vd_step_gb300 import vd


class OnGpu:
    """What the checks ask of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, device
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.at

    def data_ptr(self):
        return 4096

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)


def test_tensors_on_two_gpus_are_refused(monkeypatch):
    class NoLibrary:
        def __getattr__(self, name):
            def call(*a):
                raise AssertionError(f"{name} reached")
            return call
    monkeypatch.setattr(vd, "lib", NoLibrary)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vd, "_current_raw_stream", lambda device: 0)
    tree = object.__new__(vd.Tree)
    spec = type("Spec", (), dict(n_heads=4, head_dim=64, qkv_dim=512, vocab=100))
    tree.h, tree.model = 1, type("M", (), dict(h=1, spec=spec))()
    pool = type("P", (), dict(h=1))()
    tree.num_nodes, tree.num_seqs = 3, 2
    q = [OnGpu((3, 4, 64), torch.bfloat16, d) for d in (0, 1)]
    qkv = [OnGpu((3, 512), torch.bfloat16, d) for d in (0, 1)]
    t, n, o = ([OnGpu(s, torch.int32, d) for d in (0, 1)] for s in ((3,), (2,), (2, 5)))
    calls = [lambda: tree.attention(pool, 0, q[1], q[0]), lambda: tree.attention(pool, 0, q[0], q[1]),
             lambda: tree.rope_kv(pool, 0, qkv[1], q[0]), lambda: tree.rope_kv(pool, 0, qkv[0], q[1]),
             lambda: tree.step(pool, OnGpu((3, 100), torch.float32, 1)),
             lambda: tree.accept(pool, t[1], t[0], n[0], o[0]), lambda: tree.accept(pool, t[0], t[1], n[0], o[0]),
             lambda: tree.accept(pool, t[0], t[0], n[1], o[0]), lambda: tree.accept(pool, None, t[0], n[0], o[1])]
    try:
        for i, call in enumerate(calls):
            with pytest.raises(vd.VDError) as e:
                call()
                pytest.fail(f"call {i} was taken")
            assert e.value.code == vd.VD_ERR_INVALID_ARG
    finally:
        tree.h = None  # nothing for close() to destroy
