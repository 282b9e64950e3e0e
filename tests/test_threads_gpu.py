"""Calls that two host threads make at the same time, each on its own stream, model and workspace: kernels that both use
with different amounts of shared memory."""

import ctypes
import subprocess

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import vd
from tree_scenario import TreeScenario, make_tree, tree_spec

pytestmark = pytest.mark.gpu

# Two threads that do nothing but call (Python's own would take turns between the calls).  Every 256 calls a thread
# waits for its stream through `sync`.
CALLER = r"""
#include <atomic>
#include <cstdint>
#include <cstddef>
#include <thread>
namespace {
std::atomic<int> ready;
template <typename F>
void loop(int n, int* rc, F f) {
  ready.fetch_add(1);
  while (ready.load() < 2) {}
  for (int k = 0; k < n && !*rc; ++k) *rc = f(k);
}
template <typename F, typename G>
void both(int n, int* rc, F f, G g) {
  ready = 0;
  std::thread a([&] { loop(n, rc, f); }), b([&] { loop(n, rc + 1, g); });
  a.join();
  b.join();
}
}
using Tree = int (*)(void*, void*, int32_t, const void*, void*, void*);
using Sample = int (*)(const void*, int32_t, int32_t, int64_t, const void*, const void*, void*, void*, void*, size_t, void*);
using Sync = int (*)(void*);
struct TreeCall { void *t, *pool; const void* q; void *out, *stream; };
struct SampleCall { const void* x; int64_t V; const void *s, *f; void *tok, *ws; size_t bytes; void* stream; };
extern "C" void trees(int n, Tree f, Sync sync, const TreeCall* c, int* rc) {
  auto job = [&](const TreeCall& c) { return [&](int k) {
    const int r = f(c.t, c.pool, 0, c.q, c.out, c.stream);
    return r ? r : k % 256 == 255 ? sync(c.stream) : 0; }; };
  both(n, rc, job(c[0]), job(c[1]));
}
extern "C" void samples(int n, Sample f, Sync sync, const SampleCall* c, int* rc) {
  auto job = [&](const SampleCall& c) { return [&](int k) {
    const int r = f(c.x, 1, (int32_t)c.V, c.V, c.s, c.f, c.tok, nullptr, c.ws, c.bytes, c.stream);
    return r ? r : k % 256 == 255 ? sync(c.stream) : 0; }; };
  both(n, rc, job(c[0]), job(c[1]));
}
"""

VP = ctypes.c_void_p


class TreeCall(ctypes.Structure):
    _fields_ = [(n, VP) for n in ("t", "pool", "q", "out", "stream")]


class SampleCall(ctypes.Structure):
    _fields_ = [("x", VP), ("V", ctypes.c_int64), ("s", VP), ("f", VP), ("tok", VP), ("ws", VP),
                ("bytes", ctypes.c_size_t), ("stream", VP)]


@pytest.fixture(scope="module")
def caller(tmp_path_factory):
    ready()
    d = tmp_path_factory.mktemp("caller")
    (d / "caller.cpp").write_text(CALLER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", str(d / "caller.cpp"), "-o",
                    str(d / "libcaller.so")], check=True)
    return ctypes.CDLL(str(d / "libcaller.so"))


@ctypes.CFUNCTYPE(ctypes.c_int, VP)
def sync(stream):
    torch.cuda.ExternalStream(stream).synchronize()
    return 0


def at_once(call, entry, calls, n):
    rc = (ctypes.c_int * 2)()
    call(n, ctypes.cast(entry, VP), sync, calls, rc)
    torch.cuda.synchronize()
    assert list(rc) == [0, 0], vd.lib().vd_last_error()


def test_trees_of_two_models_with_short_and_long_tails(caller):
    # tails of 198 and of 12 rows: 99 KB and 6 KB of shared memory
    scenarios = [TreeScenario(tree_spec(8, 2, 128), [(31, make_tree("star", 167))], seed=1),
                 TreeScenario(tree_spec(8, 2, 128), [(4, make_tree("random", 8, 2))], seed=2)]
    want = [sc.attention() for sc in scenarios]
    outs = [torch.full_like(sc.q, float("nan")) for sc in scenarios]
    streams = [torch.cuda.Stream() for _ in scenarios]
    torch.cuda.synchronize()
    calls = (TreeCall * 2)(*[TreeCall(sc.tree.h, sc.pool.h, sc.q.data_ptr(), o.data_ptr(), s.cuda_stream)
                             for sc, o, s in zip(scenarios, outs, streams)])
    at_once(caller.trees, vd.lib().vd_op_tree_attention, calls, 6000)
    for o, w in zip(outs, want):
        np.testing.assert_array_equal(bits(o), bits(w))


def test_choices_from_two_large_vocabularies(caller):
    calls, keep = (SampleCall * 2)(), []
    for k, V in enumerate((1 << 21, 1400000)):
        x = torch.randn((1, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(V))
        want, tok = (torch.full((1,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        s, f = np.array([(3, V, 0.8, 0)], vd.SAMPLER), np.array([(50, 0.9, 0, 0)], vd.FILTER)
        ws, stream = vd.sample_workspace(1, V), torch.cuda.Stream()
        vd.sample(x, s, f, want, workspace=ws)
        calls[k] = SampleCall(x.data_ptr(), V, s.ctypes.data, f.ctypes.data, tok.data_ptr(), ws.data_ptr(), ws.nbytes,
                              stream.cuda_stream)
        keep.append((x, s, f, ws, stream, want, tok))
    torch.cuda.synchronize()
    at_once(caller.samples, vd.lib().vd_op_sample, calls, 2000)
    for *_, want, tok in keep:
        assert torch.equal(tok, want)
