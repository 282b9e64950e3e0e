"""Rotary positions against float64: layouts, rotated parts, scalings, types,
strides, far positions; the model's RoPE + K/V write with a set rope."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from gpu_util import bits, f64, ready
from invariant_vd_step_gb300 import synth, vd
from test_rotary import SCALINGS, frequencies

pytestmark = pytest.mark.gpu

TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
# half a step of each type, relative, and its smallest subnormal's half
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def reference(x, pos, rot, layout, theta, scaling, inverse):
    """float64 rotation of x [T][H][hd] and the bound of each element's float32 error before its last rounding."""
    f, mag = frequencies(rot, theta, scaling)
    ang = np.array([[float((Fraction(int(p)) * Fraction(float(v)) / TWO_PI) % 1) * 2 * math.pi for v in f] for p in pos])
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    if inverse:
        s, mag = -s, 1 / mag
    half = rot // 2
    i1 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i2 = i1 + (half if layout == "half" else 1)
    y, err = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = mag * (x1 * c - x2 * s), mag * (x2 * c + x1 * s)
    # sincospi within 2 ulp (2^-22), its argument's rounding (pi/4 2^-24), the magnitude's and its product's
    # rounding, the products' and the sum's: below 2^-21 of mag (|x1| + |x2|); the frequency's own last bit (host
    # pow) times the position on top
    e = mag * (np.abs(x1) + np.abs(x2)) * (2.0 ** -21 + np.abs(pos.astype(np.float64))[:, None, None] * f * 2.0 ** -51)
    err[..., i1], err[..., i2] = e, e
    return y, err


def check(got, want, err, dtype):
    tol = err + HALF_STEP[dtype] * (np.abs(want) + err) + SMALLEST[dtype]
    d = np.abs(f64(got.contiguous()) - want)
    assert np.all(d <= tol), f"max excess {(d - tol).max():.3g}"


CASES = [  # head_dim, rot_dim, layout
    (64, 0, "half"), (128, 0, "half"), (128, 64, "half"), (96, 0, "interleaved"), (96, 64, "interleaved"),
    (256, 128, "interleaved"), (80, 20, "half"), (18, 6, "interleaved"), (2, 0, "half"), (512, 512, "half"),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("hd,rot,layout", CASES)
def test_rotation_vs_float64(hd, rot, layout, dtype):
    ready()
    for k, (scaling, inverse, T, H) in enumerate([(None, False, 1, 1), ("linear", True, 5, 3), ("bands", False, 67, 9),
                                                   ("yarn", True, 33, 40), ("yarn", False, 130, 2)]):
        sc = SCALINGS.get(scaling)
        rope = vd.Rope(hd, rot, layout, 5e5, sc)
        g = torch.Generator().manual_seed(k)
        x = torch.randn((T, H, hd), generator=g).to(dtype).cuda()
        pos = torch.randint(-200, 200000, (T,), generator=g, dtype=torch.int32)
        pos[0] = 0 if T == 1 else 2 ** 31 - 1
        if T > 1:
            pos[1] = -2 ** 31
        out = rope.apply(x, pos.cuda(), inverse=inverse)
        want, err = reference(f64(x), pos.numpy(), rot or hd, layout, 5e5, sc, inverse)
        check(out, want, err, dtype)
        if (rot or hd) < hd:
            assert torch.equal(out[..., rot:], x[..., rot:])
        # in place, and from / into strided rows whose other elements stay as they are: the same bits
        y = x.clone()
        assert rope.apply(y, pos.cuda(), y, inverse=inverse) is y
        np.testing.assert_array_equal(bits(y), bits(out))
        for pad, shift in ((8, 0), (3, 1)):
            xs = torch.full((T, H + 2, hd + pad), 7.0, dtype=dtype, device="cuda")
            ys = xs.clone()
            xv, yv = xs[:, 1:H + 1, shift:shift + hd], ys[:, :H, shift:shift + hd]
            xv.copy_(x)
            rope.apply(xv, pos.cuda(), yv, inverse=inverse)
            np.testing.assert_array_equal(bits(yv), bits(out))
            ys[:, :H, shift:shift + hd] = 7.0
            assert (ys == 7.0).all()


def test_zero_sizes_side_stream_and_capture():
    ready()
    rope = vd.Rope(128, scaling=SCALINGS["bands"])
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    rope.apply(e, torch.empty(0, dtype=torch.int32, device="cuda"))
    rope.apply(torch.empty((4, 0, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
    x = torch.randn((300, 8, 128), device="cuda").bfloat16()
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    want = rope.apply(x, pos)
    y, s, g = torch.empty_like(x), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        rope.apply(x, pos, y)
    x.copy_(x.flip(0))
    want2 = rope.apply(x, pos)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2) and not torch.equal(want, want2)


def test_refusals():
    ready()
    rope = vd.Rope(64)
    x = torch.zeros((4, 2, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [
        lambda: rope.apply(x.double(), pos),
        lambda: rope.apply(x, pos.long()),
        lambda: rope.apply(x, pos[:3]),
        lambda: rope.apply(x[..., :32], pos),
        lambda: rope.apply(x.transpose(1, 2).contiguous().transpose(1, 2), pos),      # elements of a row not contiguous
        lambda: rope.apply(x, pos, x[:1].expand(4, 2, 64)),                            # rows of y overlap
        lambda: rope.apply(x, pos, torch.zeros(4 * 64 + 64, device="cuda").as_strided((4, 2, 64), (64, 64, 1))),
        lambda: rope.apply(x, pos, x.view(-1).as_strided((4, 2, 64), (64, 256, 1))),   # in place, other strides
        lambda: rope.apply(x, pos.cpu()),
        lambda: rope.apply(x, pos, x.bfloat16()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(vd.VDError):
            call()
            pytest.fail(f"call {i} was taken")


ROPES = [dict(layout="half", scaling=SCALINGS["bands"]), dict(layout="interleaved"),
         dict(layout="interleaved", rot_dim=32, scaling=SCALINGS["yarn"]), dict(layout="half", rot_dim=16)]


@pytest.mark.parametrize("kw", ROPES, ids=str)
def test_model_rope_equals_the_op(kw):
    """rope_kv of a model with a set rope: q and K bit for bit the op's, V untouched; the local layers use theirs."""
    ready()
    spec = synth.TINY.with_(sliding_window=8, local_global_period=2)
    W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=1).items()}
    model = vd.Model(spec, W, max_tokens=64, max_seqs=2, max_logit_rows=4, max_context=256)
    pool = vd.KVPool(model, 20)
    rope, local = vd.Rope(64, theta=5e5, **kw), vd.Rope(64, theta=1e4)
    model.set_rope(rope, local)
    T, Hq, Hkv, hd = 40, 4, 2, 64
    qkv = synth.make_normal_bf16((T, (Hq + 2 * Hkv) * hd), seed=3).cuda()
    pt = synth.page_permutation(20, seed=1)[:16]
    b = vd.StepBatch([(np.zeros(T, np.int32), 101, pt)])
    rows = qkv.view(T, Hq + 2 * Hkv, hd)
    pos = torch.arange(101, 101 + T, dtype=torch.int32, device="cuda")
    k, v = (torch.empty((101 + T, Hkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for layer, r in ((0, local), (1, rope)):
        q = torch.empty((T, Hq, hd), dtype=torch.bfloat16, device="cuda")
        model.rope_kv(pool, layer, b, qkv, q)
        model.copy_kv(pool, layer, pt, 101 + T, k, v)
        want = r.apply(rows[:, :Hq + Hkv], pos)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(q), bits(want[:, :Hq]))
        np.testing.assert_array_equal(bits(k[101:]), bits(want[:, Hq:]))
        np.testing.assert_array_equal(bits(v[101:]), bits(rows[:, Hq + Hkv:]))


def test_default_rope_keeps_the_models_results_near_and_graphs_follow_a_new_rope():
    ready()
    spec = synth.TINY
    W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=1).items()}
    toks = synth.make_tokens(40, spec.vocab, seed=2)

    def run(rope, graphs=0, again=None):
        m = vd.Model(spec, W, max_tokens=64, max_seqs=2, max_logit_rows=4, max_context=64)
        p = vd.KVPool(m, 4)
        m.set_graph_mode(graphs)
        if rope is not None:
            m.set_rope(rope)
        out = torch.empty((1, spec.vocab), device="cuda")
        b = vd.StepBatch([(toks, 0, np.arange(4, dtype=np.int32))], logit_rows=[39])
        for _ in range(3 if graphs else 1):
            m.step(p, b, out)
        if again is not None:
            m.set_rope(again)
            for _ in range(3):
                m.step(p, b, out)
        torch.cuda.synchronize()
        assert m.device_status() == 0
        return out
    table, same = run(None), run(vd.Rope(64, theta=spec.rope_theta))
    # cos and sin differ in their last bit at most (the table rounds float64, the op's are within 2 ulp), far below
    # the bf16 rounding of q and k: the step's stated tolerance holds with room
    assert torch.all((table - same).abs() <= 2e-2 + 1e-2 * table.abs())
    scaled = vd.Rope(64, theta=spec.rope_theta, scaling=SCALINGS["linear"])
    want = run(scaled)
    assert not torch.equal(want, same)
    assert torch.equal(run(None, graphs=2, again=scaled), want)  # captured graphs do not outlive the rope


def test_outputs_and_workspaces_made_by_a_call_belong_to_its_stream():
    """Memory that torch still has in use on the current stream is not handed to a call on another one."""
    ready()
    side, x = torch.cuda.Stream(), torch.randn((64, 8, 64), device="cuda", dtype=torch.bfloat16)
    pos, rope = torch.arange(64, dtype=torch.int32, device="cuda"), vd.Rope(64)
    want = rope.apply(x, pos)
    logits = torch.randn((4, 5000), device="cuda")
    s, f = [(1, k, 1.0) for k in range(4)], [(0, 0.9, 0.0)] * 4
    tok, tok_side = (torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(2))
    vd.sample(logits, s, f, tok)
    torch.cuda.synchronize()
    held = torch.empty_like(x)
    freed = held.data_ptr()
    del held  # the current stream's allocator would hand this block out next
    got = rope.apply(x, pos, stream=side)
    assert got.data_ptr() != freed
    vd.sample(logits, s, f, tok_side, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(tok_side, tok)
