"""Norm and rotation of heads against the formula in 64 bits.

Tolerance, in half steps u = 2^-24 of (|r_a| + |r_b|) * scale for a turned
pair: r holds three roundings (1/rms, x times it, times the weight), cos and
sin are off by 4 u (the angle's rest below pi/4 rounded once, Taylor sums of a
few roundings, their ends below 0.1 u), the scale, the product and the sum
round once each: 10 u.  A dim that does not turn has r's 3 u."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from gpu_util import gpu, need_gpu, say

pytestmark = gpu

U = 2.0 ** -24
EPS = 1e-6


def reference(x, w, pos, freq, axis, adjacent, scale, eps=EPS):
    """(y, tolerance) in 64 bits of x [T][H][D]; angles in 80."""
    x = x.astype(np.float64)
    t, _, dim = x.shape
    r = x if w is None else x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w.astype(np.float64)
    y, tol = r.copy(), 3 * U * np.abs(r)
    for i in range(len(freq)):
        if not 0 <= axis[i] < len(pos):
            continue
        a = pos[axis[i]].astype(np.longdouble) * np.longdouble(freq[i])
        two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
        a = (a - np.rint(a / two_pi) * two_pi).astype(np.float64)[:, None]
        p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + len(freq))
        y[:, :, p] = scale * (r[:, :, p] * np.cos(a) - r[:, :, q] * np.sin(a))
        y[:, :, q] = scale * (r[:, :, q] * np.cos(a) + r[:, :, p] * np.sin(a))
        tol[:, :, p] = tol[:, :, q] = 10 * U * abs(scale) * (np.abs(r[:, :, p]) + np.abs(r[:, :, q]))
    return y, tol


def freqs(rot, base=1e4):
    return (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


def check(qmv, t, heads, kv, dim, rot, axes=1, adjacent=False, norm=True, scale=1.0, place="out", pos=None,
          axis=None, pad=0):
    say(f"heads T {t} {heads}+{kv} of {dim}, rot {rot}, axes {axes}, adjacent {adjacent}, norm {norm}, {place}")
    rng = np.random.default_rng(t * 1000 + heads + dim)
    qkv = rng.standard_normal((t, (heads + 2 * kv) * dim + pad)).astype(np.float32) * 2
    freq = freqs(rot)
    if pos is None:
        pos = rng.integers(0, 200000, (axes, t)).astype(np.int32)
    if axis is None:
        axis = (np.arange(rot // 2) * axes // max(1, rot // 2)).astype(np.int32)
    qw, kw = ((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    dev = torch.from_numpy(qkv).cuda()
    q = dev[:, :heads * dim].unflatten(1, (heads, dim))
    k = dev[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim)) if kv else None
    before = dev.clone()
    kwargs = dict(q_weight=torch.from_numpy(qw).cuda() if norm else None,
                  k_weight=torch.from_numpy(kw).cuda() if norm and kv else None, eps=EPS,
                  pair_axis=torch.from_numpy(axis).cuda(), interleaved=adjacent, scale=scale)
    if place == "out":
        kwargs["q_out"] = torch.full((t, heads, dim), 7.0, device="cuda")
        kwargs["k_out"] = torch.full((t, kv, dim), 7.0, device="cuda") if kv else None
    qo, ko = qmv.head_norm_rope(q, k, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), **kwargs)
    torch.cuda.synchronize()
    off = pos[0] < 0
    for name, got, src, w in (("q", qo, qkv[:, :heads * dim].reshape(t, heads, dim), qw),
                              ("k", ko, qkv[:, heads * dim:(heads + kv) * dim].reshape(t, kv, dim), kw)):
        if got is None:
            assert kv == 0
            continue
        got = got.cpu().numpy()
        y, tol = reference(src, w if norm else None, pos, freq, axis, adjacent, scale)
        y[off] = src[off] if place == "in" else 7.0
        tol[off] = 0
        err = np.abs(got - y)
        assert np.all(err <= tol), (name, float((err - tol).max()), np.argwhere(err > tol)[:3])
    if place == "out":
        assert torch.equal(dev, before)
    else:  # nothing but q and k is written
        assert torch.equal(dev[:, (heads + kv) * dim:], before[:, (heads + kv) * dim:])


@pytest.mark.parametrize("dim", [4, 8, 12, 16, 20, 32, 44, 64, 80, 96, 100, 128, 160, 192, 256])
@pytest.mark.parametrize("adjacent", [False, True])
def test_head_sizes(dim, adjacent):
    qmv = need_gpu()
    for rot in sorted({dim, dim // 2 // 2 * 2, 2, dim - 2}):
        check(qmv, 3, 5, 2, dim, rot, adjacent=adjacent)


@pytest.mark.parametrize("t,heads,kv", [(1, 1, 0), (1, 1, 1), (1, 32, 8), (7, 3, 5), (65, 28, 4), (700, 12, 12),
                                        (3000, 8, 1), (5, 130, 3)])
@pytest.mark.parametrize("place", ["in", "out"])
def test_batches(t, heads, kv, place):
    qmv = need_gpu()
    check(qmv, t, heads, kv, 64, 64, place=place, pad=12)
    check(qmv, t, heads, kv, 128, 96, adjacent=True, place=place)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_axes_scale_and_no_norm(axes):
    qmv = need_gpu()
    check(qmv, 33, 6, 2, 128, 128, axes=axes, scale=1.3)
    check(qmv, 33, 6, 2, 80, 40, axes=axes, norm=False, adjacent=True, scale=-0.5)
    # axes in turn, some pairs on none
    axis = np.array([(i % (axes + 2)) - 1 for i in range(32)], dtype=np.int32)
    check(qmv, 9, 4, 1, 64, 64, axes=axes, axis=axis)
    check(qmv, 9, 4, 1, 64, 64, axes=axes, axis=axis, adjacent=True, norm=False)


def test_rows_of_no_sequence_and_far_positions():
    qmv = need_gpu()
    for place in ("in", "out"):
        pos = np.array([[3, -1, 0, -2**31, 5]], dtype=np.int32)
        check(qmv, 5, 4, 2, 64, 64, pos=pos, place=place)
    pos = np.array([[0, 1, 2**20, 2**24 + 1, 2**31 - 1, 2**31 - 127, 1234567891]], dtype=np.int32)
    check(qmv, 7, 4, 2, 128, 128, pos=pos)
    # other axes turn back where they are negative
    pos = np.stack([np.arange(6), -np.arange(6) * 77777, np.full(6, -2**31)]).astype(np.int32)
    check(qmv, 6, 4, 2, 96, 96, axes=3, pos=pos)


def test_the_most_tokens():
    qmv = need_gpu()
    check(qmv, 65536, 1, 1, 16, 16)
    check(qmv, 300, 257, 31, 32, 24, adjacent=True)


def test_values_at_the_ends():
    """Rows of zeros, of values whose squares leave fp32's range either way."""
    qmv = need_gpu()
    x = torch.ones(4, 2, 64, device="cuda")
    x[0] = 0.0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, :, 5] = 1e25
    w = torch.full((64,), 2.0, device="cuda")
    y, _ = qmv.head_norm_rope(x.clone(), None, None, None, q_weight=w, eps=EPS)
    r, tol = reference(x.cpu().numpy(), w.cpu().numpy(), np.zeros((1, 4), np.int32), np.zeros(0), [], False, 1.0)
    assert np.all(np.abs(y.cpu().numpy() - r) <= tol)
    # what does not turn stays as it is, an infinity too
    x = torch.randn(2, 1, 32, device="cuda")
    x[0, 0, 20], x[1, 0, 31] = float("inf"), float("-inf")
    y, _ = qmv.head_norm_rope(x.clone(), None, torch.tensor([5, 6], dtype=torch.int32, device="cuda"),
                              torch.ones(8, device="cuda"))
    assert torch.equal(y[:, :, 16:], x[:, :, 16:]) and torch.isfinite(y[:, :, :16]).all()


def test_only_one_weight():
    qmv = need_gpu()
    q, k = torch.randn(3, 3, 32, device="cuda"), torch.randn(3, 2, 32, device="cuda")
    w = torch.rand(32, device="cuda") + 0.5
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    f = torch.from_numpy(freqs(32)).cuda()
    a = dict(pos=pos, inv_freq=f, eps=EPS)
    both = qmv.head_norm_rope(q.clone(), k.clone(), q_weight=w, k_weight=w, **a)
    none = qmv.head_norm_rope(q.clone(), k.clone(), **a)
    one = qmv.head_norm_rope(q.clone(), k.clone(), q_weight=w, **a)
    two = qmv.head_norm_rope(q.clone(), k.clone(), k_weight=w, **a)
    assert torch.equal(one[0], both[0]) and torch.equal(one[1], none[1])
    assert torch.equal(two[0], none[0]) and torch.equal(two[1], both[1])


def test_two_streams_and_a_graph():
    qmv = need_gpu()
    q, k = torch.randn(50, 8, 128, device="cuda"), torch.randn(50, 2, 128, device="cuda")
    w = torch.rand(128, device="cuda") + 0.5
    f = torch.from_numpy(freqs(128)).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    want = qmv.head_norm_rope(q, k, pos, f, w, w, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [qmv.head_norm_rope(q, k, pos, f, w, w, q_out=torch.empty_like(q), k_out=torch.empty_like(k), stream=s)
           for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmv.head_norm_rope(q, k, pos, f, w, w, q_out=qo, k_out=ko)
    for rep in range(4):
        q.normal_()
        pos += 1000
        want = qmv.head_norm_rope(q, k, pos, f, w, w, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]), rep


def test_large_angles():
    """Frequencies far above one: the place in the circle from exact fractions."""
    qmv = need_gpu()
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    pos = np.array([1, 7, -1, 65535, 2**24 + 3, 2**31 - 1], dtype=np.int32)
    freq = np.array([1.0, 3.7, -41.3, 1e3, 123457.0, 3e6, -7.7e8, 2.0**32], dtype=np.float32)
    x = np.random.default_rng(5).standard_normal((6, 3, 16)).astype(np.float32)
    y, _ = qmv.head_norm_rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda())
    y = y.cpu().numpy().astype(np.float64)
    for t, p in enumerate(pos):
        for i, f in enumerate(freq):
            a = int(p) * Fraction(float(f))
            w = 0.0 if p < 0 else float(a - round(a / two_pi) * two_pi)  # such a row stays as it is
            u, v = x[t, :, i].astype(np.float64), x[t, :, i + 8].astype(np.float64)
            tol = 10 * U * (np.abs(u) + np.abs(v))
            assert np.all(np.abs(y[t, :, i] - (u * np.cos(w) - v * np.sin(w))) <= tol), (t, i)
            assert np.all(np.abs(y[t, :, i + 8] - (v * np.cos(w) + u * np.sin(w))) <= tol), (t, i)


@pytest.mark.parametrize("dim", [36, 40, 48, 68, 80, 96, 132, 160, 192])
def test_large_batches_of_heads_that_leave_lanes_idle(dim):
    """More than 8 MB of outputs, where a lane may have several vectors of a head."""
    qmv = need_gpu()
    t = (9 << 20) // (49 * dim * 4)
    check(qmv, t, 40, 9, dim, dim, axes=2, place="in", pad=4)
    check(qmv, t, 40, 9, dim, dim // 2 // 2 * 2, adjacent=True)
    check(qmv, t, 48, 1, dim, dim - 2, norm=False, scale=1.2)
    check(qmv, 2 * t, 3, 22, dim, 32, axes=3)


@pytest.mark.parametrize("t,heads,dim", [(3, 2, 64), (4, 5, 256), (1600, 16, 96)])
def test_normed_heads_with_infinities(t, heads, dim):
    """1 / sqrt(inf) is 0: finite dims become 0, the infinite ones and their partners no numbers.  Other heads are as
    they were without the infinity, a head with a NaN is NaN throughout."""
    qmv = need_gpu()
    x = torch.randn(t, heads, dim, device="cuda")
    w = torch.rand(dim, device="cuda") + 0.5
    rot = 32
    f = torch.from_numpy(freqs(rot)).cuda()
    pos = torch.arange(1, t + 1, dtype=torch.int32, device="cuda")
    want, _ = qmv.head_norm_rope(x.clone(), None, pos, f, w)
    x[0, 0, 3], x[t - 1, 1, dim - 1], x[1, 1, 0] = float("inf"), float("-inf"), float("nan")
    y, _ = qmv.head_norm_rope(x.clone(), None, pos, f, w)
    bad = torch.isnan(y)
    gone = torch.zeros_like(bad)
    gone[0, 0, [3, 3 + rot // 2]] = True
    gone[t - 1, 1, dim - 1] = True
    gone[1, 1] = True
    assert torch.equal(bad, gone)
    zero = torch.zeros_like(bad)
    zero[0, 0] = zero[t - 1, 1] = True
    assert (y[zero & ~gone] == 0).all()
    kept = ~(zero | gone)
    assert torch.equal(y[kept], want[kept])


@pytest.mark.parametrize("dim,rot", [(64, 0), (64, 64), (96, 32), (256, 256)])
def test_normed_heads_at_the_end_of_the_range(dim, rot):
    """Values of up to the largest fp32 number, whose mean's inverse lies below the smallest normal one."""
    qmv = need_gpu()
    rng = np.random.default_rng(dim + rot)
    top = float(np.finfo(np.float32).max)
    for t in (3, (9 << 20) // (20 * dim * 4)):
        x = (rng.uniform(-1, 1, (t, 20, dim)) * top * rng.uniform(0.2, 1.0, (t, 20, 1))).astype(np.float32)
        x[:, :, 5] = rng.choice([-top, top], (t, 20))
        x[:, ::3, 7] = 1e-3
        w = (1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)
        pos = rng.integers(0, 9999, (1, t)).astype(np.int32)
        f = freqs(rot)
        y, _ = qmv.head_norm_rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(pos).cuda(),
                                  torch.from_numpy(f).cuda(), q_weight=torch.from_numpy(w).cuda())
        r, tol = reference(x, w, pos, f, [0] * len(f), False, 1.0)
        err = np.abs(y.cpu().numpy() - r)
        # a quotient below the smallest normal number has that number's half step 2^-150 beside its own
        assert np.all(err <= tol + 2.0 ** -148), float((err - tol).max())
