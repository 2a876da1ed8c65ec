"""Low-rank adapters against the formula in 64 bits.

Tolerance, in half steps u = 2^-24: weights are exact as fp32 numbers, so only
sums round.  A lane adds its products in turn, at most m = 8 * ceil(k / 512) of
them (8 columns of each 512, if one slice has them all), then 6 steps over the
wave and up to 15 over the slices: h is off by (m + 21) u of its terms' sizes
S_h.  The second product sums 8 terms in a lane, 5 steps over the lanes, the
scale and the base: 15 u of its own terms.  Together less than (m + 40) u *
|scale| * sum |b| S_h, and u of the base."""
import numpy as np
import pytest
import torch

from gpu_util import gpu, need_gpu, say

pytestmark = gpu

U = 2.0 ** -24
KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def reference(x, a, b, base, ids, ranks, scales):
    """(y, tolerance) in 64 bits for one item."""
    k = x.shape[1]
    x, y = x.double(), base.double().clone()
    tol = U * y.abs()
    m = 8 * -(-k // 512) + 40
    for e in sorted(set(ids.tolist())):
        if not 0 <= e < a.shape[0]:
            continue
        r = int(ranks[e])
        rows = ids == e
        ae, be = a[e, :r].double().t().contiguous(), b[e, :, :r].double().t().contiguous()
        y[rows] += float(scales[e]) * ((x[rows] @ ae) @ be)
        tol[rows] += m * U * abs(float(scales[e])) * ((x[rows].abs() @ ae.abs()) @ be.abs())
    return y, tol


def check(qmv, t, k, outs, rank, adapters, ids, kind="bf16", ranks=None, scaled=True, base="other", pad=0, ws=None):
    say(f"lora T {t} K {k} N {outs} rank {rank} of {adapters} adapters {kind} ranks {ranks} base {base} pad {pad}")
    g = torch.Generator().manual_seed(t * 31 + k + rank)
    dt = KINDS[kind]
    x = torch.randn(t, k + 4 * pad, generator=g)[:, :k]
    ranks_ = torch.full((adapters,), rank, dtype=torch.int32) if ranks is None else torch.tensor(ranks).int()
    scales = torch.randn(adapters, generator=g)
    items, want = [], []
    ids = torch.tensor(ids, dtype=torch.int32)
    cut = ranks_.clamp(0, rank)
    dev_x = torch.empty(t, k + 4 * pad, device="cuda")[:, :k]
    dev_x.copy_(x)
    for n in outs:
        a = (torch.randn(adapters, rank, k, generator=g) / k ** 0.5).to(dt)
        b = torch.randn(adapters, n, rank, generator=g).to(dt)
        for e in range(adapters):  # what lies past an adapter's rank is not a number
            a[e, cut[e]:] = float("nan")
            b[e, :, cut[e]:] = float("nan")
        y0 = torch.randn(t, n, generator=g)
        want.append(reference(x, a, b, y0 if base != "none" else torch.zeros_like(y0), ids, cut,
                              scales if scaled else torch.ones(adapters)))
        wide = torch.full((t + 1, n + pad), 5.0, device="cuda")  # a row and columns that stay
        y = wide[:t, :n]
        if base == "same":
            y.copy_(y0)
        items.append((a.cuda(), b.cuda(), None if base == "none" else y if base == "same" else y0.cuda(), y, wide))
    got = qmv.lora(dev_x, ids.cuda(), [i[:4] for i in items], ranks=None if ranks is None else ranks_.cuda(),
                   scales=scales.cuda() if scaled else None, ws=ws)
    torch.cuda.synchronize()
    for (y, tol), o, item in zip(want, got, items):
        err = (o.double().cpu() - y).abs()
        assert torch.all(err <= tol), (float((err / tol.clamp(min=1e-300)).max()), torch.argwhere(err > tol)[:3])
        wide = item[4]
        assert torch.all(wide[t:] == 5.0) and torch.all(wide[:, o.shape[1]:] == 5.0)
    return got


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 64, 72, 128, 256])
def test_ranks_and_types(rank, kind):
    qmv = need_gpu()
    check(qmv, 3, 512, [100], rank, 4, [2, 0, 2], kind)
    check(qmv, 10, 264, [65, 7], rank, 3, [0, 0, 1, 1, 1, -1, 0, 2, 0, 9], kind, ranks=[1, rank - 3, rank])


@pytest.mark.parametrize("k", [8, 16, 520, 2048, 2056, 4096, 5120, 14336])
def test_lengths(k):
    qmv = need_gpu()
    check(qmv, 1, k, [33], 16, 1, [0])
    check(qmv, 5, k, [130], 8, 2, [1, 0, 1, 1, 1], "f16", pad=3)


@pytest.mark.parametrize("t", [1, 2, 3, 7, 8, 9, 16, 63, 64, 65, 130, 500])
@pytest.mark.parametrize("pattern", ["one", "own", "mixed", "runs", "short runs", "any"])
def test_tokens(t, pattern):
    qmv = need_gpu()
    ids = {"one": [1] * t, "own": [i % 20 for i in range(t)], "mixed": [-1 if i % 4 == 3 else (7 * i) % 5 for i in range(t)],
           "runs": [i * 6 // t for i in range(t)], "short runs": [i // 5 % 20 for i in range(t)],
           "any": [(i * i + i // 3) % 23 - 2 for i in range(t)]}[pattern]
    check(qmv, t, 256, [48, 300], 16, 20, ids, "bf16", ranks=[16, 3, 0, 8, 13] * 4, base="same")


def test_many_rows_and_items():
    qmv = need_gpu()
    check(qmv, 16, 1024, [14336, 8192], 64, 16, list(range(16)))
    check(qmv, 64, 512, [9000], 8, 2, [i % 3 - 1 for i in range(64)], "f32")
    check(qmv, 4, 128, [1, 2, 3, 5, 64, 65, 127, 500], 24, 3, [0, 1, 2, 0], "f16")
    check(qmv, 300, 128, [5000], 32, 2, [i // 150 for i in range(300)], "bf16", base="none", scaled=False)


def test_the_most_tokens():
    qmv = need_gpu()
    check(qmv, 4096, 64, [70, 33], 8, 7, [i // 613 - 1 for i in range(4096)], "f16", base="same")
    check(qmv, 4095, 32, [9], 16, 300, [(i * 7) % 300 for i in range(4095)], "bf16", ranks=[1 + i % 16 for i in range(300)])


def test_columns_of_one_buffer():
    """The items' outputs as columns of the same rows, in place, and a row stride on base alone."""
    qmv = need_gpu()
    t, k, r = 6, 128, 8
    g = torch.Generator().manual_seed(1)
    x, ids = torch.randn(t, k, generator=g), torch.tensor([0, 1, 1, -1, 0, 0], dtype=torch.int32)
    outs = [50, 7, 20]
    ab = [(torch.randn(2, r, k, generator=g), torch.randn(2, n, r, generator=g)) for n in outs]
    whole0 = torch.randn(t, 80, generator=g)
    want = [reference(x, a, b, whole0[:, at:at + b.shape[1]], ids, [r, r], [1.0, 1.0])
            for (a, b), at in zip(ab, (0, 50, 57))]
    whole, other = whole0.cuda(), whole0.cuda()
    dab = [(a.cuda(), b.cuda()) for a, b in ab]
    cols = [whole[:, 0:50], whole[:, 50:57], whole[:, 57:77]]
    qmv.lora(x.cuda(), ids.cuda(), [(a, b, c, c) for (a, b), c in zip(dab, cols)])
    apart = qmv.lora(x.cuda(), ids.cuda(), [(a, b, other[:, at:at + b.shape[1]], None) for (a, b), at in zip(dab, (0, 50, 57))])
    for c, o, (y, tol) in zip(cols, apart, want):
        assert torch.all((c.double().cpu() - y).abs() <= tol) and torch.equal(c, o)
    assert torch.equal(whole[:, 77:].cpu(), whole0[:, 77:])


def test_no_adapter_at_all():
    qmv = need_gpu()
    for base in ("same", "other", "none"):
        check(qmv, 9, 64, [77], 8, 2, [-1, 2, 100, -5, 2**31 - 1, -2**31, 5, 5, 5], base=base, pad=1)
        check(qmv, 2, 64, [77], 8, 2, [0, 1], ranks=[0, -4], base=base)
    check(qmv, 2, 64, [77], 8, 2, [0, 1], ranks=[100, 8])  # a rank past the pool's counts as the pool's


def test_offsets_past_32_bits():
    """A pool of more than 2^31 weights: the last adapter's lie past them."""
    qmv = need_gpu()
    e, r, k, n = 600, 256, 16384, 64
    a = torch.zeros(e, r, k, dtype=torch.float16, device="cuda")
    b = torch.zeros(e, n, r, dtype=torch.float16, device="cuda")
    a[e - 1].normal_()
    b[e - 1].normal_()
    x = torch.randn(2, k, device="cuda")
    y, = qmv.lora(x, torch.tensor([e - 1, 0], dtype=torch.int32, device="cuda"), [(a, b, None, None)])
    want, tol = reference(x.cpu(), a[e - 1:].cpu(), b[e - 1:].cpu(), torch.zeros(2, n),
                          torch.tensor([0, -1]), [r], [1.0])
    assert torch.all((y.double().cpu() - want).abs() <= tol) and not y[1].any()


def test_graph_and_streams():
    """Two graphs that share a workspace, replayed in turn with eager work
    between, and calls on a stream of their own, give the eager results."""
    qmv = need_gpu()
    t, k, n, r, e = 12, 1024, 700, 16, 4
    a = torch.randn(e, r, k, device="cuda").half()
    b = torch.randn(e, n, r, device="cuda").half()
    x, base = torch.randn(t, k, device="cuda"), torch.randn(t, n, device="cuda")
    ids = torch.randint(-1, e, (t,), dtype=torch.int32, device="cuda")
    ws = torch.empty(qmv.lora_workspace_bytes(1, r, t), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty(t, n, device="cuda") for _ in range(2)], []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qmv.lora(x, ids, [(a, b, base, o)], ws=ws)
        graphs.append(graph)
    side = torch.cuda.Stream()
    for rep in range(6):
        x.normal_()
        ids.random_(-1, e)
        want, = qmv.lora(x, ids, [(a, b, base, None)])
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[rep % 2], want), rep
        other, = qmv.lora(x, ids, [(a, b, base, None)], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(other, want), rep


def test_one_workspace_for_every_batch():
    """Sized for the most items, rank and rows, in calls of fewer: those of some take more slices than those of more."""
    qmv = need_gpu()
    ws = torch.empty(qmv.lora_workspace_bytes(3, 64, 256), dtype=torch.uint8, device="cuda")
    for t in (256, 34, 1, 252, 64, 100, 9, 2):
        ws.fill_(255)
        for outs, rank, k in (([70, 33, 500], 64, 1536), ([300], 16, 4096), ([40, 50], 40, 256)):
            check(qmv, t, k, outs, rank, 5, [i * 7 // 3 % 6 for i in range(t)], ws=ws)
