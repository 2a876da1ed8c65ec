"""Routing by scores, bias and groups against the formula in 64 bits.  Ids are
equal; weights are made in 64 bits and rounded to fp32 once, half a step 2^-24
of their size (and 1e-12 for exp and sums in 64 bits)."""
import numpy as np
import pytest
import torch

from gpu_util import gpu, need_gpu, say

pytestmark = gpu


def reference(l, top_k, scoring, bias, groups, top_groups, best, renorm, scale):
    """l: logits in 64 bits [T][E]."""
    t, e = l.shape
    if scoring == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    c = s + (0 if bias is None else bias.astype(np.float64))
    size = e // groups
    ids = np.zeros((t, top_k), np.int32)
    w = np.zeros((t, top_k))
    for i in range(t):
        cand = range(e)
        if groups > 1:
            worth = [np.sort(c[i, g * size:(g + 1) * size])[-best:].sum() for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            cand = [x for g in kept for x in range(g * size, (g + 1) * size)]
        ids[i] = sorted(cand, key=lambda x: (-c[i, x], x))[:top_k]
        w[i] = s[i, ids[i]]
        if renorm:
            w[i] /= w[i].sum()
    return ids, w * scale


def check(qmv, x, wr, top_k, scoring="softmax", bias=None, groups=1, top_groups=1, best=2, renorm=True, scale=1.0,
          ws=None, xq=None, pad=0):
    t, k = x.shape
    e = wr.shape[0]
    say(f"gate T {t} K {k} E {e} top {top_k} {scoring} bias {bias is not None} groups {top_groups}/{groups}:{best} renorm {renorm}")
    l = x.astype(np.float64) @ wr.astype(np.float64).T
    ids, w = reference(l, top_k, scoring, bias, groups, top_groups, best, renorm, scale)
    dx = torch.zeros(t, k + pad, device="cuda")[:, :k]
    dx.copy_(torch.from_numpy(x))
    logits = torch.empty(t, e, device="cuda")
    gi, gw = qmv.router_gate(dx, torch.from_numpy(wr).cuda(), top_k, scoring=scoring,
                             bias=None if bias is None else torch.from_numpy(bias).cuda(), n_groups=groups,
                             top_groups=top_groups, group_best=best, renorm=renorm, scale=scale, logits=logits, ws=ws,
                             xq=xq)
    torch.cuda.synchronize()
    assert np.array_equal(gi.cpu().numpy(), ids)
    err = np.abs(gw.cpu().numpy().astype(np.float64) - w)
    assert np.all(err <= (2.0 ** -24 + 1e-12) * np.abs(w)), float(err.max())
    lerr = np.abs(logits.cpu().numpy().astype(np.float64) - l)
    assert np.all(lerr <= 2.0 ** -24 * np.abs(l) + 1e-12 * (np.abs(x).astype(np.float64) @ np.abs(wr).T))
    if ws is not None:
        assert not ws[:256].any()
    return gi, gw


def make(t, k, e, seed=0):
    rng = np.random.default_rng(seed + t * 7 + k + e)
    x = rng.standard_normal((t, k)).astype(np.float32)
    return x, (rng.standard_normal((e, k)) / k ** 0.5).astype(np.float32), (0.1 * rng.standard_normal(e)).astype(np.float32)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 16, 33, 64])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_tokens(t, scoring):
    qmv = need_gpu()
    x, wr, bias = make(t, 512, 128)
    ws = torch.zeros(qmv.router_gate_workspace_bytes(64, 256), dtype=torch.uint8, device="cuda")
    check(qmv, x, wr, 8, scoring, ws=ws)
    check(qmv, x, wr, 8, scoring, bias, 8, 4, scale=2.5, ws=ws, pad=8)
    check(qmv, x, wr, 6, scoring, bias, 4, 2, 1, renorm=False, ws=ws)


@pytest.mark.parametrize("e,groups", [(1, 1), (2, 1), (3, 3), (8, 4), (60, 1), (63, 7), (64, 64), (65, 13), (160, 8), (256, 8),
                                      (384, 1), (1000, 8), (1024, 64), (1024, 1)])
def test_experts(e, groups):
    qmv = need_gpu()
    x, wr, bias = make(5, 256, e)
    size = e // groups
    for top_groups in sorted({1, max(1, groups // 2), groups}):
        for top_k in sorted({1, min(16, size * top_groups), min(7, size * top_groups)}):
            check(qmv, x, wr, top_k, "sigmoid", bias, groups, top_groups, min(2, size))
            check(qmv, x, wr, top_k, "softmax", None, groups, top_groups, 1, renorm=False)


@pytest.mark.parametrize("k", [4, 28, 2044, 2048, 2052, 4096, 7168, 16388])
def test_lengths(k):
    qmv = need_gpu()
    x, wr, bias = make(6, k, 96)
    check(qmv, x, wr, 8, "sigmoid", bias, 4, 2)


def test_ties_go_to_the_lower_index():
    """Equal experts and equal groups: sums of small whole numbers are exact in any order."""
    qmv = need_gpu()
    rng = np.random.default_rng(3)
    x = rng.integers(-3, 4, (9, 64)).astype(np.float32)
    rows = (rng.integers(-2, 3, (6, 64)) / 64).astype(np.float32)
    wr = rows[rng.integers(0, 6, 48)]
    for scoring in ("softmax", "sigmoid"):
        check(qmv, x, wr, 12, scoring)
        check(qmv, x, np.concatenate([wr[:8]] * 6), 8, scoring, None, 6, 3)
    check(qmv, x, np.zeros_like(wr), 16, "sigmoid")
    # scores that round to one: choices are equal, order by index
    check(qmv, np.abs(x) + 1, np.full((40, 64), 10, np.float32), 5, "sigmoid", None, 4, 2)


def test_bias_that_forbids():
    qmv = need_gpu()
    x, wr, bias = make(4, 128, 64)
    bias[::2] = -np.inf
    check(qmv, x, wr, 8, "sigmoid", bias, 4, 2)
    bias[:] = -np.inf  # none is left: the lowest ones
    gi, _ = qmv.router_gate(torch.from_numpy(x).cuda(), torch.from_numpy(wr).cuda(), 8, bias=torch.from_numpy(bias).cuda())
    assert torch.equal(gi.cpu(), torch.arange(8, dtype=torch.int32).expand(4, 8))


def test_no_numbers():
    """Ids are in range and different whatever the logits are."""
    qmv = need_gpu()
    x, wr, _ = make(5, 64, 96)
    x[0, 3], x[1, 5], x[2, 7] = np.nan, np.inf, -np.inf
    x[3] = 1e38
    for scoring in ("softmax", "sigmoid"):
        for groups in (1, 8):
            gi, gw = qmv.router_gate(torch.from_numpy(x).cuda(), torch.from_numpy(wr * 1e6).cuda(), 8, scoring=scoring,
                                     n_groups=groups, top_groups=max(1, groups // 2))
            ids = gi.cpu().numpy()
            assert ids.min() >= 0 and ids.max() < 96 and all(len(set(r)) == 8 for r in ids)
            assert torch.isfinite(gw[4]).all()


def test_scores_that_vanish():
    """exp(-l) beyond fp64 gives scores of 0: equal weights."""
    qmv = need_gpu()
    x = np.full((1, 64), 100, np.float32)
    gi, gw = qmv.router_gate(torch.from_numpy(x).cuda(), torch.full((32, 64), -1.0, device="cuda"), 4, scoring="sigmoid",
                             scale=3.0)
    assert gi.cpu().tolist() == [[0, 1, 2, 3]] and torch.equal(gw.cpu(), torch.full((1, 4), 0.75))


@pytest.mark.parametrize("t,k,e", [(1, 4096, 40), (2, 1056, 40), (7, 64, 40), (64, 2048, 40), (4, 4128, 5), (3, 96, 4),
                                   (40, 288, 17)])
def test_q8_of_x(t, k, e):
    qmv = need_gpu()
    x, wr, _ = make(t, k, e)
    xq = torch.zeros(qmv.act_bytes(t, k), dtype=torch.uint8, device="cuda")
    check(qmv, x, wr, 4, xq=xq)
    want = qmv.quantize_act(torch.from_numpy(x).cuda())
    for a, b in zip(qmv.act_fields(xq, t, k), qmv.act_fields(want, t, k)):
        assert torch.equal(a, b)


def test_graphs_streams_and_one_workspace():
    qmv = need_gpu()
    x, wr, bias = make(20, 512, 64)
    x, wr, bias = (torch.from_numpy(v).cuda() for v in (x, wr, bias))
    ws = torch.zeros(qmv.router_gate_workspace_bytes(20, 64), dtype=torch.uint8, device="cuda")
    kw = dict(scoring="sigmoid", bias=bias, n_groups=4, top_groups=2)
    out, graphs = [], []
    for t in (20, 3):
        o = (torch.empty(t, 6, dtype=torch.int32, device="cuda"), torch.empty(t, 6, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmv.router_gate(x[:t], wr, 6, ids=o[0], weights=o[1], ws=ws, **kw)
        out.append(o)
        graphs.append(g)
    side = torch.cuda.Stream()
    for rep in range(8):
        x.normal_()
        i = rep % 2
        want = qmv.router_gate(x[:out[i][0].shape[0]], wr, 6, **kw)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out[i], want)), rep
        other = qmv.router_gate(x[:out[i][0].shape[0]], wr, 6, stream=side, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, want)), rep
    assert not ws[:256].any()


def test_ties_among_many_experts():
    """As above where a lane has several experts, as many as there are."""
    qmv = need_gpu()
    rng = np.random.default_rng(8)
    x = rng.integers(-3, 4, (6, 32)).astype(np.float32)
    rows = (rng.integers(-2, 3, (5, 32)) / 32).astype(np.float32)
    for e in (130, 256, 520, 1024):
        wr = rows[rng.integers(0, 5, e)]
        for t in (2, 6):
            check(qmv, x[:t], wr, 16, "softmax")
            check(qmv, x[:t], wr, 16, "sigmoid", None, e // 26 if e % 26 == 0 else 8, 2)
            check(qmv, x[:t], np.zeros_like(wr), 16, "sigmoid", None, 2, 1)


def test_one_workspace_for_every_batch():
    """Sized for the most tokens and experts, in calls of fewer, with one launch and with two."""
    qmv = need_gpu()
    ws = torch.zeros(qmv.router_gate_workspace_bytes(64, 384), dtype=torch.uint8, device="cuda")
    for t in (64, 26, 48, 3, 40, 1, 31, 5):
        for e, k in ((384, 1280), (128, 2052), (16, 5120)):
            x, wr, bias = make(t, k, e)
            check(qmv, x, wr, 8, "sigmoid", bias, ws=ws)
    assert not ws[:256].any()
