"""Log probabilities, entropy and alternatives against the formula in 64 bits.

Ids are equal.  Tolerances in half steps u = 2^-24: e^d has d (rounded once, |d| u)
times log2 e (rounded twice) and the hardware's exponential (2 u): (3 |d| + 3) u
of itself, which is (3 mean|d| + 3) u of the sum, mean|d| under the
probabilities being at most ln V < 17.  All terms of the sums have one sign; a
lane adds at most V / 1024 + 16 terms in turn, rescales (3 roundings) at most
every 16 of them, and joins 16 times: the sums are off by
N = V / 1024 * 1.2 + 140 half steps of themselves.  A log probability is off by N u and
its own rounding, the entropy by 2 N u (1 + entropy)."""
import numpy as np
import pytest
import torch

from gpu_util import gpu, need_gpu, say

pytestmark = gpu

U = 2.0 ** -24


def reference(x, given, n, scale):
    z = x.astype(np.float64) * float(np.float32(scale))
    m = z.max(1, keepdims=True)
    m[m == -np.inf] = 0.0
    p = np.exp(z - m)
    s = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lp = z - m - np.log(s)
        lp[z == -np.inf] = -np.inf
        p = p / s
        ent = -np.where(p > 0, p * lp, 0.0).sum(1)
    ent[s[:, 0] == 0] = 0.0
    out = None
    if given is not None:
        ok = (given >= 0) & (given < x.shape[1])
        out = np.where(ok, np.take_along_axis(lp, np.where(ok, given, 0), 1), -np.inf)
    order = np.argsort(-(x.astype(np.float64)), axis=1, kind="stable")[:, :n]
    return out, ent, order.astype(np.int32), np.take_along_axis(lp, order, 1)


def close(got, want, tol):
    got = got.cpu().numpy().astype(np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    err = np.abs(got - np.where(fin, want, 0))[fin]
    lim = (tol + U * np.abs(want))[fin] if np.ndim(tol) == 0 else tol[fin]
    assert np.all(err <= lim), (float(err.max()), float(lim.min()))


def check(qmv, x, given=None, n=0, scale=1.0, pad=0, ws="both"):
    t, v = x.shape
    say(f"logprobs T {t} V {v} given {None if given is None else given.shape} top {n} scale {scale} pad {pad}")
    dx = torch.full((t, v + pad), float("nan"), device="cuda")[:, :v]
    dx.copy_(torch.from_numpy(x))
    dg = None if given is None else torch.from_numpy(given.astype(np.int32)).cuda()
    want = reference(x, given, n, scale)
    size = 1.2 * v / 1024 + 140
    for with_ws in (False, True):
        need = qmv.token_logprobs_workspace_bytes(t, v, n)
        buf = torch.zeros(need, dtype=torch.uint8, device="cuda") if with_ws else None
        if with_ws and need == 0:
            continue
        lp, ent, ids, top = qmv.token_logprobs(dx, dg, top_n=n, scale=scale, ws=buf)
        torch.cuda.synchronize()
        if given is not None:
            close(lp, want[0], size * U)
        close(ent, want[1], 2 * size * U * (1 + want[1]))
        if n:
            assert np.array_equal(ids.cpu().numpy(), want[2])
            close(top, want[3], size * U)
        else:
            assert ids is None and top is None
        if with_ws:
            assert not buf[:65536].any()


def make(t, v, seed=0, spread=3.0):
    rng = np.random.default_rng(seed + 31 * t + v)
    return (rng.standard_normal((t, v)) * spread).astype(np.float32), rng


@pytest.mark.parametrize("v", [1, 2, 3, 4, 5, 63, 100, 255, 1000, 1024, 1100, 4095, 4097, 8191, 8193, 12289, 20000, 32003, 50257,
                               152064])
def test_vocabularies(v):
    qmv = need_gpu()
    x, rng = make(3, v)
    check(qmv, x, rng.integers(0, v, (3, 2)), min(20, v))
    check(qmv, x, rng.integers(-2, v + 2, (3, 1)), min(1, v), scale=0.7, pad=3)
    check(qmv, x, None, min(32, v), pad=1)
    check(qmv, x, rng.integers(0, v, (3, 1)), 0)


@pytest.mark.parametrize("t", [1, 2, 16, 64, 256, 257, 700])
def test_rows(t):
    qmv = need_gpu()
    x, rng = make(t, 20011)
    check(qmv, x, rng.integers(0, 20011, (t, 3)), 7, scale=1.25)


def test_the_most_rows_and_tokens():
    qmv = need_gpu()
    x, rng = make(65536, 40)
    check(qmv, x, rng.integers(0, 40, (65536, 1)), 2)
    x, rng = make(2, 3_000_001)
    check(qmv, x, rng.integers(0, 3_000_001, (2, 700)), 32)


@pytest.mark.parametrize("v", [300, 5000, 60000])
def test_ties(v):
    """Few different values: the lower index first, also where all are equal or zeros differ in sign."""
    qmv = need_gpu()
    rng = np.random.default_rng(v)
    x = rng.integers(-2, 3, (4, v)).astype(np.float32)
    x[1] = 1.5
    x[2] = np.where(rng.random(v) < 0.5, 0.0, -0.0)
    x[3, :] = np.floor(np.arange(v) / 50)
    check(qmv, x, rng.integers(0, v, (4, 1)), 32)


@pytest.mark.parametrize("v", [5000, 70001, 152064])
def test_sorted_rows(v):
    """The largest lie side by side, at the end, at the start, in one stride."""
    qmv = need_gpu()
    x = np.stack([np.linspace(-9, 9, v), np.linspace(9, -9, v), np.linspace(-1, 1, v) ** 2 * 20,
                  np.where(np.arange(v) % 1024 == 7, 5 + np.arange(v) / v, np.arange(v) / v)]).astype(np.float32)
    check(qmv, x, np.zeros((4, 1), np.int64), 32)


@pytest.mark.parametrize("v", [400, 9000, 100003])
def test_forbidden_tokens(v):
    qmv = need_gpu()
    x, rng = make(6, v)
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[1] = -np.inf
    x[1, v // 2] = -3.0
    x[2] = -np.inf  # nothing is left
    x[3, : v - 5] = -np.inf
    x[4, 5:] = -np.inf
    given = rng.integers(0, v, (6, 4))
    given[1, 0] = v // 2
    given[:, 3] = -1
    check(qmv, x, given, 20)


def test_wide_ranges():
    """Logits so far apart that one token has it all, and large ones of both signs."""
    qmv = need_gpu()
    x, rng = make(4, 30000)
    x[0] *= 1e30
    x[1] += 1e6
    x[2] -= 1e6
    x[3, 77] = 3e38
    check(qmv, x, rng.integers(0, 30000, (4, 2)), 5)


def test_no_numbers():
    qmv = need_gpu()
    for v in (900, 40000):
        x, _ = make(5, v)
        x[0, 17], x[1, 30], x[2, :] = np.nan, np.inf, np.nan
        x[3, 40:60] = np.nan
        dx = torch.from_numpy(x).cuda()
        given = torch.full((5,), 3, dtype=torch.int32, device="cuda")
        for need in (0, qmv.token_logprobs_workspace_bytes(5, v, 4)):
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
            lp, ent, ids, top = qmv.token_logprobs(dx, given, top_n=4, ws=ws)
            assert torch.isnan(lp[:4]).all() and torch.isnan(ent[:4]).all() and torch.isnan(top[:4]).all()
            assert torch.isfinite(lp[4]) and torch.isfinite(ent[4]) and torch.isfinite(top[4]).all()
            order = np.argsort(-np.where(np.isnan(x), -np.inf, x.astype(np.float64)), axis=1, kind="stable")[:, :4]
            assert np.array_equal(ids.cpu().numpy(), order)


def test_rows_beyond_32_bits():
    """Rows whose offsets pass 2^31 elements."""
    qmv = need_gpu()
    t, ld = 3, (1 << 30) + 4
    base = torch.empty((t - 1) * ld + 5000, device="cuda")
    x = base.as_strided((t, 5000), (ld, 1))
    x.normal_()
    lp, ent, ids, top = qmv.token_logprobs(x, torch.zeros(t, 1, dtype=torch.int32, device="cuda"), top_n=3)
    want = reference(x.cpu().numpy(), np.zeros((t, 1), np.int64), 3, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want[2])
    close(lp, want[0], 200 * U)


def test_graphs_streams_and_one_workspace():
    qmv = need_gpu()
    t, v = 6, 50257
    x = torch.randn(t, v, device="cuda") * 3
    given = torch.randint(0, v, (t, 1), dtype=torch.int32, device="cuda")
    ws = torch.zeros(qmv.token_logprobs_workspace_bytes(t, v, 20), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for n_tok, n in ((t, 20), (2, 3)):
        o = (torch.empty(n_tok, 1, device="cuda"), torch.empty(n_tok, device="cuda"),
             torch.empty(n_tok, n, dtype=torch.int32, device="cuda"), torch.empty(n_tok, n, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmv.token_logprobs(x[:n_tok], given[:n_tok], top_n=n, logprobs=o[0], entropy=o[1], top_ids=o[2],
                               top_logprobs=o[3], ws=ws)
        outs.append(o)
        graphs.append(g)
    side = torch.cuda.Stream()
    for rep in range(8):
        x.normal_()
        given.random_(0, v)
        i = rep % 2
        n_tok, n = outs[i][2].shape
        other = torch.zeros_like(ws)
        want = qmv.token_logprobs(x[:n_tok], given[:n_tok], top_n=n, ws=other)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want)), rep
        again = qmv.token_logprobs(x[:n_tok], given[:n_tok], top_n=n, ws=other, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want)), rep
    assert not ws[:65536].any()


def test_logits_that_scale_past_the_range():
    """z beyond fp32's range is an infinity: forbidden below it, no number above it."""
    qmv = need_gpu()
    for v in (700, 60000):
        x, rng = make(4, v)
        x[0, 9] = -3e38   # one forbidden token
        x[1, 11] = 3e38   # no number
        x[2, :] = -1e38   # none is allowed
        given = np.full((4, 2), 9, np.int32)
        given[:, 1] = 20
        for need in {0, qmv.token_logprobs_workspace_bytes(4, v, 3)}:
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
            lp, ent, ids, top = (o.cpu() for o in qmv.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(given).cuda(),
                                                                     top_n=3, scale=10.0, ws=ws))
            assert lp[0, 0] == -np.inf and torch.isfinite(lp[0, 1]) and torch.isfinite(ent[0])
            assert torch.isnan(lp[1]).all() and torch.isnan(ent[1]) and torch.isnan(top[1]).all()
            assert (lp[2] == -np.inf).all() and ent[2] == 0 and (top[2] == -np.inf).all()
            assert torch.isfinite(lp[3]).all() and torch.isfinite(ent[3])
            assert ids[2].tolist() == [0, 1, 2] and ids[1, 0] == 11


def test_scaled_rows_far_from_zero():
    """Rows whose common part is large beside their spread: no term depends on it."""
    qmv = need_gpu()
    for t, v in ((3, 900), (40, 30011), (2, 70001), (5, 152064)):
        x, rng = make(t, v, 9)
        for scale in (0.7, 1.3):
            for far in (1e4, -3e5):
                check(qmv, x + np.float32(far), rng.integers(0, v, (t, 3)), 4, scale)


@pytest.mark.parametrize("t,v", [(41, 50257), (60, 152064), (83, 100003), (126, 152064), (12, 100001)])
def test_rows_in_long_parts(t, v):
    """Some tens of rows, which workgroups share in parts of several steps."""
    qmv = need_gpu()
    x, rng = make(t, v, 4)
    x[1] = np.sort(x[1])
    x[2] = np.sort(x[2])[::-1]
    x[3] = np.round(x[3])           # many equal ones
    x[4] = 0.5                      # all of them
    x[5, : v // 2] = -np.inf
    x[6, 5:] = -np.inf
    check(qmv, x, rng.integers(0, v, (t, 3)), 32, scale=0.7, pad=1)
    check(qmv, x, rng.integers(0, v, (t, 1)))
    check(qmv, x, n=1)


def test_tokens_outside_in_rows_without_numbers():
    """A row with NaN, with +inf or with a z beyond the range has no number for any given token, one outside too."""
    qmv = need_gpu()
    for v in (700, 60000):
        x, _ = make(5, v)
        x[0, 3], x[1, 4], x[2, 5] = np.nan, np.inf, 3e38
        x[3] = -1e38  # nothing is allowed
        given = np.tile(np.array([[-1, v, 2, 2**31 - 1]], np.int32), (5, 1))
        need = qmv.token_logprobs_workspace_bytes(5, v, 0)
        for ws in [None] + ([torch.zeros(need, dtype=torch.uint8, device="cuda")] if need else []):
            lp, ent, _, _ = qmv.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(given).cuda(), scale=10.0, ws=ws)
            lp = lp.cpu()
            assert torch.isnan(lp[:3]).all() and torch.isnan(ent[:3]).all()
            assert (lp[3] == -np.inf).all() and ent[3] == 0
            assert (lp[4, [0, 1, 3]] == -np.inf).all() and torch.isfinite(lp[4, 2]) and torch.isfinite(ent[4])


def microseconds(calls, n=8):
    """Each call's least time among others of its own, by replays of a graph of them, the graphs in turn."""
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(n):
                call()
    times = [[] for _ in calls]
    for _ in range(9):
        for graph, took in zip(graphs, times):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b) * 1e3 / n)
    return [min(took) for took in times]


def times_of(qmv, t, v, n):
    """Times of a call without a workspace and with one."""
    x = torch.randn(t, v, device="cuda") * 3
    need = qmv.token_logprobs_workspace_bytes(t, v, n)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out = dict(entropy=torch.empty(t, device="cuda"), top_ids=torch.empty(t, n, dtype=torch.int32, device="cuda"),
               top_logprobs=torch.empty(t, n, device="cuda"))
    whole, shared = microseconds([lambda w=w: qmv.token_logprobs(x, top_n=n, ws=w, **out) for w in (None, ws)])
    say(f"logprobs T {t} V {v} top {n}: whole rows {whole:.1f} us, with a workspace {shared:.1f}")
    return whole, shared


@pytest.mark.parametrize("t,v,n", [(41, 50257, 32), (66, 128256, 32), (106, 128256, 24), (96, 152064, 24),
                                   (126, 152064, 20), (120, 160000, 20), (64, 262144, 32), (128, 262144, 20),
                                   (200, 262144, 32)])
def test_alternatives_of_rows_in_few_parts(t, v, n):
    """Four to eleven parts a row bound the alternatives too: without a bound a row's last workgroup reads all of it
    twice, which took four to seven times the time of whole rows."""
    whole, shared = times_of(need_gpu(), t, v, n)
    assert shared < 2 * whole


def test_one_workspace_for_every_batch():
    """Sized for the most rows: calls of one part a step, of long parts, of few parts and of whole rows in turn, each
    as with a workspace of its own."""
    qmv = need_gpu()
    v = 128256
    ws = torch.zeros(qmv.token_logprobs_workspace_bytes(256, v, 0), dtype=torch.uint8, device="cuda")
    x = torch.randn(300, v, device="cuda") * 3
    given = torch.randint(0, v, (300, 2), dtype=torch.int32, device="cuda")
    for t, n in ((256, 20), (1, 20), (106, 5), (5, 32), (40, 0), (60, 32), (2, 1), (300, 3), (64, 20), (1, 0), (13, 24)):
        size = qmv.token_logprobs_workspace_bytes(t, v, n)
        want = qmv.token_logprobs(x[:t], given[:t], top_n=n, ws=torch.zeros(size, dtype=torch.uint8, device="cuda"))
        got = qmv.token_logprobs(x[:t], given[:t], top_n=n, ws=ws)
        torch.cuda.synchronize()
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want)), (t, n)
        assert not ws[:65536].any()
    for w in (40000, 32000, 500):  # and of smaller vocabularies
        want = qmv.token_logprobs(x[:20, :w], given[:20] % w, top_n=20,
                                  ws=torch.zeros(qmv.token_logprobs_workspace_bytes(20, w, 20), dtype=torch.uint8, device="cuda"))
        got = qmv.token_logprobs(x[:20, :w], given[:20] % w, top_n=20, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), w


@pytest.mark.parametrize("t,v,n", [(28, 50257, 32), (33, 50257, 16), (42, 100003, 32), (77, 100003, 1), (50, 128256, 32),
                                   (97, 128256, 5), (55, 152064, 32), (72, 152064, 20), (104, 152064, 5), (82, 262144, 16),
                                   (158, 262144, 0), (90, 500009, 20)])
def test_alternatives_of_rows_in_long_parts(t, v, n):
    """As many rows as are shared with that many alternatives, in few and long parts."""
    qmv = need_gpu()
    x, rng = make(t, v, 6)
    x[1] = np.sort(x[1])
    x[2] = np.sort(x[2])[::-1]
    x[3] = np.round(x[3])
    x[4] = 0.5
    x[5, : v // 2] = -np.inf
    x[6, 5:] = -np.inf
    x[7, v // 3: v // 3 + 200] += 50  # all of them in one part
    check(qmv, x, rng.integers(0, v, (t, 2)), n, scale=0.7, pad=1)


@pytest.mark.parametrize("t,v,n", [(41, 50257, 32), (106, 128256, 5), (66, 128256, 32), (126, 152064, 20), (96, 152064, 32),
                                   (55, 152064, 32), (100, 152064, 5), (100, 262144, 32), (200, 262144, 20), (6, 152064, 20)])
def test_a_workspace_costs_no_time(t, v, n):
    """Rows are shared only where that is not slower: a fixed number of rows had taken up to 1.7 times as long."""
    whole, shared = times_of(need_gpu(), t, v, n)
    assert shared < 1.2 * whole


@pytest.mark.parametrize("t,v", [(2, 3_000_001), (1, 1 << 24)])
def test_the_longest_rows(t, v):
    """A lane of a whole row's 512 threads adds V / 512 terms in turn and rescales (3 roundings) at most every 16 of
    them: with the rest as above, sums are off by V / 512 * 1.2 + 140 half steps at most."""
    qmv = need_gpu()
    x, rng = make(t, v, 8)
    given = rng.integers(0, v, (t, 5))
    given[0, 0], given[0, 1] = v - 1, v
    want = reference(x, given, 32, 1.25)
    size = 1.2 * v / 512 + 140
    dx, dg = torch.from_numpy(x).cuda(), torch.from_numpy(given.astype(np.int32)).cuda()
    need = qmv.token_logprobs_workspace_bytes(t, v, 32)
    assert need > 0
    for ws in (None, torch.zeros(need, dtype=torch.uint8, device="cuda")):
        lp, ent, ids, top = qmv.token_logprobs(dx, dg, top_n=32, scale=1.25, ws=ws)
        torch.cuda.synchronize()
        close(lp, want[0], size * U)
        close(ent, want[1], 2 * size * U * (1 + want[1]))
        assert np.array_equal(ids.cpu().numpy(), want[2])
        close(top, want[3], size * U)
