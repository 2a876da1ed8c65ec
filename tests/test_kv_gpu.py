"""qmv_kv_append (bit for bit) and qmv_kv_attn (within the bound of
kv_ref.attend) against the definitions, at the lengths, masks, tables and
layouts where they can go wrong."""
import numpy as np
import pytest
import torch

import kv_ref
import oracle
from gpu_util import gpu, need_gpu, say, to_dev

pytestmark = gpu


class Case:
    """A pool with scattered blocks, garbage in what no call may read, and the
    sequences of one call."""

    def __init__(self, seed, lens, counts, heads, dim, *, width=None, spare=3, uniform=None, padded=0):
        r = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        n = len(lens)
        need = [-(-max(x, 0) // 64) for x in lens]
        self.width = width or max(max(need), 1)
        self.n_blocks = sum(min(x, self.width) for x in need) + spare
        ids = r.permutation(self.n_blocks)
        self.table = r.choice(np.array([-1, -2**31, 2**31 - 1, 10**6]), (n, self.width)).astype(np.int32)
        at = 0
        self.used = np.zeros(self.n_blocks, bool)
        for s in range(n):
            m = min(need[s], self.width)
            self.table[s, :m] = ids[at:at + m]
            self.used[ids[at:at + m]] = True
            at += m
        self.codes = np.clip(np.round(r.standard_normal((self.n_blocks, 2, heads, 64 * dim)) * 35), -127, 127).astype(np.int8)
        self.scales = (r.uniform(0.5, 1.5, (self.n_blocks, 2, heads)) * 4 / 127).astype(np.float32)
        self.scales[~self.used] = np.nan
        self.heads, self.dim = heads, dim
        self.max_q = uniform or max(max(counts), 1)
        if uniform:
            self.start, self.n_tok = None, n * uniform
        else:
            self.start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
            self.n_tok = int(self.start[-1]) + padded

    def rows(self, heads, spread=1.0):
        return (self.rng.standard_normal((self.n_tok, heads, self.dim)) * spread).astype(np.float32)

    def dev(self):
        return [to_dev(x) for x in (self.codes, self.scales, self.table, self.lens)] + \
            [None if self.start is None else to_dev(self.start)]


def same_cache(c, codes, scales, what):
    got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(got_s, c.scales, equal_nan=True), what
    bad = np.argwhere(got_c != c.codes)
    assert len(bad) == 0, (what, len(bad), bad[:3])


def run_append(qmv, c, k, v, what, **kw):
    codes, scales, table, lens, start = c.dev()
    qmv.kv_append(to_dev(k), to_dev(v), codes, scales, table, lens, tok_start=start, max_q=c.max_q, **kw)
    kv_ref.append(c.codes, c.scales, c.table, c.lens, c.start, c.max_q, k, v)
    same_cache(c, codes, scales, what)


APPENDS = {  # lengths after, new tokens
    "one": ([1], [1]),
    "open block": ([70, 64, 65, 128, 3], [1, 1, 1, 1, 2]),
    "crosses": ([130, 64, 200, 97], [5, 64, 73, 33]),
    "many blocks": ([517, 300], [450, 300]),
    "ragged, empty": ([0, 40, 77, 0, 500], [0, 3, 0, 0, 128]),
    "more rows than tokens": ([2, 0, 66], [5, 3, 70]),
    "verify": ([63, 64, 65, 66, 127, 128], [6, 6, 6, 6, 6, 6]),
}


@pytest.mark.parametrize("name", sorted(APPENDS))
@pytest.mark.parametrize("heads,dim", [(1, 16), (3, 64), (2, 80), (8, 128), (1, 192), (2, 256)])
def test_append(name, heads, dim):
    qmv = need_gpu()
    say(f"append {name} {heads}x{dim}")
    lens, counts = APPENDS[name]
    c = Case(3, lens, counts, heads, dim, padded=2)
    spread = np.float32(1.0 + 3.0 * (c.rng.random() < 0.5))
    run_append(qmv, c, c.rows(heads) * spread, c.rows(heads) * 2, name)


def test_append_blocks_outside():
    """Table entries outside the pool, and positions past the table: nothing
    is written there, the rest is."""
    qmv = need_gpu()
    c = Case(4, [200, 300, 130], [150, 250, 100], 2, 96, width=3)
    c.table[0, 1] = -1
    c.table[2, 2] = c.n_blocks
    run_append(qmv, c, c.rows(2), c.rows(2), "outside")


def test_append_step_by_step():
    """A block filled token by token: its scale grows, its older codes follow
    it; then a rollback into it, and a fresh start at its first slot over a
    scale that is not a number."""
    qmv = need_gpu()
    say("append step by step")
    c = Case(5, [64, 64], [1, 1], 2, 64)
    c.scales[:] = np.nan
    codes, scales, table, lens, _ = c.dev()
    order = list(range(1, 65)) + [40, 41, 42] + [1, 2]
    for n in order:
        c.lens[:] = (n, max(n - 3, 0))
        lens.copy_(torch.from_numpy(c.lens))
        c.start, c.n_tok, c.max_q = None, 2, 1
        k, v = c.rows(2, 0.1 * n), c.rows(2, 4.0 / n)
        k[:, :, :] *= np.float32(0.0) if n in (1, 7) else np.float32(1.0)
        qmv.kv_append(to_dev(k), to_dev(v), codes, scales, table, lens)
        kv_ref.append(c.codes, c.scales, c.table, c.lens, None, 1, k, v)
        same_cache(c, codes, scales, n)


def test_append_small_and_large_values():
    qmv = need_gpu()
    c = Case(6, [70, 20, 64], [3, 20, 64], 2, 64)
    k, v = c.rows(2), c.rows(2)
    k[:3] *= np.float32(1e30)
    v[3:23] *= np.float32(1e-30)
    k[23:60] = 0.0
    v[23:] = 0.0
    run_append(qmv, c, k, v, "values")


ATTNS = {  # lengths, new tokens, query heads a kv head
    "one token": ([1], [1], 4),
    "short": ([5, 63, 64, 65, 129], [1, 1, 1, 1, 1], 3),
    "whole prompt": ([70], [70], 1),
    "verify": ([300, 64, 66, 1000], [6, 6, 6, 6], 2),
    "ragged, padded": ([0, 130, 77, 900, 64], [0, 3, 0, 9, 1], 5),
    "rows before the first token": ([2, 0, 66], [5, 3, 70], 2),
    "wide group": ([513, 200], [4, 3], 16),
    "many rows": ([400, 90], [64, 33], 5),
    "long": ([4001], [1], 8),
}


def check_attn(qmv, c, group, what, window=0, scale=None, ws=True, xq=False, q=None):
    codes, scales, table, lens, start = c.dev()
    heads = c.heads * group
    q = c.rows(heads) if q is None else q
    need = qmv.kv_attn_workspace_bytes(len(c.lens), c.n_tok, c.max_q, heads, c.heads, c.dim, c.width)
    w = torch.zeros(need, dtype=torch.uint8, device="cuda") if ws and need else None
    out = torch.full(q.shape, 5.0, device="cuda")
    buf = None
    if xq:
        buf = torch.full((qmv.act_bytes(c.n_tok, heads * c.dim),), 9, dtype=torch.uint8, device="cuda")
    kw = dict(tok_start=start, max_q=c.max_q, scale=scale, window=window, ws=w, xq=buf)
    got = qmv.kv_attn(to_dev(q), codes, scales, table, lens, out=out, **kw)
    assert got.data_ptr() == out.data_ptr()
    g = out.cpu().numpy()
    ref, tol, rows = kv_ref.attend(c.codes, c.scales, c.table, c.lens, c.start, c.max_q, q,
                                   c.dim ** -0.5 if scale is None else scale, window)
    err = np.abs(g[rows] - ref[rows])
    assert np.all(err <= tol[rows]), (what, float((err - tol[rows]).max()), np.argwhere(~(err <= tol[rows]))[:3])
    assert np.all(g[~rows] == 5.0), what  # rows of no sequence
    if w is not None:
        again = qmv.kv_attn(to_dev(q), codes, scales, table, lens, **kw)
        assert torch.equal(again[torch.from_numpy(rows)], out[torch.from_numpy(rows)]), what
        assert not w[:65536].any(), what
    if xq:
        want = oracle.quantize_act(np.ascontiguousarray(g.reshape(c.n_tok, -1)))
        for x, y in zip(qmv.act_fields(buf, c.n_tok, heads * c.dim), want):
            assert np.array_equal(x.cpu().numpy()[rows], y[rows]), what
    return g


@pytest.mark.parametrize("name", sorted(ATTNS))
@pytest.mark.parametrize("heads,dim", [(1, 16), (2, 64), (1, 80), (2, 128), (1, 192), (1, 256)])
def test_attn(name, heads, dim):
    qmv = need_gpu()
    say(f"attn {name} {heads}x{dim}")
    lens, counts, group = ATTNS[name]
    c = Case(7, lens, counts, heads, dim, padded=3 if "padded" in name else 0)
    for ws in (False, True):
        check_attn(qmv, c, group, name, ws=ws, xq=dim % 32 == 0)


@pytest.mark.parametrize("window", [1, 5, 63, 64, 65, 200, 2**40])
def test_window(window):
    qmv = need_gpu()
    c = Case(8, [700, 64, 30, 1], [7, 4, 30, 1], 2, 64)
    for ws in (False, True):
        check_attn(qmv, c, 3, window, window=window, ws=ws)


def test_blocks_outside():
    """Blocks outside the pool and positions past the table are not seen; a
    sequence with no block in the cache gives zeros."""
    qmv = need_gpu()
    c = Case(9, [300, 500, 100, 128], [2, 3, 1, 2], 2, 128, width=5)
    c.table[0, 2] = -7
    c.table[2, :] = c.n_blocks
    c.table[3, 1] = 2**31 - 1
    for ws in (False, True):
        g = check_attn(qmv, c, 4, "outside", ws=ws)
        assert not g[5].any()


def test_shared_blocks():
    """Two sequences with the same first blocks."""
    qmv = need_gpu()
    c = Case(10, [200, 330], [1, 2], 2, 64)
    c.table[1, :3] = c.table[0, :3]
    check_attn(qmv, c, 2, "shared")


def test_scores_far_apart():
    """Scores of thousands (one key takes all), of nearly nothing, a scale of
    zero and below it, rows of zeros and of very small values."""
    qmv = need_gpu()
    c = Case(11, [200, 200, 200, 200, 200], [1] * 5, 1, 64)
    q = c.rows(4)
    q[0] *= np.float32(3e4)
    q[1] *= np.float32(1e-12)
    q[2] = 0.0
    q[3, :, 5:] *= np.float32(1e-9)
    q[4] *= np.float32(1e-33)
    check_attn(qmv, c, 4, "spread", q=q)
    for scale in (0.0, -0.3, 2.5):
        check_attn(qmv, c, 4, scale, scale=scale)


def test_a_row_that_is_not_finite_stays_alone():
    qmv = need_gpu()
    say("attn nan rows")
    c = Case(12, [400, 130], [3, 3], 2, 128)
    q = c.rows(8)
    good = check_attn(qmv, c, 4, "finite", q=q)
    bad = q.copy()
    bad[1, 2, 7] = np.nan
    bad[3, 0, 100] = np.inf
    codes, scales, table, lens, start = c.dev()
    ws = torch.zeros(qmv.kv_attn_workspace_bytes(2, 6, 3, 8, 2, 128, c.width), dtype=torch.uint8, device="cuda")
    for w in (None, ws):
        g = qmv.kv_attn(to_dev(bad), codes, scales, table, lens, tok_start=start, max_q=3, ws=w).cpu().numpy()
        hit = np.zeros(g.shape[:2], bool)
        hit[1, 2] = hit[3, 0] = True
        assert np.isnan(g[hit]).all()
        assert np.allclose(g[~hit], good[~hit], rtol=1e-5, atol=1e-6)


def test_layouts():
    """Rows in the columns of a projection's output, the output among others'
    columns, and the output over q itself; on another stream."""
    qmv = need_gpu()
    say("attn layouts")
    c = Case(13, [90, 65], [2, 2], 2, 64)
    heads, d = 6, 64
    codes, scales, table, lens, start = c.dev()
    wide = torch.randn(4, (heads + 4) * d, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q, k, v = (wide[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, heads), (heads, heads + 2), (heads + 2, heads + 4)))
    codes2, scales2 = codes.clone(), scales.clone()
    qmv.kv_append(k, v, codes, scales, table, lens, tok_start=start, max_q=2)
    qmv.kv_append(k.contiguous(), v.contiguous(), codes2, scales2, table, lens, tok_start=start, max_q=2)
    assert torch.equal(codes, codes2)
    ref = qmv.kv_attn(q.contiguous(), codes, scales, table, lens, tok_start=start, max_q=2)
    host = torch.full((4, 500), 2.0, device="cuda")
    out = host[:, 100:100 + heads * d].unflatten(1, (heads, d))
    qmv.kv_attn(q, codes, scales, table, lens, tok_start=start, max_q=2, out=out)
    assert torch.equal(out, ref) and (host[:, :100] == 2).all() and (host[:, 100 + heads * d:] == 2).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qmv.kv_attn(q, codes, scales, table, lens, tok_start=start, max_q=2, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    qmv.kv_attn(q, codes, scales, table, lens, tok_start=start, max_q=2, out=q)
    assert torch.equal(q, ref)


def test_far_blocks():
    """A pool of more than 2^32 bytes: block offsets pass 32 bits."""
    qmv = need_gpu()
    heads, dim = 8, 128
    n_blocks = (5 << 30) // (2 * heads * 64 * dim)
    c = Case(14, [150, 64], [40, 1], heads, dim)
    small_codes, small_scales, table, lens, start = c.dev()
    codes = torch.empty((n_blocks, 2, heads, 64 * dim), dtype=torch.int8, device="cuda")
    scales = torch.empty((n_blocks, 2, heads), device="cuda")
    off = n_blocks - c.n_blocks
    codes[off:], scales[off:] = small_codes, small_scales
    far = torch.where((table >= 0) & (table < c.n_blocks), table + off, -1).int()
    near = torch.where((table >= 0) & (table < c.n_blocks), table, -1).int()
    k, v, q = to_dev(c.rows(heads)), to_dev(c.rows(heads)), to_dev(c.rows(2 * heads))
    kw = dict(tok_start=start, max_q=40)
    qmv.kv_append(k, v, codes, scales, far, lens, **kw)
    qmv.kv_append(k, v, small_codes, small_scales, near, lens, **kw)
    assert torch.equal(codes[off:], small_codes)
    assert torch.equal(qmv.kv_attn(q, codes, scales, far, lens, **kw),
                       qmv.kv_attn(q, small_codes, small_scales, near, lens, **kw))


@pytest.mark.parametrize("heads,dim,group,tokens", [(4, 256, 8, 1), (2, 128, 8, 1), (4, 64, 2, 3), (1, 16, 4, 16)])
def test_many_sequences_shared_by_length(heads, dim, group, tokens):
    """Sequences of no token to many, their workgroups counted by length: some
    short enough for one, some not, lanes without a sequence."""
    qmv = need_gpu()
    for n in (2, 48, 63, 64, 65):
        say(f"attn {n} sequences {heads}x{dim}")
        r = np.random.default_rng(n)
        lens = r.integers(0, 700, n)
        lens[: min(n, 3)] = (0, 2500, 1)[: min(n, 3)]
        counts = r.integers(0, tokens + 1, n)
        counts[1] = tokens
        c = Case(20 + n, lens.tolist(), counts.tolist(), heads, dim)
        check_attn(qmv, c, group, (n, dim))


@pytest.mark.parametrize("dim", [32, 48, 96, 112, 144, 160, 176, 208, 224, 240])
def test_other_dims(dim):
    """Each multiple of 16, with few rows, more than 16 and more than 32."""
    qmv = need_gpu()
    for lens, counts, group in (([200, 65], [1, 3], 2), ([900, 130], [9, 4], 3), ([700, 90], [64, 20], 2)):
        c = Case(dim, lens, counts, 2, dim)
        for ws in (False, True):
            check_attn(qmv, c, group, (dim, group), ws=ws, xq=dim % 32 == 0)


@pytest.mark.parametrize("lens,counts,group", [
    ([9000], [3], 8),            # 24 rows, one sequence: every group the same parts
    ([5000, 64, 0, 1300], [9, 9, 0, 2], 8),  # up to 72 rows, parts by length, some one part
    ([2500], [80], 4),           # row blocks of one sequence
])
def test_rows_joined_by_a_second_launch(lens, counts, group):
    """More than 16 rows over many blocks: the sums of several workgroups, the
    output over q itself, and a captured call replayed with others between."""
    qmv = need_gpu()
    say(f"attn joined {lens} {counts}")
    c = Case(31, lens, counts, 2, 64)
    q = c.rows(2 * group)
    for window in (0, 700):
        check_attn(qmv, c, group, (lens, window), window=window, xq=True, q=q)
    codes, scales, table, seq, start = c.dev()
    need = qmv.kv_attn_workspace_bytes(len(lens), c.n_tok, c.max_q, 2 * group, 2, 64, c.width)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    kw = dict(tok_start=start, max_q=c.max_q, ws=ws)
    x = to_dev(q)
    want = qmv.kv_attn(x, codes, scales, table, seq, **kw)
    over = x.clone()
    qmv.kv_attn(over, codes, scales, table, seq, out=over, **kw)
    assert torch.equal(over, want)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        qmv.kv_attn(x, codes, scales, table, seq, out=out, **kw)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(qmv.kv_attn(x, codes, scales, table, seq, **kw), want)


@pytest.mark.parametrize("dim", [64, 192])
def test_value_scales_far_apart(dim):
    """Blocks whose values differ by many powers of two, and blocks of zeros."""
    qmv = need_gpu()
    c = Case(33, [1500, 900], [2, 20], 2, dim)
    c.scales[:, 1] *= np.float32(2.0) ** c.rng.integers(-60, 40, c.scales[:, 1].shape).astype(np.float32)
    c.scales[:, 1][c.rng.random(c.scales[:, 1].shape) < 0.2] = 0.0
    for ws in (False, True):
        check_attn(qmv, c, 3, dim, ws=ws)


@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 40, 2**33])
def test_the_widest_windows(window):
    """Windows about the largest whole number, rows before the first token in
    the same call: those see nothing, the others all of theirs."""
    qmv = need_gpu()
    c = Case(34, [3, 130, 70], [10, 5, 70], 2, 64)
    for ws in (False, True):
        check_attn(qmv, c, 2, window, window=window, ws=ws)


@pytest.mark.parametrize("uniform", [1, 40])
def test_append_at_half_steps(uniform):
    """Values at and one step beside the middle between two codes, with scales
    that are no power of two, very small and very large ones too."""
    qmv = need_gpu()
    for e in (0, -3, -98, -103, 98, 103):
        c = Case(40, [uniform, 64 + uniform], [uniform] * 2, 2, 64, uniform=uniform)
        d = (np.float32(2.0) ** e * c.rng.uniform(1, 2, (2 * uniform, 2, 64))).astype(np.float32)
        d[:] = d[:1, :1, :1]
        n = c.rng.integers(-127, 127, d.shape)
        k = ((n + np.float32(0.5)) * d).astype(np.float32)
        k = np.nextafter(k, np.where(c.rng.random(d.shape) < 0.5, k, np.float32(0))).astype(np.float32)
        k[..., 0] = 127 * d[..., 0]
        run_append(qmv, c, k, np.ascontiguousarray(k[:, ::-1, ::-1]), e)


def test_a_run_longer_than_the_integer_sums_hold():
    """Equal weights over 9375 blocks of the largest codes: nothing but their
    number makes a wave add its integer sums up."""
    qmv = need_gpu()
    say("attn long equal")
    c = Case(50, [600000], [1], 1, 16)
    c.codes[:, 1] = np.where(c.codes[:, 1] >= 0, 127, -127)
    c.codes[:, 1, :, ::3] = 127
    c.scales[:, 1] = c.scales[0, 1]
    q = np.zeros((1, 2, 16), np.float32)
    q[0, 1] = c.rng.standard_normal(16) * 1e-3
    for ws in (False, True):
        check_attn(qmv, c, 2, "long", ws=ws, q=q)


def test_calls_on_two_streams():
    """Calls of two shapes at once, each with its own workspace."""
    qmv = need_gpu()
    say("attn two streams")
    jobs = []
    for seed, lens, counts, group in ((51, [3000, 70, 900], [1, 1, 1], 8), (52, [4000], [12], 4)):
        c = Case(seed, lens, counts, 4, 128)
        codes, scales, table, seq, start = c.dev()
        q = to_dev(c.rows(4 * group))
        ws = torch.zeros(qmv.kv_attn_workspace_bytes(len(lens), c.n_tok, c.max_q, 4 * group, 4, 128, c.width),
                         dtype=torch.uint8, device="cuda")
        args = (q, codes, scales, table, seq)
        kw = dict(tok_start=start, max_q=c.max_q, ws=ws)
        jobs.append((args, kw, qmv.kv_attn(*args, **kw), torch.cuda.Stream(), torch.empty_like(q)))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, kw, _, stream, out in jobs:
            qmv.kv_attn(*args, out=out, stream=stream, **kw)
    torch.cuda.synchronize()
    for _, _, want, _, out in jobs:
        assert torch.equal(out, want)


def test_two_graphs_share_a_workspace():
    """Captured calls of two shapes with one workspace, replayed in turn."""
    qmv = need_gpu()
    say("attn two graphs")
    jobs, need = [], 0
    for seed, lens, group in ((53, [5000], 8), (54, [2000, 10, 600], 4)):
        c = Case(seed, lens, [1] * len(lens), 2, 128)
        need = max(need, qmv.kv_attn_workspace_bytes(len(lens), c.n_tok, 1, 2 * group, 2, 128, c.width))
        jobs.append((c, to_dev(c.rows(2 * group))))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for c, q in jobs:
        codes, scales, table, seq, start = c.dev()
        want = qmv.kv_attn(q, codes, scales, table, seq, tok_start=start, ws=ws)
        out = torch.empty_like(q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            qmv.kv_attn(q, codes, scales, table, seq, tok_start=start, ws=ws, out=out)
        graphs.append((graph, out, want, (codes, scales, table, seq, start)))
    for _ in range(4):
        for graph, out, _, _ in graphs:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in graphs:
            assert torch.equal(out, want)
        assert not ws[:65536].any()


def attend_far(c, q, scale):
    """(out, tol) where scores lie so far apart that the largest take all: the
    mean of the values of the keys that have it.  Weights of one are rounded
    to 33 u of the block's largest, sums and joins as in kv_ref.attend."""
    u = 2.0 ** -24
    kk, vv = kv_ref.split(c.codes, c.dim)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for s, (t0, n) in enumerate(kv_ref.rows_of(c.start, len(c.lens), q.shape[0], c.max_q)):
        length = int(c.lens[s])
        ids = c.table[s, :-(-length // 64)]
        kf = kk[ids] * c.scales[ids].astype(np.float64)[:, 0, :, None, None]
        vf = vv[ids] * c.scales[ids].astype(np.float64)[:, 1, :, None, None]
        for i in range(n):
            for h in range(q.shape[1]):
                g = h // (q.shape[1] // c.heads)
                score = (kf[:, g].reshape(-1, c.dim) @ q[t0 + i, h].astype(np.float64)) * scale * np.log2(np.e)
                score[length - n + i + 1:] = -np.inf
                top = score.max()
                won = score >= top - 1e-6 * abs(top)
                rest = score[~won].max()
                assert top - rest > 40 + 1e-5 * abs(top), (i, h, top, rest)  # weights below 2^-40 are nothing
                v = vf[:, g].reshape(-1, c.dim)
                blocks = np.unique(np.flatnonzero(won) // 64)
                a = np.abs(v).reshape(-1, 64, c.dim)[blocks].sum((0, 1)) / won.sum()
                out[t0 + i, h] = v[won].mean(0)
                tol[t0 + i, h] = 33 * u * a + 4 * (len(ids) + 73) * u * np.abs(v[won]).mean(0)
    return out, tol


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 1), (128, 3), (192, 1), (256, 3)])
def test_the_largest_scores(dim, new, order):
    """Scores up to 1e30 and down to -1e30 over many blocks a wave, where an
    fp32 step of a score is more than what its weight's field has to spare,
    later more than the whole field: one key, or a few alike, take all."""
    qmv = need_gpu()
    say(f"attn far scores {dim} {new} {order}")
    c = Case(60, [2500, 1300], [new, 1], 1, dim)
    kk, _ = kv_ref.split(c.codes, dim)
    kk[...] = 0
    kk[..., 0] = c.rng.integers(62, 126, kk.shape[:-1])
    kk[..., 7, 0], kk[..., 11, 0] = 127, 127
    kk[..., 5, 0], kk[..., 60, 0] = 60, 60
    c.scales[:, 1] = 2.0 ** c.rng.uniform(-3, 3, c.scales[:, 1].shape)
    for s in range(2):
        n = -(-int(c.lens[s]) // 64)
        at = {"rising": np.arange(n), "falling": np.arange(n)[::-1], "mixed": c.rng.permutation(n)}[order]
        c.scales[c.table[s, :n], 0, 0] = 0.02 * (1 + 0.02 * at)
    scale = dim ** -0.5
    far = np.array([2e4, 7e4, 2e5, 3e6, 1e9, 1e20, 1e30])
    q = np.zeros((c.n_tok, 14, dim), np.float32)
    q[..., 0] = np.concatenate([far, -far]) / (127 * c.scales[:, 0][c.used].max() * scale * np.log2(np.e))
    codes, scales, table, lens, start = c.dev()
    ref, tol = attend_far(c, q, scale)
    need = qmv.kv_attn_workspace_bytes(2, c.n_tok, new, 14, 1, dim, c.width)
    for ws in (None, torch.zeros(need, dtype=torch.uint8, device="cuda")):
        got = qmv.kv_attn(to_dev(q), codes, scales, table, lens, tok_start=start, max_q=new, ws=ws).cpu().numpy()
        bad = np.argwhere(~(np.abs(got - ref) <= tol))
        assert len(bad) == 0, (len(bad), bad[:3], got[tuple(bad[0])], ref[tuple(bad[0])])


@pytest.mark.parametrize("dim", [64, 128, 160])
def test_large_scores_among_others(dim):
    """Rows with scores of up to 1e5 beside ordinary ones in the same waves,
    many blocks a wave; and a row whose scores leave fp32, which is not to
    touch the others."""
    qmv = need_gpu()
    c = Case(61, [8000, 700], [2, 1], 1, dim)
    q = c.rows(8)
    q[0, 1] *= np.float32(1e4)
    q[0, 2] *= np.float32(3e4)
    q[0, 5] *= np.float32(100)
    q[2, :4] *= np.float32(3e4)
    for ws in (False, True):
        good = check_attn(qmv, c, 8, dim, q=q, ws=ws)
    q[1, 3] = np.float32(3e38)
    codes, scales, table, lens, start = c.dev()
    got = qmv.kv_attn(to_dev(q), codes, scales, table, lens, tok_start=start, max_q=2, scale=30.0).cpu().numpy()
    q[1, 3] = 0.0
    want = qmv.kv_attn(to_dev(q), codes, scales, table, lens, tok_start=start, max_q=2, scale=30.0).cpu().numpy()
    keep = np.ones(good.shape[:2], bool)
    keep[1, 3] = False
    assert np.isfinite(want).all()
    assert np.abs(got - want)[keep].max() <= 1e-4 * np.abs(want).max()


@pytest.mark.parametrize("new", [1, 40])
def test_append_behind_a_scale_of_zero(new):
    """Codes under a scale of zero stand for zeros, whatever they are: they
    are zeros when the scale grows."""
    qmv = need_gpu()
    say(f"append behind zero scales {new}")
    c = Case(62, [50 + new, 9 + new], [new, new], 2, 80)
    c.scales[c.table[:, 0], 0, 1] = 0.0
    c.scales[c.table[:, 0], 1, 0] = 0.0
    k, v = c.rows(2), c.rows(2)
    before = c.codes.copy()
    codes, scales, table, lens, start = c.dev()
    qmv.kv_append(to_dev(k), to_dev(v), codes, scales, table, lens, tok_start=start, max_q=new)
    kv_ref.append(c.codes, c.scales, c.table, c.lens, c.start, c.max_q, k, v)
    for part, h in ((0, 1), (1, 0)):
        for s, old in enumerate((50, 9)):
            assert kv_ref.split(before, 80)[part][c.table[s, 0], h, :old].any()
            kv_ref.split(c.codes, 80)[part][c.table[s, 0], h, :old] = 0
    same_cache(c, codes, scales, new)


@pytest.mark.parametrize("lens,counts,group", [
    ([1300], [1], 6),  # 21 blocks: 3 parts of 8 for eight waves, 6 of 4 for four
    ([2500], [1], 1),  # 40 blocks: 5 or 10 parts
    ([700], [1], 3),   # 11 blocks: 2 or 3 parts
    ([2000, 190], [1, 1], 3), ([1800, 130, 1349], [3, 1, 2], 5)])
def test_joins_of_odd_rows_and_parts(lens, counts, group):
    """Rows times parts of no multiple of four: what is summed lies behind
    that many factors."""
    qmv = need_gpu()
    for dim in (16, 48, 128, 256):
        say(f"attn join {lens} {dim}")
        c = Case(63, lens, counts, 1, dim)
        check_attn(qmv, c, group, (lens, dim))


def test_a_run_whose_integer_sums_would_wrap():
    """Equal weights over 18000 blocks, 2250 a wave without a workspace.  A
    weight is then kTop / kUnit = 64 * 2^16 - 128 * 2^8 + 0, so a block of codes
    127 adds 64 * 128 * 127 to the sum of the middle digit: 2064 blocks are
    more than 2^31 if nothing adds the sums up before."""
    qmv = need_gpu()
    say("attn wrap")
    blocks = 18000
    assert (blocks // 8) * 64 * 128 * 127 > 2**31
    c = Case(64, [64 * 5], [1], 1, 16)
    ids = c.table[0].copy()
    _, vv = kv_ref.split(c.codes, 16)
    vv[..., ::3], vv[..., 1::3] = 127, -127
    c.scales[:, 1] = c.scales[ids[0], 1]
    c.table = np.tile(ids, blocks // 5).reshape(1, blocks)
    c.lens[:], c.width = 64 * blocks, blocks
    q = np.zeros((1, 2, 16), np.float32)
    q[0, 1] = c.rng.standard_normal(16) * 1e-3
    for ws in (False, True):
        check_attn(qmv, c, 2, "wrap", ws=ws, q=q)


@pytest.mark.parametrize("lens,counts", [([700, 64], [1, 1]), ([4000], [5])])
def test_q8_output_alone(lens, counts):
    """The C call without an fp32 output writes the same Q8 blocks."""
    import ctypes
    qmv = need_gpu()
    say(f"attn q8 alone {lens}")
    c = Case(65, lens, counts, 2, 64)
    codes, scales, table, seq, start = c.dev()
    heads, k = 8, 8 * 64
    q = to_dev(c.rows(heads))
    need = qmv.kv_attn_workspace_bytes(len(lens), c.n_tok, c.max_q, heads, 2, 64, c.width)
    ws = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
    want, got = (torch.full((qmv.act_bytes(c.n_tok, k),), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
    qmv.kv_attn(q, codes, scales, table, seq, tok_start=start, max_q=c.max_q, xq=want, ws=ws)
    kv = qmv._kv(codes, scales, table, seq, start, c.n_tok, c.max_q, 64)
    st = qmv.lib().qmv_kv_attn(ctypes.byref(kv), q.data_ptr(), k, heads, 64 ** -0.5, 0, None, 0, got.data_ptr(),
                               ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(got, want)
