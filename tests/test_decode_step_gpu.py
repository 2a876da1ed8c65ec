"""One decode step through the library's own chain: norm -> q/k/v projections
-> adapters -> norm and rotation of the heads -> cache append -> attention ->
output projection with residual and its adapters -> norm -> gate -> routed
experts -> norm -> output head -> log probabilities; a prompt chunk, verify
batches and single tokens.  Every stage is compared with its reference on the
GPU's own output of the stage before; captured in a graph, the step gives the
eager one's bits, with ids, positions and lengths changed between replays."""
import numpy as np
import pytest
import torch

import kv_ref
import oracle
import synth
import test_gate_gpu
import test_heads_gpu
import test_logprobs_gpu
import test_lora_gpu
from gpu_util import assert_y, gpu, need_gpu, say, to_dev, x_host

pytestmark = gpu

H, HEADS, KVH, D = 512, 8, 2, 64
NQ, NKV = HEADS * D, KVH * D
E, TOP_K, FF, GROUPS = 16, 4, 256, 4
V = 3001
RANK, ADAPTERS = 16, 5
EPS = 1e-5


class Step:
    def __init__(self, qmv, seqs, width, rows):
        self.qmv, self.seqs = qmv, seqs
        rng = np.random.default_rng(7)
        fmt = {"q": synth.Q4_K, "k": synth.Q4_K, "v": synth.Q4_K, "o": synth.Q4_K}
        self.host = {n: synth.make_weights(f, r, k, f"step/{n}").data
                     for (n, f), (r, k) in zip(fmt.items(), ((NQ, H), (NKV, H), (NKV, H), (H, NQ)))}
        self.host["gu"] = synth.make_weights(synth.IQ4_XS, E * 2 * FF, H, "step/gu").data
        self.host["dn"] = synth.make_weights(synth.IQ4_XS, E * H, FF, "step/dn").data
        self.host["head"] = synth.make_weights(synth.Q8_0, V, H, "step/head").data
        self.w = {n: to_dev(a) for n, a in self.host.items()}
        self.norms = [(1 + 0.2 * rng.standard_normal(H)).astype(np.float32) for _ in range(3)]
        self.hn = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
        self.dn, self.dhn = [to_dev(a) for a in self.norms], [to_dev(a) for a in self.hn]
        self.freq = test_heads_gpu.freqs(D)
        self.dfreq = to_dev(self.freq)
        g = torch.Generator().manual_seed(5)
        self.ad = [((torch.randn(ADAPTERS, RANK, k, generator=g) / k ** 0.5).bfloat16(),
                    (0.3 * torch.randn(ADAPTERS, n, RANK, generator=g)).bfloat16())
                   for n, k in ((NQ, H), (NKV, H), (NKV, H), (H, NQ))]
        self.dad = [(a.cuda(), b.cuda()) for a, b in self.ad]
        self.ranks = torch.tensor([16, 4, 0, 9, 16], dtype=torch.int32)
        self.lscale = torch.tensor([1.0, 2.0, 1.0, 0.5, -1.0])
        self.dranks, self.dlscale = self.ranks.cuda(), self.lscale.cuda()
        self.router = (rng.standard_normal((E, H)) / H ** 0.5).astype(np.float32)
        self.bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        self.drouter, self.dbias = to_dev(self.router), to_dev(self.bias)
        blocks = seqs * width
        self.codes = torch.zeros((blocks, 2, KVH, 64 * D), dtype=torch.int8, device="cuda")
        self.scales = torch.full((blocks, 2, KVH), float("nan"), device="cuda")
        self.table = torch.randperm(blocks, generator=g).view(seqs, width).int().cuda()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        q = qmv

        def ws(n):
            return torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")

        self.ws = {"attn": ws(q.kv_attn_workspace_bytes(seqs, rows, rows, HEADS, KVH, D, width)),
                   "lora": ws(q.lora_workspace_bytes(3, RANK, rows)), "gate": ws(q.router_gate_workspace_bytes(rows, E)),
                   "gu": ws(q.moe_workspace_bytes(synth.IQ4_XS, E, 2 * FF, H, rows, TOP_K)),
                   "dn": ws(q.moe_workspace_bytes(synth.IQ4_XS, E, H, FF, rows, TOP_K))}

    def buffers(self, t):
        q = self.qmv

        def f(*shape):
            return torch.empty(*shape, device="cuda")

        def xq(rows, k):
            return torch.zeros(q.act_bytes(rows, k), dtype=torch.uint8, device="cuda")

        return {"y1": f(t, H), "x1": xq(t, H), "q": f(t, NQ), "k": f(t, NKV), "v": f(t, NKV),
                "base": f(t, NQ + 2 * NKV), "rot": f(t, NQ + NKV), "att": f(t, HEADS, D), "attq": xq(t, NQ), "o": f(t, H),
                "obase": f(t, H), "y2": f(t, H), "x2": xq(t, H),
                "ids": torch.empty(t, TOP_K, dtype=torch.int32, device="cuda"), "rw": f(t, TOP_K),
                "hq": xq(t * TOP_K, FF), "ff": f(t, H), "r3": f(t, H), "x3": xq(t, H), "logits": f(t, V), "lp": f(t, 1),
                "ent": f(t), "top": torch.empty(t, 5, dtype=torch.int32, device="cuda"), "tlp": f(t, 5)}

    def run(self, b, x, pos, ad, given, start, max_q):
        """One step on the residual stream x [T][H]; every product stays in b."""
        q, t = self.qmv, x.shape[0]
        kv = (self.codes, self.scales, self.table, self.lens)
        q.rmsnorm_quantize(x, self.dn[0], EPS, y_out=b["y1"], xq=b["x1"])
        q.matvec_batch(synth.Q4_K, [(self.w[n], r, b[n], None) for n, r in (("q", NQ), ("k", NKV), ("v", NKV))], H,
                       b["x1"], t)
        for n, at in (("q", 0), ("k", NQ), ("v", NQ + NKV)):
            b["base"][:, at:at + b[n].shape[1]].copy_(b[n])  # what the references start from
        q.lora(b["y1"], ad, [(*w, y, y) for w, y in zip(self.dad, (b["q"], b["k"], b["v"]))], ranks=self.dranks,
               scales=self.dlscale, ws=self.ws["lora"])
        b["rot"][:, :NQ].copy_(b["q"])
        b["rot"][:, NQ:].copy_(b["k"])
        qh, kh = b["q"].unflatten(1, (HEADS, D)), b["k"].unflatten(1, (KVH, D))
        q.head_norm_rope(qh, kh, pos, self.dfreq, self.dhn[0], self.dhn[1], eps=EPS)
        q.kv_append(kh, b["v"].unflatten(1, (KVH, D)), *kv, tok_start=start, max_q=max_q)
        q.kv_attn(qh, *kv, tok_start=start, max_q=max_q, out=b["att"], xq=b["attq"], ws=self.ws["attn"])
        q.matvec_batch(synth.Q4_K, [(self.w["o"], H, b["o"], x)], NQ, b["attq"], t)
        b["obase"].copy_(b["o"])
        q.lora(b["att"].view(t, NQ), ad, [(*self.dad[3], b["o"], b["o"])], ranks=self.dranks, scales=self.dlscale,
               ws=self.ws["lora"])
        q.rmsnorm_quantize(b["o"], self.dn[1], EPS, y_out=b["y2"], xq=b["x2"])
        q.router_gate(b["y2"], self.drouter, TOP_K, scoring="sigmoid", bias=self.dbias, n_groups=GROUPS, top_groups=2,
                      scale=1.5, ids=b["ids"], weights=b["rw"], ws=self.ws["gate"])
        q.moe_gate_up_swiglu(synth.IQ4_XS, self.w["gu"], E, FF, H, b["x2"], b["ids"], self.ws["gu"], hq=b["hq"])
        q.moe_matvec(synth.IQ4_XS, self.w["dn"], E, H, FF, b["hq"], True, b["ids"], b["rw"], self.ws["dn"], y=b["ff"])
        q.rmsnorm_quantize(b["ff"], self.dn[2], EPS, residual=b["o"], sum_out=b["r3"], xq=b["x3"])
        q.matvec(synth.Q8_0, self.w["head"], V, H, b["x3"], t, y=b["logits"])
        q.token_logprobs(b["logits"], given, top_n=5, logprobs=b["lp"], entropy=b["ent"], top_ids=b["top"],
                         top_logprobs=b["tlp"])


def check(step, b, x, pos, ad, given, codes, scales, start, max_q):
    """Every stage of a step that has run, against its reference."""
    qmv, t = step.qmv, x.shape[0]
    g = {n: v.cpu().numpy() for n, v in b.items()}

    def q8(name, rows, k):
        return tuple(f.cpu().numpy() for f in qmv.act_fields(b[name], rows, k))

    q1 = q8("x1", t, H)
    base = [g["base"][:, :NQ], g["base"][:, NQ:NQ + NKV], g["base"][:, NQ + NKV:]]
    for n, y in zip("qkv", base):
        yr, mag = oracle.matvec(synth.Q4_K, step.host[n], H, *q1)
        assert_y(y, yr, mag, n)
    ranks = step.ranks
    after = (g["rot"][:, :NQ], g["rot"][:, NQ:], g["v"])
    ids = torch.from_numpy(ad)
    for (a, w), y0, y in zip(step.ad, base, after):
        want, tol = test_lora_gpu.reference(torch.from_numpy(g["y1"]), a, w, torch.from_numpy(y0), ids, ranks, step.lscale)
        assert torch.all((torch.from_numpy(y).double() - want).abs() <= tol)
    for n, src, w, heads in (("q", g["rot"][:, :NQ], step.hn[0], HEADS), ("k", g["rot"][:, NQ:], step.hn[1], KVH)):
        want, tol = test_heads_gpu.reference(src.reshape(t, heads, D), w, pos[None], step.freq, [0] * (D // 2), False, 1.0,
                                             EPS)
        assert np.all(np.abs(g[n].reshape(t, heads, D) - want) <= tol), n
    table, lens = step.table.cpu().numpy(), step.lens.cpu().numpy()
    kv_ref.append(codes, scales, table, lens, start, max_q, g["k"].reshape(t, KVH, D), g["v"].reshape(t, KVH, D))
    assert np.array_equal(codes, step.codes.cpu().numpy())
    assert np.array_equal(scales, step.scales.cpu().numpy(), equal_nan=True)
    ref, tol, rows = kv_ref.attend(codes, scales, table, lens, start, max_q, g["q"].reshape(t, HEADS, D), D ** -0.5, 0)
    assert rows.all() and np.all(np.abs(g["att"] - ref) <= tol)
    yr, mag = oracle.matvec(synth.Q4_K, step.host["o"], NQ, *q8("attq", t, NQ))
    assert_y(g["obase"], yr + x, mag + np.abs(x), "o")
    want, tol = test_lora_gpu.reference(torch.from_numpy(g["att"].reshape(t, NQ)), *step.ad[3], torch.from_numpy(g["obase"]),
                                        ids, ranks, step.lscale)
    assert torch.all((torch.from_numpy(g["o"]).double() - want).abs() <= tol)
    l = g["y2"].astype(np.float64) @ step.router.astype(np.float64).T
    want_ids, want_w = test_gate_gpu.reference(l, TOP_K, "sigmoid", step.bias, GROUPS, 2, 2, True, 1.5)
    assert np.array_equal(g["ids"], want_ids)
    assert np.all(np.abs(g["rw"] - want_w) <= (2.0 ** -24 + 1e-12) * want_w)
    qs, d, s = q8("hq", t * TOP_K, FF)
    yr, mag = oracle.moe_matvec(synth.IQ4_XS, step.host["dn"], E, H, FF, qs, d, s, g["ids"], g["rw"], True)
    assert_y(g["ff"], yr, mag, "experts")
    assert np.array_equal(g["r3"], g["ff"] + g["o"])
    yr, mag = oracle.matvec(synth.Q8_0, step.host["head"], H, *q8("x3", t, H))
    assert_y(g["logits"], yr, mag, "head")
    want = test_logprobs_gpu.reference(g["logits"], given, 5, 1.0)
    n = 1.2 * V / 1024 + 140
    test_logprobs_gpu.close(b["lp"], want[0], n * test_logprobs_gpu.U)
    test_logprobs_gpu.close(b["ent"], want[1], 2 * n * test_logprobs_gpu.U * (1 + want[1]))
    assert np.array_equal(g["top"], want[2])
    test_logprobs_gpu.close(b["tlp"], want[3], n * test_logprobs_gpu.U)


def test_steps():
    qmv = need_gpu()
    step = Step(qmv, 2, 3, 16)
    for i, counts in enumerate(([16, 0], [0, 13], [5, 6], [1, 1], [0, 1])):
        t = sum(counts)
        say(f"decode step {i} {counts}")
        step.lens += torch.tensor(counts, dtype=torch.int32, device="cuda")
        lens = step.lens.cpu().numpy()
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        pos = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, counts)]).astype(np.int32)
        ad = np.array([s * 3 - 1 + i % 3 for s, c in enumerate(counts) for _ in range(c)], dtype=np.int32)
        given = np.random.default_rng(i).integers(0, V, (t, 1))
        x = x_host(t, H, f"step/x{i}")
        codes, scales = step.codes.cpu().numpy(), step.scales.cpu().numpy()
        b = step.buffers(t)
        step.run(b, to_dev(x), to_dev(pos), to_dev(ad), to_dev(given.astype(np.int32)), to_dev(start), max(counts))
        torch.cuda.synchronize()
        check(step, b, x, pos, ad, given, codes, scales, start, max(counts))
    for name in ("attn", "gate"):
        assert not step.ws[name][:256].any()


@pytest.mark.parametrize("seqs", [1, 6])
def test_step_in_a_graph(seqs):
    qmv = need_gpu()
    say(f"decode step graph, {seqs} sequences")
    one, eager = Step(qmv, seqs, 4, seqs), Step(qmv, seqs, 4, seqs)
    x = torch.empty(seqs, H, device="cuda").normal_()
    pos = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    ad = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    given = torch.zeros(seqs, 1, dtype=torch.int32, device="cuda")
    b, e = one.buffers(seqs), eager.buffers(seqs)
    graphs = []
    for _ in range(2):  # two graphs on the same workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one.run(b, x, pos, ad, given, None, 1)
        graphs.append(g)
    for rep in range(8):
        x.normal_()
        ad.random_(-1, ADAPTERS)
        given.random_(0, V)
        one.lens += 1
        eager.lens += 1
        pos.copy_(one.lens - 1)
        eager.run(e, x, pos, ad, given, None, 1)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        for n in b:
            assert torch.equal(b[n], e[n]), (rep, n)
        assert torch.equal(one.codes, eager.codes)
