"""The attention half of a decode layer through the library's own chain:
residual + norm + Q8 -> q/k/v projections in one launch -> cache append ->
attention, with its Q8 blocks -> output projection + residual, over a prompt,
a verify batch and single tokens; then the same captured in a graph.  Every
stage is compared with its reference on the GPU's output of the stage before."""
import numpy as np
import pytest
import torch

import kv_ref
import oracle
import synth
from gpu_util import assert_y, gpu, need_gpu, say, to_dev, x_host

pytestmark = gpu

H, HEADS, KVH, D = 512, 8, 2, 64
NQ, NKV = HEADS * D, KVH * D
EPS = 1e-5


class Layer:
    def __init__(self, qmv, seqs, width, most):
        self.qmv, self.seqs = qmv, seqs
        self.host = {n: synth.make_weights(synth.Q4_K, rows, k, f"layer/{n}").data
                     for n, rows, k in (("q", NQ, H), ("k", NKV, H), ("v", NKV, H), ("o", H, NQ))}
        self.w = {n: to_dev(a) for n, a in self.host.items()}
        self.norm_host = 1.0 + 0.2 * x_host(1, H, "layer/norm")[0]
        self.norm = to_dev(self.norm_host)
        blocks = seqs * width
        self.codes = torch.empty((blocks, 2, KVH, 64 * D), dtype=torch.int8, device="cuda")
        self.codes.random_(-128, 128, generator=torch.Generator("cuda").manual_seed(2))
        self.scales = torch.full((blocks, 2, KVH), float("nan"), device="cuda")
        self.table = torch.randperm(blocks, generator=torch.Generator().manual_seed(3)).view(seqs, width).int().cuda()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(max(qmv.kv_attn_workspace_bytes(seqs, most, most, HEADS, KVH, D, width), 1),
                              dtype=torch.uint8, device="cuda")

    def buffers(self, t):
        q = self.qmv
        return {"r": torch.empty(t, H, device="cuda"), "q": torch.empty(t, NQ, device="cuda"),
                "k": torch.empty(t, NKV, device="cuda"), "v": torch.empty(t, NKV, device="cuda"),
                "out": torch.empty(t, HEADS, D, device="cuda"), "y": torch.empty(t, H, device="cuda"),
                "xq": torch.empty(q.act_bytes(t, H), dtype=torch.uint8, device="cuda"),
                "oq": torch.empty(q.act_bytes(t, NQ), dtype=torch.uint8, device="cuda")}

    def run(self, x, res, b, start, max_q, ws=None):
        """One step on x, res [T][H]; every product stays in b."""
        q, t = self.qmv, x.shape[0]
        q.rmsnorm_quantize(x, self.norm, EPS, residual=res, sum_out=b["r"], xq=b["xq"])
        qs, ks, vs = b["q"], b["k"], b["v"]
        q.matvec_batch(synth.Q4_K, [(self.w["q"], NQ, qs, None), (self.w["k"], NKV, ks, None),
                                    (self.w["v"], NKV, vs, None)], H, b["xq"], t)
        kv = (self.codes, self.scales, self.table, self.lens)
        q.kv_append(ks.unflatten(1, (KVH, D)), vs.unflatten(1, (KVH, D)), *kv, tok_start=start, max_q=max_q)
        q.kv_attn(qs.unflatten(1, (HEADS, D)), *kv, tok_start=start, max_q=max_q, out=b["out"], xq=b["oq"],
                  ws=self.ws if ws is None else ws)
        q.matvec_batch(synth.Q4_K, [(self.w["o"], H, b["y"], b["r"])], NQ, b["oq"], t)


def check_step(lay, x, res, counts, what):
    """One step against the references; counts: new tokens of each sequence."""
    t, n = x.shape[0], len(counts)
    codes, scales = lay.codes.cpu().numpy(), lay.scales.cpu().numpy()
    table, lens = lay.table.cpu().numpy(), lay.lens.cpu().numpy()
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    b = lay.buffers(t)
    lay.run(to_dev(x), to_dev(res), b, to_dev(start), max(counts))
    g = {k: v.cpu().numpy() for k, v in b.items()}
    r = x + res
    assert np.array_equal(g["r"], r), what
    r64 = r.astype(np.float64)
    y64 = r64 / np.sqrt((r64 * r64).mean(1, keepdims=True) + EPS) * lay.norm_host.astype(np.float64)
    qs, d, s = (f.cpu().numpy() for f in lay.qmv.act_fields(b["xq"], t, H))
    # a code is the nearest whole number, or the other one beside a half step that fp32 cannot tell
    got = qs.reshape(t, -1, 32) * d.astype(np.float64)[..., None]
    assert np.all(np.abs(got.reshape(t, H) - y64) <= np.repeat(d, 32, 1) * (0.5 + 2e-4)), what
    for name in "qkv":
        yr, mag = oracle.matvec(synth.Q4_K, lay.host[name], H, qs, d, s)
        assert_y(g[name], yr, mag, f"{what} {name}")
    kv_ref.append(codes, scales, table, lens, start, max(counts), g["k"].reshape(t, KVH, D),
                  g["v"].reshape(t, KVH, D))
    assert np.array_equal(codes, lay.codes.cpu().numpy()), what
    assert np.array_equal(scales, lay.scales.cpu().numpy(), equal_nan=True), what
    ref, tol, rows = kv_ref.attend(codes, scales, table, lens, start, max(counts),
                                   g["q"].reshape(t, HEADS, D), D ** -0.5, 0)
    assert rows.all() and np.all(np.abs(g["out"] - ref) <= tol), what
    qs, d, s = (f.cpu().numpy() for f in lay.qmv.act_fields(b["oq"], t, NQ))
    for x_, y_ in zip((qs, d, s), oracle.quantize_act(g["out"].reshape(t, NQ))):
        assert np.array_equal(x_, y_), what
    yr, mag = oracle.matvec(synth.Q4_K, lay.host["o"], NQ, qs, d, s)
    assert_y(g["y"], yr + r, mag + np.abs(r), f"{what} output")


def test_layer_steps():
    qmv = need_gpu()
    lay = Layer(qmv, 2, 5, 16)
    for i, counts in enumerate(([16, 16], [16, 3], [16, 16], [16, 16], [6, 5], [1, 1], [1, 1])):
        if sum(counts) > 16:  # the projections take 16 rows: sequence by sequence
            parts = [[counts[0], 0], [0, counts[1]]]
        else:
            parts = [counts]
        for j, c in enumerate(parts):
            say(f"layer step {i} {c}")
            lay.lens += torch.tensor(c, dtype=torch.int32, device="cuda")
            x, res = x_host(sum(c), H, f"layer/x{i}{j}"), x_host(sum(c), H, f"layer/r{i}{j}") * np.float32(2.0)
            check_step(lay, x, res, c, f"step {i}.{j}")


@pytest.mark.parametrize("seqs,width", [(1, 40), (3, 12)])
def test_layer_in_a_graph(seqs, width):
    """Replays, with the lengths advanced on the device between them and eager
    work on another cache, give the bits of eager steps; two graphs share the
    workspace one after the other."""
    qmv = need_gpu()
    say(f"layer graph {seqs}x{width}")
    lay, eager = Layer(qmv, seqs, width, 1), Layer(qmv, seqs, width, 1)
    for a in (lay, eager):  # a context to begin with
        a.codes.random_(-127, 128, generator=torch.Generator("cuda").manual_seed(5))
        a.scales.fill_(0.02)
        a.lens.fill_(width * 64 - 70)
        a.lens[0] += 3
    x, res = torch.empty(seqs, H, device="cuda"), torch.empty(seqs, H, device="cuda")
    b, e = lay.buffers(seqs), eager.buffers(seqs)
    one = torch.ones_like(lay.lens)
    x.normal_(generator=torch.Generator("cuda").manual_seed(6))
    res.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            lay.lens += one
            lay.run(x, res, b, None, 1)
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(6):
        x.normal_()
        eager.lens += one
        eager.run(x, res, e, None, 1, ws=eager.ws)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        for name in b:
            if name in ("xq", "oq"):
                k = H if name == "xq" else NQ
                assert all(torch.equal(p, q) for p, q in zip(qmv.act_fields(b[name], seqs, k),
                                                             qmv.act_fields(e[name], seqs, k))), (rep, name)
            else:
                assert torch.equal(b[name], e[name]), (rep, name)
        assert torch.equal(lay.codes, eager.codes) and torch.equal(lay.scales, eager.scales), rep
    assert not lay.ws[:65536].any()
