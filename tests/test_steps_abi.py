"""Refusals of the steps around a layer's matvecs: every call here returns
from host validation, so these run without a GPU."""
import ctypes

import pytest
import torch

import quantized_decode_gemv_qmv_amd as q

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000000  # 256-byte aligned, never dereferenced by host validation
NAN, INF = float("nan"), float("inf")


def heads(**kw):
    a = dict(pos=FAKE, freq=FAKE, axis=None, axes=1, rot=64, adjacent=0, scale=1.0, q=FAKE, ldq=256, heads=4,
             qw=FAKE, k=FAKE, ldk=128, kv=2, kw=FAKE, t=3, dim=64, eps=1e-6, qo=FAKE, ldqo=256, ko=FAKE, ldko=128)
    a.update(kw)
    rope = q._Rope(a["pos"], a["freq"], a["axis"], a["axes"], a["rot"], a["adjacent"], a["scale"])
    return q.lib().qmv_head_norm_rope(ctypes.byref(rope), a["q"], a["ldq"], a["heads"], a["qw"], a["k"], a["ldk"],
                                      a["kv"], a["kw"], a["t"], a["dim"], a["eps"], a["qo"], a["ldqo"], a["ko"],
                                      a["ldko"], None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
    (dict(k=None, ko=None, kv=0), INVALID), (dict(kv=0), INVALID), (dict(kv=-1), INVALID), (dict(heads=0), INVALID),
    (dict(t=0), INVALID), (dict(dim=0), INVALID), (dict(dim=62, rot=60), INVALID), (dict(rot=-2), INVALID),
    (dict(rot=63), INVALID), (dict(rot=66), INVALID), (dict(axes=0), INVALID), (dict(adjacent=2), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(eps=-1.0), INVALID),
    (dict(ldq=252), INVALID), (dict(ldqo=252), INVALID), (dict(ldk=124), INVALID), (dict(ldko=124), INVALID),
    (dict(t=65537), UNSUPPORTED), (dict(heads=16385, ldq=1 << 21, ldqo=1 << 21), UNSUPPORTED),
    (dict(kv=1025, ldk=1 << 17, ldko=1 << 17), UNSUPPORTED),
    (dict(dim=260, ldq=2048, ldqo=2048, ldk=2048, ldko=2048), UNSUPPORTED), (dict(axes=5), UNSUPPORTED),
    (dict(q=FAKE + 4), MISALIGNED), (dict(qo=FAKE + 8), MISALIGNED), (dict(k=FAKE + 4), MISALIGNED),
    (dict(ko=FAKE + 4), MISALIGNED), (dict(ldq=257), MISALIGNED), (dict(ldqo=258), MISALIGNED),
    (dict(ldk=129), MISALIGNED), (dict(ldko=130), MISALIGNED), (dict(qw=FAKE + 4), MISALIGNED),
    (dict(kw=FAKE + 8), MISALIGNED), (dict(pos=FAKE + 2), MISALIGNED), (dict(freq=FAKE + 1), MISALIGNED),
    (dict(axis=FAKE + 2), MISALIGNED)])
def test_heads_refusals(change, status):
    assert heads(**change) == status


def test_heads_binding_refusals():
    x = torch.zeros(2, 4, 64)
    for call in (lambda: q.head_norm_rope(x, None, None, None),          # not on the GPU
                 lambda: q.head_norm_rope(x.view(2, 256), None, None, None)):
        with pytest.raises(ValueError):
            call()
    assert q.lib().qmv_head_norm_rope(None, FAKE, 256, 4, None, None, 0, 0, None, 1, 64, 1e-6, FAKE, 256, None, 0,
                                      None) == INVALID


def lora(**kw):
    a = dict(kind=0, a=FAKE, b=FAKE, n=100, base=None, ldb=0, y=FAKE, ldy=100, items=1, x=FAKE, ldx=64, t=3, k=64,
             ids=FAKE, adapters=4, rank=16, ranks=None, scales=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    arr = (q._LoraItem * 9)(*[q._LoraItem(a["a"], a["b"], a["n"], a["base"], a["ldb"], a["y"], a["ldy"])] * 9)
    return q.lib().qmv_lora(a["kind"], arr if a["items"] is not None else None, a["items"] or 1, a["x"], a["ldx"],
                            a["t"], a["k"], a["ids"], a["adapters"], a["rank"], a["ranks"], a["scales"], a["ws"],
                            a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(kind=3), INVALID), (dict(kind=-1), INVALID), (dict(items=None), INVALID), (dict(items=-1), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(y=None), INVALID), (dict(n=0), INVALID),
    (dict(ldy=99), INVALID), (dict(base=FAKE, ldb=99), INVALID), (dict(x=None), INVALID), (dict(ids=None), INVALID),
    (dict(ws=None), INVALID), (dict(t=0), INVALID), (dict(k=0), INVALID), (dict(k=60), INVALID), (dict(ldx=60), INVALID),
    (dict(adapters=0), INVALID), (dict(rank=0), INVALID), (dict(rank=12), INVALID),
    (dict(items=9), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(t=4097), UNSUPPORTED),
    (dict(k=65544, ldx=65544), UNSUPPORTED), (dict(n=262145, ldy=262145), UNSUPPORTED),
    (dict(adapters=2**31), UNSUPPORTED),
    (dict(a=FAKE + 8), MISALIGNED), (dict(b=FAKE + 2), MISALIGNED), (dict(y=FAKE + 2), MISALIGNED),
    (dict(base=FAKE + 1, ldb=100), MISALIGNED), (dict(x=FAKE + 4), MISALIGNED), (dict(ldx=65), MISALIGNED),
    (dict(ids=FAKE + 2), MISALIGNED), (dict(ranks=FAKE + 2), MISALIGNED), (dict(scales=FAKE + 1), MISALIGNED),
    (dict(ws=FAKE + 64), MISALIGNED), (dict(wsb=100), WORKSPACE), (dict(wsb=0), WORKSPACE)])
def test_lora_refusals(change, status):
    assert lora(**change) == status


def test_lora_overlaps():
    """Items that write the same values, or another's base, are refused; columns of the same rows are not."""
    def call(items, t=3):
        arr = (q._LoraItem * len(items))(*[q._LoraItem(FAKE, FAKE, n, b, lb, y, ly) for n, b, lb, y, ly in items])
        return q.lib().qmv_lora(0, arr, len(items), FAKE, 64, t, 64, FAKE, 4, 16, None, None, FAKE, 1 << 40, None)

    y = FAKE + (1 << 20)
    bad = [[(100, None, 0, y, 100), (100, None, 0, y, 100)],
           [(100, None, 0, y, 200), (100, None, 0, y + 4 * 99, 200)],
           [(100, None, 0, y + 4 * 99, 200), (100, None, 0, y, 200)],
           [(100, None, 0, y, 200), (101, None, 0, y + 400, 200)],
           [(100, None, 0, y, 200), (100, None, 0, y + 400, 201)],
           [(100, y + 4, 100, y, 100)], [(100, y, 101, y, 100)],
           [(100, None, 0, y, 100), (100, y, 100, y + (1 << 20), 100)],
           [(100, y + (1 << 20), 100, y, 100), (100, None, 0, y + (1 << 20), 100)]]
    for items in bad:
        assert call(items) == INVALID, items
    if torch.cuda.is_available():
        return  # right ones would run on these addresses
    good = [[(100, None, 0, y, 200), (100, None, 0, y + 400, 200)], [(100, y, 100, y, 100)],
            [(100, y, 100, y, 100), (50, y + 1200, 50, y + 1200, 50)],
            [(100, y, 200, y, 200), (100, y + 400, 200, y + 400, 200)]]
    for items in good:
        assert call(items) == 5, items  # QMV_ERR_HIP: the launch found no device


def test_lora_workspace_and_binding():
    f = q.lora_workspace_bytes
    assert f(1, 16, 1) >= 64 and f(8, 256, 4096) >= 8 * 256 * 4096 * 4
    for bad in ((0, 16, 1), (9, 16, 1), (1, 0, 1), (1, 12, 1), (1, 264, 1), (1, 16, 0), (1, 16, 4097)):
        assert f(*bad) == 0, bad
    x, ids = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32)
    a, b = torch.zeros(3, 8, 64), torch.zeros(3, 5, 8)
    for items in ([], [(a, b, None, None)], [(a, b[:, :, :7], None, None)], [(a[0], b, None, None)],
                  [(a.long(), b, None, None)]):
        with pytest.raises(ValueError):
            q.lora(x, ids, items)


def gate(**kw):
    a = dict(scoring=0, bias=None, groups=4, top_groups=2, best=2, renorm=1, scale=1.0, x=FAKE, ldx=64, t=3, k=64,
             w=FAKE, e=32, top_k=8, gate=1, ids=FAKE, weights=FAKE, logits=None, xq=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    g = q._Gate(a["scoring"], a["bias"], a["groups"], a["top_groups"], a["best"], a["renorm"], a["scale"])
    return q.lib().qmv_router_gate(a["x"], a["ldx"], a["t"], a["k"], a["w"], a["e"], a["top_k"],
                                   ctypes.byref(g) if a["gate"] else None, a["ids"], a["weights"], a["logits"],
                                   a["xq"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(gate=None), INVALID), (dict(ids=None), INVALID),
    (dict(weights=None), INVALID), (dict(ws=None), INVALID), (dict(t=0), INVALID), (dict(k=0), INVALID),
    (dict(k=62), INVALID), (dict(ldx=60), INVALID), (dict(ldx=66), INVALID), (dict(e=0), INVALID),
    (dict(top_k=0), INVALID), (dict(top_k=17), INVALID), (dict(top_k=33, groups=1, top_groups=1), INVALID),
    (dict(xq=FAKE, k=36, ldx=36), INVALID), (dict(scoring=2), INVALID), (dict(scoring=-1), INVALID),
    (dict(renorm=2), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(groups=0), INVALID),
    (dict(groups=5), INVALID), (dict(groups=-4), INVALID), (dict(top_groups=0), INVALID), (dict(top_groups=5), INVALID),
    (dict(best=0), INVALID), (dict(best=3), INVALID), (dict(groups=32, top_groups=32), INVALID),
    (dict(t=65), UNSUPPORTED), (dict(k=(1 << 24) + 4, ldx=1 << 25), UNSUPPORTED),
    (dict(e=1028), UNSUPPORTED), (dict(top_k=17, groups=1, top_groups=1), UNSUPPORTED),
    (dict(e=130, groups=65, top_groups=65), UNSUPPORTED),
    (dict(x=FAKE + 4), MISALIGNED), (dict(w=FAKE + 8), MISALIGNED), (dict(bias=FAKE + 2), MISALIGNED),
    (dict(ids=FAKE + 1), MISALIGNED), (dict(weights=FAKE + 2), MISALIGNED), (dict(logits=FAKE + 2), MISALIGNED),
    (dict(xq=FAKE + 64), MISALIGNED), (dict(ws=FAKE + 128), MISALIGNED), (dict(wsb=q.router_gate_workspace_bytes(3, 32) - 1), WORKSPACE),
    (dict(wsb=0), WORKSPACE)])
def test_gate_refusals(change, status):
    assert gate(**change) == status


def test_gate_workspace_and_binding():
    f = q.router_gate_workspace_bytes
    assert f(3, 32) >= 256 + 3 * 32 * 8 and f(64, 1024) >= 64 * 1024 * 8
    for bad in ((0, 32), (65, 32), (1, 0), (1, 1025)):
        assert f(*bad) == 0, bad
    x, w = torch.zeros(2, 64), torch.zeros(8, 64)
    for call in (lambda: q.router_gate(x, w, 2), lambda: q.router_gate(x, w[:, :32], 2),
                 lambda: q.router_gate(x, w, 2, scoring="max")):
        with pytest.raises(ValueError):
            call()


def logprobs(**kw):
    a = dict(x=FAKE, ld=1000, t=3, v=1000, scale=1.0, given=FAKE, n=1, lp=FAKE, ent=FAKE, top=5, ids=FAKE, tl=FAKE,
             ws=None, wsb=0)
    a.update(kw)
    return q.lib().qmv_token_logprobs(a["x"], a["ld"], a["t"], a["v"], a["scale"], a["given"], a["n"], a["lp"],
                                      a["ent"], a["top"], a["ids"], a["tl"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(given=None), INVALID), (dict(lp=None), INVALID), (dict(ids=None), INVALID),
    (dict(tl=None), INVALID), (dict(n=-1), INVALID), (dict(n=0, top=0, ent=None), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(ld=999), INVALID),
    (dict(t=0), INVALID), (dict(v=0), INVALID), (dict(top=-1), INVALID), (dict(top=11, v=10), INVALID),
    (dict(t=65537), UNSUPPORTED), (dict(v=(1 << 24) + 1, ld=1 << 25), UNSUPPORTED), (dict(top=33), UNSUPPORTED),
    (dict(n=65537), UNSUPPORTED),
    (dict(x=FAKE + 2), MISALIGNED), (dict(given=FAKE + 1), MISALIGNED), (dict(lp=FAKE + 2), MISALIGNED),
    (dict(ent=FAKE + 3), MISALIGNED), (dict(ids=FAKE + 2), MISALIGNED), (dict(tl=FAKE + 1), MISALIGNED),
    (dict(ws=FAKE + 64, wsb=1 << 30), MISALIGNED), (dict(ws=FAKE, wsb=100, v=100000, ld=100000), WORKSPACE)])
def test_logprob_refusals(change, status):
    assert logprobs(**change) == status


def test_logprob_workspace_and_binding():
    f = q.token_logprobs_workspace_bytes
    assert f(1, 152064, 20) > 65536 and f(5000, 152064, 20) == 0 and f(1, 30000, 20) == 0
    for bad in ((0, 152064, 0), (1, 0, 0), (1, 152064, -1), (1, 152064, 33), (65537, 152064, 0), (1, (1 << 24) + 1, 0)):
        assert f(*bad) == 0, bad
    x = torch.zeros(2, 64)
    g = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: q.token_logprobs(x), lambda: q.token_logprobs(x, g[:1]),
                 lambda: q.token_logprobs(x, logprobs=torch.zeros(2)), lambda: q.token_logprobs(x, top_ids=g)):
        with pytest.raises(ValueError):
            call()


def test_heads_overlaps():
    """Outputs that share values with an input that is not theirs, or with each other, are refused."""
    y = FAKE + (1 << 20)
    apart = dict(k=FAKE + (1 << 16), qo=y, ko=y + (1 << 16))
    bad = [dict(qo=FAKE + 16), dict(qo=FAKE, ldqo=260), dict(ko=FAKE + (1 << 16), ldko=132), dict(ko=FAKE + (1 << 16) + 64),
           dict(qo=FAKE + (1 << 16)), dict(ko=FAKE + 1024), dict(ko=y + 1024), dict(qo=y, ko=y),
           dict(k=FAKE + 4 * 256, ldq=384, ldk=384, qo=FAKE, ldqo=384, ko=FAKE + 4 * 252, ldko=384),
           dict(k=FAKE + 4 * 256, ldq=384, ldk=384, qo=FAKE + 4 * 256, ldqo=384, ko=FAKE, ldko=384)]
    for change in bad:
        assert heads(**{**apart, **change}) == INVALID, change
    if torch.cuda.is_available():
        return  # right ones would run on these addresses
    good = [{}, dict(qo=FAKE, ko=FAKE + (1 << 16)), dict(qo=FAKE, ldqo=260, t=1), dict(k=None, kv=0, kw=None, ko=None),
            dict(k=FAKE + 4 * 256, ldq=384, ldk=384, qo=FAKE, ldqo=384, ko=FAKE + 4 * 256, ldko=384),
            dict(k=FAKE + 4 * 256, ldq=384, ldk=384, qo=y, ldqo=384, ko=y + 4 * 256, ldko=384)]
    for change in good:
        assert heads(**{**apart, **change}) == 5, change  # QMV_ERR_HIP: the launch found no device


def never_falls(sizes):
    assert all(b >= a > 0 for a, b in zip(sizes, sizes[1:])), sizes


def test_lora_workspace_covers_smaller_calls():
    """A workspace sized once, for the largest call, is enough for every smaller one."""
    f = q.lora_workspace_bytes
    for items, rank in ((1, 8), (2, 64), (3, 16), (8, 256), (5, 200)):
        never_falls([f(items, rank, t) for t in range(1, 4097)])
    for t in (1, 7, 34, 252, 700):
        for items in range(1, 9):
            never_falls([f(items, r, t) for r in range(8, 257, 8)])
        for r in (8, 16, 64, 256):
            never_falls([f(items, r, t) for items in range(1, 9)])
    # what a call takes: tiles of 32 bytes for each 64 tokens, and h of each slice of k
    for items, rank in ((1, 8), (2, 64), (3, 16), (8, 256), (5, 200)):
        for t in range(1, 4097):
            groups = items * -(-rank // 16) * max(min(t, 8), -(-t // 4))
            assert f(items, rank, t) >= -(-t // 64) * 2048 + 4 * items * rank * t * min(16, -(-512 // groups)), (items, rank, t)
    if torch.cuda.is_available():
        return  # right calls would run on these addresses
    for items, rank, most in ((2, 64, 256), (3, 16, 700), (1, 16, 64)):
        for t in range(1, most + 1):
            assert lora(items=1, t=t, rank=rank, wsb=f(items, rank, most)) == 5, (rank, t)  # found no device


def test_gate_workspace_covers_smaller_calls():
    f = q.router_gate_workspace_bytes
    for e in (1, 16, 60, 128, 256, 384, 1024):
        never_falls([f(t, e) for t in range(1, 65)])
        for t in range(1, 65):
            slices = max(1, min(8, 256 // (-(-t // 16) * -(-e // 16))))
            assert f(t, e) >= 256 + 8 * t * e * slices, (t, e)
    for t in (1, 26, 48, 64):
        never_falls([f(t, e) for e in range(1, 1025)])
    if torch.cuda.is_available():
        return
    for t in range(1, 65):
        assert gate(t=t, e=384, groups=1, top_groups=1, wsb=f(64, 384)) == 5, t


def test_logprob_workspace_covers_smaller_calls():
    f = q.token_logprobs_workspace_bytes
    assert q.MAX_SHARED_ROWS == 256 and f(257, 152064, 20) == 0
    for v in (32769, 40000, 45056, 50257, 128256, 152064, 262144, 1000003, 1 << 24):
        never_falls([f(t, v, 20) for t in range(1, 257)])
        assert len({f(64, v, n) for n in range(33)}) == 1
        for t in range(1, min(256, v // 1200) + 1):  # counters, keys and sums of a row's parts
            most = -(-v // 4096)
            parts = -(-v // (4096 * min(-(-t * most // 512), most // 4)))
            assert f(t, v, 20) >= 65536 + t * parts * (32 * 8 + 16), (t, v)
    for t in (1, 40, 256):
        never_falls([f(t, v, 0) for v in range(32769, 1 << 20, 997)])
    if torch.cuda.is_available():
        return
    for t in (*range(1, 130), 256, 300, 2000):
        assert logprobs(t=t, v=128256, ld=128256, ws=FAKE, wsb=f(128, 128256, 20)) == 5, t
