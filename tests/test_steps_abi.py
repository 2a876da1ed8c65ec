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
