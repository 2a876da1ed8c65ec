"""The norm's, the cache's and the attention's refusals: every call here
returns from host validation, so these run without a GPU."""
import ctypes

import pytest
import torch

import quantized_decode_gemv_qmv_amd as q

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 0x10000000  # 256-byte aligned, never dereferenced by host validation
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(x=FAKE, ldx=64, res=None, ldr=0, t=2, k=64, w=FAKE, eps=1e-5, s=None, lds=0, y=None, ldy=0, xq=FAKE)
    a.update(kw)
    return q.lib().qmv_rmsnorm_quantize(a["x"], a["ldx"], a["res"], a["ldr"], a["t"], a["k"], a["w"], a["eps"],
                                        a["s"], a["lds"], a["y"], a["ldy"], a["xq"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(xq=None), INVALID), (dict(t=0), INVALID),
    (dict(k=0), INVALID), (dict(k=48, ldx=48), INVALID), (dict(ldx=60), INVALID), (dict(res=FAKE, ldr=60), INVALID),
    (dict(s=FAKE, lds=32), INVALID), (dict(y=FAKE, ldy=32), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(t=65537), UNSUPPORTED), (dict(k=65568, ldx=65568), UNSUPPORTED),
    (dict(x=FAKE + 4), MISALIGNED), (dict(ldx=65), MISALIGNED), (dict(w=FAKE + 8), MISALIGNED),
    (dict(xq=FAKE + 16), MISALIGNED), (dict(res=FAKE + 4, ldr=64), MISALIGNED), (dict(res=FAKE, ldr=66), MISALIGNED),
    (dict(s=FAKE + 4, lds=64), MISALIGNED), (dict(s=FAKE, lds=65), MISALIGNED), (dict(y=FAKE + 4, ldy=64), MISALIGNED),
    (dict(y=FAKE, ldy=65), MISALIGNED)])
def test_norm_refusals(change, status):
    assert norm(**change) == status


def kv(**kw):
    a = dict(codes=FAKE, scales=FAKE, n_blocks=9, n_kv_heads=2, head_dim=64, block_table=FAKE, table_width=4,
             seq_lens=FAKE, tok_start=None, n_seqs=3, n_tok=6, max_q=2)
    a.update({k: v for k, v in kw.items() if k in a})
    return q._Kv(**a)


CACHE = [
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(n_blocks=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=72), INVALID), (dict(table_width=0), INVALID),
    (dict(n_seqs=0), INVALID), (dict(n_tok=0), INVALID), (dict(max_q=0), INVALID), (dict(n_tok=5), INVALID),
    (dict(head_dim=272), UNSUPPORTED), (dict(n_kv_heads=1025), UNSUPPORTED), (dict(n_blocks=2**31), UNSUPPORTED),
    (dict(n_seqs=65536, n_tok=65536, max_q=1), UNSUPPORTED), (dict(n_tok=65537, tok_start=FAKE), UNSUPPORTED),
    (dict(max_q=65537, tok_start=FAKE), UNSUPPORTED), (dict(table_width=2**24 + 1), UNSUPPORTED),
    (dict(codes=FAKE + 8), MISALIGNED), (dict(scales=FAKE + 2), MISALIGNED), (dict(block_table=FAKE + 2), MISALIGNED),
    (dict(seq_lens=FAKE + 1), MISALIGNED), (dict(tok_start=FAKE + 2), MISALIGNED)]


def append(**kw):
    a = dict(k=FAKE, ldk=2048, v=FAKE, ldv=2048)
    a.update({k: v for k, v in kw.items() if k in a})
    return q.lib().qmv_kv_append(ctypes.byref(kv(**kw)), a["k"], a["ldk"], a["v"], a["ldv"], None)


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ldk=124), INVALID), (dict(ldv=124), INVALID),
    (dict(k=FAKE + 4), MISALIGNED), (dict(v=FAKE + 8), MISALIGNED), (dict(ldk=129), MISALIGNED),
    (dict(ldv=130), MISALIGNED)])
def test_append_refusals(change, status):
    assert append(**change) == status
    assert q.lib().qmv_kv_append(None, FAKE, 2048, FAKE, 2048, None) == INVALID


def attn(**kw):
    a = dict(q=FAKE, ldq=2048, n_heads=4, scale=0.125, window=0, out=FAKE, ldo=2048, xq=None, ws=None, wsb=0)
    a.update({k: v for k, v in kw.items() if k in a})
    return q.lib().qmv_kv_attn(ctypes.byref(kv(**kw)), a["q"], a["ldq"], a["n_heads"], a["scale"], a["window"],
                               a["out"], a["ldo"], a["xq"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ldq=252), INVALID), (dict(ldo=252), INVALID),
    (dict(n_heads=0), INVALID), (dict(n_heads=3), INVALID), (dict(window=-1), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(xq=FAKE, head_dim=80), INVALID), (dict(n_heads=16386), UNSUPPORTED),
    (dict(q=FAKE + 4), MISALIGNED), (dict(ldq=257), MISALIGNED), (dict(out=FAKE + 8), MISALIGNED),
    (dict(ldo=258), MISALIGNED), (dict(xq=FAKE + 64), MISALIGNED),
    # more workgroups than one launch has
    (dict(n_seqs=65535, n_kv_heads=1024, n_heads=1024, n_tok=65535, max_q=1, ldq=65536, ldo=65536), UNSUPPORTED),
    (dict(table_width=64, ws=FAKE, wsb=1000), WORKSPACE),
    (dict(table_width=64, ws=FAKE + 64, wsb=1 << 40), MISALIGNED)])
def test_attn_refusals(change, status):
    assert attn(**change) == status
    assert q.lib().qmv_kv_attn(None, FAKE, 2048, 4, 0.1, 0, FAKE, 2048, None, None, 0, None) == INVALID


def test_workspace_sizes():
    f = q.kv_attn_workspace_bytes
    assert f(1, 1, 1, 32, 8, 128, 64) > 65536
    assert f(48, 48, 1, 64, 8, 128, 64) > 65536  # shared by length
    assert f(200, 200, 1, 64, 8, 128, 64) == 0   # enough sequences: none is shared
    assert f(1, 1, 1, 32, 8, 128, 1) == 0     # one block has nothing to share
    for bad in ((0, 1, 1, 32, 8, 128, 64), (1, 0, 1, 32, 8, 128, 64), (1, 1, 0, 32, 8, 128, 64),
                (1, 1, 1, 33, 8, 128, 64), (1, 1, 1, 32, 0, 128, 64), (1, 1, 1, 32, 8, 100, 64),
                (1, 1, 1, 32, 8, 128, 0), (1, 1, 1, 16392, 8, 128, 64)):
        assert f(*bad) == 0, bad


def test_binding_refuses_host_tensors_and_shapes():
    x, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError):
        q.rmsnorm_quantize(x, w)
    with pytest.raises(ValueError):
        q.rmsnorm_quantize(x.view(1, 2, 64), w)
    codes, scales = torch.zeros(3, 2, 1, 64 * 64, dtype=torch.int8), torch.zeros(3, 2, 1)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.kv_append(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), codes, scales, table, lens)
    with pytest.raises(ValueError):
        q.kv_append(torch.zeros(1, 64), torch.zeros(1, 64), codes, scales, table, lens)
    with pytest.raises(ValueError):
        q.kv_attn(torch.zeros(1, 2, 64), codes, scales, table, lens)
    with pytest.raises(ValueError):
        q.kv_attn(torch.zeros(1, 64), codes, scales, table, lens)


def test_more_threads_than_a_launch_has():
    """Groups of eight waves: 2^23 of them are 2^32 threads."""
    big = dict(n_seqs=65535, n_tok=65535, max_q=1, n_heads=10240, ldq=10240 * 64, ldo=10240 * 64)
    assert attn(n_kv_heads=160, **big) == UNSUPPORTED


@pytest.mark.parametrize("n_tok,k", [(1, 32), (3, 96), (2, 4096)])
def test_act_fields_of_a_buffer_without_padding(n_tok, k):
    """The fields end before act_bytes; a buffer that ends with them holds
    them all, one byte less does not."""
    _, at = q.act_offsets(n_tok, k)
    end = at + 4 * n_tok * (k // 32)
    buf = torch.arange(q.act_bytes(n_tok, k)).to(torch.uint8)
    want = q.act_fields(buf, n_tok, k)
    for part in (buf[:end].clone(), buf[:end]):
        assert all(torch.equal(a.view(torch.int8), b.view(torch.int8)) for a, b in zip(q.act_fields(part, n_tok, k), want))
    with pytest.raises((ValueError, RuntimeError)):
        q.act_fields(buf[:end - 1], n_tok, k)
