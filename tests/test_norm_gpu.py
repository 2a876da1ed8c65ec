"""qmv_rmsnorm_quantize against its definition in 64 bits and the oracle.

r = x + residual is one fp32 addition: exact.  y = (r inv) weight takes three
roundings to fp32 (inv, and two products), each off by at most 2^-24 of the
value: |y - y64| <= 3.01 2^-24 |y64|, plus one step of the subnormals for
values that end there.  The Q8 blocks are an integer decision on y, so they
are compared bit for bit with the oracle's quantization of the GPU's y."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import gpu, need_gpu, say, to_dev, x_host

pytestmark = gpu

EPS32 = 2.0 ** -24
EPS = 1e-5


def check(qmv, x, w, res=None, eps=EPS, what="", **kw):
    t, k = x.shape
    y = torch.full((t, k), 7.0, device="cuda")
    r, xq = qmv.rmsnorm_quantize(to_dev(x), to_dev(w), eps, residual=None if res is None else to_dev(res), y_out=y, **kw)
    r_ref = x if res is None else x + res
    assert np.array_equal(r.cpu().numpy(), r_ref), what
    r64 = r_ref.astype(np.float64)
    y64 = r64 / np.sqrt((r64 * r64).mean(1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64)
    y_h = y.cpu().numpy()
    assert np.all(np.abs(y_h - y64) <= 3.01 * EPS32 * np.abs(y64) + 2.0 ** -149), what
    for got, want in zip(qmv.act_fields(xq, t, k), oracle.quantize_act(y_h)):
        assert np.array_equal(got.cpu().numpy(), want), what
    return y_h


# widths of every way a row is split over threads (one wave, 256, 512 and 1024
# threads, by width alone), with a ragged last vector and the largest; row
# counts from one to more than the device holds at once
@pytest.mark.parametrize("t,k", [(1, 32), (3, 96), (1, 4096), (5, 4128), (16, 5120), (2, 14336), (3, 16416), (2, 65536),
                                 (1, 49184), (1025, 32), (1030, 992), (1024, 4096), (513, 4128), (515, 16384),
                                 (2050, 2080)])
@pytest.mark.parametrize("residual", [False, True])
def test_shapes(t, k, residual):
    qmv = need_gpu()
    say(f"norm {t}x{k} residual={residual}")
    x = x_host(t, k, f"norm/x{t}x{k}")
    res = x_host(t, k, f"norm/r{t}x{k}") * np.float32(5.0) if residual else None
    w = 1.0 + x_host(1, k, f"norm/w{k}")[0] * np.float32(0.3)
    check(qmv, x, w, res, what=f"{t}x{k}")


def test_values():
    """Rows of zeros, a row with one value, large and small rows side by side
    (their squares leave fp32's range), weights of zero and below it."""
    qmv = need_gpu()
    k = 256
    x = x_host(7, k, "norm/values")
    x[0] = 0.0
    x[1] = 0.0
    x[1, 77] = 3.0
    x[2] *= np.float32(1e30)
    x[3] *= np.float32(1e-25)
    x[4, 32:64] = 0.0
    w = x_host(1, k, "norm/vw")[0]
    w[5:40] = 0.0
    y = check(qmv, x, w, what="values")
    assert not y[0].any() and not y[4, 32:64].any()
    check(qmv, x, w, eps=1e-20, what="small eps")


def test_strides_and_in_place():
    qmv = need_gpu()
    t, k = 6, 160
    say("norm strided, in place")
    wide = to_dev(x_host(t, 3 * k, "norm/wide"))
    x, res = wide[:, k:2 * k], wide[:, 2 * k:]
    w = to_dev(x_host(1, k, "norm/sw")[0])
    r0, q0 = qmv.rmsnorm_quantize(x.contiguous(), w, EPS, residual=res.contiguous())
    out = torch.full((t, 2 * k), 3.0, device="cuda")
    r1, q1 = qmv.rmsnorm_quantize(x, w, EPS, residual=res, sum_out=out[:, :k], y_out=out[:, k:])
    assert r1.data_ptr() == out.data_ptr() and torch.equal(r0, out[:, :k])
    for a, b in zip(qmv.act_fields(q0, t, k), qmv.act_fields(q1, t, k)):
        assert torch.equal(a, b)
    for target in ("x", "residual"):
        c = wide.clone()
        xs, rs = c[:, k:2 * k], c[:, 2 * k:]
        r2, q2 = qmv.rmsnorm_quantize(xs, w, EPS, residual=rs, sum_out=xs if target == "x" else rs,
                                      y_out=rs if target == "x" else xs)
        assert torch.equal(r2, r0) and torch.equal(c[:, :k], wide[:, :k])
        assert torch.equal(rs if target == "x" else xs, out[:, k:])
        for a, b in zip(qmv.act_fields(q0, t, k), qmv.act_fields(q2, t, k)):
            assert torch.equal(a, b)
    # without a residual x itself comes back, or its copy in sum_out
    r3, _ = qmv.rmsnorm_quantize(x, w, EPS)
    assert r3.data_ptr() == x.data_ptr()
    copy = torch.empty(t, k, device="cuda")
    assert torch.equal(qmv.rmsnorm_quantize(x, w, EPS, sum_out=copy)[0], x)


def test_rows_do_not_depend_on_each_other_or_the_split():
    """A row gives the same bits alone and among many (other thread counts)."""
    qmv = need_gpu()
    for k in (2048, 4096, 16384):
        t = 1030
        x = torch.randn(t, k, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        w = torch.rand(k, device="cuda") + 0.5
        _, many = qmv.rmsnorm_quantize(x, w, EPS)
        for row in (0, 517, t - 1):
            _, one = qmv.rmsnorm_quantize(x[row], w, EPS)
            for a, b in zip(qmv.act_fields(many, t, k), qmv.act_fields(one, 1, k)):
                assert torch.equal(a[row], b[0]), (k, row)


def test_a_row_without_its_dimension():
    """A 1-D x takes 1-D residuals and outputs, and may be its own output."""
    qmv = need_gpu()
    say("norm 1-D")
    k = 96
    x, res, w = (to_dev(x_host(1, k, f"norm/1d{i}")[0]) for i in range(3))
    r0, q0 = qmv.rmsnorm_quantize(x.view(1, k), w, EPS, residual=res.view(1, k), y_out=(y0 := torch.empty(1, k, device="cuda")))
    s, y = torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    r, q = qmv.rmsnorm_quantize(x, w, EPS, residual=res, sum_out=s, y_out=y)
    assert torch.equal(s, r0[0]) and torch.equal(y, y0[0]) and r.data_ptr() == s.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(qmv.act_fields(q, 1, k), qmv.act_fields(q0, 1, k)))
    c = x.clone()
    qmv.rmsnorm_quantize(c, w, EPS, residual=res, sum_out=c)
    assert torch.equal(c, r0[0])
