"""Oracle pins of the layer norm and of the 4-bit format: worked values, the norm's gradient against
differences, and the host arithmetic and refusals of their entry points (no GPU)."""
import os

import numpy as np
import pytest
import torch

from lm_head_cross_pg_amd import abi, build
from oracle import oracle as ora

P = 0x10000      # a 16-byte aligned "device" address: validation never reads it
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        build.build()
    return abi.load()


def no_gpu():
    return not torch.cuda.is_available()


# ------------------------------------------------------------------------------------------ format
def test_levels_ties_and_saturation():
    """At scale 1 (largest magnitude in [3.5, 7)): every border between levels goes to the even code, the
    values next to it to their own side, and everything from 5 on to 6."""
    x = np.zeros((1, 32))
    row = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, 0.74, 1.26, 1.74, 2.51, 3.49, 5.01, 6.99, -0.25, -5.0, -6.5]
    x[0, :len(row)] = row
    val, code, e = ora.quantize_rows_mx4(x)
    assert e[0, 0] == 0
    want = [0, 1, 1, 2, 2, 4, 4, 0.5, 0.5, 1.5, 1.5, 3, 3, 6, 6, -0.0, -4, -6]
    np.testing.assert_array_equal(val[0, :len(row)], want)
    assert code[0, 15] == 8 and code[0, 16] == 8 + 6 and code[0, 0] == 0 and code[0, 14] == 7


def test_block_exponents():
    tops = {7.0: 1, 6.999: 0, 3.5: 0, 3.499: -1, 1.0: -2, 2.0 ** 100: 98, 2.0 ** 127: 125, 7 * 2.0 ** 125: 125, 1.99 * 2.0 ** 127: 125, 2.0 ** -125: -127, 2.0 ** -140: -127, 0.0: -127}
    x = np.zeros((len(tops), 32))
    x[:, 3] = list(tops)
    _, _, e = ora.quantize_rows_mx4(x)
    np.testing.assert_array_equal(e[:, 0], list(tops.values()))
    bad = np.zeros((2, 40))
    bad[0, 1], bad[1, 39] = np.nan, -np.inf
    val, code, e = ora.quantize_rows_mx4(bad)
    assert np.isnan(val[0, :32]).all() and (val[0, 32:] == 0).all() and e[0, 0] == 128 and e[0, 1] == -127
    assert np.isnan(val[1, 32:]).all() and (val[1, :32] == 0).all() and not code.any()


def test_row_bytes(lib):
    for D, cb, sb in ((1, 32, 16), (64, 32, 16), (65, 64, 16), (512, 256, 16), (513, 288, 32), (1 << 20, 1 << 19, 1 << 15)):
        assert (abi.pg_mx4_code_bytes(D), abi.pg_mx4_scale_bytes(D)) == (cb, sb)
    for D in (0, -5, (1 << 20) + 1):
        with pytest.raises(abi.PgError, match="PG_ERR_SHAPE"):
            abi.pg_mx4_code_bytes(D)
        with pytest.raises(abi.PgError, match="PG_ERR_SHAPE"):
            abi.pg_mx4_scale_bytes(D)


# -------------------------------------------------------------------------------------------- norm
def test_norm_worked_row():
    """x = (1, 2, 3, 4): mean 2.5, variance 1.25; eps 0, weight 2, bias 1."""
    y = ora.layer_norm([[1.0, 2.0, 3.0, 4.0]], np.full(4, 2.0), np.ones(4), 0.0)
    np.testing.assert_allclose(y[0], 1 + 2 * np.array([-1.5, -0.5, 0.5, 1.5]) / np.sqrt(1.25), rtol=1e-15)


@pytest.mark.parametrize("masked", [False, True])
def test_norm_gradient_against_differences(masked):
    """Central differences of f = sum(dy * y): error of order h^2 f''' / 6 with third derivatives of order
    1 here, plus the rounding 1e-16 |f| / h: below 1e-8 at h = 1e-5."""
    rng = np.random.default_rng(2)
    T, D, eps, h = 3, 7, 1e-3, 1e-5
    x, dy, w, b = rng.standard_normal((T, D)), rng.standard_normal((T, D)), 1 + rng.random(D), rng.random(D)
    mask = np.array([1, 0, 1], np.uint8) if masked else None
    on = np.ones(T, bool) if mask is None else mask != 0
    f = lambda x, w, b: float(np.sum((dy * ora.layer_norm(x, w, b, eps))[on]))  # noqa: E731
    dx, dw, db = ora.layer_norm_backward(x, w, dy, eps, mask)
    for got, args, k in ((dx, (x, w, b), 0), (dw, (x, w, b), 1), (db, (x, w, b), 2)):
        num = np.zeros_like(got)
        for i in np.ndindex(got.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][i] += h
            down[k][i] -= h
            num[i] = (f(*up) - f(*down)) / (2 * h)
        np.testing.assert_allclose(got, num, atol=1e-8)


# ---------------------------------------------------------------------------------------- refusals
def norm(lib, **kw):
    a = dict(x=P, dx=0, w=P, b=P, m=None, T=256, D=64, eps=1e-5, y=P, dy=0) | kw
    return lib.pg_layernorm_fwd(a["x"], a["dx"], a["w"], a["b"], a["m"], a["T"], a["D"], a["eps"], a["y"], a["dy"], None)


def norm4(lib, **kw):
    a = dict(x=P, dx=0, w=P, b=P, m=None, T=256, D=64, eps=1e-5, c=P, s=P) | kw
    return lib.pg_layernorm_fwd_mx4(a["x"], a["dx"], a["w"], a["b"], a["m"], a["T"], a["D"], a["eps"], a["c"], a["s"],
                                    None)


def grad(lib, **kw):
    a = dict(x=P, tx=0, w=P, m=None, dy=P, tdy=1, T=256, D=64, eps=1e-5, dx=P, tdx=1, dw=P, db=P, ws=P, wsb=BIG) | kw
    return lib.pg_layernorm_bwd(a["x"], a["tx"], a["w"], a["m"], a["dy"], a["tdy"], a["T"], a["D"], a["eps"], a["dx"],
                                a["tdx"], a["dw"], a["db"], a["ws"], a["wsb"], None)


def quant(lib, **kw):
    a = dict(x=P, t=0, m=None, T=256, D=64, c=P, s=P) | kw
    return lib.pg_quantize_mx4(a["x"], a["t"], a["m"], a["T"], a["D"], a["c"], a["s"], None)


def dequant(lib, **kw):
    a = dict(c=P, s=P, T=256, D=64, out=P, t=0) | kw
    return lib.pg_dequantize_mx4(a["c"], a["s"], a["T"], a["D"], a["out"], a["t"], None)


def head(lib, **kw):
    a = dict(hc=P, hs=P, ec=P, es=P, y=P, m=None, T=256, D=64, V=512, c=30.0, nats=P, lse=P, ws=P, wsb=BIG) | kw
    return lib.pg_lmhead_ce_fwd_mx4(a["hc"], a["hs"], a["ec"], a["es"], a["y"], a["m"], a["T"], a["D"], a["V"], a["c"],
                                    a["nats"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [norm, norm4, grad, quant, dequant, head])
def test_refused_shapes(lib, call):
    for kw in (dict(T=-1), dict(T=(1 << 31) - 255), dict(D=0), dict(D=(1 << 20) + 1)):
        assert call(lib, **kw) == -2, kw
    if no_gpu():
        assert call(lib) == -7 and call(lib, T=(1 << 31) - 256) == -7   # valid: only the device is missing


@pytest.mark.parametrize("call,required,aligned", [
    (norm, "x y", "x w b m y"), (norm4, "x c s", "x w b m c s"), (grad, "x dy ws", "x w m dy dx dw db ws"),
    (quant, "x c s", "x m c s"), (dequant, "c s out", "c s out"),
    (head, "hc hs ec es y nats ws", "hc hs ec es y m nats lse ws")])
def test_refused_pointers(lib, call, required, aligned):
    for k in required.split():
        assert call(lib, **{k: None}) == -1, k
    for k in aligned.split():
        assert call(lib, **{k: P + 8}) == -6, k
    if no_gpu():
        for k in set(aligned.split()) - set(required.split()):
            assert call(lib, **{k: None}) == -7, k   # the others may be left out


def test_refused_numbers_and_types(lib):
    for eps in (-1e-5, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == norm4(lib, eps=eps) == grad(lib, eps=eps) == -4
    assert head(lib, c=-1.0) == head(lib, c=float("inf")) == -4
    assert head(lib, V=0) == head(lib, V=(1 << 20) + 1) == -2
    assert norm(lib, dx=2) == norm(lib, dy=7) == norm4(lib, dx=2) == quant(lib, t=2) == dequant(lib, t=-1) == -3
    assert grad(lib, tx=2) == grad(lib, tdy=2) == grad(lib, tdx=2) == -3
    for call, op, T, D, V in ((grad, abi.PG_OP_LN_BWD, 256, 64, 1), (grad, abi.PG_OP_LN_BWD, 256, 4096, 1),
                              (head, abi.PG_OP_FWD_MX4, 256, 64, 512)):
        need = abi.workspace_bytes(op, T, D, V)
        assert need > 0 and call(lib, T=T, D=D, wsb=need - 1) == -5
    if no_gpu():
        assert norm(lib, T=0, x=None, y=None) == -7   # no rows: nothing to point at


def test_binding_refuses_mismatched_tensors(monkeypatch):
    """Shapes and types are checked before the library is called."""
    monkeypatch.setattr(abi, "load", lambda *a, **k: pytest.fail("the library was called"))
    T, D, V = 8, 100, 16
    x, y, w, m = torch.zeros(T, D), torch.zeros(T, D), torch.zeros(D), torch.ones(T, dtype=torch.uint8)
    c, s = torch.zeros((T, 64), dtype=torch.uint8), torch.zeros((T, 16), dtype=torch.uint8)
    ec, es = torch.zeros((V, 64), dtype=torch.uint8), torch.zeros((V, 16), dtype=torch.uint8)
    t, n = torch.zeros(T, dtype=torch.int32), torch.zeros(T)
    cases = [
        (lambda: abi.pg_layernorm_fwd(x.double(), w, w, None, 1e-5, y), "x has dtype"),
        (lambda: abi.pg_layernorm_fwd(x.t(), w, w, None, 1e-5, y), "x must be contiguous"),
        (lambda: abi.pg_layernorm_fwd(x, w[:3], w, None, 1e-5, y), "weight has 3 elements"),
        (lambda: abi.pg_layernorm_fwd(x, w, w.double(), None, 1e-5, y), "bias has dtype"),
        (lambda: abi.pg_layernorm_fwd(x, w, w, m[:2], 1e-5, y), "score_mask has 2"),
        (lambda: abi.pg_layernorm_fwd(x, w, w, None, 1e-5, y[:4]), "y has shape"),
        (lambda: abi.pg_layernorm_fwd(x, w, w, None, 1e-5, y), "is on cpu"),
        (lambda: abi.pg_layernorm_fwd_mx4(x, w, w, None, 1e-5, c[:, :32].contiguous(), s), "codes has shape"),
        (lambda: abi.pg_layernorm_fwd_mx4(x, w, w, None, 1e-5, c, s[:4]), "scales has shape"),
        (lambda: abi.pg_layernorm_bwd(x, w, None, y[:, :5].contiguous(), 1e-5, y, w, w), "dy has shape"),
        (lambda: abi.pg_layernorm_bwd(x, w, None, y, 1e-5, y.double(), w, w), "dx has dtype"),
        (lambda: abi.pg_layernorm_bwd(x, w, None, y, 1e-5, y, w[:9], w), "dweight has 9"),
        (lambda: abi.pg_layernorm_bwd(x, w, None, y, 1e-5, y, w, w), "is on cpu"),
        (lambda: abi.pg_quantize_mx4(x, None, c.to(torch.int8), s), "codes has dtype"),
        (lambda: abi.pg_quantize_mx4(x, None, c, s.t()), "scales has shape"),
        (lambda: abi.pg_dequantize_mx4(c, s[:, :8].contiguous(), y), "scales has shape"),
        (lambda: abi.pg_lmhead_ce_fwd_mx4(c, s, ec, es, t, None, 200, 30.0, n), "hidden_codes has shape"),
        (lambda: abi.pg_lmhead_ce_fwd_mx4(c, s, ec, es[:3], t, None, D, 30.0, n), "embed_scales has shape"),
        (lambda: abi.pg_lmhead_ce_fwd_mx4(c, s, ec, es, t.long(), None, D, 30.0, n), "target has dtype"),
        (lambda: abi.pg_lmhead_ce_fwd_mx4(c, s, ec, es, t, None, D, 30.0, n[:2]), "nats has 2"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()
