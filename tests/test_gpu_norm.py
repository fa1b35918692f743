"""Layer norm forward and backward on the GPU against the float64 oracle.

Tolerances (u = 2^-24, half a float32 step; half a bf16 step is 2^-8, relative):
  forward   the values are formed in float64 and rounded to float32, then to y's type: half a step of y's
            type, with 2^-14 of that for the first rounding, plus the float64 error: 2^-53 times a few
            hundred operations on terms of size |xh w| + |b|, below 1e-12 of it
  backward  in float32 from float64 statistics. xh has three roundings, g one; a sum over D adds
            n = 8 K + 6 <= 38 terms one after another (8 K in a lane, 6 exchanges), and errors of at most
            n + 4 half steps of the sum of magnitudes: with A1 = mean |g|, A2 = mean |g xh|,
            |error of dx| <= u r (6 (|g| + |c1| + |xh c2|) + 44 A1 + 48 |xh| A2), and half a step of
            dx's type of |dx|
  sums      dw and db add at most R rows in a lane, 2 exchanges and 16 waves in float32, the rest in
            float64: (R + 24) u of the sum of magnitudes (xh's three roundings and the product's among
            the 24) and u of the result
"""
import numpy as np
import pytest
import torch

from lm_head_cross_pg_amd import abi
from oracle import oracle as ora
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def states(T, D, dtype, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, D), generator=g) * torch.exp(0.4 * torch.randn(D, generator=g)) + offset
    return x.to(dtype), 1 + 0.1 * torch.randn(D, generator=g), 0.1 * torch.randn(D, generator=g)


def mask_of(kind, T, seed=0):
    if kind is None:
        return None
    m = (torch.rand(T, generator=torch.Generator().manual_seed(seed)) < 0.4).to(torch.uint8)
    if kind == "empty":
        m[:] = 0
    if kind == "one":
        m[:] = 0
        m[T // 2] = 1
    return m


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def f64(t):
    return t.double().cpu().numpy()


def check_forward(x, w, b, mask, eps, dtype_y):
    T, D = x.shape
    print(f"[case] norm T={T} D={D} {x.dtype}->{dtype_y} w={w is not None} b={b is not None} "
          f"mask={None if mask is None else int(mask.sum())}", flush=True)
    y = torch.full((T, D), 777.0, dtype=dtype_y, device="cuda")
    xd, wd, bd, md = cuda(x, w, b, mask)
    abi.pg_layernorm_fwd(xd, wd, bd, md, eps, y)
    torch.cuda.synchronize()
    got = f64(y)
    ref = ora.layer_norm(f64(x), None if w is None else f64(w), None if b is None else f64(b), eps)
    size = np.abs(ora.layer_norm(f64(x), None, None, eps)) * (1.0 if w is None else np.abs(f64(w)))
    if b is not None:
        size = size + np.abs(f64(b))
    on = np.ones(T, bool) if mask is None else mask.numpy() != 0
    tol = HALF[dtype_y] * (1 + 2.0 ** -14) * np.abs(ref) + 1e-12 * size
    if dtype_y == BF:
        tol += U * np.abs(ref)
    assert np.all(np.abs(got - ref)[on] <= tol[on])
    assert np.all(got[~on] == 776.0 if dtype_y == BF else got[~on] == 777.0)   # bf16 holds 776, not 777
    return y


@pytest.mark.parametrize("D", [1, 2, 7, 8, 31, 64, 100, 128, 129, 255, 256, 257, 511, 512, 1001, 1024, 1025, 2047, 2048,
                               2049, 2560, 4100, 8192, 8193, 9001])
@pytest.mark.parametrize("tx,ty", [(BF, BF), (F, F), (F, BF), (BF, F)])
def test_forward_widths_and_types(D, tx, ty):
    x, w, b = states(5, D, tx, D)
    check_forward(x, w, b, None, 1e-5, ty)


@pytest.mark.parametrize("T", [1, 3, 4, 17, 1000, 9000])
@pytest.mark.parametrize("kind", [None, "random", "empty", "one"])
@pytest.mark.parametrize("D", [40, 200, 512, 3001])
def test_forward_rows_and_masks(T, kind, D):
    x, w, b = states(T, D, BF, T)
    check_forward(x, w, b, mask_of(kind, T), 1e-5, BF)


def test_forward_without_parameters_and_bool_mask():
    x, w, b = states(33, 96, F, 1)
    check_forward(x, None, None, None, 1e-5, F)
    check_forward(x, w, None, None, 0.0, F)
    check_forward(x, None, b, mask_of("random", 33).bool(), 1e-3, F)


def test_forward_far_mean_and_extreme_values():
    """A mean 10^4 deviations away keeps its digits (the input's own are all there are); values near the
    end of float32 do not overflow; equal values give the bias."""
    x, w, b = states(9, 512, F, 2, offset=1e4)
    check_forward(x, w, b, None, 1e-5, F)
    check_forward(x * 2.0 ** 110, w, b, None, 1e-5, F)
    check_forward(torch.full((3, 130), 2.5), *states(3, 130, F, 3)[1:], None, 1e-5, F)
    check_forward(torch.full((2, 1), -4.0), torch.tensor([3.0]), torch.tensor([0.5]), None, 1e-5, F)


def test_forward_nan_and_infinite_rows_stay_alone():
    for D in (64, 600, 2500):
        x, w, b = states(6, D, F, 4)
        good = check_forward(x.clone(), w, b, None, 1e-5, F)
        x[1, 3], x[4, D - 1] = float("nan"), float("inf")
        y = torch.empty_like(x).cuda()
        abi.pg_layernorm_fwd(*cuda(x, w, b), None, 1e-5, y)
        assert torch.isnan(y[1]).all() and torch.isnan(y[4]).all()
        assert torch.equal(y[[0, 2, 3, 5]], good[[0, 2, 3, 5]])


# -------------------------------------------------------------------------------------- backward
def rows_per_lane(T, D):
    """Rows a lane adds in float32, at most: the launch has at most 256 workgroups of 4 waves or more."""
    per = 4 * (4 if D <= 128 else 2 if D <= 256 else 1)
    return max(1, -(-T // (min(256, -(-T // per)) * per)))


def check_backward(x, w, dy, mask, eps=1e-5, dtype_dx=F, want=("dx", "dw", "db")):
    T, D = x.shape
    print(f"[case] norm backward T={T} D={D} {x.dtype},{dy.dtype}->{dtype_dx} w={w is not None} "
          f"mask={None if mask is None else int(mask.sum())} {want}", flush=True)
    xd, wd, md, dyd = cuda(x, w, mask, dy)
    dx = torch.full((T, D), float("nan"), dtype=dtype_dx, device="cuda") if "dx" in want else None
    dw, db = (torch.full((D,), float("nan"), device="cuda") if k in want else None for k in ("dw", "db"))
    abi.pg_layernorm_bwd(xd, wd, md, dyd, eps, dx, dw, db)
    torch.cuda.synchronize()
    X, DY, W = f64(x), f64(dy), np.ones(D) if w is None else f64(w)
    on = np.ones(T, bool) if mask is None else mask.numpy() != 0
    rdx, rdw, rdb = ora.layer_norm_backward(X, W, DY, eps, None if mask is None else mask.numpy())
    d = X - X.mean(1, keepdims=True)
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    xh, g = d * r, DY * W
    c1, c2 = np.abs(g.mean(1, keepdims=True)), np.abs((g * xh).mean(1, keepdims=True))
    tol = U * r * (6 * (np.abs(g) + c1 + np.abs(xh) * c2) + 44 * np.abs(g).mean(1, keepdims=True)
                   + 48 * np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True)) + HALF[dtype_dx] * np.abs(rdx) + 1e-40
    if dx is not None:
        got = f64(dx)
        assert np.all(got[~on] == 0)
        assert np.all(np.abs(got - rdx)[on] <= tol[on])
    n = rows_per_lane(T, D) + 24
    for got, ref, mag in ((dw, rdw, np.abs(DY * xh)[on].sum(0)), (db, rdb, np.abs(DY)[on].sum(0))):
        if got is not None:
            assert np.all(np.abs(f64(got) - ref) <= n * U * mag + U * np.abs(ref) + 1e-40)
    return dx, dw, db


def gradients(T, D, dtype, seed):
    return torch.randn((T, D), generator=torch.Generator().manual_seed(seed + 77)).to(dtype) / 64


@pytest.mark.parametrize("D", [1, 2, 7, 8, 31, 64, 129, 255, 257, 512, 1001, 1024, 2047, 2048, 2049, 2560, 4100, 8192, 8193])
@pytest.mark.parametrize("tx,ty,tdx", [(BF, F, F), (BF, BF, BF), (F, F, BF), (F, BF, F)])
def test_backward_widths_and_types(D, tx, ty, tdx):
    x, w, _ = states(6, D, tx, D)
    check_backward(x, w, gradients(6, D, ty, D), None, dtype_dx=tdx)


@pytest.mark.parametrize("T", [1, 2, 15, 700, 9001])
@pytest.mark.parametrize("kind", [None, "random", "empty", "one"])
@pytest.mark.parametrize("D", [24, 200, 512, 2600])
def test_backward_rows_and_masks(T, kind, D):
    x, w, _ = states(T, D, BF, T)
    check_backward(x, w, gradients(T, D, F, T), mask_of(kind, T))


def test_backward_other_types_and_missing_outputs():
    x, w, _ = states(40, 300, BF, 5)
    for tx in (BF, F):
        for ty in (BF, F):
            for tdx in (BF, F):
                check_backward(x.to(tx), w, gradients(40, 300, ty, 5), None, dtype_dx=tdx)
                check_backward(x.to(tx).repeat(1, 8), w.repeat(8), gradients(40, 2400, ty, 5), None, dtype_dx=tdx)
    for D in (300, 2400):
        x, w, _ = states(40, D, BF, 6)
        dy = gradients(40, D, F, 6)
        full = check_backward(x, None, dy, None)
        for want in (("dx",), ("dw",), ("db",), ("dw", "db"), ("dx", "db")):
            part = check_backward(x, None, dy, None, want=want)
            for a, b in zip(full, part):
                assert b is None or torch.equal(a, b)


def test_backward_no_rows():
    for D in (64, 3000):
        w = torch.ones(D, device="cuda")
        x = torch.empty((0, D), device="cuda")
        dw, db = torch.full((D,), 5.0, device="cuda"), torch.full((D,), 5.0, device="cuda")
        abi.pg_layernorm_bwd(x, w, None, x, 1e-5, x.clone(), dw, db)
        assert not dw.any() and not db.any()
        abi.pg_layernorm_fwd(x, w, w, None, 1e-5, x.clone())


def test_backward_nan_rows():
    for D in (96, 2100):
        x, w, _ = states(5, D, F, 7)
        dy = gradients(5, D, F, 7)
        x[1, 2], dy[3, 9] = float("nan"), float("inf")
        dx, dw, db = (torch.empty(s, device="cuda") for s in ((5, D), (D,), (D,)))
        abi.pg_layernorm_bwd(*cuda(x, w), None, dy.cuda(), 1e-5, dx, dw, db)
        # an infinite dy makes the means of its row infinite: -inf where the sign of xh lets it, else NaN
        assert torch.isnan(dx[1]).all() and not torch.isfinite(dx[3]).any() and torch.isfinite(dx[[0, 2, 4]]).all()
        assert torch.isnan(dw).all() and torch.isfinite(db).sum() == D - 1
        mask = torch.tensor([1, 0, 1, 0, 1], dtype=torch.uint8, device="cuda")
        abi.pg_layernorm_bwd(*cuda(x, w), mask, dy.cuda(), 1e-5, dx, dw, db)   # unscored: they do not matter
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
        assert not dx[[1, 3]].any()


def test_gradient_against_differences():
    """f = sum(dy y) with the GPU's own forward in float32: a step h moves f by h dx, f's own rounding is
    u times the sum of its terms' magnitudes, and the curvature costs about h^2 per term."""
    T, D, eps, h = 4, 48, 1e-2, 2.0 ** -7
    x, w, b = states(T, D, F, 8)
    dy = gradients(T, D, F, 8)
    dx, dw, db = check_backward(x, w, dy, None, eps)

    def f(x, w, b):
        y = torch.empty((T, D), device="cuda")
        abi.pg_layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), None, eps, y)
        return float((y.double().cpu() * dy.double()).sum())

    noise = 4 * U * float(dy.abs().sum()) / h + 40 * h * h * float(dy.abs().max())
    for k, got in ((0, dx), (1, dw), (2, db)):
        for i in ((0, 0), (1, 5), (3, 47)) if k == 0 else ((0,), (17,), (47,)):
            up, down = [t.clone() for t in (x, w, b)], [t.clone() for t in (x, w, b)]
            up[k][i] += h
            down[k][i] -= h
            assert abs((f(*up) - f(*down)) / (2 * h) - float(got[i])) <= noise


def test_repeatable_on_another_stream_and_in_a_graph():
    """The same bits each time: on a side stream, and replayed from a graph with eager work between."""
    T, D = 3000, 512
    x, w, b = states(T, D, BF, 9)
    dy = gradients(T, D, F, 9)
    xd, wd, bd, dyd = cuda(x, w, b, dy)
    y, dx, dw, db = (torch.empty(s, device="cuda") for s in ((T, D), (T, D), (D,), (D,)))
    ws = torch.empty(abi.workspace_bytes(abi.PG_OP_LN_BWD, T, D, 1), dtype=torch.uint8, device="cuda")

    def step():
        abi.pg_layernorm_fwd(xd, wd, bd, None, 1e-5, y)
        abi.pg_layernorm_bwd(xd, wd, None, dyd, 1e-5, dx, dw, db, ws)

    step()
    first = [t.clone() for t in (y, dx, dw, db)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (y, dx, dw, db):
            t.fill_(float("nan"))
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in (y, dx, dw, db):
            t.fill_(float(k))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw, db)))
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("D", [96, 512, 2600])
def test_two_calls_at_once(D):
    """Forward and backward on two streams with nothing between them, workspaces of their own (one given, one
    allocated by the call on a stream that is not the current one): the bits of the calls one by one."""
    T = 4000
    ins = []
    for seed in (20, 21):
        x, w, b = states(T, D, BF, seed)
        ins.append(cuda(x, w, b, gradients(T, D, F, seed)))

    def run(i, stream, ws):
        x, w, b, dy = ins[i]
        out = [torch.empty((T, D), device="cuda"), torch.empty((T, D), device="cuda"), torch.empty(D, device="cuda"),
               torch.empty(D, device="cuda")]
        torch.cuda.synchronize()
        for _ in range(5):
            abi.pg_layernorm_fwd(x, w, b, None, 1e-5, out[0], stream=stream)
            abi.pg_layernorm_bwd(x, w, None, dy, 1e-5, *out[1:], ws, stream=stream)
        return out

    want = [run(0, None, None), run(1, None, None)]
    torch.cuda.synchronize()
    want = [[t.clone() for t in o] for o in want]
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = torch.empty(abi.workspace_bytes(abi.PG_OP_LN_BWD, T, D, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = [run(0, s0.cuda_stream, ws), run(1, s1.cuda_stream, None)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_past_32_bit_offsets():
    """2.3 x 10^9 values: the last rows of the forward and the backward are those of a call on them alone, and
    dw, db of a mask that leaves only them too."""
    T, D, K = 4_500_000, 512, 96
    x = torch.empty((T, D), dtype=BF, device="cuda")
    x[:T - K] = 1.0
    tail, w, b = states(K, D, BF, 22)
    x[T - K:] = tail.cuda()
    w, b = w.cuda(), b.cuda()
    dy = torch.zeros((T, D), dtype=BF, device="cuda")
    dy[T - K:] = gradients(K, D, BF, 22).cuda()
    y = torch.empty_like(x)
    abi.pg_layernorm_fwd(x, w, b, None, 1e-5, y)
    small = torch.empty((K, D), dtype=BF, device="cuda")
    abi.pg_layernorm_fwd(x[T - K:].contiguous(), w, b, None, 1e-5, small)
    assert torch.equal(y[T - K:], small) and torch.equal(y[0], b.to(BF))
    del y
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[T - K:] = 1
    dx, dw, db = torch.empty_like(x), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    abi.pg_layernorm_bwd(x, w, mask, dy, 1e-5, dx, dw, db)
    sdx, sdw, sdb = torch.empty((K, D), dtype=BF, device="cuda"), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    abi.pg_layernorm_bwd(x[T - K:].contiguous(), w, None, dy[T - K:].contiguous(), 1e-5, sdx, sdw, sdb)
    assert torch.equal(dx[T - K:], sdx) and not dx[:T - K].any()
    # the rows fall to other lanes: each adds at most one of them here and there, the rest in float64
    mag = dy[T - K:].double().abs().sum(0)
    assert float(((db - sdb).double().abs() - 2 * U * db.double().abs() - 40 * U * mag).max()) <= 0


def test_many_rows_keep_the_sums_digits():
    """2^23 rows of equal sign: db is a sum of equal values, whose float32 running sum alone would be off by
    far more than the (512 + 24) u that lanes of at most 512 rows allow."""
    T, D = 1 << 23, 16
    x = torch.randn((T, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(BF)
    dy = torch.full((T, D), 0.1, device="cuda")
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    abi.pg_layernorm_bwd(x, None, None, dy, 1e-5, None, dw, db)
    want = T * float(torch.tensor(0.1))
    assert float((db.double() - want).abs().max()) <= (512 + 24) * U * want
