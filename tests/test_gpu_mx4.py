"""The 4-bit format and the head on it, on the GPU, against the float64 oracle: codes and scales bit for
bit, the values they stand for exactly, and the head within tolerances that are worked out at each test."""
import numpy as np
import pytest
import torch

from lm_head_cross_pg_amd import abi
from oracle import oracle as ora
from tests.gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def room(T, D, fill=0xAB):
    return (torch.full((T, abi.pg_mx4_code_bytes(D)), fill, dtype=torch.uint8, device="cuda"),
            torch.full((T, abi.pg_mx4_scale_bytes(D)), fill, dtype=torch.uint8, device="cuda"))


def packed(codes, exps):
    """The bytes of oracle codes [T, D] and exponents [T, blocks], padding included."""
    T, D = codes.shape
    wide = np.zeros((T, 64 * -(-D // 64)), np.uint8)
    wide[:, :D] = codes
    scales = np.zeros((T, 16 * -(-D // 512)), np.uint8)
    scales[:, :exps.shape[1]] = exps + 127
    return wide[:, 0::2] | (wide[:, 1::2] << 4), scales


def f64(t):
    return t.double().cpu().numpy()


def rows(T, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, D), generator=g) * torch.exp2(torch.randint(-6, 7, (T, -(-D // 32)), generator=g).float()
                                                     ).repeat_interleave(32, 1)[:, :D]
    return (x * scale).to(dtype)


def check_quantise(x, mask=None):
    T, D = x.shape
    print(f"[case] quantise T={T} D={D} {x.dtype} mask={None if mask is None else int(mask.sum())}", flush=True)
    codes, scales = room(T, D)
    abi.pg_quantize_mx4(x.cuda(), None if mask is None else mask.cuda(), codes, scales)
    torch.cuda.synchronize()
    val, oc, oe = ora.quantize_rows_mx4(f64(x))
    ec, es = packed(oc, oe)
    on = np.ones(T, bool) if mask is None else mask.numpy() != 0
    np.testing.assert_array_equal(scales.cpu().numpy()[on], es[on])
    np.testing.assert_array_equal(codes.cpu().numpy()[on], ec[on])
    assert np.all(codes.cpu().numpy()[~on] == 0xAB) and np.all(scales.cpu().numpy()[~on] == 0xAB)
    for dtype in (BF, F):
        if mask is None:
            out = torch.empty((T, D), dtype=dtype, device="cuda")
            abi.pg_dequantize_mx4(codes, scales, out)
            np.testing.assert_array_equal(f64(out), val)
    return codes, scales, val


@pytest.mark.parametrize("D", [1, 2, 7, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 256, 300, 512, 513, 1000, 1024, 2050])
@pytest.mark.parametrize("dtype", [BF, F])
def test_quantise_bit_exact(D, dtype):
    check_quantise(rows(7, D, dtype, D))


@pytest.mark.parametrize("T,D", [(1, 512), (3, 64), (2000, 96), (5001, 512), (300, 1500)])
def test_quantise_rows_and_masks(T, D):
    x = rows(T, D, BF, T)
    check_quantise(x)
    for p in (0.0, 0.4):
        check_quantise(x, (torch.rand(T, generator=torch.Generator().manual_seed(T)) < p).to(torch.uint8))


def test_quantise_ties_and_borders():
    """Every multiple of a sixteenth up to 7 and its float32 neighbours, in blocks whose largest magnitude
    is 4 (scale 1), 6.9 (scale 1) and 7 (scale 2), at exponents from the smallest to the largest."""
    k = np.arange(0, 65) / 16.0
    near = np.unique(np.concatenate([k, np.nextafter(k.astype(np.float32), np.float32(9)),
                                     np.nextafter(k.astype(np.float32), np.float32(-9))]).astype(np.float32))
    near = near[np.abs(near) <= 4]
    blocks = []
    for top in (4.0, 6.9, 7.0):
        for i in range(0, len(near), 31):
            v = np.zeros(32, np.float32)
            v[1:1 + len(near[i:i + 31])] = near[i:i + 31]
            v[0] = top
            blocks.append(v)
            blocks.append(-v)
    x = np.stack(blocks)
    for e in (-126, -100, -1, 0, 3, 100, 124):
        check_quantise(torch.from_numpy(np.ldexp(x, e).astype(np.float32)))


def test_quantise_small_zero_nan_and_infinite_blocks():
    x = torch.zeros((12, 96))
    x[0, :] = 2.0 ** -149
    x[1, 5] = 2.0 ** -126
    x[2, :32] = -0.0
    x[3, 40] = float("nan")
    x[4, 0], x[4, 95] = float("inf"), -float("inf")
    x[5] = torch.finfo(F).max
    x[6] = torch.linspace(-1, 1, 96) * 2.0 ** -125
    x[7] = torch.linspace(-1, 1, 96) * 2.0 ** -130
    check_quantise(x)
    check_quantise(x.to(BF))


def test_dequantise_every_code_and_scale():
    """All 16 codes under all 256 scale bytes, in both types: exact, infinite past the type, NaN at 255."""
    codes = torch.arange(16, dtype=torch.uint8).repeat(2)[None].repeat(256, 1)
    c = torch.zeros((256, 32), dtype=torch.uint8)
    c[:, :16] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    s = torch.zeros((256, 16), dtype=torch.uint8)
    s[:, 0] = torch.arange(256)
    level = np.concatenate([ora.MX4_LEVELS, -ora.MX4_LEVELS])
    want = level[codes.numpy()] * np.exp2(np.arange(256.0) - 127)[:, None]
    want[255] = np.nan
    want[np.abs(want) >= 2.0 ** 128] = np.inf * np.sign(want[np.abs(want) >= 2.0 ** 128])
    for dtype in (BF, F):
        out = torch.empty((256, 32), dtype=dtype, device="cuda")
        abi.pg_dequantize_mx4(c.cuda(), s.cuda(), out)
        np.testing.assert_array_equal(f64(out), want)


# --------------------------------------------------------------------------- norm straight to 4 bits
@pytest.mark.parametrize("D", [1, 31, 64, 100, 128, 200, 256, 300, 512, 700, 1024, 1500, 2048, 2100])
@pytest.mark.parametrize("dtype", [BF, F])
def test_norm_to_4_bits_is_norm_then_quantise(D, dtype):
    """Bit for bit the float32 norm followed by the quantiser, unscored rows left as they were."""
    for T, masked in ((1, False), (37, False), (500, True)):
        print(f"[case] norm to 4 bits T={T} D={D} {dtype}", flush=True)
        x = rows(T, D, dtype, D + T).cuda()
        g = torch.Generator().manual_seed(D)
        w, b = (1 + 0.1 * torch.randn(D, generator=g)).cuda(), torch.randn(D, generator=g).cuda()
        m = (torch.rand(T, generator=g) < 0.5).to(torch.uint8).cuda() if masked else None
        y = torch.empty((T, D), device="cuda")
        want, got = room(T, D), room(T, D)
        abi.pg_layernorm_fwd(x, w, b, m, 1e-5, y)
        abi.pg_quantize_mx4(y, m, *want)
        abi.pg_layernorm_fwd_mx4(x, w, b, m, 1e-5, *got)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# ---------------------------------------------------------------------------------------------- head
def head_inputs(T, D, V, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    h, e = gain * torch.randn((T, D), generator=g), torch.randn((V, D), generator=g) / D ** 0.5
    hq, eq = room(T, D), room(V, D)
    abi.pg_quantize_mx4(h.cuda(), None, *hq)
    abi.pg_quantize_mx4(e.cuda(), None, *eq)
    H, E = torch.empty((T, D), device="cuda"), torch.empty((V, D), device="cuda")
    abi.pg_dequantize_mx4(*hq, H)
    abi.pg_dequantize_mx4(*eq, E)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    return hq, eq, y, f64(H), f64(E)


def tolerance(H, E, c, V):
    """Of nats and lse. A logit: products are exact, D additions in float32, D u of the sum of magnitudes A.
    The softcap: exp2, fma and rcp, each within two steps, act on s log2 e = M + K / (1 + e), |K| = 2 M:
    12 u M. The sum of V positive terms: two steps each for exp2 and V u for the additions at the very
    most. log2 (two steps of a value up to 64) and the last difference: 2^-16. nats is a difference of two
    such values."""
    A = float(np.max(np.abs(H).sum(1))) * float(np.max(np.abs(E)))
    A = min(A, float(np.sqrt((H * H).sum(1).max() * (E * E).sum(1).max()) * 1.0))   # Cauchy-Schwarz
    M = (c if c > 0 else A) * 1.4427
    return 2 * (H.shape[1] * U * A + 12 * U * M + (V + 4) * U + 2.0 ** -16)


def check_head(T, D, V, c, seed=0, gain=1.0, mask=None, sample=None, inputs=None):
    hq, eq, y, H, E = inputs or head_inputs(T, D, V, seed, gain)
    print(f"[case] 4-bit head T={T} D={D} V={V} c={c} gain={gain} mask={None if mask is None else int(mask.sum())}",
          flush=True)
    nats, lse = (torch.full((T,), -5.0, device="cuda") for _ in range(2))
    m = None if mask is None else mask.cuda()
    abi.pg_lmhead_ce_fwd_mx4(*hq, *eq, y.cuda(), m, D, c, nats, lse)
    torch.cuda.synchronize()
    at = np.arange(T) if sample is None else np.unique(np.asarray(sample))
    on, ol = ora.forward(H[at], E, y.numpy()[at], c, None if mask is None else mask.numpy()[at])
    n, l = f64(nats), f64(lse)
    tol = tolerance(H, E, c, V)
    assert np.max(np.abs(n[at] - on), initial=0) <= tol and np.max(np.abs(l[at] - ol), initial=0) <= tol
    assert np.all(n >= 0)
    if mask is not None:
        off = mask.numpy() == 0
        assert not n[off].any() and not l[off].any()
    only = torch.full((T,), -5.0, device="cuda")
    abi.pg_lmhead_ce_fwd_mx4(*hq, *eq, y.cuda(), m, D, c, only)       # without lse: the same nats
    assert torch.equal(only, nats)
    return nats, lse


@pytest.mark.parametrize("D", [1, 32, 33, 64, 65, 100, 128, 190, 256, 300, 320, 384, 448, 512, 513, 640, 768, 1000, 1024,
                               1025, 2048, 2100])
@pytest.mark.parametrize("c,gain", [(30.0, 1.0), (30.0, 8.0), (0.0, 1.0)])
def test_head_widths(D, c, gain):
    check_head(70, D, 333, c, D, gain)


@pytest.mark.parametrize("T", [1, 15, 16, 17, 129, 1023, 1040, 8191, 8192, 8193, 16385, 65535, 65536, 65537])
@pytest.mark.parametrize("part", [0.02, 0.5, 1.0])
def test_head_selects_scored_rows(T, part):
    """Every count of rows that a wave, a piece of the mask and a workgroup end in, any nonzero byte scoring."""
    g = torch.Generator().manual_seed(T)
    value = torch.tensor([1, 2, 128, 255], dtype=torch.uint8)[torch.randint(0, 4, (T,), generator=g)]
    mask = torch.where(torch.rand(T, generator=g) < part, value, torch.zeros_like(value))
    at = np.unique(np.concatenate([np.arange(min(T, 40)), np.arange(max(0, T - 40), T),
                                   torch.randint(0, T, (200,), generator=g).numpy()]))
    check_head(T, 33, 70, 30.0, T, mask=mask, sample=at)


@pytest.mark.parametrize("scored", [130, 300, 900, 1500, 2000])
@pytest.mark.parametrize("D,V", [(200, 5003), (640, 5003), (1100, 5003), (64, 1291)])
@pytest.mark.parametrize("c", [30.0, 0.0])
def test_head_splits_without_tiles(scored, D, V, c):
    """Splits of the vocabulary whose share of tiles is empty (40 tiles over 21 splits are 20 splits of two and
    one of none) next to a last tile that is not whole: every row of the vocabulary counts once."""
    T = scored + 70
    mask = (torch.arange(T) >= 70).to(torch.uint8)
    check_head(T, D, V, c, scored, mask=mask, sample=np.arange(60, T, 37))


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 1000, 8192, 8193])
@pytest.mark.parametrize("c", [30.0, 0.0])
def test_head_vocabularies(V, c):
    nats, _ = check_head(33, 128, V, c, V, 4.0)
    if V == 1:
        assert not nats.any()      # the only token has probability one, exactly


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 127, 128, 129, 255, 257, 1000, 4133])
@pytest.mark.parametrize("masked", [False, True])
def test_head_rows(T, masked):
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.4).to(torch.uint8) if masked else None
    check_head(T, 512, 1000, 30.0, T, 8.0, mask)


@pytest.mark.parametrize("c,gain", [(0.0, 8.0), (5.0, 8.0), (15.0, 8.0), (40.0, 30.0), (41.0, 8.0), (300.0, 8.0), (0.005, 1.0),
                                    (30.0, 0.01), (30.0, 3.0), (30.0, 1000.0)])
def test_head_caps(c, gain):
    check_head(300, 512, 700, c, 3, gain)


def test_head_many_rows():
    rng = np.random.default_rng(0)
    check_head(70000, 64, 96, 30.0, 5, 4.0, sample=np.append(rng.choice(70000, 300), [0, 69999]))


def test_head_full_size():
    rng = np.random.default_rng(1)
    at = np.append(rng.choice(65536, 100), [0, 65535])
    ins = head_inputs(65536, 512, 8192, 6, 8.0)
    nats, lse = check_head(65536, 512, 8192, 30.0, sample=at, inputs=ins)
    mask = (torch.arange(65536) % 2048 >= 1984).to(torch.uint8)
    n2, l2 = check_head(65536, 512, 8192, 30.0, mask=mask, sample=np.nonzero(mask.numpy())[0][:64], inputs=ins)
    on = mask.cuda() != 0
    # the vocabulary is split where few rows are scored: the same terms, added in another order
    assert torch.allclose(n2[on], nats[on], rtol=0, atol=1e-4) and torch.allclose(l2[on], lse[on], rtol=0, atol=1e-4)


def test_head_masks_that_leave_little():
    T, D, V = 5000, 96, 200
    ins = head_inputs(T, D, V, 7)
    for at in ([], [0], [T - 1], [3, 1000, 1001, 4999], list(range(256, 512))):
        mask = torch.zeros(T, dtype=torch.uint8)
        mask[at] = 255
        check_head(T, D, V, 30.0, mask=mask, inputs=ins)
        check_head(T, D, V, 0.0, mask=mask.bool().to(torch.uint8), inputs=ins)


@pytest.mark.parametrize("c", [30.0, 0.0])
def test_head_poisoned_rows(c):
    """A target outside the vocabulary, a block of NaNs in a row's states: that row is NaN and no other. A
    block of NaNs in the embedding: every scored row. Unscored rows are 0 whatever they hold."""
    T, D, V = 200, 160, 300
    hq, eq, y, H, E = head_inputs(T, D, V, 8)
    want, wl = check_head(T, D, V, c, inputs=(hq, eq, y, H, E))
    y2 = y.clone()
    y2[3], y2[77], y2[130] = -1, V, 2 ** 31 - 1
    hs = hq[1].clone()
    hs[50, 4] = 255
    nats, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    abi.pg_lmhead_ce_fwd_mx4(hq[0], hs, *eq, y2.cuda(), None, D, c, nats, lse)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[3, 77, 130, 50]] = True
    assert torch.isnan(nats[bad]).all() and torch.equal(nats[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])
    assert torch.isnan(lse[50])
    mask = (~bad).to(torch.uint8)
    abi.pg_lmhead_ce_fwd_mx4(hq[0], hs, *eq, y2.cuda(), mask, D, c, nats, lse)
    assert not nats[bad].any() and not lse[bad].any() and torch.isfinite(nats).all()
    es = eq[1].clone()
    es[299, 0] = 255
    abi.pg_lmhead_ce_fwd_mx4(*hq, eq[0], es, y.cuda(), mask, D, c, nats, lse)
    assert torch.isnan(nats[~bad]).all() and torch.isnan(lse[~bad]).all() and not nats[bad].any()


def test_head_no_rows():
    D, V = 64, 50
    _, eq, _, _, _ = head_inputs(1, D, V, 9)
    abi.pg_lmhead_ce_fwd_mx4(*room(0, D), *eq, torch.empty(0, dtype=torch.int32, device="cuda"), None, D, 30.0,
                             torch.empty(0, device="cuda"))
    torch.cuda.synchronize()


def test_head_agrees_with_the_bf16_head():
    """pg_lmhead_ce_fwd on the dequantised rows (bf16 holds them exactly): the same logits up to the order of
    float32 sums, so each side is within the tolerance of the definition."""
    for c in (30.0, 0.0):
        hq, eq, y, H, E = head_inputs(700, 512, 1500, 10, 8.0)
        nats, lse = check_head(700, 512, 1500, c, inputs=(hq, eq, y, H, E))
        hb, eb = torch.empty((700, 512), dtype=BF, device="cuda"), torch.empty((1500, 512), dtype=BF, device="cuda")
        abi.pg_dequantize_mx4(*hq, hb)
        abi.pg_dequantize_mx4(*eq, eb)
        n2, l2 = torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
        abi.pg_lmhead_ce_fwd(hb, eb, y.cuda(), None, c, n2, l2)
        tol = 2 * tolerance(H, E, c, 1500)
        assert float((n2 - nats).abs().max()) <= tol and float((l2 - lse).abs().max()) <= tol


def test_repeatable_on_another_stream_and_in_a_graph():
    """The whole scoring run (norm to 4 bits, head, bits per byte) gives the same bits eagerly, on a side
    stream, and from a graph replayed with eager work between."""
    T, D, V = 2000, 512, 1000
    g = torch.Generator().manual_seed(11)
    x, w, b = torch.randn((T, D), generator=g).to(BF).cuda(), 8 * torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    _, eq, _, _, _ = head_inputs(1, D, V, 11)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    blen = torch.randint(1, 9, (V,), generator=g, dtype=torch.int32).cuda()
    for mask in (None, (torch.rand(T, generator=g) < 0.3).to(torch.uint8).cuda()):
        hq = room(T, D)
        nats, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        out = torch.empty(4, dtype=torch.float64, device="cuda")
        ws = torch.empty(abi.workspace_bytes(abi.PG_OP_FWD_MX4, T, D, V), dtype=torch.uint8, device="cuda")
        wb = torch.empty(abi.workspace_bytes(abi.PG_OP_BPB, T, 1, V), dtype=torch.uint8, device="cuda")

        def step():
            abi.pg_layernorm_fwd_mx4(x, w, b, mask, 1e-5, *hq)
            abi.pg_lmhead_ce_fwd_mx4(*hq, *eq, y, mask, D, 30.0, nats, lse, ws)
            abi.pg_bpb_reduce(nats, y, mask, blen, None, V, out, wb)

        step()
        first = [t.clone() for t in (nats, lse, out)]
        val = torch.empty((T, D), device="cuda")
        ev = torch.empty((V, D), device="cuda")
        abi.pg_dequantize_mx4(*eq, ev)
        h = ora.quantize_rows_mx4(ora.layer_norm(f64(x), f64(w), f64(b), 1e-5).astype(np.float32))[0]
        onats, _ = ora.forward(h, f64(ev), y.cpu().numpy(), 30.0, None if mask is None else mask.cpu().numpy())
        want = ora.bpb(onats, y.cpu().numpy(), blen.cpu().numpy(), None if mask is None else mask.cpu().numpy())
        assert abs(float(out[3]) - want[3]) <= 1e-5 * want[3] and float(out[2]) == want[2]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ws.fill_(0xFF)
            nats.fill_(-1)
            step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (nats, lse, out)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for k in range(3):
            nats.fill_(float(k))
            ws.fill_(k)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, (nats, lse, out)))
            step()
            torch.cuda.synchronize()


def test_two_calls_at_once():
    """The head on two streams with nothing between them, one workspace given and one allocated by the call:
    the bits of the calls one by one."""
    T, D, V = 3000, 512, 2000
    ins = [head_inputs(T, D, V, s, 4.0) for s in (30, 31)]
    ys = [i[2].cuda() for i in ins]
    torch.cuda.synchronize()

    def run(i, stream, ws):
        nats, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        torch.cuda.synchronize()
        for _ in range(5):
            abi.pg_lmhead_ce_fwd_mx4(*ins[i][0], *ins[i][1], ys[i], None, D, 30.0, nats, lse, ws, stream=stream)
        return nats, lse

    want = [run(0, None, None), run(1, None, None)]
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = torch.empty(abi.workspace_bytes(abi.PG_OP_FWD_MX4, T, D, V), dtype=torch.uint8, device="cuda")
    got = [run(0, s0.cuda_stream, ws), run(1, s1.cuda_stream, None)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_past_32_bit_offsets():
    """9 x 10^6 rows (2.3 x 10^9 bytes of codes, 4.6 x 10^9 values): quantised, read back and scored, the last
    rows as in calls on them alone."""
    T, D, V, K = 9_000_000, 512, 96, 200
    x = torch.empty((T, D), dtype=BF, device="cuda")
    x[:T - K] = 0.5
    x[T - K:] = rows(K, D, BF, 40).cuda()
    codes, scales = (torch.empty((T, n), dtype=torch.uint8, device="cuda") for n in (256, 16))
    abi.pg_quantize_mx4(x, None, codes, scales)
    sc, ss = room(K, D)
    abi.pg_quantize_mx4(x[T - K:].contiguous(), None, sc, ss)
    assert torch.equal(codes[T - K:], sc) and torch.equal(scales[T - K:], ss)
    abi.pg_dequantize_mx4(codes, scales, x)
    out = torch.empty((K, D), dtype=BF, device="cuda")
    abi.pg_dequantize_mx4(sc, ss, out)
    assert torch.equal(x[T - K:], out) and bool((x[0] == 0.5).all())
    del x
    _, eq, _, _, _ = head_inputs(1, D, V, 41)
    y = torch.zeros(T, dtype=torch.int32, device="cuda")
    nats = torch.empty(T, device="cuda")
    abi.pg_lmhead_ce_fwd_mx4(codes, scales, *eq, y, None, D, 30.0, nats)
    small = torch.empty(K, device="cuda")
    abi.pg_lmhead_ce_fwd_mx4(sc, ss, *eq, y[:K].contiguous(), None, D, 30.0, small)
    # one split either way (one tile of vocabulary): the same operations on each row
    assert torch.equal(nats[T - K:], small)


def test_head_widest_vocabulary_and_states():
    """V = 2^20 for few rows (the splits go past 64), and D = 2^16."""
    check_head(3, 32, 1 << 20, 30.0, 50)
    check_head(5, 1 << 16, 70, 30.0, 51)
    mask = torch.tensor([1, 0, 1, 1, 0], dtype=torch.uint8)
    check_head(5, 64, 1 << 18, 0.0, 52, mask=mask)


def test_captured_head_follows_its_mask():
    """A captured masked call replayed after the mask's bytes have changed: the rows that it scores now, and as
    many splits as their number makes."""
    T, D, V = 5000, 96, 1500
    hq, eq, y, H, E = head_inputs(T, D, V, 60, 4.0)
    y = y.cuda()
    nats, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(abi.workspace_bytes(abi.PG_OP_FWD_MX4, T, D, V), dtype=torch.uint8, device="cuda")
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")

    def call():
        abi.pg_lmhead_ce_fwd_mx4(*hq, *eq, y, mask, D, 30.0, nats, lse, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = torch.Generator().manual_seed(61)
    for part in (1.0, 0.5, 0.0, 0.01, 0.9):
        m = (torch.rand(T, generator=g) < part).to(torch.uint8)
        mask.copy_(m)
        nats.fill_(-1.0)
        lse.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        got = nats.clone(), lse.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], nats) and torch.equal(got[1], lse)
        on, ol = ora.forward(H, E, y.cpu().numpy(), 30.0, m.numpy())
        tol = tolerance(H, E, 30.0, V)
        assert np.max(np.abs(f64(nats) - on)) <= tol and np.max(np.abs(f64(lse) - ol)) <= tol
