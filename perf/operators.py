"""Cases of the final norm and of the tied head in microscaled 4-bit floating point, for measuring.

Five operators, each with a plain form (elementary torch operations) and the library's own calls:

  norm   layer norm of the model's last hidden states, what the tied head reads
  grad   its backward: the gradient of the states, of the gain and of the bias
  quant  rows to 4 bits and back: the fake quantisation that quantisation-aware training runs on
         the tied embedding at every step
  score  norm, 4-bit states and the 4-bit head in a row: states in, nats and log-sum-exps out
  head   the 4-bit head alone, on states and an embedding that are held in 4 bits

The 4-bit format: 32 consecutive values of a row share a scale 2^e, one byte e + 127 (255 = NaN), and
each value is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, two to a byte, the first in the low half.
A row is padded with zeros to 64 values (32 bytes of codes) and to 16 scale bytes. e is the one for which
the block's largest magnitude lies in [3.5, 7) 2^e, held to -127 .. 125; values above 6 2^e become 6 2^e,
which is off by less than half the grid's last step.
"""
import math

import torch

own = False

EPS = 1e-5
WINDOW, STRIDE = 2048, 64   # sliding-window evaluation: the last 64 rows of each window are scored
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token's state in front of the head: latency
        {"name": "norm_token", "op": "norm", "T": 1, "D": 512, "x": "f32", "y": "bf16", "mask": "none"},
        # the states of a training batch of the head's main workload
        {"name": "norm_batch", "op": "norm", "T": 65536, "D": 512, "x": "bf16", "y": "bf16", "mask": "none"},
        # the same batch backward: the head's float32 gradient in, the states' gradient out
        {"name": "grad_batch", "op": "grad", "T": 65536, "D": 512, "x": "bf16", "y": "f32", "dx": "f32", "mask": "none"},
        # a short batch of a float32 residual stream of an odd width, gradients in bf16
        {"name": "grad_ragged", "op": "grad", "T": 2047, "D": 1001, "x": "f32", "y": "bf16", "dx": "bf16", "mask": "none"},
        # the tied embedding of the main workload, quantised and read back at every training step
        {"name": "quant_embed", "op": "quant", "T": 8192, "D": 512, "x": "bf16", "y": "bf16"},
        # float32 master weights of a large matrix
        {"name": "quant_master", "op": "quant", "T": 32768, "D": 1024, "x": "f32", "y": "f32"},
        # scoring a single token after a quantised model
        {"name": "score_token", "op": "score", "T": 1, "D": 512, "V": 8192, "x": "f32", "cap": 30.0, "gain": 8.0,
         "mask": "none"},
        # a whole batch of the main workload, logits of a trained model's size
        {"name": "score_batch", "op": "score", "T": 65536, "D": 512, "V": 8192, "x": "bf16", "cap": 30.0, "gain": 8.0,
         "mask": "none"},
        # the head of a single token
        {"name": "head_token", "op": "head", "T": 1, "D": 512, "V": 8192, "cap": 30.0, "gain": 8.0, "mask": "none"},
        # the head of the main workload
        {"name": "head_batch", "op": "head", "T": 65536, "D": 512, "V": 8192, "cap": 30.0, "gain": 8.0, "mask": "none"},
        # one batch of sliding-window evaluation: 32 windows, 64 rows of each scored
        {"name": "head_window", "op": "head", "T": 65536, "D": 512, "V": 8192, "cap": 30.0, "gain": 8.0, "mask": "window"},
        # odd sizes throughout, no softcap, logits of a model at its start
        {"name": "head_ragged", "op": "head", "T": 3001, "D": 200, "V": 5003, "cap": 0.0, "gain": 1.0, "mask": "random"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half the widths are multiples of 64 as models have, the others are anything."""
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.5 else max(64, min(hi // 64 * 64, 64 * round(d / 64)))


def draw(rng):
    op = rng.choice(("norm", "grad", "quant", "score", "head"))
    kind = lambda: rng.choice(("bf16", "f32"))  # noqa: E731
    mask = rng.choice(("none", "none", "window", "random"))
    if op in ("norm", "grad", "quant"):
        D = _width(rng, 8, 4096)
        c = {"op": op, "T": _log_int(rng, 1, min(65536, 65536 * 512 // D)), "D": D, "x": kind(), "y": kind()}
        if op == "grad":
            c["dx"] = kind()
        if op != "quant":
            c["mask"] = mask
        return c
    D, V = _width(rng, 16, 1024), _log_int(rng, 16, 16384)
    T = _log_int(rng, 1, min(65536, 65536 * 512 * 8192 // (max(64, -(-D // 64) * 64) * V)))
    c = {"op": op, "T": T, "D": D, "V": V, "cap": rng.choice((30.0, 30.0, 15.0, 50.0, 0.0)),
         "gain": rng.choice((1.0, 8.0)), "mask": mask}
    if op == "score":
        c["x"] = kind()
    return c


def _window(T):
    return min(WINDOW, T)


def _scored(case):
    """Rows that a case's mask scores (on average, where it is drawn)."""
    T = case["T"]
    if case.get("mask", "none") == "none":
        return T
    if case["mask"] == "random":
        return T / 2
    L = _window(T)
    first = max(0, L - STRIDE)
    return (T // L) * (L - first) + max(0, T % L - first)


def work(case):
    size = {"bf16": 2, "f32": 4}
    op, T, D, n = case["op"], case["T"], case["D"], _scored(case)
    mask = 0 if case.get("mask", "none") == "none" else T
    row4 = (-(-D // 32)) * 17              # a row in 4 bits: 16 bytes of codes and a scale for each 32 values
    if op == "norm":
        return {"bytes": n * D * (size[case["x"]] + size[case["y"]]) + 8 * D + mask, "flops": 9 * n * D}
    if op == "grad":
        return {"bytes": n * D * (size[case["x"]] + size[case["y"]]) + T * D * size[case["dx"]] + 12 * D + mask,
                "flops": 18 * n * D}
    if op == "quant":
        return {"bytes": T * D * (size[case["x"]] + size[case["y"]]) + 2 * T * row4, "flops": 6 * T * D}
    V = case["V"]
    states = n * (row4 if op == "head" else D * size[case["x"]])
    return {"bytes": states + V * row4 + 4 * n + 8 * T + mask, "flops": 2 * n * D * V + 8 * n * V}


# ----------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _states(g, T, D, dtype):
    """A residual stream: channels of unlike size, a small common offset."""
    x = torch.randn((T, D), generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(D, generator=g, device="cuda"))
    x += 0.3 * torch.randn(D, generator=g, device="cuda")
    return (1.7 * x).to(dtype)


def _mask(g, case):
    T, kind = case["T"], case.get("mask", "none")
    if kind == "none":
        return None
    if kind == "window":
        L = _window(T)
        return (torch.arange(T, device="cuda") % L >= L - STRIDE).to(torch.uint8)
    return (torch.rand(T, generator=g, device="cuda") < 0.5).to(torch.uint8)


def _packed(values):
    """Rows in 4 bits, as a checkpoint of a quantised model holds them: codes and scale bytes."""
    code, e = _quantised(values)
    T, B = e.shape
    code = torch.nn.functional.pad(code.reshape(T, B * 32), (0, (B & 1) * 32))
    scale = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -B % 16))
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scale.contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op, T, D = case["op"], case["T"], case["D"]
    s = {"op": op, "D": D, "mask": _mask(g, case)}
    if op == "quant":
        s["x"] = (0.02 * torch.randn((T, D), generator=g, device="cuda")).to(DT[case["x"]])
        s["codes"], s["scales"] = _rows4(T, D)
        s["y"] = torch.empty((T, D), dtype=DT[case["y"]], device="cuda")
        return s
    if op != "head":
        s["x"] = _states(g, T, D, DT[case["x"]])
        s["weight"] = case.get("gain", 1.0) * (1 + 0.1 * torch.randn(D, generator=g, device="cuda"))
        s["bias"] = case.get("gain", 1.0) * 0.1 * torch.randn(D, generator=g, device="cuda")
    if op == "norm":
        s["y"] = torch.zeros((T, D), dtype=DT[case["y"]], device="cuda")
    if op == "grad":
        s["dy"] = (torch.randn((T, D), generator=g, device="cuda") / T).to(DT[case["y"]])
        s["dx"] = torch.empty((T, D), dtype=DT[case["dx"]], device="cuda")
        s["dweight"], s["dbias"] = (torch.empty(D, device="cuda") for _ in range(2))
    if op in ("score", "head"):
        V = case["V"]
        s["softcap"] = case["cap"]
        s["embed"], s["embed_scales"] = _packed(0.02 * torch.randn((V, D), generator=g, device="cuda"))
        if op == "head":
            s["codes"], s["scales"] = _packed(case["gain"] * torch.randn((T, D), generator=g, device="cuda"))
        else:
            s["codes"], s["scales"] = _rows4(T, D)
        s["target"] = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["nats"], s["lse"] = (torch.empty(T, device="cuda") for _ in range(2))
    s["workspace"] = {}
    return s


def _rows4(T, D):
    """Room for T rows of D values in 4 bits."""
    return (torch.zeros((T, 32 * -(-D // 64)), dtype=torch.uint8, device="cuda"),
            torch.zeros((T, 16 * -(-D // 512)), dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------------------- plain form
def _norm(x, weight, bias):
    d = x - x.mean(1, keepdim=True)
    return d * torch.rsqrt((d * d).mean(1, keepdim=True) + EPS) * weight + bias


def _quantised(x):
    """Codes [rows, blocks, 32] and exponents [rows, blocks] of float32 rows."""
    T, D = x.shape
    x = torch.nn.functional.pad(x, (0, -D % 32)).reshape(T, -1, 32)
    top = x.abs().amax(2)
    m, e = torch.frexp(top)                       # top = m 2^e, m in [0.5, 1)
    e = e - 3 + (m >= 0.875).to(e.dtype)
    e = torch.where(top > 0, e, -127).clamp(-127, 125)
    a = torch.ldexp(x.abs(), -e[:, :, None])      # exact: a power of two
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.minimum(torch.round(a / step) * step, torch.full_like(a, 6.0))
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return code | (torch.signbit(x).to(torch.uint8) << 3), e


def _values(code, e):
    """What codes and exponents stand for, in float32: rows of whole blocks."""
    a = torch.tensor(LEVELS, device=code.device)[(code & 7).long()]
    return torch.ldexp(torch.where(code > 7, -a, a), e[:, :, None]).flatten(1)


def _unpacked(codes, scales):
    T, B = codes.shape[0], codes.shape[1] // 16
    code = torch.stack((codes & 15, codes >> 4), 2).reshape(T, B, 32)
    return _values(code, scales[:, :B].to(torch.int32) - 127)


def _cross_entropy(h, e, target, cap, mask):
    z = h @ e.t()
    s = cap * torch.tanh(z / cap) if cap > 0 else z
    top = s.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(s - top).sum(1, keepdim=True)))[:, 0]
    nats = lse - s.gather(1, target.long()[:, None])[:, 0]
    if mask is not None:
        nats, lse = (torch.where(mask != 0, v, torch.zeros_like(v)) for v in (nats, lse))
    return nats, lse


def _plain(s):
    op, mask = s["op"], s["mask"]
    if op == "norm":
        y = _norm(s["x"].float(), s["weight"], s["bias"]).to(s["y"].dtype)
        return y if mask is None else torch.where(mask[:, None] != 0, y, s["y"])
    if op == "grad":
        x, dy = s["x"].float(), s["dy"].float()
        d = x - x.mean(1, keepdim=True)
        r = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        xh, g = d * r, dy * s["weight"]
        dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if mask is not None:
            on = mask[:, None] != 0
            dx, dy = torch.where(on, dx, 0.0), torch.where(on, dy, 0.0)
        # sums over all rows: in 64 bits
        return (dx.to(s["dx"].dtype), (dy * xh).sum(0, dtype=torch.float64).float(),
                dy.sum(0, dtype=torch.float64).float())
    if op == "quant":
        return _values(*_quantised(s["x"].float()))[:, :s["D"]].to(s["y"].dtype)
    if op == "score":
        # in 64 bits up to the float32 values that are quantised: next to a border of the 4-bit
        # grid one rounding more moves a value by a whole step
        h = _values(*_quantised(_norm(s["x"].double(), s["weight"].double(), s["bias"].double()).float()))
    else:
        h = _unpacked(s["codes"], s["scales"])
    e = _unpacked(s["embed"], s["embed_scales"])
    return _cross_entropy(torch.nn.functional.pad(h, (0, e.shape[1] - h.shape[1])), e, s["target"], s["softcap"], mask)


# ------------------------------------------------------------------------------------- own kernels
def _workspace(s, abi, op, T, D, V):
    """The caller's workspace, allocated once for its sizes."""
    if op not in s["workspace"]:
        s["workspace"][op] = torch.empty(max(256, abi.workspace_bytes(op, T, D, V)), dtype=torch.uint8, device="cuda")
    return s["workspace"][op]


def _own(s):
    from lm_head_cross_pg_amd import abi
    op, mask, D = s["op"], s["mask"], s["D"]
    if op == "norm":
        abi.pg_layernorm_fwd(s["x"], s["weight"], s["bias"], mask, EPS, s["y"])
        return s["y"]
    if op == "grad":
        ws = _workspace(s, abi, abi.PG_OP_LN_BWD, s["x"].shape[0], D, 1)
        abi.pg_layernorm_bwd(s["x"], s["weight"], mask, s["dy"], EPS, s["dx"], s["dweight"], s["dbias"], ws)
        return s["dx"], s["dweight"], s["dbias"]
    if op == "quant":
        abi.pg_quantize_mx4(s["x"], None, s["codes"], s["scales"])
        abi.pg_dequantize_mx4(s["codes"], s["scales"], s["y"])
        return s["y"]
    if op == "score":
        abi.pg_layernorm_fwd_mx4(s["x"], s["weight"], s["bias"], mask, EPS, s["codes"], s["scales"])
    ws = _workspace(s, abi, abi.PG_OP_FWD_MX4, s["codes"].shape[0], D, s["embed"].shape[0])
    abi.pg_lmhead_ce_fwd_mx4(s["codes"], s["scales"], s["embed"], s["embed_scales"], s["target"], mask, D,
                             s["softcap"], s["nats"], s["lse"], ws)
    return s["nats"], s["lse"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------- in 64 bits
_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)   # between neighbouring levels: ties to the even code


def _exact_norm(x, weight, bias):
    x = x.double()
    n = x.shape[1]
    mean = x.sum(1) / n
    var = ((x - mean[:, None]) ** 2).sum(1) / n
    return (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None], 1 / torch.sqrt(var + EPS)


def _exact_rounded(x):
    """Rows as the nearest values of the 4-bit format, in float64, by comparing with every border."""
    T, D = x.shape
    x = torch.cat((x.double(), torch.zeros((T, -D % 32), dtype=torch.float64, device=x.device)), 1).view(T, -1, 32)
    top = x.abs().max(2).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2   # one off at most
    e = torch.where(top >= 7 * torch.exp2(e), e + 1, e)
    e = torch.where(top >= 7 * torch.exp2(e), e + 1, e)
    e = torch.where(top < 3.5 * torch.exp2(e), e - 1, e)
    unit = torch.exp2(torch.where(top > 0, e.clamp(-127, 125), -127.0))[:, :, None]
    at = torch.tensor(_BORDERS, dtype=torch.float64, device=x.device)
    at[0::2] = torch.nextafter(at[0::2], at[0::2] + 1)                  # a tie there goes down
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    q = level[torch.searchsorted(at, (x.abs() / unit).contiguous(), right=True)]
    return (torch.sign(x) * q * unit).flatten(1)[:, :D]


def _exact_rows(codes, scales, D):
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=codes.device)
    k = torch.arange(D, device=codes.device)
    nibble = (codes.long()[:, k // 2] >> (4 * (k % 2))) & 15
    return table[nibble] * torch.exp2(scales.double()[:, k // 32] - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op, D, mask = case["op"], case["D"], s["mask"]
    on = None if mask is None else mask.bool()
    if op == "norm":
        y = _exact_norm(s["x"], s["weight"], s["bias"])[0] * s["weight"].double() + s["bias"].double()
        return y if on is None else y * on[:, None]
    if op == "grad":
        xh, r = _exact_norm(s["x"], s["weight"], None)
        dy = s["dy"].double() if on is None else s["dy"].double() * on[:, None]
        g = dy * s["weight"].double()
        dx = (g - g.sum(1, keepdim=True) / D - xh * ((g * xh).sum(1, keepdim=True) / D)) * r[:, None]
        return dx, (dy * xh).sum(0), dy.sum(0)
    if op == "quant":
        return _exact_rounded(s["x"])
    if op == "score":
        y = _exact_norm(s["x"], s["weight"], s["bias"])[0] * s["weight"].double() + s["bias"].double()
        h = _exact_rounded(y.float())
    else:
        h = _exact_rows(s["codes"], s["scales"], D)
    e, cap = _exact_rows(s["embed"], s["embed_scales"], D), case["cap"]
    nats, lse = [], []
    for rows in torch.split(torch.arange(case["T"], device="cuda"), 8192):
        z = torch.mm(h[rows], e.t())
        if cap > 0:
            z = cap * torch.tanh(z / cap)
        total = torch.logsumexp(z, 1)
        lse.append(total)
        nats.append(total - z[torch.arange(len(rows), device="cuda"), s["target"][rows].long()])
    nats, lse = torch.cat(nats), torch.cat(lse)
    return (nats, lse) if on is None else (nats * on, lse * on)
