"""The sliding-window driver from the model's last states on: the final norm in front of the bf16 and of
the 4-bit head, and score-first training of the norm and the embedding, batch by batch against the
oracle. nats and gradients of the bf16 head within the parity tolerances; the norm's gradients against
the oracle's norm backward of the GPU's own dH; the SGD steps bit for bit."""
import numpy as np
import pytest
import torch

from lm_head_cross_pg_amd import abi
from lm_head_cross_pg_amd.window_eval import SlidingWindowEval
from oracle import oracle as ora
from tests.gpu_helpers import BPB_RTOL, GRAD_RL2, NATS_ATOL, ensure_lib, rel_l2
from tests.test_gpu_mx4 import tolerance

pytestmark = pytest.mark.gpu
N, D, V, WINDOW, STRIDE, CAP = 700, 128, 300, 64, 16, 30.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def f64(t):
    return t.double().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def setup(seed, x_dtype):
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    blen = torch.randint(1, 9, (V,), generator=g, dtype=torch.int32).cuda()
    embed = (0.1 * torch.randn((V, D), generator=g)).to(torch.bfloat16).cuda()
    weight, bias = (2 + 0.2 * torch.randn(D, generator=g)).cuda(), (0.2 * torch.randn(D, generator=g)).cuda()

    def states(w0, nw):
        gg = torch.Generator().manual_seed(seed + 1000 + w0)
        return (3 * torch.randn((nw * WINDOW, D), generator=gg) + 0.5).to(x_dtype).cuda()

    return tokens, blen, embed, weight, bias, states


def totals(drv, nats, targets, blen):
    sn, sb, n, bpb = drv.result()
    want = ora.bpb(np.concatenate(nats), np.concatenate(targets), blen.cpu().numpy())
    assert n == N - 1 == want[2] and sb == want[1]
    assert abs(sn - want[0]) <= BPB_RTOL * want[0] and abs(bpb - want[3]) <= BPB_RTOL * want[3]


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("per_batch", [3, 7])
def test_norm_then_bf16_head(x_dtype, per_batch):
    tokens, blen, embed, weight, bias, states = setup(1, x_dtype)
    drv = SlidingWindowEval(tokens, blen, V, D, WINDOW, STRIDE, per_batch, CAP, final_norm=(weight, bias))
    nats, targets = [], []
    for w0, nw in drv.batches():
        x = states(w0, nw)
        print(f"[case] driver norm {x_dtype} w0={w0} nw={nw}", flush=True)
        n = drv.step(x, embed, w0, nw)
        on = drv.mask[:nw * WINDOW].cpu().numpy() != 0
        y = drv.target[:nw * WINDOW].cpu().numpy()
        h = f64(bf16(ora.layer_norm(f64(x), f64(weight), f64(bias))))
        ref, _ = ora.forward(h[on], f64(embed), y[on], CAP)
        assert n == on.sum() and np.max(np.abs(f64(drv.nats[:nw * WINDOW])[on] - ref)) <= NATS_ATOL
        nats.append(ref)
        targets.append(y[on])
    totals(drv, nats, targets, blen)


@pytest.mark.parametrize("norm", [True, False])
def test_mx4_head(norm):
    tokens, blen, embed, weight, bias, states = setup(2, torch.bfloat16)
    ec = torch.empty((V, abi.pg_mx4_code_bytes(D)), dtype=torch.uint8, device="cuda")
    es = torch.empty((V, abi.pg_mx4_scale_bytes(D)), dtype=torch.uint8, device="cuda")
    abi.pg_quantize_mx4(embed, None, ec, es)
    E = ora.quantize_rows_mx4(f64(embed))[0]
    drv = SlidingWindowEval(tokens, blen, V, D, WINDOW, STRIDE, 5, CAP, mx4_head=True,
                            final_norm=(weight, bias) if norm else None)
    nats, targets = [], []
    for w0, nw in drv.batches():
        x = states(w0, nw)
        print(f"[case] driver 4-bit norm={norm} w0={w0} nw={nw}", flush=True)
        n = drv.step_mx4(x, ec, es, w0, nw)
        on = drv.mask[:nw * WINDOW].cpu().numpy() != 0
        y = drv.target[:nw * WINDOW].cpu().numpy()
        h = ora.layer_norm(f64(x), f64(weight), f64(bias)).astype(np.float32) if norm else f64(x)
        h = ora.quantize_rows_mx4(h)[0]
        ref, _ = ora.forward(h[on], E, y[on], CAP)
        assert n == on.sum()
        assert np.max(np.abs(f64(drv.nats[:nw * WINDOW])[on] - ref)) <= tolerance(h[on], E, CAP, V)
        nats.append(ref)
        targets.append(y[on])
    totals(drv, nats, targets, blen)
    with pytest.raises(ValueError, match="step_mx4"):
        drv.step(states(0, 1), embed, 0, 1)


@pytest.mark.parametrize("ttt_lr,norm_lr,keep", [(2.0, 0.5, False), (0.0, 0.5, True), (2.0, 0.0, True), (2.0, 0.0, False)])
def test_training_from_the_last_states(ttt_lr, norm_lr, keep):
    tokens, blen, embed, weight, bias, states = setup(3, torch.float32)
    master = embed.float()
    drv = SlidingWindowEval(tokens, blen, V, D, WINDOW, STRIDE, 6, CAP, ttt_lr=ttt_lr,
                            embed_master=master if ttt_lr else None, keep_dhidden=keep, final_norm=(weight, bias),
                            norm_lr=norm_lr)
    for w0, nw in drv.batches():
        x, rows = states(w0, nw), nw * WINDOW
        print(f"[case] driver training lr={ttt_lr} norm_lr={norm_lr} keep={keep} w0={w0} nw={nw}", flush=True)
        w_before, b_before, e_before = weight.clone(), bias.clone(), embed.clone()
        n = drv.step(x, embed, w0, nw)
        mask = drv.mask[:rows].cpu().numpy()
        on, y = mask != 0, drv.target[:rows].cpu().numpy()
        h = f64(bf16(ora.layer_norm(f64(x), f64(w_before), f64(b_before))))
        ref, _ = ora.forward(h, f64(e_before), y, CAP, mask)
        assert np.max(np.abs(f64(drv.nats[:rows]) - ref)) <= NATS_ATOL
        dH, dE = ora.backward(h, f64(e_before), y, CAP, 1.0 / n, mask)
        assert rel_l2(f64(drv.dE), dE) <= GRAD_RL2
        if norm_lr or keep:
            got = f64(drv.dH[:rows])
            assert rel_l2(got, dH) <= GRAD_RL2
            rdx, rdw, rdb = ora.layer_norm_backward(f64(x), f64(w_before), got, 1e-5, mask)
            if keep:
                assert rel_l2(f64(drv.dX[:rows]), rdx) <= 1e-5 and not f64(drv.dX[:rows])[~on].any()
        if norm_lr:
            dw, db = drv.dnorm
            assert rel_l2(f64(dw), rdw) <= 1e-5 and rel_l2(f64(db), rdb) <= 1e-5
            for p, before, grad in ((weight, w_before, dw), (bias, b_before, db)):
                u = (np.float32(norm_lr) * grad.cpu().numpy()).astype(np.float32)
                np.testing.assert_array_equal(p.cpu().numpy(), before.cpu().numpy() - u)
        else:
            assert torch.equal(weight, w_before) and torch.equal(bias, b_before)
        assert torch.equal(embed, e_before) == (ttt_lr == 0.0)
    assert abs(drv.result()[2] - (N - 1)) == 0


def test_driver_refusals():
    tokens, blen, embed, weight, bias, states = setup(4, torch.float32)
    make = lambda **kw: SlidingWindowEval(tokens, blen, V, D, WINDOW, STRIDE, **kw)  # noqa: E731
    for kw, msg in ((dict(mx4_head=True, int8_head=True), "4-bit head"), (dict(mx4_head=True, norm_lr=1.0, final_norm=(weight, bias)), "4-bit head"),
                    (dict(int8_head=True, final_norm=(weight, bias)), "int8 head"), (dict(norm_lr=1.0), "norm_lr needs"),
                    (dict(norm_lr=1.0, final_norm=(None, None)), "norm_lr needs"),
                    (dict(mx4_head=True, ttt_lr=1.0, embed_master=embed.float()), "4-bit head")):
        with pytest.raises(ValueError, match=msg):
            make(**kw)
    with pytest.raises(ValueError, match="mx4_head=True"):
        make().step_mx4(states(0, 1), None, None, 0, 1)
