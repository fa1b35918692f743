"""Sliding-window evaluation of a token stream, with optional score-first test-time training of the
tied embedding, driven through the library's C ABI (include/pg_lmhead.h).

Windows of ``window`` tokens advance by ``stride`` over the stream; each scores only the predictions
no earlier window scored (parameter-golf README leaderboard, "Sliding Window Eval" row, stride 64).
Batches of ``windows_per_batch`` windows are scored one after another, and the bits per byte
accumulate over all of them on the device. With ``ttt_lr > 0`` each batch, once scored, also yields
the gradient of its mean loss with respect to the tied embedding (the hidden states' gradient only
with ``keep_dhidden``), and the embedding takes one SGD step on it before the next batch is
scored: score-first test-time training, every chunk adapted on only after it has been
scored (README leaderboard, "Legal Score-First TTT" rows, and the row that trains in phases on
validation chunks already scored).

The driver can take the model's last states instead of the final norm's output: with ``final_norm`` it
runs the norm on the rows a batch scores, and with ``norm_lr > 0`` the norm's gain and bias take an SGD
step of their own after each scored batch.

This module only sequences calls: the schedule's arithmetic, the rows of each batch, the forward,
the backward, the sums and the update all run in the library. The hidden states of each batch
come from the caller (the model run on each window).
"""
from __future__ import annotations

from typing import Iterator, Optional, Tuple

import torch

from . import abi


class SlidingWindowEval:
    def __init__(self, tokens: torch.Tensor, byte_len: torch.Tensor, V: int, D: int, window: int = 2048,
                 stride: int = 64, windows_per_batch: int = 32, softcap: float = 30.0, ttt_lr: float = 0.0,
                 embed_master: Optional[torch.Tensor] = None, keep_dhidden: bool = False,
                 int8_head: bool = False, mx4_head: bool = False,
                 final_norm: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
                 norm_eps: float = 1e-5, norm_lr: float = 0.0):
        """keep_dhidden: with ttt_lr > 0, also compute the gradient of the hidden states of each
        batch (into self.dH). The embedding step needs only dE, so by default dH is left out and
        its product is not run.
        int8_head: score the per-row int8 form of the tied embedding (pg_quantize_q8) with
        step_int8, as a model evaluated after quantisation is (README leaderboard, "Mixed Quant +
        Sliding Window Eval": int8 embeddings); evaluation only, no test-time training.
        mx4_head: score the 4-bit form of the tied embedding (pg_quantize_mx4) with step_mx4, the states
        of the scored rows brought to 4 bits too; evaluation only.
        final_norm: (weight, bias) of the final layer norm, float32 [D] each or None. The hidden states
        given to step and step_mx4 are then the model's last states (bf16 or float32), and the norm runs
        on the rows a batch scores, with norm_eps.
        norm_lr: with final_norm, after each scored batch one SGD step of weight and bias (in place,
        where given) on the gradient of the batch's mean loss; ttt_lr may be 0 then, which leaves the
        embedding as it is. With keep_dhidden, self.dX is the gradient of the batch's last states."""
        if ttt_lr and embed_master is None:
            raise ValueError("score-first TTT needs float32 master weights of the embedding (embed_master)")
        if ttt_lr and int8_head:
            raise ValueError("test-time training updates a bf16 embedding; the int8 head is evaluation only")
        if mx4_head and (ttt_lr or norm_lr or int8_head):
            raise ValueError("the 4-bit head is evaluation only, and takes the place of the int8 head")
        if int8_head and final_norm is not None:
            raise ValueError("the int8 head takes the final norm's output: final_norm is for the other heads")
        if norm_lr and (final_norm is None or all(t is None for t in final_norm)):
            raise ValueError("norm_lr needs the final norm's weight or bias")
        self.int8_head, self.mx4_head = bool(int8_head), bool(mx4_head)
        self.final_norm, self.norm_eps, self.norm_lr = final_norm, float(norm_eps), float(norm_lr)
        self.tokens, self.byte_len, self.V, self.D = tokens, byte_len, int(V), int(D)
        self.window, self.stride, self.per_batch = int(window), int(stride), int(windows_per_batch)
        self.softcap, self.ttt_lr, self.embed_master = float(softcap), float(ttt_lr), embed_master
        self.keep_dhidden = bool(keep_dhidden)
        self.n_windows = abi.pg_window_count(tokens.numel(), self.window, self.stride)
        dev = tokens.device
        rows = self.per_batch * self.window
        self.target = torch.empty(rows, dtype=torch.int32, device=dev)
        self.mask = torch.empty(rows, dtype=torch.uint8, device=dev)
        self.nats = torch.empty(rows, dtype=torch.float32, device=dev)
        self.lse = torch.empty(rows, dtype=torch.float32, device=dev)
        # running sums (nats, bytes, predictions) and their bits per byte: NaN (0 / 0) until a batch
        # with predictions has been scored, as for a stream too short to predict anything
        self.out = torch.tensor([0.0, 0.0, 0.0, float("nan")], dtype=torch.float64, device=dev)
        train = bool(self.ttt_lr or self.norm_lr)
        op = (abi.PG_OP_FWD_BWD if train else abi.PG_OP_FWD_Q8 if self.int8_head else
              abi.PG_OP_FWD_MX4 if self.mx4_head else abi.PG_OP_FWD)
        self.ws = torch.empty(max(abi.workspace_bytes(op, rows, self.D, self.V), 256), dtype=torch.uint8, device=dev)
        self.ws_bpb = torch.empty(max(abi.workspace_bytes(abi.PG_OP_BPB, rows, 1, self.V), 256), dtype=torch.uint8,
                                  device=dev)
        self.dH = self.dX = None
        if train:
            if self.keep_dhidden or self.norm_lr:
                self.dH = torch.empty((rows, self.D), dtype=torch.float32, device=dev)
            self.dE = torch.empty((self.V, self.D), dtype=torch.float32, device=dev)
        if self.mx4_head:
            self.codes = torch.zeros((rows, abi.pg_mx4_code_bytes(self.D)), dtype=torch.uint8, device=dev)
            self.scales = torch.zeros((rows, abi.pg_mx4_scale_bytes(self.D)), dtype=torch.uint8, device=dev)
        elif final_norm is not None:
            self.normed = torch.zeros((rows, self.D), dtype=torch.bfloat16, device=dev)
            if train and (self.keep_dhidden or self.norm_lr):
                self.ws_norm = torch.empty(abi.workspace_bytes(abi.PG_OP_LN_BWD, rows, self.D, 1), dtype=torch.uint8,
                                           device=dev)
                if self.keep_dhidden:
                    self.dX = torch.empty((rows, self.D), dtype=torch.float32, device=dev)
            if self.norm_lr:
                self.dnorm = tuple(None if t is None else torch.empty_like(t) for t in final_norm)
                # the SGD step also writes a bf16 copy, which nothing reads here
                self.norm_bf16 = torch.empty(self.D, dtype=torch.bfloat16, device=dev)

    def batches(self) -> Iterator[Tuple[int, int]]:
        """(first window, number of windows) of each batch, in order."""
        for w0 in range(0, self.n_windows, self.per_batch):
            yield w0, min(self.per_batch, self.n_windows - w0)

    def scored(self, first_window: int, n_windows: int) -> int:
        return abi.pg_window_scored(self.tokens.numel(), self.window, self.stride, first_window, n_windows)

    def step(self, hidden: torch.Tensor, embed: torch.Tensor, first_window: int, n_windows: int) -> int:
        """Score one batch. hidden: [n_windows * window, D] bf16, row (b, r) the hidden state of
        input position (first_window + b) stride + r in its window (only scored rows are read); with
        final_norm the model's last states, bf16 or float32.
        embed: the bf16 tied embedding [V, D], updated in place by the SGD step when ttt_lr > 0.
        Returns the number of predictions the batch scored."""
        rows = n_windows * self.window
        tgt, msk, nats, lse = self.target[:rows], self.mask[:rows], self.nats[:rows], self.lse[:rows]
        if self.mx4_head:
            raise ValueError("a driver built with mx4_head=True scores with step_mx4 (its workspace)")
        abi.pg_window_rows(self.tokens, self.window, self.stride, first_window, n_windows, tgt, msk)
        n = self.scored(first_window, n_windows)
        states = hidden
        if self.final_norm is not None:
            weight, bias = self.final_norm
            hidden = self.normed[:rows]
            abi.pg_layernorm_fwd(states, weight, bias, msk, self.norm_eps, hidden)
        if (self.ttt_lr or self.norm_lr) and n > 0:
            # the batch's scores and the gradients of its mean loss come from the same embedding and
            # norm; the updates reach only later batches
            dH = self.dH[:rows] if self.dH is not None else None
            abi.pg_lmhead_ce_fwd_bwd(hidden, embed, tgt, msk, self.softcap, 1.0 / n, nats, lse, dH, self.dE, self.ws)
            abi.pg_bpb_accumulate(nats, tgt, msk, self.byte_len, None, self.V, self.out, self.ws_bpb)
            if self.final_norm is not None and dH is not None:
                dX = self.dX[:rows] if self.dX is not None else None
                grads = self.dnorm if self.norm_lr else (None, None)
                abi.pg_layernorm_bwd(states, weight, msk, dH, self.norm_eps, dX, *grads, self.ws_norm)
                for param, grad in zip(self.final_norm, grads):
                    if grad is not None:
                        abi.pg_sgd_step_bf16(param, grad, self.norm_lr, self.norm_bf16)
            if self.ttt_lr:
                abi.pg_sgd_step_bf16(self.embed_master, self.dE, self.ttt_lr, embed)
        else:
            abi.pg_lmhead_ce_fwd(hidden, embed, tgt, msk, self.softcap, nats, lse, self.ws)
            abi.pg_bpb_accumulate(nats, tgt, msk, self.byte_len, None, self.V, self.out, self.ws_bpb)
        return n

    def step_int8(self, hidden: torch.Tensor, embed_q8: torch.Tensor, embed_scale: torch.Tensor,
                  first_window: int, n_windows: int) -> int:
        """Score one batch on the int8 head (embed_q8 [V, D] int8, embed_scale [V] float32, from
        pg_quantize_q8); hidden as for step. Returns the number of predictions the batch scored."""
        if not self.int8_head:
            raise ValueError("step_int8 needs a driver built with int8_head=True (its workspace)")
        rows = n_windows * self.window
        tgt, msk, nats, lse = self.target[:rows], self.mask[:rows], self.nats[:rows], self.lse[:rows]
        abi.pg_window_rows(self.tokens, self.window, self.stride, first_window, n_windows, tgt, msk)
        n = self.scored(first_window, n_windows)
        abi.pg_lmhead_ce_fwd_q8(hidden, embed_q8, embed_scale, tgt, msk, self.softcap, nats, lse, self.ws)
        abi.pg_bpb_accumulate(nats, tgt, msk, self.byte_len, None, self.V, self.out, self.ws_bpb)
        return n

    def step_mx4(self, hidden: torch.Tensor, embed_codes: torch.Tensor, embed_scales: torch.Tensor,
                 first_window: int, n_windows: int) -> int:
        """Score one batch on the 4-bit head (embed_codes and embed_scales from pg_quantize_mx4); hidden
        as for step, bf16 or float32. Returns the number of predictions the batch scored."""
        if not self.mx4_head:
            raise ValueError("step_mx4 needs a driver built with mx4_head=True (its workspace)")
        rows = n_windows * self.window
        tgt, msk, nats, lse = self.target[:rows], self.mask[:rows], self.nats[:rows], self.lse[:rows]
        abi.pg_window_rows(self.tokens, self.window, self.stride, first_window, n_windows, tgt, msk)
        n = self.scored(first_window, n_windows)
        codes, scales = self.codes[:rows], self.scales[:rows]
        if self.final_norm is not None:
            abi.pg_layernorm_fwd_mx4(hidden, *self.final_norm, msk, self.norm_eps, codes, scales)
        else:
            abi.pg_quantize_mx4(hidden, msk, codes, scales)
        abi.pg_lmhead_ce_fwd_mx4(codes, scales, embed_codes, embed_scales, tgt, msk, self.D, self.softcap, nats, lse,
                                 self.ws)
        abi.pg_bpb_accumulate(nats, tgt, msk, self.byte_len, None, self.V, self.out, self.ws_bpb)
        return n

    def result(self):
        """(sum of nats, sum of bytes, predictions scored, bits per byte) over the batches so far."""
        return self.out.cpu().tolist()
