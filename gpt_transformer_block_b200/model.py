"""Device-memory holders around the C ABI (PyTorch allocates; the library computes).

GPTStack   weights, fp32 gradient buffers and the step workspace of a whole
           stack; ``step(idx, targets)`` enqueues one gpt_stack_step.
BlockRunner one block's saved-activation and scratch workspaces for
           gpt_block_forward / gpt_block_backward.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import (BF16, F32, WS_BLOCK_SAVED, WS_BLOCK_SCRATCH, WS_LM_HEAD, WS_STACK, _device, _flat, _rows, block_grads,
               block_weights, gpt_block_backward, gpt_block_forward, gpt_stack_step, gptb_gemm_bf16, gptb_policy_loss,
               gptb_policy_loss_workspace_bytes, gptb_token_logprobs, gptb_workspace_bytes, lm_head_xent, make_config,
               model_grads, model_weights)


def storage_torch_dtype(c: dict) -> torch.dtype:
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def to_device_weights(c: dict, w: dict, device="cuda") -> dict:
    """Copy synthetic (CPU fp32) weights to the device in the storage dtype."""
    dt = storage_torch_dtype(c)

    def mat(t):
        return t.to(device=device, dtype=dt).contiguous()

    out = {"layers": []}
    for lw in w["layers"]:
        d = {k: mat(lw[k]) for k in ("w_qkv", "w_o", "w_fc", "w_proj")}
        d["lambdas"] = torch.tensor([lw["resid_lambda"], lw["x0_lambda"]], dtype=torch.float32, device=device)
        if "w_ve_gate" in lw:
            d["w_ve_gate"] = mat(lw["w_ve_gate"])
            d["ve_table"] = mat(lw["ve_table"])
        out["layers"].append(d)
    for k in ("wte", "w_lm", "w_smear_gate"):
        if k in w:
            out[k] = mat(w[k])
    for k in ("smear_lambda", "backout_lambda"):
        if k in w:
            out[k] = torch.tensor([w[k]], dtype=torch.float32, device=device)
    return out


def zero_grads_like(c: dict, dw: dict) -> dict:
    """fp32 gradient buffers matching the device weights."""
    g = {"layers": []}
    for lw in dw["layers"]:
        g["layers"].append({k: torch.zeros(v.shape, dtype=torch.float32, device=v.device) for k, v in lw.items()})
    for k in ("wte", "w_lm", "w_smear_gate", "smear_lambda", "backout_lambda"):
        if k in dw:
            g[k] = torch.zeros(dw[k].shape, dtype=torch.float32, device=dw[k].device)
    return g


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


class GPTStack:
    """One stack's weights, gradients and step workspace on the current device."""

    def __init__(self, c: dict, weights: dict, device="cuda"):
        self.c = c
        self.cfg = make_config(c)
        self.device = torch.device(device)
        self.w = to_device_weights(c, weights, device)
        self.g = zero_grads_like(c, self.w)
        self.ws = _ws(gptb_workspace_bytes(self.cfg, WS_STACK), self.device)
        self.loss = torch.zeros(1, dtype=torch.float32, device=self.device)
        self._mw = model_weights(self.w)
        self._mg = model_grads(self.g)

    def zero_grad(self):
        for lg in self.g["layers"]:
            for v in lg.values():
                v.zero_()
        for k, v in self.g.items():
            if k != "layers":
                v.zero_()

    def step(self, idx: torch.Tensor, targets: torch.Tensor, stream=None) -> torch.Tensor:
        """Forward + backward of the whole stack; grads accumulate; returns the loss tensor."""
        gpt_stack_step(self.cfg, self._mw, idx, targets, self.loss, self._mg, self.ws, stream)
        return self.loss


class BlockRunner:
    """Workspaces for one block's forward/backward through the C ABI."""

    def __init__(self, c: dict, device="cuda"):
        self.c = c
        self.cfg = make_config(c)
        self.device = torch.device(device)
        self.saved = _ws(gptb_workspace_bytes(self.cfg, WS_BLOCK_SAVED), self.device)
        self.scratch = _ws(gptb_workspace_bytes(self.cfg, WS_BLOCK_SCRATCH), self.device)

    def forward(self, layer, lw: dict, x, x0, idx, x_out, stream=None):
        gpt_block_forward(self.cfg, layer, block_weights(lw), x, x0, idx, x_out, self.saved, self.scratch, stream)

    def backward(self, layer, lw: dict, x, x0, idx, dx_out, dx, dx0_accum, lg: dict, dx_extra=None,
                 stream=None):
        gpt_block_backward(self.cfg, layer, block_weights(lw), x, x0, idx, self.saved, dx_out, dx_extra, dx,
                           dx0_accum, block_grads(lg), self.scratch, stream)


def lm_head(c: dict, h, w_lm, targets, dh, dw_lm, stream=None):
    """lm_head_xent through the C ABI with a fresh workspace; returns the loss tensor."""
    cfg = make_config(c)
    ws = _ws(gptb_workspace_bytes(cfg, WS_LM_HEAD), h.device)
    loss = torch.zeros(1, dtype=torch.float32, device=h.device)
    lm_head_xent(cfg, h, w_lm, targets, loss, dh, dw_lm, ws, stream)
    return loss


def _matrix(name: str, t, rows: int, cols: int, dtype, dev) -> int:
    """The row stride of t, a [rows, cols] matrix as the GEMM takes it (contiguous rows, 16-byte boundaries)."""
    if t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, wanted [{rows}, {cols}]")
    at, ld = _rows(name, t, cols, dtype, dev, rows)
    if at % 16 or ld * t.element_size() % 16 or ld < cols:
        raise ValueError(f"{name}: rows on 16-byte boundaries are wanted (address {at}, row stride {ld})")
    return ld


def _head(h, w_lm, rows_per_chunk):
    """(device, rows, d, vocab, row strides of h and w_lm) of an lm_head over h."""
    dev = _device("h", h)
    if h.dim() != 2 or w_lm.dim() != 2:
        raise ValueError(f"h, w_lm: matrices are wanted, not {tuple(h.shape)}, {tuple(w_lm.shape)}")
    if rows_per_chunk < 1:
        raise ValueError(f"rows_per_chunk: {rows_per_chunk}")
    (N, d), V = h.shape, w_lm.shape[0]
    if d % 8 or V % 8 or not d or not V:
        raise ValueError(f"d and the vocabulary have to be multiples of 8, not {d}, {V}")
    return dev, N, d, V, _matrix("h", h, N, d, torch.bfloat16, dev), _matrix("w_lm", w_lm, V, d, torch.bfloat16, dev)


def _current(dev):
    """dev as the current device, on whose current stream every launch of a call is made."""
    return contextlib.nullcontext() if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def lm_head_logprobs(h, w_lm, tokens, rows_per_chunk=8192):
    """Log-probabilities [N] of the given tokens (int32 [N]) under logits h w_lm^T (bf16 h [N, d], w_lm [V, d], column
    ranges of wider arrays are fine; d and V multiples of 8), a chunk of rows at a time, on the current stream of the
    tensors' device: what the sampling and the reference policy hand to lm_head_policy.  ValueError where an argument
    does not fit, before anything is launched."""
    dev, N, d, V, ldh, ldw = _head(h, w_lm, rows_per_chunk)
    _flat("tokens", tokens, torch.int32, dev, N)
    with _current(dev):
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        z = torch.empty(min(N, rows_per_chunk), V, dtype=torch.bfloat16, device=dev)
        for i in range(0, N, rows_per_chunk):
            n = min(rows_per_chunk, N - i)
            gptb_gemm_bf16(h[i:i + n], 0, ldh, w_lm, 0, ldw, z, 0, V, n, V, d)
            gptb_token_logprobs(z[:n], tokens[i:i + n], logp[i:i + n])
    return logp


def lm_head_policy(h, w_lm, actions, weights, advantages, logp_old, logp_ref, clip_lo, clip_hi, beta, dh, dw_lm,
                   rows_per_chunk=8192):
    """The lm_head with the clipped policy loss in the place of the cross entropy: logits h w_lm^T of bf16 h [N, d] and
    w_lm [V, d] (d and V multiples of 8), gptb_policy_loss over them, and the gradients dh (bf16 [N, d], overwritten; may
    be h itself) and dw_lm (fp32 [V, d], accumulated); the matrices may be column ranges of wider arrays.  A chunk of rows at a time,
    the gradient over the logits, so the [N, V] logits never exist whole; on the current stream of the tensors' device.
    A row of weight 0 adds nothing, whatever its h and its other values are; its dh is 0.
    Returns (stats [3]: loss, KL, clipped weight; logp [N]).  ValueError where an argument does not fit, before anything
    is launched."""
    dev, N, d, V, ldh, ldw = _head(h, w_lm, rows_per_chunk)
    lddh = _matrix("dh", dh, N, d, torch.bfloat16, dev)
    lddw = _matrix("dw_lm", dw_lm, V, d, torch.float32, dev)
    _flat("actions", actions, torch.int32, dev, N)
    for name, t in (("weights", weights), ("advantages", advantages), ("logp_old", logp_old), ("logp_ref", logp_ref)):
        if t is not None or name != "logp_ref":
            _flat(name, t, torch.float32, dev, N)
    if not 0 <= clip_lo <= 1 or not clip_hi >= 0 or not math.isfinite(beta) or (beta and logp_ref is None):
        raise ValueError(f"clip borders {clip_lo}, {clip_hi}, beta {beta} (with a beta logp_ref is needed)")
    with _current(dev):
        stats = torch.zeros(3, dtype=torch.float32, device=dev)
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        part = torch.empty(3, dtype=torch.float32, device=dev)
        rows = max(1, min(N, rows_per_chunk))
        z = torch.empty(rows, V, dtype=torch.bfloat16, device=dev)
        ws = _ws(gptb_policy_loss_workspace_bytes(rows), dev)
        for i in range(0, N, rows_per_chunk):
            n, at = min(rows_per_chunk, N - i), slice(i, min(N, i + rows_per_chunk))
            gptb_gemm_bf16(h[at], 0, ldh, w_lm, 0, ldw, z, 0, V, n, V, d)
            gptb_policy_loss(z[:n], actions[at], weights[at], advantages[at], logp_old[at],
                             None if logp_ref is None else logp_ref[at], clip_lo, clip_hi, beta, z[:n], logp[at], part, ws)
            # (0 times a NaN is NaN: what a row of weight 0 holds must not meet the gradient's zeros)
            hw = torch.where((weights[at] != 0)[:, None], h[at], 0)
            gptb_gemm_bf16(z, 1, V, hw, 1, d, dw_lm, 1, lddw, V, d, n)
            gptb_gemm_bf16(z, 0, V, w_lm, 1, ldw, dh[at], 0, lddh, n, d, V)
            stats += part
    return stats, logp


__all__ = ["GPTStack", "BlockRunner", "to_device_weights", "zero_grads_like", "lm_head", "lm_head_logprobs",
           "lm_head_policy", "BF16", "F32"]
