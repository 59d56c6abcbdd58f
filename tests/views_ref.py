"""64-bit reference of the view-cache operators: one view and one head at a time, and the
bounds on a kernel's error that follow from its roundings."""

from __future__ import annotations

import torch

NEG = float("-inf")
U32 = 2.0 ** -24            # half a step of fp32, relative
U16 = torch.finfo(torch.bfloat16).eps / 2  # of bf16: 2^-8


def views(q_off, own_off):
    for b in range(len(q_off) - 1):
        yield b, slice(q_off[b], q_off[b + 1]), slice(own_off[b], own_off[b + 1])


def seen(nq, nk, causal, device):
    """[nq, nk]: does query i see own key j."""
    if not causal:
        return torch.ones(nq, nk, dtype=torch.bool, device=device)
    i, j = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)[None]
    return j - nk <= i - nq


def scores(q, kp, ko, rows, cols, h, hk, causal, scale):
    k = torch.cat((kp[:, hk], ko[cols, hk])).double()
    qd = q[rows, h].double()
    s = scale * (qd @ k.T)
    size = scale * (qd.abs() @ k.abs().T)  # what its rounding errors go by
    see = seen(qd.shape[0], ko[cols].shape[0], causal, q.device)
    s[:, kp.shape[0]:].masked_fill_(~see, NEG)
    return s, size


def attend(q, kp, vp, ko, vo, q_off, own_off, causal=False, scale=0.125):
    """out, lse and the bounds on a kernel's error in each, all float64; rows of no view are NaN.

    A score is a sum of 64 exact products kept in fp32: an error of at most 64 roundings of the sum of their
    magnitudes, two units each where the tensor core cuts off instead of rounding; its scaling adds two.  The
    exponential is within 4e-6, the weight for the product with V is rounded to bf16, the result to bf16.  A sum of n weights
    takes at most n / 16 + 64 roundings of its total on the way (chains of a key tile, then tiles, then parts).
    """
    H, Hk = q.shape[1], kp.shape[1]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64, device=q.device)
    tol_out, tol_lse = out.clone(), lse.clone()
    for b, rows, cols in views(q_off, own_off):
        for h in range(H):
            hk = h // (H // Hk)
            s, size = scores(q, kp, ko, rows, cols, h, hk, causal, scale)
            n = s.shape[1]
            if n == 0 or s.shape[0] == 0:
                out[rows, h], lse[rows, h], tol_out[rows, h], tol_lse[rows, h] = 0, NEG, 0, 0
                continue
            v = torch.cat((vp[:, hk], vo[cols, hk])).double()
            z = torch.logsumexp(s, 1)
            none = z == NEG
            p = torch.where(none[:, None], torch.zeros_like(s), (s - z[:, None]).exp())
            out[rows, h] = p @ v
            lse[rows, h] = z
            top = torch.where(p > 0, size, torch.zeros_like(size)).amax(1)
            rel = 2 * (130 * U32 * top) + 4e-6 + (n / 16 + 64) * U32  # weight against weight, and their sum
            tol_out[rows, h] = (U16 + rel)[:, None] * (p @ v.abs()) * 1.01 + U16 * out[rows, h].abs() * 1.01 + 1e-30
            tol_lse[rows, h] = torch.where(none, torch.zeros_like(z), rel + 8 * U32 * (z.abs() + top))
    return out, lse, tol_out, tol_lse
