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


def weights(q, kp, ko, q_off, own_off, lse, acc=None, decay=1.0, causal=False, scale=0.125):
    """acc_out and the bounds on a kernel's error in it; own tokens of no view are NaN.

    Weight against weight as in attend; the log sum is given, its product with log2(e) and the difference to the
    score are rounded.
    """
    H, Hk, P = q.shape[1], kp.shape[1], kp.shape[0]
    w = torch.full((Hk, P + ko.shape[0]), float("nan"), dtype=torch.float64, device=q.device)
    w[:, :P] = 0
    tol = w.clone()
    for b, rows, cols in views(q_off, own_off):
        own = slice(P + cols.start, P + cols.stop)
        w[:, own], tol[:, own] = 0, 0
        for h in range(H):
            hk = h // (H // Hk)
            s, size = scores(q, kp, ko, rows, cols, h, hk, causal, scale)
            z = lse[rows, h].double()[:, None]
            p = torch.where((z == NEG) | (s == NEG), torch.zeros_like(s), (s - z).exp())
            rel = 130 * U32 * size + 4e-6 + 4 * U32 * (z.abs() + s.abs().nan_to_num(0, 0, 0) + 64) + (q.shape[0] * (H // Hk) / 64 + 64) * U32
            rel = torch.where(p > 0, rel, torch.zeros_like(rel))
            for at, cut in ((slice(0, P), slice(0, P)), (own, slice(P, None))):
                w[hk, at] += p[:, cut].sum(0)
                tol[hk, at] += (p * rel)[:, cut].sum(0) * 1.01
    if acc is not None and decay:
        w[:, :P] += decay * acc[:, :P].double()
        tol[:, :P] += 4 * U32 * (w[:, :P].abs() + decay * acc[:, :P].double().abs())
    return w, tol + 1e-30


def evict(acc, ids, keep, recent_from):
    """source[h][slot]: the slot whose token ends up in `slot`, for slots below `keep`."""
    out = []
    for a, i in zip(acc.double().tolist(), ids.tolist()):
        key = [float("inf") if t >= recent_from else (NEG if x != x else x) for x, t in zip(a, i)]
        kept = set(sorted(range(len(key)), key=lambda s: (-key[s], s))[:keep])
        movers = iter(sorted(s for s in kept if s >= keep))
        out.append([s if s in kept else next(movers) for s in range(keep)])
    return torch.tensor(out, dtype=torch.int64).reshape(len(out), keep)
