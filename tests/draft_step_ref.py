"""Plain fp64 forms (numpy) of the draft step's operators: the 8-bit norm, the 8-bit
product, the beam selection and the reordering of states.  They share no code with
the kernels and follow the definitions in include/spec_verify.h literally."""
import numpy as np
import torch


def f64(t):
    """A torch tensor's exact values as float64."""
    return t.detach().cpu().to(torch.float64).numpy()


def q8_rows(x, residual=None, weight=None, eps=None):
    """(q, scale, sum, normed) in fp64; eps None: no norm (scale = max / 127)."""
    s = x if residual is None else x + residual
    p = s if weight is None else s * weight[None, :]
    top = np.abs(p).max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        q = np.where(top > 0, np.rint(p * 127 / top), 0.0)
        rms = np.ones_like(top) if eps is None else np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
        scale = np.where(top > 0, top / (127 * rms), 0.0)
        normed = np.where(top > 0, p / rms, 0.0)
    bad = ~np.isfinite(p).all(axis=1)
    q[bad] = 0
    scale[bad] = np.nan
    normed[bad] = np.nan
    return q, scale[:, 0], s, normed


def q8_matmul(a, a_scale, w, w_scale):
    # float64 holds these integer sums exactly (below 2^31)
    return (a.astype(np.float64) @ w.astype(np.float64).T) * a_scale[:, None] * w_scale[None, :]


def beam_keys(logits, scores, temperature, frozen=None, pad_token=0):
    """[B, W, V] keys (-inf: no candidate) and the status bits of each sequence."""
    B, W, V = logits.shape
    keys = np.full((B, W, V), -np.inf)
    status = np.zeros(B, np.int64)
    for b in range(B):
        T = float(temperature[b])
        ok = T == 0 or (np.isfinite(T) and T >= np.float32(1e-6))
        if not ok:
            status[b] |= 4
        for w in range(W):
            sc = scores[b, w]
            if np.isnan(sc) or sc == np.inf:
                status[b] |= 64
                continue
            if sc == -np.inf:
                continue
            if frozen is not None and frozen[b, w]:
                keys[b, w, pad_token] = sc
                continue
            if not ok:
                continue
            row = logits[b, w]
            if np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
                status[b] |= 2
                continue
            if T == 0:
                keys[b, w, int(np.argmax(row))] = sc
            else:
                z = row / T
                m = z.max()
                keys[b, w] = sc + (z - (m + np.log(np.exp(z - m).sum())))
    return keys, status


def beam_select(keys, K):
    """(parent, token, key), ties to the lower (beam, token)."""
    B, W, V = keys.shape
    parent, token, key = np.full((B, K), -1), np.full((B, K), -1), np.full((B, K), -np.inf)
    for b in range(B):
        flat = keys[b].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:K]
        order = order[flat[order] > -np.inf]
        n = len(order)
        parent[b, :n], token[b, :n], key[b, :n] = order // V, order % V, flat[order]
    return parent, token, key


def reorder(src, parent, out, lengths=None):
    """out (a copy is returned) with the live tokens of the chosen parents."""
    out = out.clone()
    L, B, W, H, S, D = src.shape
    for b in range(B):
        n = S if lengths is None else min(S, max(0, int(lengths[b])))
        for k in range(parent.shape[1]):
            p = int(parent[b, k])
            if 0 <= p < W:
                out[:, b, k, :, :n] = src[:, b, p, :, :n]
    return out
