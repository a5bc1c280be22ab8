"""Plain fp64 CPU oracle of the router, the gate gradient and gradient clipping.

TEST INFRASTRUCTURE ONLY, like ``lrm_oracle``: written from the formulas
("Expert Parallel Math Deep": importance P_e, load f_e, the auxiliary loss
E sum f_e P_e; the z loss is the mean squared log-partition; the softmax's
Jacobian), with none of the CUDA library's code.
"""

from __future__ import annotations

import numpy as np

__all__ = ["router_forward", "router_backward", "gate_grad", "clip"]


def top_k(logits, k: int) -> np.ndarray:
    """The k largest per row, descending, ties to the lower column, NaN below -inf."""
    T, E = logits.shape
    x = np.where(np.isnan(logits), -np.inf, logits)
    out = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        # last key is the primary one: value descending (NaN last), then column
        out[t] = np.lexsort((np.arange(E), np.isnan(logits[t]), -x[t]))[:k]
    return out


def router_forward(logits, k: int, renorm: bool, aux_coef: float = 0.0, z_coef: float = 0.0, valid=None) -> dict:
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids = top_k(l, k)
    m = np.full(T, 0.0)
    s = np.zeros(T)
    p = np.zeros((T, E))
    alpha = np.zeros((T, k))
    counted = np.zeros(T, dtype=bool)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(T):
            dead = bool(np.all(l[t] == -np.inf))
            if dead or (valid is not None and not valid[t]):
                continue
            counted[t] = True
            m[t] = np.fmax.reduce(l[t])
            if m[t] == -np.inf or np.isnan(m[t]):
                m[t] = 0.0
            e = np.exp(l[t] - m[t])
            s[t] = e.sum()
            p[t] = e / s[t]
            alpha[t] = e[ids[t]] / (e[ids[t]].sum() if renorm else s[t])
    Tc = int(counted.sum())
    counts = np.bincount(ids[counted].reshape(-1), minlength=E)
    f = counts / (Tc * k) if Tc else np.zeros(E)
    P = p[counted].sum(0) / Tc if Tc else np.zeros(E)
    lse = m[counted] + np.log(s[counted])
    aux = E * float((f * P).sum())
    z = float((lse ** 2).sum() / Tc) if Tc else 0.0
    return dict(expert_idx=ids, alpha=alpha, row_stats=np.stack([m, s], 1), counts=counts, f=f, P=P, aux=aux, z=z,
                loss=aux_coef * aux + z_coef * z, tokens=Tc, p=p, counted=counted)


def router_backward(logits, ids, alpha, f, Tc: int, dgate, renorm: bool, aux_coef: float, z_coef: float,
                    counted) -> np.ndarray:
    """dL/dlogits with dgate[t, j] = alpha dL/dalpha, from the Jacobians: the
    balance loss through p, the z loss through lse, the gates through the
    softmax over the slots (renorm) or over all experts."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    for t in np.flatnonzero(counted):
        m = l[t].max()
        s = np.exp(l[t] - m).sum()
        p = np.exp(l[t] - m) / s
        dp = aux_coef * E / Tc * np.asarray(f, dtype=np.float64)
        g = p * (dp - (p * dp).sum()) + 2.0 * z_coef / Tc * (m + np.log(s)) * p
        if dgate is not None:
            d = np.asarray(dgate[t], dtype=np.float64)
            if renorm:
                g[ids[t]] += d - np.asarray(alpha[t], dtype=np.float64) * d.sum()
            else:
                g[ids[t]] += d
                g -= p * d.sum()
        out[t] = g
    return out


def gate_grad(dphi_rows, phi_rows, sel_ids, N: int) -> np.ndarray:
    """<dphi_c[r], phi_c[r]> at pair sel_ids[r], zeros elsewhere."""
    out = np.zeros(N)
    out[np.asarray(sel_ids, dtype=np.int64)] = (np.asarray(dphi_rows, np.float64) * np.asarray(phi_rows, np.float64)).sum(1)
    return out


def clip(tensors, max_norm: float):
    """(norm, coef, clipped tensors); squares summed scaled by the largest magnitude."""
    flat = [np.asarray(t, dtype=np.float64).reshape(-1) for t in tensors]
    big = max([np.abs(x).max() for x in flat if x.size], default=0.0)
    if not np.isfinite(big):
        return big, 1.0, flat
    norm = big * np.sqrt(sum(((x / big) ** 2).sum() for x in flat if x.size)) if big > 0 else 0.0
    coef = max_norm / norm if norm > max_norm else 1.0
    return float(norm), float(coef), [x * coef for x in flat]
