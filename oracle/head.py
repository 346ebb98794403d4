"""fp64 oracle of the 8-bit product, the teacher's top logits and the
distillation loss (plain numpy; test infrastructure only).

  s_t = clip max|x_t| / 127, a = clamp(rint(x / s_t), -127, 127)   (fp32)
  y_to = s_t w_o (sum_k a_tk (q_ok - z_o)) + b_o
  L = w T^2 [ sum_k p_k (log p_k - log q_k) + r (log r - log q_r) ]
  dL/ds_j = w T [ c_j q_j - p_j ],  c_j = P on the list, P - r / q_r off it
"""
from __future__ import annotations

import numpy as np

REST_MIN = 2.0 ** -16


def quantize_rows(x, clip=1.0):
    """(codes int64, scales fp32, sums); the grid is decided in fp32."""
    x = np.asarray(x, np.float32)
    n = x.shape[0]
    codes = np.zeros(x.shape, np.int64)
    scale = np.zeros(n, np.float32)
    for i in range(n):
        if not np.all(np.isfinite(x[i])):
            scale[i] = np.nan
            continue
        m = np.max(np.abs(x[i]))
        s = np.float32(np.float32(np.float32(clip) * m) / np.float32(127))
        scale[i] = s
        if s > 0:
            codes[i] = np.clip(np.rint(x[i] / s), -127, 127).astype(np.int64)
    return codes, scale, codes.sum(1)


def product(codes, scale, w, w_scale, w_zero=None, bias=None):
    """fp64 y and the exact integer sums."""
    w = np.asarray(w, np.int64)
    # fp64 holds these sums exactly (below 2^53)
    acc = (codes.astype(np.float64) @ w.T.astype(np.float64)).astype(np.int64)
    if w_zero is not None:
        acc = acc - codes.sum(1)[:, None] * np.asarray(w_zero, np.int64)[None, :]
    y = acc * scale.astype(np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :]
    return y, acc


def top_logits(logits, k, temperature=1.0):
    """(values, index, lse): descending, equal values by lowest index, a NaN
    first."""
    z = np.asarray(logits, np.float64)
    n, v = z.shape
    values, index, lse = np.empty((n, k)), np.empty((n, k), np.int64), np.empty(n)
    for i in range(n):
        # Python's sort is stable: equal keys stay in index order
        order = sorted(range(v), key=lambda j: (0, 0.0) if np.isnan(z[i, j]) else (1, -z[i, j]))
        index[i] = order[:k]
        values[i] = z[i, order[:k]]
        m = np.max(z[i])
        if m == np.inf:  # (a NaN in the row makes m NaN)
            lse[i] = np.inf
            continue
        m = 0.0 if m == -np.inf else m
        with np.errstate(divide="ignore"):
            lse[i] = m / temperature + np.log(np.sum(np.exp((z[i] - m) / temperature)))
    return values, index, lse


def distill(logits, values, index, t_lse=None, temperature=1.0, weight=None):
    """(loss, gradient, stats), row by row from the definition; stats: the
    largest logit m, log sum exp((s - m) / T), log of the mass off the list."""
    s = np.asarray(logits, np.float64)
    n, v = s.shape
    T = float(temperature)
    loss, grad = np.zeros(n), np.zeros((n, v))
    stats = np.zeros((n, 3))
    with np.errstate(divide="ignore", invalid="ignore"):
        for i in range(n):
            w = 1.0 if weight is None else float(weight[i])
            m = np.max(s[i])
            if m == -np.inf:
                log_q, q, log_sum = np.full(v, -np.inf), np.zeros(v), -np.inf
            else:
                # the largest goes off first: next to it the sum's logarithm
                # would be lost where the logits are large
                e = np.exp((s[i] - m) / T)
                log_sum = np.log(np.sum(e))
                log_q, q = (s[i] - m) / T - log_sum, e / np.sum(e)
            # the teacher's mass on each column of the list
            entries = [(int(j), float(t) / T) for j, t in zip(index[i], values[i]) if 0 <= j < v]
            if t_lse is not None:
                log_p = [t - float(t_lse[i]) for _, t in entries]
            elif entries:
                tm = max(t for _, t in entries)
                z = 0.0 if tm == -np.inf else tm + np.log(sum(np.exp(t - tm) for _, t in entries))
                log_p = [t - z for _, t in entries]
            else:
                log_p = []
            total = sum(np.exp(lp) for lp in log_p)
            r = 0.0
            if t_lse is not None and 1.0 - total > REST_MIN:
                r = 1.0 - total
            on = np.zeros(v, bool)
            on[[j for j, _ in entries]] = True
            # against the largest off the list: its mass may lie far below
            # what a number can hold beside 1
            m_off = np.max(s[i][~on], initial=-np.inf)
            if m_off == -np.inf:
                log_q_off, share = -np.inf, np.zeros(v)
            else:
                e_off = np.where(on, 0.0, np.exp((np.where(on, m_off, s[i]) - m_off) / T))
                log_q_off = (m_off - m) / T + np.log(np.sum(e_off)) - log_sum
                share = e_off / np.sum(e_off)  # q_j / q_r
            stats[i] = m, log_sum, log_q_off
            if w == 0.0:
                continue
            value = 0.0
            for (j, _), lp in zip(entries, log_p):
                p = np.exp(lp)
                if p > 0:
                    value += p * (lp - log_q[j])
                grad[i, j] -= p
            if r > 0:
                value += r * (np.log(r) - log_q_off)
            P = total + r
            grad[i] += q * P - r * share
            loss[i] = w * T * T * value
            grad[i] *= w * T
    return loss, grad, stats
