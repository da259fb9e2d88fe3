"""CPU oracle for the operators around the expert block: the norms before and
after it with the combine, the residual scale and their gradients, and the
routing's balance loss, per-expert counts and gradients.

TEST INFRASTRUCTURE ONLY: the tests and the smoke check import it.  The
definitions written out in float64 with numpy, token by token, without blocking
or fusion; it shares no code with the library.  Pinned by
tests/test_block_oracle.py to finite differences, torch's float64 autograd and
closed forms.
"""
from __future__ import annotations

import numpy as np


def norm(x, w, eps):
    """x * (mean(x^2) + eps)^(-1/2) * w of each row."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return x * r * np.asarray(w, np.float64)


def norm_backward(d, x, w, eps):
    """The gradients of norm for the gradient d of its result: (dx, dw summed over the rows, the
    magnitude of dx's terms, the magnitude of dw's)."""
    d, x, w = (np.asarray(a, np.float64) for a in (d, x, w))
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    unit = x * r
    dx = r * (d * w - unit * np.mean(d * w * unit, axis=-1, keepdims=True))
    mag = r * (np.abs(d * w) + np.abs(unit) * np.mean(np.abs(d * w * unit), axis=-1, keepdims=True))
    return dx, (d * unit).sum(0), mag, np.abs(d * unit).sum(0)


def combine(proj, gates):
    """(h, sum of |terms|): sum_s gates[t, s] * proj[t, s, :] over the slots whose gate is not 0."""
    T, k, N = proj.shape
    h, mag = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for s in range(k):
            if gates[t, s] != 0:
                h[t] += gates[t, s] * proj[t, s].astype(np.float64)
                mag[t] += np.abs(gates[t, s] * proj[t, s].astype(np.float64))
    return h, mag


def combine_norm(proj, gates, w_post, x, scale, eps):
    """The block's output before rounding: x + scale * (norm of) the combine."""
    h, _ = combine(proj, gates)
    u = h if w_post is None else norm(h, w_post, eps)
    return np.asarray(x, np.float64) + scale * u


def combine_norm_backward(dx_out, dxn, x_out, w_next, proj, gates, w_post, scale, eps):
    """The gradients of combine_norm and of the next norm of the stored x_out: a dict of dx, dproj,
    dgates, dw_post, dw_next (None where there is no such weight), and of dh and G's magnitudes
    for the tolerances (mag_dx, mag_dh, mag_post, mag_next)."""
    T, k, N = proj.shape
    g = np.zeros((T, N)) if dx_out is None else np.asarray(dx_out, np.float64).copy()
    mag_g = np.abs(g)
    out = {"dw_post": None, "dw_next": None, "mag_post": None, "mag_next": None}
    if dxn is not None:
        dn, out["dw_next"], mag, out["mag_next"] = norm_backward(dxn, x_out, w_next, eps)
        g, mag_g = g + dn, mag_g + mag
    h, mag_h = combine(proj, gates)
    dh, mag_dh = scale * g, np.abs(scale) * mag_g
    if w_post is not None:
        w = np.asarray(w_post, np.float64)
        r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
        big = r * mag_h  # at least |h^|
        # how far h's own rounding moves r
        lift = 1.0 + (np.abs(h) * mag_h).sum(-1, keepdims=True) / np.maximum((h * h).sum(-1, keepdims=True), 1e-300)
        out["mag_post"] = (mag_dh * big * lift).sum(0)
        mag_dh = lift * r * (mag_dh * np.abs(w) + big * np.mean(mag_dh * np.abs(w) * big, axis=-1, keepdims=True))
        dh, out["dw_post"], _, _ = norm_backward(dh, h, w_post, eps)
    dproj, dgates, mag_dgates = np.zeros((T, k, N)), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            if gates[t, s] != 0:
                row = proj[t, s].astype(np.float64)
                dproj[t, s] = gates[t, s] * dh[t]
                dgates[t, s] = dh[t] @ row
                mag_dgates[t, s] = mag_dh[t] @ np.abs(row)
    out.update(dx=g, mag_dx=mag_g, dproj=dproj, mag_dproj=np.abs(gates)[:, :, None] * mag_dh[:, None, :],
               dgates=dgates, mag_dgates=mag_dgates)
    return out


def _sequence(t, seq_offsets):
    """The sequence that holds token t, or None."""
    for s in range(len(seq_offsets) - 1):
        if seq_offsets[s] <= t < seq_offsets[s + 1]:
            return s
    return None


def softmax(l):
    """(probabilities, log-sum-exp) of one row with a finite maximum."""
    m = l.max()
    e = np.exp(l - m)
    return e / e.sum(), m + np.log(e.sum())


def counted(logits, ids, seq_offsets):
    """Per token: its sequence if it is counted (it lies in one, has a valid slot and a logit above
    -inf), else None."""
    T, E = logits.shape
    where = []
    for t in range(T):
        s = _sequence(t, seq_offsets)
        ok = s is not None and any(0 <= i < E for i in ids[t]) and bool(np.any(logits[t] > -np.inf))
        where.append(s if ok else None)
    return where


def balance(logits, ids, seq_offsets):
    """(counts [S, E], tokens [S + 2], losses [2]) of float64 logits; seq_offsets ascending."""
    T, E = logits.shape
    k, S = ids.shape[1], len(seq_offsets) - 1
    counts, n = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    p_sum, z2 = np.zeros((S, E)), 0.0
    for t, s in enumerate(counted(logits, ids, seq_offsets)):
        if s is None:
            continue
        p, z = softmax(logits[t])
        n[s] += 1
        p_sum[s] += p
        z2 += z * z
        for i in ids[t]:
            if 0 <= i < E:
                counts[s, i] += 1
    used = int((n > 0).sum())
    loss = sum(E * float((counts[s] / (k * n[s])) @ (p_sum[s] / n[s])) for s in range(S) if n[s]) / max(used, 1)
    return counts, np.concatenate([n, [n.sum(), used]]), np.array([loss, z2 / max(int(n.sum()), 1)])


def route_backward(logits, ids, gates, dgates, seq_offsets, dlosses):
    """(dlogits [T, E], the magnitude of its terms).  dgates None: no gradient through the gates;
    dlosses None: none through the losses (seq_offsets is then not used)."""
    T, k = ids.shape
    E = logits.shape[1]
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    if dlosses is not None:
        where = counted(logits, ids, seq_offsets)
        counts, tokens, _ = balance(logits, ids, seq_offsets)
        n_all, used = max(int(tokens[-2]), 1), max(int(tokens[-1]), 1)
    for t in range(T):
        if dlosses is not None:
            s = where[t]
            if s is None:
                continue
            p, z = softmax(logits[t])
            n = int(tokens[s])
            c = (counts[s] - counts[s].mean()) * E / (used * k * n * n) * dlosses[0]
            b = dlosses[1] * 2.0 / n_all * z
            out[t] += p * (c - p @ c + b)
            mag[t] += p * (np.abs(c) + p @ np.abs(c) + abs(b))
        if dgates is not None:
            slots = [q for q in range(k) if 0 <= ids[t, q] < E and gates[t, q] != 0]
            mean = sum(gates[t, q] * dgates[t, q] for q in slots)
            mean_mag = sum(abs(gates[t, q] * dgates[t, q]) for q in slots)
            for q in slots:
                out[t, ids[t, q]] += gates[t, q] * (dgates[t, q] - mean)
                mag[t, ids[t, q]] += gates[t, q] * (abs(dgates[t, q]) + mean_mag)
    return out, mag
