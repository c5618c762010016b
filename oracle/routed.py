"""Oracle of the routed layers, in numpy and FP64, from the definitions in include/w4a16.h.

TEST INFRASTRUCTURE ONLY: shares no code with the CUDA library. 16-bit values come in and go out
as float64 (the caller widens and rounds), maps as integers.
"""
import numpy as np


def sort(ids, E):
    """(offsets [E + 1], rows [R], slots [T, k]) of ids [T, k]: choice by choice, expert by expert."""
    flat = np.asarray(ids).reshape(-1)
    slots = np.full(flat.size, -1, dtype=np.int64)
    offsets = np.zeros(E + 1, dtype=np.int64)
    rows = []
    for e in range(E):
        offsets[e] = len(rows)
        for i in np.flatnonzero(flat == e):
            slots[i] = len(rows)
            rows.append(i)
    offsets[E] = len(rows)
    return offsets, np.asarray(rows, dtype=np.int64), slots.reshape(np.asarray(ids).shape)


def combine(Ys, slots, weights):
    """(Y [T, H], sum of the magnitudes of its terms)."""
    T, k = slots.shape
    Y = np.zeros((T, Ys.shape[1]))
    Yabs = np.zeros_like(Y)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < T * k:
                w = 1.0 if weights is None else float(weights[t, j])
                term = w * Ys[slots[t, j]]
                Y[t] += term
                Yabs[t] += np.abs(term)
    return Y, Yabs


def combine_grad(dY, Ys, slots, weights):
    """(dYs {row: values}, dweights [T, k], sum of the magnitudes of each weight's terms)."""
    T, k = slots.shape
    dYs, dw, dwabs = {}, np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = int(slots[t, j])
            if 0 <= s < T * k:
                dYs[s] = (1.0 if weights is None else float(weights[t, j])) * dY[t]
                dw[t, j] = dY[t] @ Ys[s]
                dwabs[t, j] = np.abs(dY[t]) @ np.abs(Ys[s])
    return dYs, dw, dwabs


def lora(A, La, Lb, scale, row_adapter):
    """The adapters' term of the layer, delta [M, N], and the magnitudes an error bound needs: per
    output sum_j |s T_j Lb_nj|, sum_j |s Lb_nj| sum_k |A_k La_jk| and max_j |s T_j| sum_j |Lb_nj|."""
    M, N = A.shape[0], Lb.shape[1]
    out = [np.zeros((M, N)) for _ in range(4)]
    for m in range(M):
        a = int(row_adapter[m])
        if not 0 <= a < La.shape[0]:
            continue
        s = float(scale[a])
        T = La[a] @ A[m]
        out[0][m] = s * (Lb[a] @ T)
        out[1][m] = abs(s) * (np.abs(Lb[a]) @ np.abs(T))
        out[2][m] = abs(s) * (np.abs(Lb[a]) @ (np.abs(La[a]) @ np.abs(A[m])))
        out[3][m] = abs(s) * np.abs(T).max() * np.abs(Lb[a]).sum(1)
    return out
