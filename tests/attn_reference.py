"""Attention in fp64 with modified scores, and the error bound its kernels are held to.

Bound of one output element.  With u the half step of the dtype (eps / 2), the
exact weights w_j, A = sum w_j |v_j| / sum w_j and n keys seen:

* a score (log2 units) is off by e_y: its dot product's roundings, at most
  D / 4 partial sums of at most S = log2(e) scale max_j sum_d |q_d k_jd| each
  (tensor-core sums may truncate: a whole step, 2^-23), the roundings of its
  scaling, penalty and exponent argument (6 of 2^-24 max |y|) and the cap
  (C 2^-21 with the approximate functions, C 2^-22 with tanhf);
* a weight is off by ln 2 e_y + 2^-22 (the approximate exp2) relatively, once in
  the numerator and once in the sum, and each of their fp32 sums of at most
  n / 16 + 64 terms in a row adds that many steps of 2^-24;
* 16-bit dtypes round each weight to the dtype for P V (u A), fp16 besides
  flushes what lies below its range (2^-25 of a weight of at least 1 each, n of
  them at most), and round the output (u |out|).
"""
from __future__ import annotations

import math

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOG2E = math.log2(math.e)


def seen_mask(P, N, window, prefix, docs):
    """[N, P + N] truth values: which keys the rows of a sequence with P cached tokens see."""
    p = np.arange(P, P + N)[:, None]
    j = np.arange(P + N)[None]
    seen = j <= p
    if window:
        seen &= j > p - window
    seen |= j < prefix
    if docs is not None:
        d = np.maximum(np.asarray(docs), docs[0])[:, None]
        seen &= j >= d
    return seen


def attention64(q, k, v, scale, mask, cap=0.0, slopes=None, P=0, dtype="f32"):
    """One sequence: q [H_q, N, D], k, v [H_kv, T, D] (fp64 numpy), mask [N, T].

    Returns (out, tolerance), both [H_q, N, D]."""
    H_q, N, D = q.shape
    g = H_q // k.shape[0]
    u = 0.0 if dtype == "f32" else torch.finfo(DT[dtype]).eps / 2
    out, tol = np.zeros_like(q), np.zeros_like(q)
    j = np.arange(k.shape[1])
    for h in range(H_q):
        kh, vh = k[h // g], v[h // g]
        for i in range(N):
            m = mask[i]
            if not m.any():
                continue
            qi, km, vm = q[h, i], kh[m], vh[m]
            y = km @ qi * scale
            S = LOG2E * scale * (np.abs(km) @ np.abs(qi)).max()
            if cap:
                y = cap * np.tanh(y / cap)
            if slopes is not None:
                y = y - slopes[h] * np.abs(P + i - j[m])
            y = y * LOG2E
            w = np.exp2(y - y.max())
            out[h, i] = w @ vm / w.sum()
            A = w @ np.abs(vm) / w.sum()
            n = m.sum()
            e_y = D / 4 * 2.0 ** -23 * S + 6 * 2.0 ** -24 * np.abs(y).max()
            e_y += cap * LOG2E * (2.0 ** -22 if dtype == "f32" else 2.0 ** -21)
            rel = 2 * (math.log(2) * e_y + 2.0 ** -22 + (n / 16 + 64) * 2.0 ** -24)
            tol[h, i] = A * (rel + u) + u * np.abs(out[h, i])
            if dtype == "f16":
                tol[h, i] += n * 2.0 ** -25 * np.abs(vm).max(axis=0) + 2.0 ** -25
    return out, tol


def assert_near(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))),
                           np.argwhere(bad)[:3].tolist())
