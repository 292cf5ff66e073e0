"""Reference and error bound of the layer with its epilogue, in fp64 (no GPU work here; imported by the tests).

``act_rows`` evaluates, for rows of one layer,

    v = s_x s_w (C_x C_w^T) + (X L1) L2 + bias,   y = act(v) [x v of the second half] + residual

from the codes' definition, and beside y a bound on |kernel - y| that arithmetic fixes, with u = 2^-24:

* the integer sum is exact and exact as fp32 (below 2^24); s_x s_w and its product round twice:  2 u |a|;
* T is an fp32 sum of d exact products (gamma_d sum |x||l1|) carried in bf16 parts (2^-16 |t| with two, 2^-24 |t| with
  three), its product with L2 an fp32 sum of parts * r_pad exact products, which may be accumulated on top of the
  dequantised sum:  gamma_(parts r_pad + 2) (sum |t||l2| + |a|);
* two more additions (low-rank term, bias):  2 u (|a| + |l| + |b|);
* activation: slopes are at most 1.13.  exp(-w) has a relative error of |w| 2^-23 from its rounded argument; it enters
  1 / (1 + exp(-w)) with weight sigmoid(-w), and the erf form as the factor of Phi(-|v|); a reciprocal and the few
  products around it add 8 2^-23 |y|, the polynomial of the erf form 0.75e-7 |v|;
* product of the halves and the residual's addition: one rounding each;
* the final rounding: half a step of Y's type, eps / 2 relative to the value.
"""

from __future__ import annotations

import math

import numpy as np
import torch

import oracle.tq_oracle as tqo

U = 2.0 ** -24
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def gamma(k):
    return k * U / (1.0 - k * U)


def _sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def act_value(v, act):
    """(act(v), absolute error of its evaluation)."""
    if act == "none":
        return v, np.zeros_like(v)
    if act == "relu":
        return np.maximum(v, 0.0), np.zeros_like(v)
    if act == "gelu":
        erfc = np.vectorize(math.erfc, otypes=[np.float64])
        y = 0.5 * v * erfc(-v * math.sqrt(0.5))
        tail = 0.5 * np.abs(v) * erfc(np.abs(v) * math.sqrt(0.5))
        return y, 2.0 ** -23 * (0.5 * v * v * tail + 8 * np.abs(y)) + 0.75e-7 * np.abs(v)
    # the argument of the tanh form is itself rounded a few times: 3 |w|
    w, times = (v, 1.0) if act == "silu" else (2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3), 3.0)
    y = v * _sigmoid(w)
    return y, 2.0 ** -23 * np.abs(y) * (times * np.abs(w) * _sigmoid(-w) + 8.0)


def act_rows(x, w_codes, s_w, l1=None, l2=None, bias=None, act="none", gated=False, residual=None, y_dtype="bf16"):
    """x n x d (fp32 values), w_codes m x d/2 packed, s_w m, l1 d x r and l2 r x m (bf16 values) -> (y, bound), fp64."""
    x = np.asarray(x, dtype=np.float32)
    n, d = x.shape
    cx, sx = tqo.quantize_rows(x, 4)
    cw = tqo.unpack_int4(np.asarray(w_codes))
    acc = cx.astype(np.int64) @ cw.astype(np.int64).T
    a = acc.astype(np.float64) * sx.astype(np.float64)[:, None] * np.asarray(s_w, dtype=np.float64)[None, :]
    lr, d_lr = np.zeros_like(a), np.zeros_like(a)
    if l1 is not None:
        xb = torch.from_numpy(x).bfloat16().double().numpy()
        l1, l2 = np.asarray(l1, dtype=np.float64), np.asarray(l2, dtype=np.float64)
        r = l1.shape[1]
        rp = 32
        while rp < r:
            rp *= 2
        parts = 2 if y_dtype == "bf16" else 3
        t = xb @ l1
        lr = t @ l2
        mag = np.abs(t) @ np.abs(l2)
        d_t = gamma(d + 16) * (np.abs(xb) @ np.abs(l1)) + (2.0 ** -16 if parts == 2 else 2.0 ** -24) * np.abs(t)
        d_lr = d_t @ np.abs(l2) + gamma(parts * rp + 2) * (mag + d_t @ np.abs(l2) + np.abs(a))
    b = np.zeros(a.shape[1]) if bias is None else np.asarray(bias, dtype=np.float64)
    v = a + lr + b[None, :]
    d_v = 2 * U * np.abs(a) + d_lr + 2.01 * U * (np.abs(a) + np.abs(lr) + d_lr + np.abs(b)[None, :])
    h = v.shape[1] // 2 if gated else v.shape[1]
    y, d_y = act_value(v[:, :h], act)
    d_y = d_y + 1.13 * d_v[:, :h]
    if gated:
        up, d_up = v[:, h:], d_v[:, h:]
        d_y = d_y * (np.abs(up) + d_up) + np.abs(y) * d_up
        y = y * up
        d_y = d_y + U * (np.abs(y) + d_y)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
        d_y = d_y + U * (np.abs(y) + d_y)
    half = 2.0 ** -8 if y_dtype == "bf16" else U
    return y, d_y + half * (np.abs(y) + d_y) + 2.0 ** -126


def assert_within(y_gpu, y, bound, what=""):
    y_gpu = np.asarray(y_gpu, dtype=np.float64)
    assert y_gpu.shape == y.shape, (what, y_gpu.shape, y.shape)
    assert np.isfinite(y_gpu).all(), what
    if not y.size:
        return
    ratio = np.abs(y_gpu - y) / bound
    at = np.unravel_index(int(ratio.argmax()), ratio.shape)
    print(f"  {what} max |Y - Y_ref| / bound = {ratio[at]:.3f} at {at}", flush=True)
    assert ratio[at] <= 1.0, (what, at, y_gpu[at], y[at], bound[at])
