"""float64 CPU oracle of the operators around an adapted linear: block-scaled E4M3 quantisation
and the frozen product over it, layer norm with its backward pass, the orthogonalised update.
Plain and slow; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

from .lora_oracle import e4m3_decode, e4m3_encode

BLOCK = 128


def quantize_blocks(x, rows: int, cols: int):
    """E4M3 codes of x [R, C] and one float32 scale per rows x cols block; the scaling is float32
    arithmetic by definition (r = 448 (1 / amax), x r, amax (1 / 448); 1 where r is not finite)."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    nr, nc = -(-R // rows), -(-C // cols)
    codes = np.zeros((R, C), np.uint8)
    scales = np.ones((nr, nc), np.float32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for i in range(nr):
            for j in range(nc):
                b = x[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols]
                amax = np.float32(np.max(np.abs(b)))
                r = np.float32(448.0) * (np.float32(1.0) / amax)
                if amax > 0 and np.isfinite(r):
                    scales[i, j] = amax * (np.float32(1.0) / np.float32(448.0))
                else:
                    r = np.float32(1.0)
                codes[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols] = e4m3_encode(b * r)
    return codes, scales


def dequantize_blocks(codes, scales, rows: int, cols: int):
    v = e4m3_decode(codes).astype(np.float64)
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, 0), cols, 1)
    return v * s[:v.shape[0], :v.shape[1]]


def block_product(x, W8, sw, transposed: bool):
    """(Y, sum of |terms|) of the product of x, quantised in 1 x 128 blocks, and the weight."""
    c, s = quantize_blocks(x, 1, BLOCK)
    xd = dequantize_blocks(c, s, 1, BLOCK)
    w = dequantize_blocks(W8, sw, BLOCK, BLOCK)
    if not transposed:
        w = w.T
    return xd @ w, np.abs(xd) @ np.abs(w)


def norm_forward(x, gamma, beta, eps: float, rms: bool):
    x = np.asarray(x, np.float64)
    mean = np.zeros((x.shape[0], 1)) if rms else x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    y = (x - mean) * rstd * np.asarray(gamma, np.float64)
    return (y if beta is None else y + np.asarray(beta, np.float64)), mean[:, 0], rstd[:, 0]


def norm_backward(x, gamma, dy, eps: float, rms: bool):
    """(dX, dgamma, dbeta) from the inputs alone."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    _, mean, rstd = norm_forward(x, gamma, None, eps, rms)
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * np.asarray(gamma, np.float64)
    dx = g - xhat * (g * xhat).mean(1, keepdims=True)
    if not rms:
        dx -= g.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * xhat).sum(0), dy.sum(0)


def newton_schulz(u, coef=(3.4445, -4.7750, 2.0315), steps: int = 5):
    """(X, largest gain): the sequence from u / ||u||, and the largest ratio of a singular value's
    image to itself over the matrix's singular values."""
    a, b, c = coef
    u = np.asarray(u, np.float64)
    x = u.T if u.shape[0] > u.shape[1] else u
    n = np.linalg.norm(x)
    if n == 0:
        return np.zeros_like(u), 0.0
    x = x / n
    sv = np.linalg.svd(x, compute_uv=False)
    f = sv.copy()
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
        f = f * (a + b * f ** 2 + c * f ** 4)
    live = sv > 1e-12
    gain = float(np.max(np.abs(f[live] / sv[live])))
    return (x.T if u.shape[0] > u.shape[1] else x), gain


def muon_update(p, g, m, *, c, lr, kind, mu=0.95, wd=0.01, ratio=1.0, coef=(3.4445, -4.7750, 2.0315),
                steps=5, nesterov=True, adjust="aspect"):
    """(p, m) after one update of a matrix [rows, cols]; kind 'A' or 'B'."""
    p, g, m = (np.asarray(v, np.float64) for v in (p, g, m))
    m = mu * m + c * g
    u = c * g + mu * m if nesterov else m
    x, _ = newton_schulz(u, coef, steps)
    rows, cols = p.shape
    s = np.sqrt(max(1.0, rows / cols)) if adjust == "aspect" else 0.2 * np.sqrt(max(rows, cols))
    if kind == "A":
        return p - lr * s * x - lr * wd * p, m
    return p - lr * ratio * s * x, m
