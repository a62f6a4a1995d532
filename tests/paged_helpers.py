"""Plain fp64 forms of the paged-cache operators (numpy, from the definitions) and the
error bounds that their fp32 / bf16 kernels are held to."""

from __future__ import annotations

import numpy as np

from oracle import jetlong_oracle as jo

BF16_HALF = 2.0 ** -8  # half a step of bf16 relative to the value
EPS = 1e-6


def norm_rope(x, w, positions, base, eps=EPS):
    """x [T, H, D] fp64, w [D] or None, positions [T]."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return jo.rope_rotate(x, np.asarray(positions)[:, None], base)


def norm_rope_tol(y):
    """bf16 rounding, and fp32 arithmetic on the pair (x, y): the mean of squares (D terms), the
    root, two products and one sum, under 2^-18 of the pair's length together, and the angle's
    2^-23 rad."""
    h = y.shape[-1] // 2
    pair = np.hypot(y[..., :h], y[..., h:])
    return BF16_HALF * np.abs(y) + 2.0 ** -18 * np.concatenate([pair, pair], -1)


def rule(L, w0, W, mode):
    G = jo.group_size(L, W)
    shift = w0 - w0 // G if mode == jo.MODE_SELF_EXTEND else 0
    return G, (L - 1) // G + shift


def decode_rows(q, k, v, pos, L, w0, W, base, mode=jo.MODE_SELF_EXTEND, scale=None):
    """One KV head: q [r, D] (rotated at L - 1), keys k / v [n, D] at positions pos [n] (all below L).
    Returns o [r, D], lse [r] and the bound on each score's error (hi + lo operands)."""
    r, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    if len(pos) == 0:
        return np.zeros((r, D)), np.full(r, -np.inf), 0.0
    G, target = rule(L, w0, W, mode)
    s = q @ k.T
    if G > 1 and w0 < L:
        qr = jo.rope_rotate(q, target - (L - 1), base)
        kr = jo.rope_rotate(k, pos // G - pos, base)
        s = np.where((L - 1 - pos < w0)[None, :], s, qr @ kr.T)
    s = s * scale
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    # each operand of a product carries 2^-17 (hi + lo), the fp32 sum of 2 D products 2^-16 at most;
    # a rotated pair's parts are bounded by the pair's length
    h = D // 2
    qa, ka = np.hypot(q[:, :h], q[:, h:]), np.hypot(k[:, :h], k[:, h:])
    err = abs(scale) * 2 * (qa @ ka.T).max() * 2.0 ** -15
    return p @ v / l, (m + np.log(l))[:, 0], err


def assert_decode(o, lse, want_o, want_lse, err, vmax, what=""):
    """o: bf16 rounding + a change of e^err either way of every weight; lse: err + fp32 rounding."""
    o, lse = np.asarray(o, np.float64), np.asarray(lse, np.float64)
    live = np.isfinite(want_lse)
    assert np.array_equal(np.isfinite(lse), live) and np.all(lse[~live] == -np.inf), what
    assert np.all(o[~live] == 0), what
    dl = np.abs(lse[live] - want_lse[live])
    assert np.all(dl <= err + 2.0 ** -20 * (1 + np.abs(want_lse[live]))), f"{what}: lse off by {dl.max():.2e}"
    do = np.abs(o - want_o)
    tol = BF16_HALF * np.abs(want_o) + (2 * err + 2.0 ** -16) * vmax
    assert np.all(do <= tol), f"{what}: o off by {do.max():.2e}"


def summary(k, page_size, base):
    """k [n, D]: the valid keys of one page, rows 0 .. n - 1."""
    t = np.arange(k.shape[0])
    return jo.rope_rotate(k, page_size // 2 - t, base).mean(0)


def select(q, summaries, L, page_size, w0, W, sink, top_k, base, mode=jo.MODE_SELF_EXTEND):
    """One KV head: q [r, D], summaries [pages, D] (fp64 values of bf16), in page order."""
    if L == 0:
        return []
    last = (L - 1) // page_size
    band = min(max(0, L - w0) // page_size, last)
    sink = min(sink, band)
    G, target = rule(L, w0, W, mode)
    cand = np.arange(sink, band)
    kept = list(range(sink)) + list(range(band, last + 1))
    if top_k and len(cand):
        c = cand * page_size + page_size // 2
        qr = jo.rope_rotate(q, target - (L - 1), base)
        s = (qr @ jo.rope_rotate(summaries[cand], c // G - c, base).T).max(0).astype(np.float32)
        order = sorted(range(len(cand)), key=lambda i: (-s[i] if s[i] == s[i] else -np.inf, i))
        kept += [int(cand[i]) for i in order[:top_k]]
    return sorted(kept)
