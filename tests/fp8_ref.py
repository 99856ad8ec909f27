"""64-bit numpy reference of the scored routing and the 8-bit float operators, with
the error bounds the GPU results are held to.  Shares no code with the library."""
import numpy as np

B = 128
U = 2.0 ** -24   # unit roundoff of fp32


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-a if s else a)
    return v


E4M3 = _e4m3_table()
_POS = E4M3[:0x7F]           # 0 .. 448 ascending
_MID = (_POS[1:] + _POS[:-1]) / 2


def decode(codes):
    return E4M3[np.asarray(codes, np.uint8)]


def encode(v):
    """Nearest e4m3 code, ties to the even code, |v| <= 448 (64-bit)."""
    a = np.abs(np.asarray(v, np.float64))
    lo = np.searchsorted(_MID, a, side="left")     # a <= mid[lo]: code lo, unless a tie sends it up
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    return np.where(np.signbit(v), code | 0x80, code).astype(np.uint8)


def near_midpoint(v, dv):
    """Where a value uncertain by dv could round to another code, and the step it could move by."""
    a = np.abs(v)
    i = np.clip(np.searchsorted(_POS, a, side="right") - 1, 0, len(_POS) - 2)
    mid, step = _MID[i], _POS[i + 1] - _POS[i]
    return np.abs(a - mid) <= dv, step


def nb(n):
    return (n + B - 1) // B


def quantize(x):
    """codes uint8 [T][K], scales fp64 [T][K/128] of 64-bit x."""
    T, K = x.shape
    q, d = np.zeros((T, K), np.uint8), np.zeros((T, nb(K)))
    for b in range(nb(K)):
        v = x[:, b * B:(b + 1) * B]
        a = np.abs(v).max(axis=1, keepdims=True)
        af = np.maximum(a, 2.0 ** -116)
        q[:, b * B:(b + 1) * B] = np.where(a > 0, encode(v * 448.0 / af), 0)
        d[:, b] = np.where(a > 0, af / 448.0, 0.0)[:, 0]
    return q, d


def dequant_w(q, s):
    N, K = q.shape
    return decode(q) * np.repeat(np.repeat(s.astype(np.float64), B, 0)[:N], B, 1)[:, :K]


def dequant_x(q, d):
    return decode(q) * np.repeat(np.asarray(d, np.float64), B, 1)[:, :q.shape[1]]


def _group_max(v):
    """Largest magnitude of each eight consecutive columns."""
    return np.abs(np.pad(v, ((0, 0), (0, -v.shape[1] % 8)))).reshape(v.shape[0], -1, 8).max(axis=2)


def matmul(xq, xs, wq, ws, fast=False):
    """y and its error bound: the products of a block summed in fp32 (128 roundings), a scale product, one fma
    per block.  fast: the 8-bit matrix unit, which aligns eight consecutive products to the largest and truncates
    below 2^-13 of its exponent; the largest itself (eight significant bits) loses nothing, the other seven less
    than 2^-13 of it each."""
    x, w = dequant_x(xq, xs), dequant_w(wq, ws)
    bound = (B + nb(xq.shape[1]) + 4) * U * (np.abs(x) @ np.abs(w).T)
    if fast:
        bound = bound + 7 * 2.0 ** -13 * (_group_max(x) @ _group_max(w).T)
    return x @ w.T, bound


def expert(xq, xs, gate, up, down, fast=False):
    """One expert's y rows and their bound: fp32 sums, and the codes of h that rounding could move."""
    g, dg = matmul(xq, xs, *gate, fast)
    u, du = matmul(xq, xs, *up, fast)
    sig = 1 / (1 + np.exp(-g))
    h = g * sig * u
    # |silu'| <= 1.1; the device's exponential and reciprocal: e^-g within (|g| + 4) ulp, 1/x within 2
    dh = 1.1 * dg * np.abs(u) + np.abs(g * sig) * du + 1.1 * dg * du + (np.abs(g) + 10) * 2 * U * np.abs(h)
    q, d = quantize(h)
    ab = np.repeat(d * 448.0, B, 1)
    da = np.repeat(dh.reshape(h.shape[0], -1, B).max(axis=2), B, 1)
    safe = np.where(ab > 0, ab, 1.0)
    quot = h * 448.0 / safe
    rho = da / safe
    dq = (dh * 448.0 / safe + np.abs(quot) * (rho + 8 * U)) * 1.01
    hit, step = near_midpoint(quot, dq)
    hv = dequant_x(q, d)
    dv = np.where(hit, step * ab / 448.0, 0.0) + np.abs(hv) * (rho + 2 * U) * 1.01
    w = dequant_w(*down)
    y, dy = matmul(q, d, *down, fast)
    return y, dy + dv @ np.abs(w).T * 1.01


def route(logits, k, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, bias=None):
    l = np.asarray(logits, np.float64)
    if score == "softmax":
        s = np.exp(l - l.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    else:
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-l))
    T, E = l.shape
    c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    alive = np.ones((T, E), bool)
    if n_group > 1:
        S = E // n_group
        with np.errstate(invalid="ignore"):
            gs = np.sort(c.reshape(T, n_group, S), axis=2)[:, :, ::-1][:, :, :group_top].sum(axis=2)
        keep = np.argsort(-gs, axis=1, kind="stable")[:, :topk_group]
        ga = np.zeros((T, n_group), bool)
        np.put_along_axis(ga, keep, True, 1)
        alive = np.repeat(ga, S, 1)
    # dropped experts after every kept one, -inf biased ones included
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -c, ~alive), axis=1)
    idx = order[:, :k]
    w = np.take_along_axis(s, idx, 1)
    if renorm:
        t = w.sum(axis=1, keepdims=True)
        w = np.where(t > 0, w / np.where(t > 0, t, 1.0), 0.0)
    return idx.astype(np.int32), w * scale


def buckets(idx, E):
    flat = idx.reshape(-1)
    pair = np.argsort(flat, kind="stable").astype(np.int32)
    count = np.bincount(flat, minlength=E).astype(np.int32)
    offset = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    return pair, count, offset, np.nonzero(count)[0].astype(np.int32)
