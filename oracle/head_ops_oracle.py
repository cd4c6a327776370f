"""Plain fp64 definitions of the operators on given arrays (numpy): token log
probabilities with entropy and alternatives, their gradient, the block-scaled
e4m3 quantization and product.  Shares no code with the HIP path."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
BLOCK = 128


def token_logprobs(z, tokens=None, temperature=None, top_n=0, ignore_index=None):
    """dict of logprob [T, K], lse, entropy [T], top_logprob, top_id [T, top_n]
    (see ``stce_token_logprobs`` in ``include/stce.h``)."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    temp = np.ones(T) if temperature is None else np.asarray(temperature, np.float64)
    bad = ~(np.isfinite(temp) & (temp > 0)) | np.isnan(z).any(1) | (z == np.inf).any(1)
    empty = (z == -np.inf).all(1) & ~bad
    safe = np.where((bad | empty)[:, None], 0.0, z)
    s = safe / np.where(bad, 1.0, temp)[:, None]
    m = s.max(1, keepdims=True)
    d = s - m
    e = np.exp(d)
    S = e.sum(1)
    logp = d - np.log(S)[:, None]
    lse = m[:, 0] + np.log(S)
    entropy = -(np.where(e > 0, e * np.where(e > 0, logp, 0.0), 0.0)).sum(1) / S
    logp[empty] = -np.inf
    lse[empty], entropy[empty] = -np.inf, 0.0
    logp[bad], lse[bad], entropy[bad] = np.nan, np.nan, np.nan
    out = dict(lse=lse, entropy=entropy, logp=logp, bad=bad, empty=empty)
    if tokens is not None:
        tok = np.asarray(tokens)
        ok = (tok >= 0) & (tok < V)
        lp = np.take_along_axis(logp, np.where(ok, tok, 0), 1)
        lp = np.where(ok, lp, np.nan)
        if ignore_index is not None:
            lp = np.where(tok == ignore_index, 0.0, lp)
        out["logprob"] = lp
    if top_n:
        ids = np.full((T, top_n), -1, np.int64)
        tl = np.full((T, top_n), -np.inf)
        for t in range(T):
            if bad[t]:
                tl[t] = np.nan
                continue
            order = np.lexsort((np.arange(V), -z[t]))[:top_n]
            order = order[z[t, order] > -np.inf]
            ids[t, :len(order)] = order
            tl[t, :len(order)] = logp[t, order]
        out["top_id"], out["top_logprob"] = ids, tl
    return out


def token_logprobs_backward(z, tokens, g_logprob=None, g_entropy=None, g_lse=None, temperature=None,
                            ignore_index=None):
    z = np.asarray(z, np.float64)
    T, V = z.shape
    r = token_logprobs(z, None, temperature)
    temp = np.ones(T) if temperature is None else np.asarray(temperature, np.float64)
    dz = np.zeros((T, V))
    for t in range(T):
        if r["bad"][t] or r["empty"][t]:
            continue
        p = np.exp(r["logp"][t])
        if g_logprob is not None:
            for y, g in zip(tokens[t], g_logprob[t]):
                if 0 <= y < V and y != ignore_index and z[t, y] > -np.inf:
                    dz[t] -= float(g) * p
                    dz[t, y] += float(g)
        if g_entropy is not None:
            lp = np.where(p > 0, r["logp"][t], 0.0)
            dz[t] -= float(g_entropy[t]) * p * (lp + r["entropy"][t])
        if g_lse is not None:
            dz[t] += float(g_lse[t]) * p
        dz[t] /= temp[t]
    return dz


def e4m3_values():
    """The value of every e4m3 code (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v = np.where(c & 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


def e4m3_nearest(x):
    """Codes nearest to x (|x| <= 448), ties to the even code."""
    mags = e4m3_values()[:127]                       # 0 .. 448, increasing
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize_blocks(x, block="row", transpose=False):
    """(codes uint8 [Q, round_up(L, 16)], scales fp32 [Q or tiles, blocks]);
    quotients rounded to fp32 as the definition asks."""
    y = np.asarray(x, np.float32)
    y = y.T if transpose else y
    Q, L = y.shape
    rows = 1 if block == "row" else BLOCK
    nq, nl = -(-Q // rows), -(-L // BLOCK)
    codes = np.zeros((Q, -(-L // 16) * 16), np.uint8)
    scales = np.ones((nq, nl), np.float32)
    for i in range(nq):
        for j in range(nl):
            v = y[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            if not np.isfinite(v).all():
                scales[i, j] = np.nan
                continue
            a = np.float32(np.abs(v).max() * np.float32(1 / E4M3_MAX))
            scales[i, j] = a if a > 0 else np.float32(1)
            q = np.clip((v / scales[i, j]).astype(np.float32), -E4M3_MAX, E4M3_MAX)
            codes[i * rows:i * rows + v.shape[0], j * BLOCK:j * BLOCK + v.shape[1]] = e4m3_nearest(q)
    return codes, scales


def dequantize(codes, scales, rows):
    """fp64 values of codes [R, K] with a scale per `rows` rows and 128 columns."""
    v = e4m3_values()[codes]
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, 0)[:v.shape[0]], BLOCK, 1)[:, :v.shape[1]]
    return v * s


def block_matmul(a, a_scale, b, b_scale):
    """(a b^T, sum of the products' magnitudes), fp64."""
    x = dequantize(a, a_scale, 1)
    y = dequantize(b, b_scale, 1 if b_scale.shape[0] == b.shape[0] else BLOCK)
    return x @ y.T, np.abs(x) @ np.abs(y).T
