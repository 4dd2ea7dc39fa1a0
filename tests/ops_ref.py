"""Plain 64-bit references of the handle-free operators (include/beam_ops.h),
in numpy, from their definitions.  Roundings to the small formats are by
search in the sorted list of their values, ties to the even code."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def nearest_code(v, grid):
    """Code of the grid value nearest to |v| (saturating), ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    return np.where(up == down, np.where(hi % 2 == 0, hi, lo), np.where(up < down, hi, lo))


def pow2_exponent(amax, top):
    """Least k in [-127, 127] with amax <= top 2^k."""
    k = np.full(amax.shape, -127)
    for i in range(-126, 128):
        k = np.where(amax > top * 2.0 ** (i - 1), i, k)
    return k


def tensor_scale(x):
    a = np.abs(x[np.isfinite(x)]).max(initial=0.0)
    a = max(a, 2.0 ** -100)
    k = -120
    while 2688.0 * 2.0 ** k < a:
        k += 1
    return 2.0 ** k


def quantize(x, fmt, g=None):
    """x float64 [rows, K] holding FP32 values -> (signed codes as element
    values [rows, K], scale bytes [rows, K / block]).  NVFP4 quotients are
    rounded to FP32 first, as the operator defines them."""
    rows, K = x.shape
    b = x.reshape(rows, -1, BLOCK[fmt])
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    if fmt == "nvfp4":
        g32 = np.float32(g)
        if not 2.0 ** -112 <= float(g32) <= 2.0 ** 112:
            return np.zeros_like(x), np.full(amax.shape, 0x7f)
        with np.errstate(over="ignore", under="ignore", divide="ignore", invalid="ignore"):
            sb = nearest_code((amax.astype(np.float32) / (np.float32(6) * g32)).astype(np.float64), E4M3)
            d = (E4M3[sb].astype(np.float32) * g32)[..., None]
            q = np.where(d > 0, b.astype(np.float32) / np.where(d > 0, d, np.float32(1)), np.float32(0))
        e = np.copysign(E2M1[nearest_code(q.astype(np.float64), E2M1)], b)
        return np.where(bad[..., None], 0.0, e).reshape(x.shape), np.where(bad, 0x7f, sb)
    top, grid = (448.0, E4M3) if fmt == "mxfp8" else (6.0, E2M1)
    k = pow2_exponent(amax, top)
    e = np.copysign(grid[nearest_code(b * 2.0 ** -k[..., None].astype(np.float64), grid)], b)
    return np.where(bad[..., None], 0.0, e).reshape(x.shape), np.where(bad, 0xff, k + 127)


def scale_values(sb, fmt):
    if fmt == "nvfp4":
        return np.where(sb == 0x7f, np.nan, E4M3[np.minimum(sb, 126)])
    return np.where(sb == 0xff, np.nan, 2.0 ** (sb.astype(np.float64) - 127))


def values(e, sb, fmt, g=1.0):
    rows, K = e.shape
    return (e.reshape(rows, -1, BLOCK[fmt]) * scale_values(sb, fmt)[..., None]).reshape(rows, K) * g


def tile(sb):
    """Scale bytes [rows, n] in the tiled layout, zeros past the ends."""
    rows, n = sb.shape
    n4 = (n + 3) // 4
    out = np.zeros((rows + 127) // 128 * n4 * 512, np.uint8)
    for r in range(rows):
        for j in range(n):
            out[((r // 128) * n4 + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4] = sb[r, j]
    return out


def codes(e, fmt):
    """Element values to code bytes."""
    grid = E4M3 if fmt == "mxfp8" else E2M1
    c = nearest_code(e, grid) + np.signbit(e) * (128 if fmt == "mxfp8" else 8)
    return c.astype(np.uint8) if fmt == "mxfp8" else (c[:, 0::2] + 16 * c[:, 1::2]).astype(np.uint8)


def elements(c, fmt):
    if fmt == "mxfp8":
        return np.where(c & 128, -1.0, 1.0) * E4M3[np.minimum(c & 127, 126)]
    n = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    return np.where(n & 8, -1.0, 1.0) * E2M1[n & 7]


def route(logits, top_k, score, bias, n_group, topk_group, group_top, renorm, scale):
    """-> (idx, w) of float64 logits, row by row."""
    T, E = logits.shape
    idx, w = np.full((T, top_k), -1), np.zeros((T, top_k))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(T):
        l = logits[t]
        if np.isnan(l).any() or np.isnan(b).any() or (score == "softmax" and np.isposinf(l).any()):
            w[t] = np.nan
            continue
        ok = (l > -np.inf) & (b > -np.inf)
        if not (l > -np.inf).any():
            continue
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                logp = np.where(l < 0, l - np.log1p(np.exp(np.minimum(l, 0))), -np.log1p(np.exp(-np.maximum(l, 0))))
            else:
                logp = l - l.max() - np.log(np.exp(l - l.max()).sum())
        key = np.where(ok, np.exp(logp) + np.where(ok, b, 0.0), -np.inf)
        if topk_group < n_group:
            per = key.reshape(n_group, -1)
            best = -np.sort(-per, 1)[:, :group_top]
            gs = np.where(best[:, 0] > -np.inf, np.where(best > -np.inf, best, 0.0).sum(1), -np.inf)
            keep = np.argsort(-gs, kind="stable")[:topk_group]
            mask = np.zeros(n_group, bool)
            mask[keep] = True
            key = np.where(np.repeat(mask, E // n_group), key, -np.inf)
        rank = np.where(key > -np.inf, l if bias is None else key, -np.inf)
        order = np.lexsort((np.arange(E), -rank))
        order = order[key[order] > -np.inf][:top_k]
        p = logp[order]
        v = np.exp(p - p.max()) if renorm and len(p) else np.exp(p)
        if renorm and len(p):
            v = v / v.sum()
        idx[t, :len(order)], w[t, :len(order)] = order, v * scale
    return idx, w
