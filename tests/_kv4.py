"""Plain 64-bit forms of the rotary positions and of the 4-bit KV cache (numpy), for the tests."""
import numpy as np
import torch

E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def rotate(x, positions, freq, interleaved=False, inverse=False, mscale=1.0):
    """float64 [T, H, D] of x [T, H, D]."""
    y = np.array(x, dtype=np.float64)
    n = len(freq)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)[None]
    c, s = (mscale * np.cos(a))[:, None], (mscale * np.sin(a))[:, None]
    if inverse:
        s = -s
    i = np.arange(n)
    d0, d1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    x0, x1 = np.array(y[..., d0]), np.array(y[..., d1])
    y[..., d0], y[..., d1] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


def nearest(grid, x):
    """Index into the ascending grid nearest to each x >= 0; at a tie the even index; past the end the last."""
    at = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    low, high = x - grid[at - 1], grid[at] - x
    return np.where((low < high) | ((low == high) & ((at - 1) % 2 == 0)), at - 1, at)


def quantize(x, g):
    """(codes uint8 [..., D/2], scales uint8 [..., D/16]) of x [..., D]; the fp32 steps are the definition's."""
    g = np.float32(g)
    b = np.asarray(x).astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    t = np.fmax.reduce(np.abs(b), -1, initial=np.float32(0)) / (np.float32(6.0) * g)     # a NaN does not count
    sc = nearest(E4M3, t.astype(np.float64)).astype(np.uint8)
    s = (E4M3[sc].astype(np.float32) * g)[..., None]
    q = np.divide(b, s, out=np.zeros_like(b), where=s > 0)
    c = nearest(E2M1, np.abs(q).astype(np.float64)).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)
    c[np.isnan(q)] = 7                                                                   # the largest value
    c = c.reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), sc


def values(codes, scales, g):
    """The float64 values of codes [..., D/2] and scales [..., D/16]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*scales.shape, 16)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7] * E4M3[np.minimum(scales, 126)][..., None]
    return v.reshape(*scales.shape[:-1], 16 * scales.shape[-1]) * np.float64(np.float32(g))


def views(pages: torch.Tensor, page_size, D):
    """(codes [pages, heads, page_size, D/2], scales [pages, heads, page_size, D/16]) of a cache tensor."""
    cut = page_size * D // 2
    return pages[:, :, :cut].unflatten(2, (page_size, D // 2)), pages[:, :, cut:].unflatten(2, (page_size, D // 16))


def cached(pages, page_size, D, g, table_row, n):
    """float64 [heads, n, D]: the first n tokens of a sequence."""
    codes, scales = views(pages, page_size, D)
    ids = torch.as_tensor(table_row[:(n + page_size - 1) // page_size], device=pages.device, dtype=torch.long)
    v = values(codes[ids].cpu().numpy(), scales[ids].cpu().numpy(), g)         # [pages, heads, page_size, D]
    return v.transpose(1, 0, 2, 3).reshape(v.shape[1], len(ids) * page_size, D)[:, :n]


def attention(q, k, v, sm_scale, causal=True, window=0):
    """q [n, Hq, D], k and v [H, kv, D] float64 -> (o, lse, a, e): output, log sum, sum of weight times |v|, and a
    bound of the scores' size sum |q||k| * sm_scale (the largest over a row's keys), all float64."""
    n, Hq, D = q.shape
    H, kv, _ = k.shape
    o, a = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, e = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for h in range(Hq):
        kh, vh = k[h // (Hq // H)], v[h // (Hq // H)]
        for i in range(n):
            pos = kv - n + i
            last = min(kv, pos + 1) if causal else kv
            first = max(0, pos - window + 1) if window else 0
            if last <= first:
                continue
            s = kh[first:last] @ q[i, h] * sm_scale
            e[i, h] = (np.abs(kh[first:last]) @ np.abs(q[i, h])).max() * sm_scale
            w = np.exp(s - s.max())
            lse[i, h] = s.max() + np.log(w.sum())
            w /= w.sum()
            o[i, h], a[i, h] = w @ vh[first:last], w @ np.abs(vh[first:last])
    return o, lse, a, e
