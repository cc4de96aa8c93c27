"""The serving operators written out in 64 bits (numpy and torch on the CPU),
shared by their tests.  The cache's bytes are computed here byte by byte from
the layout that include/df11.h states, apart from the library."""
import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# E4M3 bytes 0 .. 126 in ascending order (127 is NaN)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest(x, grid):
    """Index of the entry of the ascending grid nearest to x >= 0, saturating; ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def to_bf16(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def quantize(x, g):
    """x (..., d) float (rounded to BF16 first) -> (codes 0..15, scale bytes, values), scale g; the scale and the
    quotients in FP32 steps, which are exact in 64 bits too when g is a power of two."""
    x = to_bf16(x)
    x = x.reshape(*x.shape[:-1], -1, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        top = np.nanmax(np.where(np.isnan(x), np.float32(0), np.abs(x)), axis=-1)
        want = np.minimum((top / np.float32(6)) / g, np.float32(448))
        sb = nearest(want.astype(np.float64), E4M3)
        step = E4M3[sb].astype(np.float32) * g
        a = np.abs(x) / step[..., None]
        a = np.where(np.isnan(x), np.inf, a)
        lv = np.where((step == 0)[..., None], 0, nearest(np.minimum(np.nan_to_num(a, nan=0.0, posinf=9.0), 9.0), LEVELS))
    neg = np.signbit(x) & ~np.isnan(x) & (step > 0)[..., None]
    val = np.where(neg, -1.0, 1.0) * LEVELS[lv] * E4M3[sb][..., None] * float(g)
    flat = (*x.shape[:-2], -1)
    return (lv | (neg.astype(np.int64) << 3)).reshape(flat).astype(np.uint8), sb.astype(np.uint8), val.reshape(flat)


class Cache:
    """The pages as bytes on the CPU, written token by token."""

    def __init__(self, n_pages, page, heads, dim, gk, gv, fill=0):
        self.n_pages, self.page, self.heads, self.dim, self.gk, self.gv = n_pages, page, heads, dim, gk, gv
        self.block = page * dim * 9 // 8
        self.bytes = np.full((n_pages, heads, self.block), fill, np.uint8)
        self.k = np.zeros((n_pages * page, heads, dim))  # what the slots hold
        self.v = np.zeros((n_pages * page, heads, dim))

    def write(self, slots, k, v):
        """k, v (t, heads, dim)."""
        P, D = self.page, self.dim
        ck, sk, vk = quantize(k, self.gk)
        cv, sv, vv = quantize(v, self.gv)
        kc, ks = P * D // 2, P * D // 16
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            p, o = divmod(int(slot), P)
            b = self.bytes[p]
            b[:, o * D // 2:(o + 1) * D // 2] = ck[t, :, 0::2] | (ck[t, :, 1::2] << 4)
            b[:, kc + o * D // 16:kc + (o + 1) * D // 16] = sk[t]
            vb = cv[t, :, 0::2] | (cv[t, :, 1::2] << 4)  # (heads, D / 2)
            for blk in range(D // 16):
                at = kc + ks + (((o // 4) * (D // 16) + blk) * 4 + o % 4) * 8
                b[:, at:at + 8] = vb[:, 8 * blk:8 * blk + 8]
                b[:, 2 * kc + ks + blk * P + o] = sv[t, :, blk]
            self.k[slot], self.v[slot] = vk[t], vv[t]


def extend(kv_lens, new_lens, free, n_free, table, page, max_tokens):
    """Token by token; a page is taken when a token starts it.  Returns table, kv_out, q_start, slots, positions,
    n_free_out."""
    table = [list(map(int, row)) for row in table]
    stack = [int(x) for x in free[:n_free]]
    kv_out, q_start, slots, pos = [], [0], [], []
    for r, (kv, new) in enumerate(zip(map(int, kv_lens), map(int, new_lens))):
        for p in range(kv, kv + new):
            if p % page == 0:
                table[r][p // page] = stack.pop()
            slots.append(table[r][p // page] * page + p % page)
            pos.append(p)
        kv_out.append(kv + new)
        q_start.append(len(slots))
    pad = max_tokens - len(slots)
    return table, kv_out, q_start, slots + [-1] * pad, pos + [0] * pad, len(stack)


def norm_rope(x, w, positions, inv_freq, rot, inter, eps):
    """x (t, heads, dim) float64 -> (y, the magnitude |a| + |b| of each element's pair after the norm)."""
    d = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    ang = np.outer(positions, inv_freq)[:, None, :]
    c, s = np.cos(ang), np.sin(ang)
    y, mag = x.copy(), np.abs(x)
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def attention(q, k, v, causal, window, scale):
    """One request: q (n, hq, d), k and v (kv, h, d), float64 tensors.  Returns o, lse and, for the error bound,
    the weighted magnitudes sum p |v| (n, hq, d), each row's largest scale * sum |q k| (n, hq), the largest |v| (hq)."""
    n, hq, d = q.shape
    kv, h = k.shape[0], k.shape[1]
    g = hq // h
    o, lse = torch.zeros(n, hq, d, dtype=torch.float64), torch.full((n, hq), -np.inf, dtype=torch.float64)
    wmag, smag, vmax = torch.zeros_like(o), torch.zeros(n, hq, dtype=torch.float64), torch.zeros(hq, dtype=torch.float64)
    if kv == 0 or n == 0:
        return o, lse, wmag, smag, vmax
    i, j = torch.arange(n)[:, None], torch.arange(kv)[None, :]
    seen = torch.ones(n, kv, dtype=torch.bool)
    if causal:
        seen = j <= kv - n + i
        if window:
            seen &= j > kv - n + i - window
    for c in range(hq):
        kk, vv = k[:, c // g], v[:, c // g]
        sc = (q[:, c] @ kk.T) * scale
        sc = torch.where(seen, sc, torch.full_like(sc, -np.inf))
        z = torch.logsumexp(sc, -1)
        p = torch.exp(sc - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
        o[:, c], lse[:, c] = p @ vv, z
        wmag[:, c] = p @ vv.abs()
        smag[:, c] = torch.where(seen, q[:, c].abs() @ kk.abs().T, torch.zeros_like(sc)).amax(-1) * abs(scale)
        vmax[c] = vv.abs().max()
    return o, lse, wmag, smag, vmax


def attention_bounds(o, lse, wmag, smag, vmax, kv, d):
    """Bounds on |o - exact| and |lse - exact| for scores summed in FP32 and probabilities rounded to FP16.

    A score is d products (exact: 8 and 6 significant bits) added in FP32 on the tensor cores, each add off by at
    most 2^-23 of the sum of magnitudes (they may truncate), then scaled (2 roundings) and reduced by the row's
    maximum (1): ds = (d + 8) 2^-23 smag, 2^-24 of the row's spread of scores, at most 2 smag, included.  Elements of
    q below 2^-24 of their row's largest vanish in FP16: within the same bound.  exp multiplies that by its argument's
    error: relative dp = ds + 2^-20 (its own 2 units in the last place and the multiplication by log2 e).  p is rounded
    to FP16: 2^-11 relative, or 2^-25 absolute when subnormal, against a row sum of at least 1 (the split of a row's
    keys only divides that by exp of a difference of maxima: still <= 1 after the join).  The products p v are
    exact in FP32, their sums and the row sum's are off by at most (kv + 64) 2^-23 of the magnitudes.  o then takes
    one rounding to BF16."""
    ds = (d + 8) * 2.0 ** -23 * smag
    rel = 2.0 ** -11 + 2 * (ds + 2.0 ** -20) + 2 * (kv + 64) * 2.0 ** -23
    bo = wmag * rel[..., None] + kv * 2.0 ** -25 * vmax[None, :, None]
    bo = bo + 2.0 ** -8 * (o.abs() + bo)
    bl = ds + 2.0 ** -20 + (kv + 64) * 2.0 ** -23 + 2.0 ** -22 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return bo, bl
