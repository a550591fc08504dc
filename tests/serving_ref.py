"""Plain 64-bit forms of the serving operators, on the CPU (numpy), for their tests."""
import numpy as np
import torch

E4M3 = np.array([(1 if i < 128 else -1) * (np.nan if (i & 127) == 127 else
                 ((1 + (i & 7) / 8) * 2.0 ** (((i >> 3) & 15) - 7) if (i >> 3) & 15 else (i & 7) / 512))
                 for i in range(256)])
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def block_byte(amax):
    """E8M0 byte of blocks whose largest finite magnitude is amax: the least X >= -126 with amax <= 448 * 2^X."""
    amax = np.asarray(amax, np.float64)
    byte = np.zeros(amax.shape, np.int64)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            X = -126
            while a > 448.0 * 2.0 ** X:
                X += 1
            byte[i] = X + 127
    return byte


def e4m3_bytes(v):
    """E4M3 bytes of float64 values: nearest, ties to even, saturating; NaN stays NaN."""
    v = np.asarray(v, np.float64)
    grid = E4M3[:127]
    a = np.minimum(np.abs(np.where(np.isnan(v), 0, v)), 448.0)
    hi = np.searchsorted(grid, a)
    lo = np.maximum(hi - 1, 0)
    mid = (grid[lo] + grid[hi]) / 2
    pick = np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)
    pick = np.where(np.isnan(v), 127, pick)
    return (pick + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def finite_amax(x, axis):
    return np.max(np.where(np.isfinite(x), np.abs(x), 0), axis=axis)


def tc_rows(flat, rows, cols):
    """[rows, cols] of a flat tensor-core-layout scale buffer."""
    katoms = -(-cols // 4)
    r, c = np.arange(rows)[:, None], np.arange(cols)[None]
    return flat[((r // 128) * katoms + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]


def tables(table, lens, new, free, head, P, max_tokens):
    table = table.copy()
    width, cu, slots, at = table.shape[1], [0], [], head
    for b in range(len(lens)):
        n, have = new[b], -(-lens[b] // P)
        for col in range(have, min(-(-(lens[b] + n) // P), width)):
            table[b, col] = free[at] if at < len(free) else -1
            at += 1
        for i in range(n):
            p = lens[b] + i
            page = table[b, p // P] if p // P < width else -1
            slots.append(page * P + p % P if page >= 0 else -1)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return table, np.minimum(cu, max_tokens), np.array(slots), min(at, len(free))


def append(x, slots, codes, byte, P):
    """x [T, H, D] float64 into codes [NP, H, P, D] and byte [NP, H], in place."""
    t, T = 0, len(slots)
    while t < T:
        n = 1
        if slots[t] < 0 or slots[t] >= codes.shape[0] * P:
            t += 1
            continue
        while t + n < T and slots[t + n] == slots[t] + n and slots[t + n] % P:
            n += 1
        page, row = slots[t] // P, slots[t] % P
        new = x[t:t + n].transpose(1, 0, 2)  # [H, n, D]
        b = block_byte(finite_amax(new, (1, 2)))
        if row:
            old = byte[page].astype(np.int64)
            b = np.maximum(b, old)
            for h in range(len(b)):
                if b[h] > old[h]:
                    codes[page, h, :row] = e4m3_bytes(E4M3[codes[page, h, :row]] * 2.0 ** float(old[h] - b[h]))
        byte[page] = b
        codes[page, :, row:row + n] = e4m3_bytes(new * 2.0 ** (127.0 - np.maximum(b, 1))[:, None, None] *
                                                 np.where(b > 0, 1.0, 2.0 ** -126)[:, None, None])
        t += n


def cache_values(codes, byte):
    return E4M3[codes] * 2.0 ** (byte.astype(np.float64) - 127)[..., None, None]


def attention(q, kc, kb, vc, vb, table, lens, cu, P, scale):
    """out [T, HQ, D] (NaN in rows of no request) and the error bound's parts: sum p |v|, and the
    largest sum |q k| * |scale| of a row."""
    T, HQ, D = q.shape
    NP, H = kb.shape
    G = HQ // H
    out = np.full((T, HQ, D), np.nan)
    spread, dots = np.zeros((T, HQ, D)), np.zeros((T, HQ, 1))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        L = lens[b] + n
        if n <= 0:
            continue
        pages = table[b, :-(-L // P)]
        seen = (pages >= 0) & (pages < NP)
        rows = np.repeat(seen, P)[:L]
        pages = np.where(seen, pages, 0)
        for h in range(H):
            k = cache_values(kc[pages, h], kb[pages, h]).reshape(-1, D)[:L]
            v = cache_values(vc[pages, h], vb[pages, h]).reshape(-1, D)[:L]
            for i in range(n):
                see = rows & (np.arange(L) <= lens[b] + i)
                for j in range(h * G, (h + 1) * G):
                    t = cu[b] + i
                    if not see.any():
                        out[t, j] = 0
                        continue
                    s = scale * (k[see] @ q[t, j])
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, j] = p @ v[see]
                    spread[t, j] = p @ np.abs(v[see])
                    dots[t, j] = abs(scale) * np.max(np.abs(k[see]) @ np.abs(q[t, j]))
    return out, spread, dots


def hadamard(x, b):
    if not b:
        return x
    h = np.ones((1, 1))
    while h.shape[0] < b:
        h = np.block([[h, h], [h, -h]])
    return (x.reshape(-1, b) @ h / np.sqrt(b)).reshape(x.shape)


def weight(codes, scales, fmt, g=1.0):
    """float64 [N, K] of codes [N, K/2] and tensor-core-layout scales."""
    N, K = codes.shape[0], codes.shape[1] * 2
    w = np.empty((N, K))
    w[:, 0::2], w[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    blk = 16 if fmt == "nvfp4" else 32
    s = tc_rows(scales, N, K // blk)
    s = E4M3[s] * g if fmt == "nvfp4" else 2.0 ** (s.astype(np.float64) - 127)
    return w * np.repeat(s, blk, 1)
