"""Plain float64 implementations (numpy) of the 8-bit cache append, the windowed verify attention over either cache and
the window release, for the tests. One request, block and head at a time, from the definitions in the header."""
import numpy as np

BLOCK = 64
MIN_EXP = -100


def e4m3_values():
    """The value of every byte; NaN at 0x7f and 0xff."""
    v = np.empty(256)
    for byte in range(256):
        e, m = (byte >> 3) & 15, byte & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[byte] = (-x if byte & 128 else x) if byte & 127 != 127 else np.nan
    return v


VALUES = e4m3_values()
_POS = VALUES[:127]


def to_e4m3(x):
    """Bytes of the nearest e4m3 values (ties to the even byte); not finite -> NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        m = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    up = np.minimum(np.searchsorted(_POS, m), 126)
    dn = np.maximum(up - 1, 0)
    a, b = m - _POS[dn], _POS[up] - m
    take = np.where((a < b) | ((a == b) & (dn % 2 == 0)), dn, up)
    take = np.where(_POS[up] == m, up, take)
    byte = take | np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), byte, 127).astype(np.uint8)


def block_scale(old, fresh, a):
    """(new scale, doublings) per head for the largest written magnitudes a."""
    s = np.where(fresh, np.float32(2.0 ** MIN_EXP), old).astype(np.float32)
    k = np.zeros(len(s), np.int64)
    for h in range(len(s)):
        with np.errstate(over="ignore"):
            while np.float32(448.0) * s[h] < np.float32(a[h]):
                s[h] *= np.float32(2.0)
                k[h] += 1
    return s, k


def append(cache, scale, x, starts, ctx, table):
    """In place: cache bytes [nb, 64, H, d] uint8, scale [nb, H] float32; x [T, H, d] float."""
    for b in range(len(ctx)):
        n = starts[b + 1] - starts[b]
        at, end = ctx[b], ctx[b] + n
        while at < end:
            page, off = at // BLOCK, at % BLOCK
            stop = min(end, (page + 1) * BLOCK)
            blk = table[b][page]
            part = np.asarray(x[starts[b] + at - ctx[b]:starts[b] + stop - ctx[b]], np.float64)
            a = np.where(np.isfinite(part), np.abs(part), 0.0).max(axis=(0, 2))
            s, k = block_scale(scale[blk], off == 0, a)
            if off:
                kept = VALUES[cache[blk, :off]] * (2.0 ** -k.astype(np.float64))[:, None]
                cache[blk, :off] = np.where(np.isnan(kept) | (k == 0)[:, None], cache[blk, :off], to_e4m3(kept))
            scale[blk] = s
            with np.errstate(invalid="ignore"):   # x / s is rounded to float32 first (the kernel's arithmetic)
                y = (part.astype(np.float32) / s[:, None]).astype(np.float64)
            cache[blk, off:off + stop - at] = to_e4m3(y)
            at = stop


def visible(t, p, window, sinks):
    return (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))


def attention(q, k_rows, v_rows, ctx, sm_scale, window, sinks):
    """One request: q [R, Hq, d], k_rows / v_rows(t) -> [len(t), Hkv, d]; float64 [R, Hq, d]. Also, for error bounds,
    sum_t p_t |v_t| of every output, the largest sum |q k| sm_scale of every row, and sum_t m_t |v_t| of every output
    with m_t the largest p within 767 visible slots of t."""
    R, Hq, d = q.shape
    t = np.arange(ctx + R)
    t = t[visible(t, ctx, window, sinks) | (t > ctx)]
    k, v = k_rows(t), v_rows(t)
    g = Hq // k.shape[1]
    out, absolute, score, near = np.empty((R, Hq, d)), np.empty((R, Hq, d)), np.empty((R, Hq, 1)), np.empty((R, Hq, d))
    for j in range(R):
        see = visible(t, ctx + j, window, sinks)
        for h in range(Hq):
            kh, vh, qh = k[see, h // g], v[see, h // g], np.asarray(q[j, h], np.float64)
            x = kh @ qh * sm_scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[j, h], absolute[j, h] = w @ vh, w @ np.abs(vh)
            wide = np.lib.stride_tricks.sliding_window_view(np.pad(w, 767), 1535).max(axis=1)
            near[j, h] = wide @ np.abs(vh)
            score[j, h] = (np.abs(kh) @ np.abs(qh)).max() * sm_scale
    return out, absolute, score, near


def release(table, seq_lens, free_list, free_count, window, sinks):
    """In place; the new free count."""
    pos = count = int(free_count)
    for b in range(len(seq_lens)):
        L = int(seq_lens[b])
        if L < 0 or L > table.shape[1] * BLOCK:
            continue
        gone = [i for i in range(table.shape[1])
                if i * BLOCK >= sinks and i * BLOCK + BLOCK - 1 <= L - window and table[b, i] >= 0]
        if gone and pos + len(gone) <= len(free_list):
            for n, i in enumerate(gone):
                free_list[pos + n] = table[b, i]
                table[b, i] = -1
            count = pos + len(gone)
        pos += len(gone)
    return count
