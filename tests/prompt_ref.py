"""Plain implementations (numpy, float64) of the block assignment and of verify attention, one request at a time from the
definitions in the header, for the tests of requests that share a prompt."""
import numpy as np

BLOCK = 64


def assign(table, seq_lens, starts, free_list, free_count, slots):
    """In place on table and slots; (taken, free count)."""
    B, max_blocks = table.shape
    taken, used, asked = np.full(B, -1, np.int64), 0, 0
    for b in range(B):
        L, n, s0 = int(seq_lens[b]), int(starts[b + 1] - starts[b]), int(starts[b])
        slots[s0:s0 + n] = -1
        if L < 0 or L + n > max_blocks * BLOCK or (n and L % BLOCK and table[b, L // BLOCK] < 0):
            continue
        missing = [i for i in range(-(-L // BLOCK), (L + n - 1) // BLOCK + 1) if table[b, i] < 0] if n else []
        asked += len(missing)
        if missing and asked > free_count:
            continue
        for i in missing:
            used += 1
            table[b, i] = free_list[free_count - used]
        taken[b] = len(missing)
        for x in range(n):
            block = int(table[b, (L + x) // BLOCK])
            slots[s0 + x] = block * BLOCK + (L + x) % BLOCK if block >= 0 else -1
    return taken, free_count - used


def path_rows(parents, R):
    """[R, R] bool: row j sees verify key i."""
    see = np.zeros((R, R), bool)
    for j in range(R):
        at = j
        while at >= 0:
            see[j, at] = True
            at = at - 1 if parents is None else int(parents[at])
    return see


def attention(q, k, v, ctx, scale, parents=None):
    """One request: q [R, Hq, d], k and v [ctx + R, Hkv, d] with the verify tokens last; float64 [R, Hq, d]. Also, for
    error bounds, sum_t p_t |v_t| of every output and the largest sum |q k| scale of every row. A key that a row does not
    see takes no part, whatever it holds."""
    R, Hq, d = q.shape
    Hkv = k.shape[1]
    see = np.concatenate([np.ones((R, ctx), bool), path_rows(parents, R)], 1)
    out, absolute, score = np.empty((R, Hq, d)), np.empty((R, Hq, d)), np.empty((R, Hq, 1))
    with np.errstate(invalid="ignore", over="ignore"):
        for j in range(R):
            kj, vj, qj = k[see[j]].astype(np.float64), v[see[j]].astype(np.float64), q[j].reshape(Hkv, -1, d).astype(np.float64)
            x = np.einsum("hgd,thd->hgt", qj, kj) * scale
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[j] = np.einsum("hgt,thd->hgd", w, vj).reshape(Hq, d)
            absolute[j] = np.einsum("hgt,thd->hgd", w, np.abs(vj)).reshape(Hq, d)
            score[j] = np.einsum("hgd,thd->hgt", np.abs(qj), np.abs(kj)).max(-1).reshape(Hq, 1) * scale
    return out, absolute, score
