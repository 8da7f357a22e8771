"""Plain numpy forms, in 64 bits, of the serving operators: page plan, 4-bit key/value cache,
attention over it, and logit adjustment."""
import numpy as np

CHUNK = 16


def plan(past, fresh, free, page, table, T, start=0):
    """(table, q_start, kv_len, position, slot, counts), request by request, token by token."""
    table = table.copy()
    R, width = table.shape
    q_start, kv_len, position, slot = [0], [], [], []
    at = start
    for r in range(R):
        p, f = max(int(past[r]), 0), max(int(fresh[r]), 0)
        have, need = -(-p // page), -(-(p + f) // page)
        for c in range(have, need):
            got = int(free[at]) if 0 <= at < len(free) else -1
            if c < width:
                table[r, c] = got
            at += 1
        for x in range(p, p + f):
            pg = int(table[r, x // page]) if x // page < width else -1
            position.append(x)
            slot.append(pg * page + x % page if pg >= 0 else -1)
        q_start.append(q_start[-1] + f)
        kv_len.append(p + f)
    counts = [q_start[-1], at]
    position = (position + [-1] * T)[:T]
    slot = (slot + [-1] * T)[:T]
    return (table, np.array(q_start), np.array(kv_len), np.array(position, dtype=np.int64),
            np.array(slot, dtype=np.int64), np.array(counts))


def quantize(x):
    """Codes, scale and zero of rows of fp32 x [..., D] (binary32 arithmetic, as defined)."""
    x = x.astype(np.float32)
    lo = np.minimum(x.min(-1, keepdims=True), np.float32(0))
    hi = np.maximum(x.max(-1, keepdims=True), np.float32(0))
    with np.errstate(over="ignore"):
        d = np.minimum((hi - lo) / np.float32(15), np.float32(65504)).astype(np.float16)
    df = d.astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(df > 0, np.float32(1) / df, np.float32(0))
    z = np.clip(np.rint(-lo * inv), 0, 15) + np.float32(0)  # +0 where a row has nothing below 0
    c = np.clip(np.rint(x * inv) + z, 0, 15)
    return c.astype(np.uint8), d[..., 0], z[..., 0].astype(np.float16)


def pack(ck, dk, zk, cv, dv, zv):
    """Cache bytes [pages][H][page * (D + 8)] of codes [pages][H][page][D] and scales, zeros
    [pages][H][page] of keys and values."""
    n, H, page, D = ck.shape
    out = np.empty((n, H, page // CHUNK, CHUNK * (D + 8)), np.uint8)
    at = 0
    for c in (ck, cv):
        c = c.reshape(n, H, page // CHUNK, CHUNK, D)
        b = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(n, H, page // CHUNK, -1)
        out[..., at:at + b.shape[-1]] = b
        at += b.shape[-1]
    for d, z in ((dk, zk), (dv, zv)):
        b = np.stack([d, z], -1).astype(np.float16).reshape(n, H, page // CHUNK, CHUNK * 2)
        out[..., at:at + CHUNK * 4] = b.view(np.uint8)
        at += CHUNK * 4
    return out.reshape(n, H, -1)


def attention(q, k, v, seen, scale):
    """out [heads][D], lse [heads], sum_j p_j * |v|_j-like weights of one query row: q [heads][D],
    k and v [n][H][D] in 64 bits, seen [n] truth values."""
    heads, D = q.shape
    H = k.shape[1]
    kk = np.repeat(k[seen], heads // H, axis=1)
    vv = np.repeat(v[seen], heads // H, axis=1)
    if not seen.any():
        return np.zeros((heads, D)), np.full(heads, -np.inf), np.zeros((0, heads))
    s = scale * np.einsum("hd,nhd->nh", q, kk)
    m = s.max(0)
    e = np.exp(s - m)
    p = e / e.sum(0)
    return np.einsum("nh,nhd->hd", p, vv), m + np.log(e.sum(0)), p


def logits(x, prompt, output, repetition, presence, frequency, bias, mask):
    """One row in 64 bits: lists of token numbers, bias a list of (token, value), mask a list of
    truth values or None."""
    x = x.astype(np.float64).copy()
    V = len(x)
    ok = [t for t in output if 0 <= t < V]
    for t in set(ok) | {t for t in prompt if 0 <= t < V}:
        x[t] = x[t] / repetition if x[t] > 0 else x[t] * repetition
    for t in set(ok):
        x[t] = x[t] - ok.count(t) * frequency - presence
    last = {t: b for t, b in bias if 0 <= t < V}
    for t, b in last.items():
        x[t] += b
    x[np.abs(x) > np.finfo(np.float32).max] *= np.inf  # results are binary32
    if mask is not None:
        x[~mask] = -np.inf
    return x
