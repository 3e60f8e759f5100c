"""The operators around a block's attention, in fp64 and in the plainest way: rotation, 4-bit chunks, attention over
them, sampled acceptance. Arrays are numpy; bf16 values come as fp64."""
import numpy as np

CHUNK = 64
# magnitudes of the eight 4-bit codes and of the 127 finite e4m3 bytes, ascending: index = code
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])


def to_bf16(x):
    """fp64 -> bf16 bits, to the nearest, ties to even (directly: no rounding to fp32 between)."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    y = np.ldexp(np.rint(np.ldexp(m, 8)), e - 8).astype(np.float32)      # 8 significant bits
    return (y.view(np.uint32) >> 16).astype(np.uint16)


def rope(x, positions, inv_freq, interleaved=False, factor=1.0, norm=None, eps=0.0):
    """x [T][H][d] -> normalised and rotated rows."""
    x = np.array(x, dtype=np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm
    if inv_freq is None:
        return x
    n = len(inv_freq)
    for t, p in enumerate(positions):
        for j in range(n):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
            angle = np.float64(p) * np.float64(inv_freq[j])
            c, s = factor * np.cos(angle), factor * np.sin(angle)
            xa, xb = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a], x[t, :, b] = xa * c - xb * s, xa * s + xb * c
    return x


def nearest(x, table):
    """Index of the table entry nearest to x >= 0: ties to the even index, past the end the last one."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    up = (table[hi] - x < x - table[lo]) | ((table[hi] - x == x - table[lo]) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def pack_rows(x, g=1.0):
    """Rows [..., d] -> (codes [..., d], scales [..., d / 16]): x / g rounded to fp32 first, as documented for the quotients."""
    x = (np.asarray(x, dtype=np.float32) / np.float32(g)).astype(np.float32)
    d = x.shape[-1]
    y = x.reshape(*x.shape[:-1], d // 16, 16)
    s = nearest((np.abs(y).max(-1) / np.float32(6)).astype(np.float64), E4M3)
    step = E4M3[s].astype(np.float32)[..., None]
    q = np.where(step > 0, np.abs(y) / np.where(step > 0, step, np.float32(1)), np.float32(0))
    codes = nearest(q.astype(np.float64), E2M1) + np.where(np.signbit(y) & (step > 0), 8, 0)
    return codes.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def write_row(record, token, codes, scales):
    """One token's row into a record (uint8 [36 d])."""
    d = codes.shape[0]
    for c in range(d):
        at = (c // 32 * CHUNK + token) * 16 + c % 32 // 2
        shift = 4 * (c % 2)
        record[at] = (record[at] & (0xF0 >> shift)) | (codes[c] << shift)
    record[32 * d + token * (d // 16):32 * d + (token + 1) * (d // 16)] = scales


def record_values(records, d):
    """Records [..., 36 d] -> values [..., 64, d] (without g). NaN scales give NaN."""
    raw = np.asarray(records)
    lead = raw.shape[:-1]
    codes = raw[..., :32 * d].reshape(*lead, d // 32, CHUNK, 16)
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*lead, d // 32, CHUNK, 32)
    both = np.moveaxis(both, -2, -3).reshape(*lead, CHUNK, d)
    v = np.where(both >= 8, -1.0, 1.0) * E2M1[both & 7]
    s = raw[..., 32 * d:].reshape(*lead, CHUNK, d // 16)
    steps = np.where((s & 127) == 127, np.nan, np.append(E4M3, np.nan)[s & 127]) * np.where(s >= 128, -1.0, 1.0)
    return v * np.repeat(steps, 16, -1)


def attend_packed_seq(q, k_pool, v_pool, ids, slots, L, gk=1.0, gv=1.0, scale=None):
    """One sequence: q [n][Hq][d] (fp64), pools uint8 [slots][Hkv][36 d]. Returns out, lse, sum_j p_j |v_j| and sum_j |v_j|."""
    n, hq, d = q.shape
    hkv = k_pool.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    out, mag, all_v = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    ids, slots = np.asarray(ids, dtype=np.int64), np.asarray(slots, dtype=np.int64)
    ok = (slots >= 0) & (slots < k_pool.shape[0]) & (ids >= 0)
    pos = (ids[ok][:, None] * CHUNK + np.arange(CHUNK)).reshape(-1)
    for h in range(hkv):
        k = record_values(k_pool[slots[ok], h], d).reshape(-1, d) * gk
        v = record_values(v_pool[slots[ok], h], d).reshape(-1, d) * gv
        for i in range(n):
            see = pos <= L - n + i
            if not see.any():
                continue
            for g in range(hq // hkv):
                x = k[see] @ q[i, h * (hq // hkv) + g] * scale
                m = x.max()
                p = np.exp(x - m)
                at = (i, h * (hq // hkv) + g)
                lse[at] = m + np.log(p.sum())
                p /= p.sum()
                out[at], mag[at], all_v[at] = p @ v[see], p @ np.abs(v[see]), np.abs(v[see]).sum(0)
    return out, lse, mag, all_v


def accept_sampled(logits, temperature, drafts, probs, uniform, noise, cu_rows):
    """Returns accepted_len, bonus, committed, and for every decision how near it was (the smallest relative gap)."""
    accepted, bonus, committed = [], [], np.full(int(cu_rows[-1]), -1, dtype=np.int64)
    gap = np.inf
    V = logits.shape[1]
    for b in range(len(cu_rows) - 1):
        r0, depth = int(cu_rows[b]), int(cu_rows[b + 1] - cu_rows[b]) - 1
        T = float(temperature[b])
        for j in range(depth + 1):
            x = np.array(logits[r0 + j], dtype=np.float64)
            if T > 0:
                x = np.where(np.isnan(x), -np.inf, x)
                top = x.max()
                with np.errstate(invalid="ignore"):
                    p = np.where(x == top, 1.0, np.exp((x - top) / T)) if top > -np.inf else np.zeros(V)
                p = p / p.sum() if p.sum() > 0 else p
            else:
                nan = np.flatnonzero(np.isnan(x))
                p = (np.arange(V) == (nan[0] if len(nan) else int(np.argmax(x)))).astype(np.float64)
            q = np.zeros(V)
            at = r0 - b + j
            if j < depth:
                d = int(drafts[at])
                if 0 <= d < V:
                    if probs is None:
                        q[d] = 1.0
                    else:
                        q = np.asarray(probs[at], dtype=np.float64)
                    lhs = float(uniform[at]) * q[d]
                    if T > 0 and max(lhs, p[d]) > 0:
                        gap = min(gap, abs(lhs - p[d]) / max(lhs, p[d]))
                    if lhs < p[d]:
                        committed[r0 + j] = d
                        continue
            if T == 0:
                token = int(np.argmax(p))
            else:
                e = np.asarray(noise[b], dtype=np.float64)
                drawn = (e > 0) & np.isfinite(e)
                e = np.where(drawn, e, 1.0)
                token = None
                for w in (np.maximum(p - q, 0.0), p):
                    race = np.where(drawn, w / e, 0.0)
                    if race.max() > 0:
                        token = int(np.argmax(race))
                        if V > 1:
                            second = np.partition(race, -2)[-2]
                            gap = min(gap, 1 - second / race.max())
                        break
                if token is None:
                    token = int(np.argmax(x))
            break
        accepted.append(j)
        bonus.append(token)
        committed[r0 + j] = token
    return np.array(accepted), np.array(bonus), committed, gap
