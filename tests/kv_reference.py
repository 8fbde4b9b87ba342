"""Plain 64-bit forms of the attention operators, token by token from their
definitions (numpy, CPU).  Shares no code with the kernels."""
import math

import numpy as np

CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def bf16(x):
    """Round to bf16 (nearest even) through fp32, as fp64."""
    u = np.asarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    nan = np.isnan(np.asarray(x, np.float64))
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(nan, np.nan, r)


def round_to(x, dtype):
    return bf16(x) if dtype == "bf16" else np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


# ------------------------------------------------------------------- batch
def build(ctx, new, T, table, free, num_blocks, bt):
    """Dict of the batch's arrays, the table after the call and the flags."""
    table = np.array(table, np.int64)
    B, width = table.shape
    cap = width * bt
    seq, pos, slots = np.full(T, -1), np.full(T, -1), np.full(T, -1)
    indptr, kv_len, flags, taken, row = [0], [], 0, 0, 0
    for i in range(B):
        if ctx[i] < 0 or new[i] < 0 or max(ctx[i], 0) + max(new[i], 0) > cap:
            flags |= 1
        c, n = min(max(int(ctx[i]), 0), cap), min(max(int(new[i]), 0), T)
        flags |= 2 * (new[i] > T)
        have, need = -(-c // bt), -(-min(c + n, cap) // bt)
        got = 0
        for b in range(have, need):
            f = taken
            taken += 1
            if f >= len(free):
                flags |= 4
                table[i, b] = -1
            else:
                got += 1
                if not 0 <= free[f] < num_blocks:
                    flags |= 8
                    table[i, b] = -1
                else:
                    table[i, b] = free[f]
        rows = min(n, T - row)
        if rows < n:
            flags |= 2
        for j in range(rows):
            p = c + j
            seq[row + j], pos[row + j] = i, p
            if p < cap:
                block = table[i, p // bt]
                if 0 <= block < num_blocks:
                    slots[row + j] = block * bt + p % bt
                elif p // bt < have:
                    flags |= 8
        row += rows
        indptr.append(row)
        kv_len.append(min(c + rows, cap, (have + got) * bt))
    return dict(q_indptr=np.array(indptr), kv_len=np.array(kv_len, np.int64), token_seq=seq, positions=pos, slots=slots,
                table=table, new_blocks=taken, flags=flags, tokens=row)


# -------------------------------------------------------------------- rope
def rotate(x, pos, freq, scale, interleaved):
    """x (T, H, D) fp64; freq (rot/2,)."""
    y = np.array(x, np.float64)
    half = len(freq)
    for t in range(x.shape[0]):
        if pos[t] < 0:
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            ang = math.fmod(float(pos[t]) * float(freq[i]), 2 * math.pi)
            c, s = math.cos(ang) * scale, math.sin(ang) * scale
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def frequencies(rot, theta, kind, factor, original, low=0.0, high=0.0):
    low = low or 1.0
    high = high or (32.0 if kind == "yarn" else 4.0)
    if kind == "ntk":
        theta = theta * factor ** (rot / max(rot - 2, 1))
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if kind == "linear":
            f /= factor
        if kind == "yarn":
            pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        if kind == "bands":
            mix = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * mix + f / factor * (1 - mix)
        out.append(f)
    return out, (0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)


# ------------------------------------------------------------------- cache
def quantise(x):
    """x (..., 32) -> (signed code indices 0..15, scale bytes): NaN as 0,
    infinities as the largest code."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    most = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.full(most.shape, -95)
    while True:  # smallest 2^e with most <= 7 * 2^e, up to 2^124
        more = (most > 7.0 * 2.0 ** e) & (e < 124)
        if not more.any():
            break
        e = e + more
    y = np.abs(np.where(np.isnan(x), 0.0, x)) / 2.0 ** e[..., None].astype(np.float64)
    idx = np.zeros(y.shape, np.int64)
    for k in range(7):  # border between codes k and k+1; ties go to the even code
        mid = (CODES[k] + CODES[k + 1]) / 2
        idx = np.where((y > mid) | ((y == mid) & (k % 2 == 1)), k + 1, idx)
    neg = np.signbit(x) & ~np.isnan(x)
    return idx + 8 * neg, e + 127


def values(code, byte):
    v = CODES[code & 7] * np.where(code >= 8, -1.0, 1.0)
    return v * 2.0 ** (np.asarray(byte, np.float64)[..., None] - 127)


def block_bytes(bt, heads, D):
    return heads * (bt // 16) * 544 * (D // 32)


def _place(D):
    """Byte and nibble of (token, dim) in a record for K and for V."""
    nc = D // 32
    t, d = np.arange(16)[:, None], np.arange(D)[None, :]
    c, r = d // 32, d % 32
    k = ((t * 4 + r // 8) * nc + c) * 4 + (r % 8) // 2, np.broadcast_to(r % 2, (16, D))
    v = 256 * nc + (((t // 4) * 16 + r % 16) * nc + c) * 4 + t % 4, np.broadcast_to(r // 16, (16, D))
    return k, v


def record_of(slot, head, bt, D):
    nc = D // 32
    return slot // bt, (head * (bt // 16) + slot % bt // 16) * 544 * nc, slot % 16


def put(data, slots, k, v, bt):
    """Write rows k, v (T, H, D) into cache bytes data (blocks, bytes) in place."""
    T, H, D = k.shape
    nc = D // 32
    (ka, kn), (va, vn) = _place(D)
    for which, (at, nib), first in ((k, (ka, kn), 512 * nc), (v, (va, vn), 528 * nc)):
        code, byte = quantise(which.reshape(T, H, nc, 32))
        code = code.reshape(T, H, D)
        for t in range(T):
            if not 0 <= slots[t] < data.shape[0] * bt:
                continue
            for h in range(H):
                b, off, u = record_of(int(slots[t]), h, bt, D)
                rec = data[b, off:off + 544 * nc]
                for n in (0, 1):
                    dims = np.nonzero(nib[u] == n)[0]
                    a = at[u][dims]
                    rec[a] = (rec[a] & (0xF0 if n == 0 else 0x0F)) | (code[t, h, dims] << (4 * n)).astype(np.uint8)
                rec[first + u * nc:first + (u + 1) * nc] = byte[t, h]


def get(data, slots, H, D, bt):
    """(k, v) values (n, H, D) at slots; zeros where a slot is no slot."""
    nc = D // 32
    (ka, kn), (va, vn) = _place(D)
    k, v = np.zeros((len(slots), H, D)), np.zeros((len(slots), H, D))
    for i, s in enumerate(slots):
        if not 0 <= s < data.shape[0] * bt:
            continue
        for h in range(H):
            b, off, u = record_of(int(s), h, bt, D)
            rec = data[b, off:off + 544 * nc].astype(np.int64)
            for out, at, nib, first in ((k, ka, kn, 512 * nc), (v, va, vn, 528 * nc)):
                code = (rec[at[u]] >> (4 * nib[u])) & 15
                out[i, h] = values(code.reshape(nc, 32), rec[first + u * nc:first + (u + 1) * nc]).reshape(D)
    return k, v


# --------------------------------------------------------------- attention
def attend_rows(q, k, v, sees, scale):
    """q (n, hq, D); k, v (L, hkv, D); row j sees keys [0, sees[j]).  Returns
    (o, |o| bound: the same sum over |v|, largest scale*sum|q||k| of a row)."""
    n, hq, D = q.shape
    G = hq // k.shape[1]
    o, a, s_abs = np.zeros((n, hq, D)), np.zeros((n, hq, D)), np.zeros((n, hq, 1))
    for j in range(n):
        L = int(sees[j])
        if L <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:L, h // G], v[:L, h // G]
            with np.errstate(invalid="ignore"):
                s = scale * (kk @ q[j, h])
                p = np.exp(s - s.max())
                p = p / p.sum()
                o[j, h] = p @ vv
                a[j, h] = p @ np.abs(vv)
                s_abs[j, h] = scale * (np.abs(kk) @ np.abs(q[j, h])).max()
    return o, a, s_abs


def attend_bound(o, a, s_abs, keys, D, dtype):
    """How far a kernel that keeps scores, sums and statistics in fp32 may be
    from o: scores off by (D + 4) roundings of their sum of absolute products
    (2^-24 each, twice for the order of the sum), which moves a weight by that
    factor; exp2 and the weighted sums by one rounding per key and a few more;
    for bf16 also the rounding of each weight (2^-8) and of the output."""
    weight = 2 * (D + 4) * 2.0 ** -24 * s_abs + (keys + 16) * 2.0 ** -23
    if dtype == "bf16":
        return (2 * weight + 2.0 ** -8) * a * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o) + 1e-37
    return 2 * weight * a + 2.0 ** -24 * np.abs(o) + 1e-37
