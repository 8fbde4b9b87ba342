"""Plain forms of the beam search operators, from their definitions (numpy and
Python, CPU, 64 bits).  Shares no code with the kernels."""
import math

import numpy as np


def candidates(x, score, length, done, eos, penalty):
    """One request: x (W, V) fp64, -inf where there is no candidate.  List of
    (rank, beam, logit, token, total, length), best first."""
    out = []
    for w in range(len(score)):
        if not np.isfinite(score[w]):
            continue
        if done[w]:
            n = int(length[w])
            out.append((score[w] / max(n, 1) ** penalty, w, 0.0, eos, float(score[w]), n))
            continue
        real = np.where(np.isnan(x[w]) | (x[w] == np.inf), -np.inf, x[w])
        if not np.isfinite(real).any():
            continue
        top = real.max()
        lse = math.log(np.exp(real - top).sum())
        n = int(length[w]) + 1
        for v in np.nonzero(np.isfinite(real))[0]:
            total = score[w] + ((real[v] - top) - lse)
            out.append((total / max(n, 1) ** penalty, w, real[v], int(v), total, n))
    out.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
    return out


def select(x, W, score, length, done, eos, penalty):
    """(parent, token, total, length, done) of every row, and the ranks in order."""
    R = len(score)
    parent, token, total, n, fin = [], [], [], [], []
    ranks = []
    for b in range(R // W):
        rows = slice(b * W, (b + 1) * W)
        best = candidates(x[rows], score[rows], length[rows], done[rows], eos, penalty)
        ranks.append(best)
        for i in range(W):
            if i < len(best):
                _, w, _, v, t, k = best[i]
                parent.append(b * W + w), token.append(v), total.append(t), n.append(k)
                fin.append(int(bool(done[b * W + w]) or (eos >= 0 and v == eos)))
            else:
                parent.append(-1), token.append(-1), total.append(-math.inf), n.append(0), fin.append(1)
    return np.array(parent), np.array(token), np.array(total), np.array(n), np.array(fin), ranks


def reorder(parent, W, kv_len, table, free, num_blocks, bt):
    """Dict of new_table, new_len, copies [(source, target, tokens)], freed, flags."""
    table, R, width = np.array(table), len(parent), np.array(table).shape[1]
    cap, flags = width * bt, 0
    new, new_len, copies, freed = np.full((R, width), -1), np.zeros(R, np.int64), [], []
    old_len = np.clip(kv_len, 0, cap)
    if (old_len != kv_len).any():
        flags |= 4
    for b in range(R // W):
        rows = range(b * W, (b + 1) * W)
        heirs, opens = [], []
        for c in rows:
            p = int(parent[c])
            if p != -1 and p not in rows:
                flags, p = flags | 2, -1
            if p < 0:
                continue
            n = int(old_len[p])
            blocks = -(-n // bt)
            new_len[c] = n
            new[c, :blocks] = table[p, :blocks]
            mine = int(table[p, blocks - 1]) if n % bt else -1
            if n % bt and (p in heirs or (0 <= mine < num_blocks and mine in opens)):
                at = len(copies)
                target = int(free[at]) if at < len(free) else -1
                if at >= len(free):
                    flags |= 8
                elif not 0 <= target < num_blocks:
                    flags, target = flags | 16, -1
                copies.append((int(table[p, blocks - 1]), target, n % bt))
                new[c, blocks - 1] = target
            heirs.append(p)
            opens.append(mine)
        held = {(j, int(table[p, j])) for p in heirs for j in range(-(-int(old_len[p]) // bt))}
        last = max(-(-int(old_len[r]) // bt) for r in rows)
        for j in range(last):
            seen = set()
            for r in rows:
                if j >= -(-int(old_len[r]) // bt):
                    continue
                i = int(table[r, j])
                if not 0 <= i < num_blocks:
                    flags |= 16 if i != -1 else 0
                    continue
                if i not in seen and (j, i) not in held:
                    freed.append(i)
                seen.add(i)
    return dict(table=new, new_len=new_len, copies=copies, freed=freed, flags=flags)
