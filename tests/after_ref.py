"""Plain 64-bit implementations of the steps after a verification, for the tests: loops
and numpy float64, from the definitions in include/spec_verify.h, without the library."""
import math

import numpy as np

import serving_ref as sref

FAR = 2.0 ** 100


def logprobs_row(row, token, T, n):
    """(logprob, entropy, rank, top tokens [n], top logprobs [n], log of the sum of
    e^(z - max)) of one row (float64)."""
    nothing = (np.full(n, -1), np.full(n, np.nan))
    x = np.where(row <= -FAR, -np.inf, row)
    if token >= len(row) or np.isnan(row).any() or (row >= FAR).any() or not np.isfinite(x).any():
        return np.nan, np.nan, -1, *nothing, 0.0
    z = x / T
    m = z.max()
    e = np.exp(z - m)
    log_s = math.log(e.sum())
    lp = z - m - log_s
    with np.errstate(invalid="ignore"):
        entropy = log_s - np.where(e > 0, e * (z - m), 0.0).sum() / e.sum()
    order = np.lexsort((np.arange(len(x)), -x))
    rank = 1 + int(np.nonzero(order == token)[0][0])
    top, val = np.full(n, -1), np.full(n, -np.inf)
    found = [v for v in order[:n] if np.isfinite(x[v])]
    top[: len(found)], val[: len(found)] = found, lp[found]
    return lp[token], entropy, rank, top, val, log_s


def logprobs(logits, tokens, T, path, n):
    B, R, V = logits.shape
    M = tokens.shape[1]
    lp, ent, log_s = np.zeros((B, M)), np.zeros((B, M)), np.zeros((B, M))
    rank, top, val = np.zeros((B, M), np.int64), np.full((B, M, n), -1), np.full((B, M, n), -np.inf)
    for b in range(B):
        for m in range(M):
            if tokens[b, m] < 0:
                continue
            r = m if path is None else 0 if m == 0 else path[b, m - 1]
            if not 0 <= r < R:
                lp[b, m], ent[b, m], rank[b, m], val[b, m] = np.nan, np.nan, -1, np.nan
                continue
            lp[b, m], ent[b, m], rank[b, m], top[b, m], val[b, m], log_s[b, m] = logprobs_row(logits[b, r], tokens[b, m], T, n)
    return lp, ent, rank, top, val, log_s


def weigh(q, lse, cache, table, lengths, weights, positions, count, path, first, scale, decay, shift, out):
    """(new weights, positions, how far the weights may be off); out: what the new
    weights' buffer holds before the call."""
    B, N, Hq, D = q.shape
    pages, Hkv, P = weights.shape
    G, W = Hq // Hkv, table.shape[1]
    new, pos, tol = out.astype(np.float64), positions.copy(), np.zeros(weights.shape)
    most = N if path is None else path.shape[1]
    for b in range(B):
        n, L = most if count is None else int(count[b]), int(lengths[b])
        if n < 0 or n > most or L < 0 or L + n > W * P:
            continue
        nodes = np.arange(n) if path is None else path[b, :n]
        if ((nodes < 0) | (nodes >= N)).any():
            continue
        t = np.arange(L + n)
        page = table[b, t // P]
        t = t[(page >= 0) & (page < pages)]
        page = table[b, t // P]
        slot = page.astype(np.int64) * P + t % P
        see = t[None] <= L + np.arange(n)[:, None]
        for h in range(Hkv):
            k = sref.q4_read(cache, slot, h, shift, 0)
            w = np.where(t < L, decay * weights[page, h, t % P].astype(np.float64), 0.0)
            d = np.where(t < L, np.abs(w) * 2.0 ** -22, 0.0)
            for i in range(n):
                for g in range(h * G, h * G + G):
                    l = float(lse[b, nodes[i], g])
                    if not math.isfinite(l):
                        continue
                    x = q[b, nodes[i], g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (k @ x)
                        e = np.where(see[i] & ~np.isnan(s), np.exp(s - l), 0.0)
                        absz = abs(scale) * (np.abs(k) @ np.abs(x) + np.abs(k).sum(-1) * np.abs(x).max() * 2.0 ** -9)
                        rel = D * 2.0 ** -23 * absz + 2.0 ** -22 * (np.abs(s) + abs(l)) + 2.0 ** -20 + 2.0 ** -24 * n * G
                    w += e
                    d += np.where(e > 0, e * rel, 0.0) + 2.0 ** -125
            new[page, h, t % P], tol[page, h, t % P] = w, d
            if pos is not None:
                fresh = t >= L
                pos[page[fresh], h, t[fresh] % P] = (L if first is None else first[b]) + t[fresh] - L
    return new, pos, tol


def evict_plan(weights, positions, table, lengths, budgets, nxt, sinks, recent, moves):
    """(moves, counts, new lengths); moves: the buffer before the call."""
    pages, Hkv, P = weights.shape
    B, W = table.shape
    moves, counts, new = moves.copy(), np.zeros((B, Hkv), np.int64), np.zeros(B, np.int64)
    for b in range(B):
        n, K = int(lengths[b]), int(budgets[b])
        if 0 <= n <= W * P and (K < 0 or n <= K):
            new[b] = n
            continue
        t = np.arange(max(0, min(n, W * P)))
        page = table[b, t // P]
        if n < 0 or n > W * P or K < 0 or min(K, n - K) > moves.shape[2] or ((page < 0) | (page >= pages)).any():
            new[b] = -1
            continue
        slot = page.astype(np.int64) * P + t % P
        new[b] = K
        for h in range(Hkv):
            w, p = weights[page, h, t % P].astype(np.float64), positions[page, h, t % P].astype(np.int64)
            w = np.where(np.isnan(w), -np.inf, w)
            isnan = np.isnan(weights[page, h, t % P])
            safe = (p < sinks) | (p >= int(nxt[b]) - recent)
            order = np.lexsort((t, np.where(safe, 0.0, -w), isnan & ~safe, ~safe))
            kept = np.zeros(n, bool)
            kept[order[:K]] = True
            src, dst = slot[K:][kept[K:]], slot[:K][~kept[:K]]
            assert len(src) == len(dst)
            counts[b, h] = len(src)
            moves[b, h, : len(src), 0], moves[b, h, : len(src), 1] = src, dst
    return moves, counts, new


def move(cache, weights, positions, moves, counts):
    cache, D, P = cache.copy(), cache.shape[3] // 36, 32 * cache.shape[2]
    weights, positions = (None if x is None else x.copy() for x in (weights, positions))
    slots = cache.shape[0] * P
    parts = sref.q4_split(cache, D)   # views
    for b in range(moves.shape[0]):
        for h in range(moves.shape[1]):
            for s, d in moves[b, h, : max(0, min(int(counts[b, h]), moves.shape[2]))]:
                if not (0 <= s < slots and 0 <= d < slots):
                    continue
                for p in parts:
                    p[d // P, h, d % P // 32, d % 32] = p[s // P, h, s % P // 32, s % 32]
                for x in (weights, positions):
                    if x is not None:
                        x[d // P, h, d % P] = x[s // P, h, s % P]
    return cache, weights, positions


def page_trim(tokens, held, ring, ring_state, table, P):
    ring, F = ring.copy(), len(ring)
    head, avail = (int(x) for x in ring_state)
    ring_ok = 0 <= head < F and 0 <= avail <= F
    new_held, status = held.copy(), np.zeros(len(tokens), np.int64)
    given = back = 0
    for b in range(len(tokens)):
        n, hd = int(tokens[b]), int(held[b])
        if not ring_ok or n < 0 or not 0 <= hd <= table.shape[1]:
            status[b] = -1
            continue
        need = -(-n // P)
        put = max(0, hd - need)
        given += put
        if put and avail + given > F:
            status[b] = -3
            continue
        for e in range(put):
            ring[(head + avail + given - put + e) % F] = table[b, need + e]
        back += put
        new_held[b] = min(hd, need)
    return new_held, np.array([head, avail + back if ring_ok else avail]), status, ring
