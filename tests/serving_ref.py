"""Plain 64-bit implementations of the serving steps around verification, for
the tests: loops and numpy float64, from the definitions in
include/spec_verify.h, without the library."""
import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def e4m3_values():
    """Values of the bytes 0..126 (increasing), by the format's definition."""
    return np.array([(b & 7) / 8 * 2.0 ** -6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


E4M3 = e4m3_values()


def nearest_even(grid, x):
    """Index of the grid value nearest to each x >= 0; halfway to the even
    index; past the end, the last."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(x >= grid[-1], len(grid) - 1, np.where(take_hi, hi, lo))


def q4_quantise(x, shift):
    """(codes [..., D] 0..15, scale bytes [..., D / 16]) of x [..., D]."""
    y = np.asarray(x, np.float64) * 2.0 ** -shift
    g = y.reshape(*y.shape[:-1], -1, 16)
    bad = ~np.isfinite(g).all(-1)
    top = np.where(bad, 0.0, np.abs(g).max(-1, initial=0.0, where=np.isfinite(g)))
    sb = nearest_even(E4M3, top / 6.0)
    s = E4M3[sb]
    safe = np.where(s > 0, s, 1.0)[..., None]
    code = nearest_even(E2M1, np.abs(np.where(np.isfinite(g), g, 0.0)) / safe) + 8 * np.signbit(g)
    code = np.where((s > 0)[..., None] & ~bad[..., None], code, 0)
    return code.reshape(y.shape).astype(np.uint8), np.where(bad, 0x7f, sb).astype(np.uint8)


def q4_split(cache, D):
    """Views (k codes, v codes, k scales, v scales) [..., 32, *] of blocks [..., 36 D]."""
    c = cache[..., : 32 * D].reshape(*cache.shape[:-1], 2, 32, D // 2)
    s = cache[..., 32 * D:].reshape(*cache.shape[:-1], 2, 32, D // 16)
    return c[..., 0, :, :], c[..., 1, :, :], s[..., 0, :, :], s[..., 1, :, :]


def q4_put(cache, slot, h, k, v, k_shift, v_shift):
    """Entry (k, v) [D] into `cache` [pages, Hkv, P / 32, 36 D] (uint8, in place)."""
    D, P = cache.shape[3] // 36, 32 * cache.shape[2]
    blk = cache[slot // P, h, slot % P // 32]
    row = slot % 32
    for half, (x, sh) in enumerate(((k, k_shift), (v, v_shift))):
        code, sb = q4_quantise(x, sh)
        at = 16 * D * half + row * (D // 2)
        blk[at: at + D // 2] = code[::2] | (code[1::2] << 4)
        at = 32 * D + 2 * D * half + row * (D // 16)
        blk[at: at + D // 16] = sb


def q4_read(cache, slots, h, shift, value):
    """float64 [n, D] of the keys (value=0) or values (1) at `slots`."""
    D, P = cache.shape[3] // 36, 32 * cache.shape[2]
    blk = cache[slots // P, h, slots % P // 32]
    row = slots % 32
    parts = q4_split(blk, D)
    n = np.arange(len(slots))
    code, sb = parts[value][n, row], parts[2 + value][n, row].astype(int)
    both = np.stack([code & 15, code >> 4], -1).reshape(len(slots), D)
    mag = E2M1[both & 7] * np.where(both >= 8, -1.0, 1.0)
    sc = np.where(sb & 127 == 127, np.nan, E4M3[np.minimum(sb & 127, 126)] * np.where(sb >= 128, -1.0, 1.0))
    return (mag.reshape(len(slots), D // 16, 16) * sc[..., None]).reshape(len(slots), D) * 2.0 ** shift


def attend(q, cache, table, lengths, k_new, v_new, see, scale, k_shift, v_shift):
    """(out, lse, mean |v| under the weights, largest scale * sum |q k|, what weights
    too small for their types may amount to), float64.  see [B, N, N] bool.
    Everything a row does not see is left out of its sums."""
    B, N, Hq, D = q.shape
    Hkv, P = cache.shape[1], 32 * cache.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((B, N, Hq, D)), np.full((B, N, Hq), -np.inf)
    absv, absz = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq))
    lost = np.zeros((B, N, Hq, D))
    for b in range(B):
        pos = np.arange(lengths[b])
        slots = table[b][pos // P].astype(np.int64) * P + pos % P
        for h in range(Hkv):
            kc, vc = (q4_read(cache, slots, h, s, i) for i, s in enumerate((k_shift, v_shift)))
            for n in range(N):
                k, v = kc, vc
                if k_new is not None:
                    idx = np.nonzero(see[b, n])[0]
                    k, v = np.concatenate([kc, k_new[b, idx, h]]), np.concatenate([vc, v_new[b, idx, h]])
                if not len(k):
                    continue
                for i in range(h * G, h * G + G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        z = scale * (k @ q[b, n, i])
                        m = z.max()
                        if m == -np.inf:
                            continue
                        # a weight is above zero, also where float64 has no number for it:
                        # times an infinity it is one, not a NaN
                        p = np.maximum(np.exp(z - m), 5e-324)
                        out[b, n, i] = p @ v / p.sum()
                        lse[b, n, i] = m + math.log(p.sum()) if np.isfinite(p.sum()) else np.nan
                        absv[b, n, i] = p @ np.abs(v) / p.sum()
                        av = np.where(np.isfinite(v), np.abs(v), 0.0)
                        lost[b, n, i] = 2.0 ** -32 * av[: len(kc)].sum(0) + 2.0 ** -125 * av[len(kc):].sum(0)
                        absz[b, n, i] = abs(scale) * (np.abs(k) @ np.abs(q[b, n, i])).max()
    return out, lse, absv, absz, lost


def mask_bits(words, n):
    """bool [..., n] of uint32 / int32 bit words."""
    w = np.asarray(words).view(np.uint32)
    return ((w[..., None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(*w.shape[:-1], -1)[..., :n].astype(bool)


def page_map(lengths, count, held, ring, ring_state, table, P, T):
    ring, table = ring.copy(), table.copy()
    F, W, B = len(ring), table.shape[1], len(lengths)
    head, avail = (int(x) for x in ring_state)
    ring_ok = 0 <= head < F and 0 <= avail <= F
    offsets = np.zeros(B + 1, np.int64)
    slots, positions = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    new_held, status = held.copy(), np.zeros(B, np.int64)
    demand = given = moved = back = 0
    old = table.copy()
    for b in range(B):
        L, n, hd = int(lengths[b]), int(count[b]), int(held[b])
        start = int(offsets[b])
        offsets[b + 1] = start + max(n, 0)
        ok = ring_ok and L >= 0 and 0 <= hd <= W and (n < 0 or (L + n <= W * P and offsets[b + 1] <= T))
        if not ok:
            status[b] = -1
            continue
        if n < 0:
            given += hd
            if hd > 0 and avail + given > F:
                status[b] = -3
                continue
            for e in range(hd):
                ring[(head + avail + given - hd + e) % F] = old[b, e]
            back += hd
            new_held[b] = 0
            continue
        take = max(0, -(-(L + n) // P) - hd)
        demand += take
        if take > 0 and demand > avail:
            status[b] = -3
            continue
        for e in range(take):
            table[b, hd + e] = ring[(head + demand - take + e) % F]
        moved += take
        new_held[b] = hd + take
        for j in range(n):
            pos = L + j
            page = int(table[b, pos // P])
            positions[start + j] = pos
            if 0 <= page < F:
                slots[start + j] = page * P + pos % P
    state = np.array([(head + moved) % F, avail - moved + back] if ring_ok else [head, avail])
    return np.minimum(offsets, T), slots, positions, new_held, state, status, table, ring


def adjust(logits, history, prompt_len, hist_len, rep, freq, pres, nodes, see, bias_tokens, bias_values, allowed):
    """(result, sum of the magnitudes that its sums went through), float64.
    see [B, R, Nt] bool: the proposed tokens of each row."""
    B, R, V = logits.shape
    out = logits.astype(np.float64)
    size = np.abs(np.where(np.isfinite(out), out, 0.0))
    for b in range(B):
        seen, made = np.zeros(V, bool), np.zeros(V, np.int64)
        if history is not None:
            n = min(max(int(hist_len[b]), 0), history.shape[1])
            for i in range(n):
                t = int(history[b, i])
                if not 0 <= t < V:
                    continue
                if prompt_len is not None and i < prompt_len[b]:
                    seen[t] = True
                else:
                    made[t] += 1
        r_, f_, p_ = (1.0 if rep is None else float(rep[b]), 0.0 if freq is None else float(freq[b]),
                      0.0 if pres is None else float(pres[b]))
        bias = np.zeros(V)
        if bias_tokens is not None:
            for t, x in zip(bias_tokens[b], bias_values[b]):
                if 0 <= t < V:
                    bias[t] += float(x)
        for r in range(R):
            n = made.copy()
            if nodes is not None:
                for j in np.nonzero(see[b, r])[0]:
                    if 0 <= nodes[b, j] < V:
                        n[nodes[b, j]] += 1
            x = out[b, r]
            hit = seen | (n > 0)
            with np.errstate(invalid="ignore"):
                x = np.where(hit, np.where(x > 0, x / r_, x * r_), x)
                x = np.where(n > 0, x - (f_ * n + p_), x) + bias
            size[b, r] = size[b, r] * max(r_, 1 / r_) + abs(f_) * n + abs(p_) + np.abs(bias)
            if allowed is not None:
                x = np.where(allowed[b, r], x, -np.inf)
            out[b, r] = x
    return out, size
