"""The serving steps around verification on the GPU against plain 64-bit
implementations (serving_ref.py).

Tolerances.  Integers, codes and scales are compared exactly.
Attention, per element: the bf16 output is off by half a step, 2^-8 |out|; a
weight is rounded to f16, 2^-11 of it, which moves numerator and (through the
unrounded sum) nothing else: 2^-11 * A with A = sum of weight * |v|; a score is a
sum of D products in fp32, off by at most D * 2^-23 * scale * sum |q k| =: dz
(2^-23: the tensor core may truncate), plus two roundings of the score itself in
the log2 domain, which changes a weight by that share, in numerator and sum:
2 * dz * A; ex2 and the sums add a few 2^-22, taken as 2^-18 * A.  So
  |d out| <= 2^-8 |out| + (2^-11 + 2 dz + 2^-18) A + U,   |d lse| <= 2 dz + 2^-20 (1 + |lse|).
U is underflow, which relative terms do not cover.  Weights of cached tokens are
f16, 2^(z - ref + 7) with a reference that is at most the largest score: f16's
smallest step is 2^-24, a weight is off by up to half of it, 2^-25, and the sum of
weights is at least 2^7, so the share is off by 2^-32 at most.  Those of fresh
entries are pairs of bf16 made from fp32, and factors between references are fp32:
what is below 2^-126 becomes 0 or 2^-126, which is off by 2^-125 at most.  Hence
U = 2^-32 * sum |v| over the cached tokens + 2^-125 * sum |v| over the fresh ones.
Logit adjustments: at most 6 fp32 roundings of intermediate sums, each 2^-24 of
the magnitudes that went in, and the output's half step."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import speculative_decoding_verification_52_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int64).to(I32).to(DEV)


def f32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.float32).to(DEV)


def bf(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.float64).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


# --- page map -----------------------------------------------------------------
def _run_map(lengths, count, held, ring, state, table, P, T):
    t_ring, t_table = i32(ring), i32(table)
    got = sv.spec_page_map(i32(lengths), i32(count), i32(held), t_ring, i32(state), t_table, P, T)
    exp = ref.page_map(lengths, count, held, ring, state, table, P, T)
    for name, g, e in zip(("offsets", "slots", "positions", "held", "state", "status", "table", "ring"), [*got, t_table, t_ring], exp):
        np.testing.assert_array_equal(g.cpu().numpy(), e, err_msg=name)
    return exp


def _pool(rng, B, W, P, F, hi):
    lengths = rng.integers(0, hi + 1, B)
    held = -(-lengths // P)
    held = np.minimum(held + rng.integers(0, 2, B), W)
    ids = rng.permutation(F)
    table = np.full((B, W), -1)
    at = 0
    for b in range(B):
        table[b, : held[b]] = ids[at: at + held[b]]
        at += held[b]
    assert at <= F
    head = int(rng.integers(0, F))
    ring = np.roll(ids, head - at)
    return lengths, held, ring, np.array([head, F - at]), table


@pytest.mark.parametrize("B,P,hi,new", [(1, 32, 0, 1), (1, 1, 5, 7), (7, 32, 100, 6), (256, 64, 500, 6), (513, 16, 40, 3),
                                        (40, 128, 700, 900), (3, 64, 0, 5000), (1025, 32, 33, 1)])
def test_page_map(B, P, hi, new):
    rng = np.random.default_rng(B * 1000 + P)
    W = -(-(hi + new) // P) + 1
    lengths, held, ring, state, table = _pool(rng, B, W, P, B * W + 3, hi)
    count = rng.integers(0, new + 1, B)
    count[rng.random(B) < 0.1] = -1
    T = int(np.maximum(count, 0).sum())
    for extra in (0, 3, 2500):
        _run_map(lengths, count, held, ring, state, table, P, T + extra)


def test_page_map_refusals_per_sequence():
    """Bad requests, a pool that runs dry, a map that is too short, ids outside
    the pool, a broken ring: the others are served, nothing of the refused moves."""
    rng = np.random.default_rng(3)
    B, P, W = 70, 16, 6
    lengths, held, ring, state, table = _pool(rng, B, W, P, 300, 30)
    count = rng.integers(0, 60, B)
    count[5] = count[60] = -1
    lengths[2], held[3], held[4], count[6] = -4, -1, W + 1, 1000
    table[8, 0] = 4000                    # not a page of the pool: its tokens get no slot
    lengths[8], held[8], count[8] = 3, 1, 8
    T = int(np.maximum(count, 0).sum())
    _run_map(lengths, count, held, ring, state, table, P, T)
    _run_map(lengths, count, held, ring, np.array([state[0], 20]), table, P, T)       # -3 from some point on
    exp = _run_map(lengths, count, held, ring, np.array([state[0], 0]), table, P, T)
    assert (exp[5] == -3).any() and (exp[5] == 0).any()
    _run_map(lengths, count, held, ring, state, table, P, T // 2)                     # places past max_tokens
    _run_map(lengths, count, held, ring, state, table, P, 0)
    for broken in ([300, 5], [-1, 5], [0, 301], [0, -2]):
        assert (_run_map(lengths, count, held, ring, np.array(broken), table, P, T)[5] == -1).all()
    count[:] = -1
    full = np.array([state[0], 300])      # a ring that already holds every id has no room for more
    assert (_run_map(lengths, count, held, ring, full, table, P, 4)[5] == -3).any()


def test_page_map_large_counts_do_not_wrap():
    big = 2 ** 31 - 1
    _run_map(np.array([5, big, 3]), np.array([big, big, 2]), np.array([1, 1, 1]), np.arange(8), np.array([2, 5]),
             np.array([[7, -1], [6, -1], [5, -1]]), 32, 10)


# --- quantise and store -----------------------------------------------------------
def _kv(rng, *shape):
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1]))[..., None]
    x[rng.random(shape) < 0.05] = 0.0
    x = np.where(rng.random(shape) < 0.05, np.round(x * 4) / 4, x)       # ties between codes
    return bf(x)


def test_page_map_of_an_empty_batch():
    """Every place is empty, so that a store behind it touches nothing."""
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    state = i32([3, 5])
    slots = torch.full((9,), 7, dtype=torch.int32, device=DEV)
    got = sv.spec_page_map(e, e, e, i32(range(8)), state, e.view(0, 4), 32, 9, slots=slots)
    assert got[0].tolist() == [0] and got[1] is slots and slots.tolist() == [-1] * 9 and got[2].tolist() == [-1] * 9
    assert got[3].numel() == 0 and got[4].tolist() == [3, 5] and got[5].numel() == 0


@pytest.mark.parametrize("D,Hkv,P,T,shift", [(128, 2, 32, 1, 0), (128, 3, 64, 77, -2), (64, 1, 32, 40, 5), (64, 5, 128, 133, 0)])
def test_store_matches_reference_bit_for_bit(D, Hkv, P, T, shift):
    rng = np.random.default_rng(T)
    pages = -(-T // P) + 3
    k, v = _kv(rng, T, Hkv, D), _kv(rng, T, Hkv, D)
    slots = rng.permutation(pages * P)[:T]
    slots[rng.random(T) < 0.1] = -1
    if T > 3:
        slots[1] = pages * P           # outside the cache
        k[2, 0, 3], v[3, 0, 40] = float("nan"), float("inf")
        k[0, 0, :16] = -0.0
    cache = rng.integers(0, 256, (pages, Hkv, P // 32, 36 * D), dtype=np.uint8)
    exp = cache.copy()
    for t in range(T):
        if 0 <= slots[t] < pages * P:
            for h in range(Hkv):
                ref.q4_put(exp, int(slots[t]), h, f64(k[t, h]), f64(v[t, h]), shift, -shift)
    c = torch.from_numpy(cache).to(DEV)
    sv.spec_kv_store_q4(k.to(DEV), v.to(DEV), i32(slots), c, k_shift=shift, v_shift=-shift)
    np.testing.assert_array_equal(c.cpu().numpy(), exp)


def test_store_every_bf16_scale():
    """Groups whose largest element runs through bf16's whole range, with values
    next to every border between two codes."""
    tops = torch.arange(0, 0x7f80, 13, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    T = tops.numel() // 8
    x = tops[: T * 8].view(T, 1, 8, 1).double().expand(T, 1, 8, 16).clone()
    frac = torch.tensor([1, 0.5, 0.25 / 6, 0.75 / 6, 1.25 / 6, 1.75 / 6, 2.5 / 6, 3.5 / 6, 5 / 6, -5 / 6, -1e-4, 0.0417, 0.125, 0.2083, -0.29, 0.83]).double()
    k = (x * frac).reshape(T, 1, 128).to(torch.bfloat16)
    v = (x * torch.rand(16, dtype=torch.float64)).reshape(T, 1, 128).to(torch.bfloat16)
    cache = np.zeros((-(-T // 32), 1, 1, 36 * 128), np.uint8)
    for t in range(T):
        ref.q4_put(cache, t, 0, f64(k[t, 0]), f64(v[t, 0]), 0, 3)
    c = sv.q4_cache(cache.shape[0], 1, 32, 128, DEV)
    sv.spec_kv_store_q4(k.to(DEV), v.to(DEV), i32(np.arange(T)), c, v_shift=3)
    np.testing.assert_array_equal(c.cpu().numpy(), cache)


@pytest.mark.parametrize("D,Hkv,P,N,use_path", [(128, 2, 32, 6, False), (64, 3, 64, 9, True), (128, 1, 32, 70, True)])
def test_commit_matches_reference(D, Hkv, P, N, use_path):
    rng = np.random.default_rng(N)
    B, W = 11, 4
    pages = B * W + 2
    table = rng.permutation(pages)[: B * W].reshape(B, W)
    lengths = rng.integers(0, W * P - N, B)
    PW = min(N, 7)
    path = np.stack([rng.permutation(N)[:PW] for _ in range(B)])
    count = rng.integers(-1, (PW if use_path else N) + 1, B)
    count[0] = 0
    lengths[1], count[1] = W * P - 1, 2           # passes the table
    lengths[2], count[2] = -1, 1
    count[3] = (PW if use_path else N) + 1        # more than there are
    table[4, lengths[4] // P], count[4] = pages, 1
    path[5, 1], count[5] = N, 2                   # outside [0, N) (with a path)
    table[6, lengths[6] // P], count[6] = -1, 1
    path[7, :2], count[7] = path[7, 0], 2         # the same node twice: appended twice
    k, v = _kv(rng, B, N, Hkv, D), _kv(rng, B, N, Hkv, D)
    cache = rng.integers(0, 256, (pages, Hkv, P // 32, 36 * D), dtype=np.uint8)
    exp, exp_len = cache.copy(), np.zeros(B, np.int64)
    for b in range(B):
        n, ln = int(count[b]), int(lengths[b])
        if n < 0:
            exp_len[b] = ln
            continue
        src = [int(path[b, j]) if use_path else j for j in range(min(n, PW if use_path else N))]
        ok = ln >= 0 and ln + n <= W * P and n == len(src) and all(0 <= s < N for s in src)
        ok = ok and all(0 <= table[b, (ln + j) // P] < pages for j in range(n))
        exp_len[b] = ln + n if ok else -1
        for j in range(n if ok else 0):
            pos = ln + j
            for h in range(Hkv):
                ref.q4_put(exp, int(table[b, pos // P]) * P + pos % P, h, f64(k[b, src[j], h]), f64(v[b, src[j], h]), 1, 0)
    c = torch.from_numpy(cache).to(DEV)
    got = sv.spec_kv_commit_q4(c, i32(table), i32(lengths), k.to(DEV), v.to(DEV), i32(count), path=i32(path) if use_path else None, k_shift=1)
    np.testing.assert_array_equal(got.cpu().numpy(), exp_len)
    np.testing.assert_array_equal(c.cpu().numpy(), exp)
    assert (exp_len == -1).sum() >= 5


# --- attention ----------------------------------------------------------------------
def _cache(rng, pages, Hkv, P, D):
    """A cache of normal entries, quantised here (shift 0)."""
    blocks = pages * Hkv * (P // 32)
    parts = []
    for _ in range(2):
        code, sb = ref.q4_quantise(rng.standard_normal((blocks, 32, D)) * np.where(rng.random(D) < 0.06, 4, 1), 0)
        parts.append((code[..., ::2] | (code[..., 1::2] << 4), sb))
    c = np.concatenate([x.reshape(blocks, -1) for x in (parts[0][0], parts[1][0], parts[0][1], parts[1][1])], 1)
    return c.reshape(pages, Hkv, P // 32, 36 * D)


def _case(seed, B, N, Hq, Hkv, D, P, lengths, tree=False, fresh=True, shifts=(0, 0)):
    rng = np.random.default_rng(seed)
    lengths = np.asarray(lengths)
    W = max(1, int(-(-lengths.max() // P)))
    pages = B * W + 2
    c = dict(rng=rng, P=P, W=W, pages=pages, D=D, shifts=shifts, lengths=lengths, table=rng.permutation(pages)[: B * W].reshape(B, W))
    c["cache"] = _cache(rng, pages, Hkv, P, D)
    for b in range(B):   # what lies behind a sequence's last token is a NaN
        pos = np.arange(lengths[b], W * P)
        slot = c["table"][b][pos // P] * P + pos % P
        for s in slot:
            blk = c["cache"][s // P, :, s % P // 32]
            for at in (32 * D, 34 * D):
                blk[:, at + s % 32 * (D // 16): at + (s % 32 + 1) * (D // 16)] = 0x7f
    c["q"] = bf(rng.standard_normal((B, N, Hq, D)) * 1.5)
    c["k"], c["v"] = (bf(rng.standard_normal((B, N, Hkv, D))) if fresh else None for _ in range(2))
    if tree:
        par = np.array([[-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, N)] for _ in range(B)])
        see = np.zeros((B, N, N), bool)
        for b in range(B):
            for i in range(N):
                j = i
                while j >= 0:
                    see[b, i, j] = True
                    j = par[b, j]
        c["parents"], c["see"] = par, see
    else:
        c["see"] = np.broadcast_to(np.tril(np.ones((N, N), bool)), (B, N, N)).copy()
    c["masks"] = None
    if tree:
        c["masks"], st = sv.spec_tree_mask(i32(par))
        assert not st.any()
    return c


def _attend(c, **kw):
    put = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    return sv.spec_attend_q4(put(c["q"]), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"]), k_new=put(c["k"]),
                             v_new=put(c["v"]), masks=c["masks"], k_shift=c["shifts"][0], v_shift=c["shifts"][1], **kw)


def _expect(c, scale=None, lengths=None):
    lengths = c["lengths"] if lengths is None else lengths
    k, v = (None if c[x] is None else f64(c[x]) for x in ("k", "v"))
    return ref.attend(f64(c["q"]), c["cache"], c["table"], lengths, k, v, c["see"], c["D"] ** -0.5 if scale is None else scale, *c["shifts"])


def _close(got, exp, D, rows=slice(None)):
    out, lse = (f64(x)[rows] for x in got)
    eo, el, av, az, lost = (x[rows] for x in exp)
    np.testing.assert_array_equal(np.isnan(out), np.isnan(eo))
    np.testing.assert_array_equal(np.isnan(lse), np.isnan(el))
    np.testing.assert_array_equal(np.isinf(out), np.isinf(eo))
    np.testing.assert_array_equal(lse == -np.inf, el == -np.inf)
    dz = D * 2.0 ** -23 * az
    fin = np.isfinite(el)
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(eo) + (2.0 ** -11 + 2 * dz[..., None] + 2.0 ** -18) * av + lost
        d = np.abs(out - eo)
        bad = np.isfinite(eo) & ~(d <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.where(bad, d / tol, 0)):.3g} times the tolerance"
        dl = np.abs(lse - el)[fin]
    assert (dl <= (2 * dz + 2.0 ** -20 * (1 + np.abs(el)))[fin]).all(), dl.max()
    np.testing.assert_array_equal(out[el == -np.inf], 0)


SHAPES = [
    # B, N, Hq, Hkv, D, P, lengths
    (1, 1, 1, 1, 128, 32, [1]),
    (1, 1, 8, 1, 64, 32, [31]),
    (2, 1, 8, 2, 128, 64, [32, 33]),
    (3, 1, 32, 8, 128, 32, [777, 0, 95]),
    (3, 6, 8, 2, 128, 64, [64, 1, 200]),
    (2, 6, 16, 2, 64, 128, [127, 129]),
    (2, 17, 3, 1, 64, 32, [50, 0]),
    (2, 33, 4, 2, 128, 96, [100, 290]),
    (1, 70, 10, 2, 64, 32, [300]),
    (5, 2, 7, 7, 128, 32, [0, 1, 2, 63, 64]),
    (2, 40, 16, 1, 128, 64, [500, 3]),
    (1, 64, 64, 1, 64, 64, [130]),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
def test_attend_matches_reference(shape, tree):
    B, N, Hq, Hkv, D, P, lengths = shape
    c = _case(sum(shape[:6]), B, N, Hq, Hkv, D, P, lengths, tree=tree)
    _close(_attend(c), _expect(c), D)


@pytest.mark.parametrize("shape", SHAPES[:6])
def test_attend_without_fresh_entries(shape):
    B, N, Hq, Hkv, D, P, lengths = shape
    c = _case(9, B, N, Hq, Hkv, D, P, lengths, fresh=False, shifts=(2, -3))
    exp = _expect(c)
    _close(_attend(c), exp, D)
    assert (exp[1][np.asarray(lengths) == 0] == -np.inf).all()


def test_attend_many_short_sequences():
    rng = np.random.default_rng(1)
    lengths = rng.integers(0, 70, 300)
    c = _case(2, 300, 3, 4, 2, 64, 32, lengths)
    _close(_attend(c), _expect(c), 64)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 1, 128), (130, 8, 4, 128), (260, 2, 1, 64)])
def test_attend_long_context(N, Hq, Hkv, D):
    """One sequence over the whole device; rows far apart in their nodes."""
    c = _case(5, 1, N, Hq, Hkv, D, 64, [4000 if N == 1 else 1500], tree=N == 130)
    _close(_attend(c), _expect(c), D)


def test_attend_masks_that_leave_nothing_and_any_bits():
    c = _case(6, 2, 40, 4, 2, 64, 32, [0, 40])
    see = c["rng"].random((2, 40, 40)) < 0.3      # no ancestors' order: any bits are obeyed
    see[:, 7] = False
    see[:, 21] = False
    w = np.zeros((2, 40, 64), np.uint64)
    w[:, :, :40] = see
    w[:, :, 40:] = 1                               # bits past N mean nothing
    words = (w.reshape(2, 40, 2, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    c["see"], c["masks"] = see, i32(words.view(np.int32))
    exp = _expect(c)
    assert (exp[1][0, 7] == -np.inf).all() and np.isfinite(exp[1][1, 7]).all()
    _close(_attend(c), exp, 64)


def test_attend_extreme_values():
    """Infinities and NaN in fresh entries reach only the rows that see them;
    scores of the largest size, queries from tiny to huge, a row of zeros."""
    c = _case(7, 2, 12, 4, 2, 128, 32, [70, 5], tree=True)
    c["v"][0, 3, 0, 5], c["v"][0, 4, 1, 100], c["k"][1, 6, 0, 2] = float("inf"), float("nan"), float("nan")
    c["v"][1, 2, 1, 0], c["k"][1, 9, 1] = float("-inf"), -1e30
    c["q"][0, 1, 2] *= 1e-30
    c["q"][0, 2, 3] = 0
    c["q"][1, 0, 1] *= 30
    c["q"][1, 3, 2] *= 1e4
    c["v"][1, 5, 0] *= 1e30                        # beyond f16
    _close(_attend(c), _expect(c), 128)


# rows of a kv head on both sides of each kernel's row tiles (32, 64 and 128 rows)
TILES = [(16, 3, 1, 128), (13, 4, 1, 128), (16, 8, 2, 128), (65, 1, 1, 128), (64, 4, 2, 128), (129, 3, 3, 128), (16, 8, 2, 64), (65, 2, 2, 64), (43, 3, 1, 64)]


@pytest.mark.parametrize("N,Hq,Hkv,D", TILES)
@pytest.mark.parametrize("tree", [False, True])
def test_attend_row_tiles(N, Hq, Hkv, D, tree):
    c = _case(60 + N, 3, N, Hq, Hkv, D, 32, [300, 0, 129], tree=tree, shifts=(1, -1))
    _close(_attend(c), _expect(c), D)


@pytest.mark.parametrize("N,Hq,Hkv,D", TILES)
def test_attend_fresh_entries_out_of_range_in_every_tile(N, Hq, Hkv, D):
    """Infinities, NaN and elements beyond f16 in the fresh entries, and queries
    whose rows need powers of two of their own."""
    c = _case(61 + N, 2, N, Hq, Hkv, D, 32, [70, 0], tree=True)
    c["v"][0, 3, 0, 5], c["v"][0, 4, Hkv - 1, D - 1], c["k"][1, 6, 0, 2] = float("inf"), float("nan"), float("nan")
    c["v"][1, N - 1, Hkv - 1, 0], c["k"][1, 9, 0] = float("-inf"), -1e30
    c["q"][0, 1, Hq - 1] *= 1e-30
    c["q"][0, 2, 0] = 0
    c["q"][1, 0, 0] *= 30
    c["v"][1, 5, 0] *= 1e30
    _close(_attend(c), _expect(c), D)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 2, 1, 128), (6, 8, 2, 64)] + TILES[1::2])
def test_attend_scores_beyond_the_weights_steps(N, Hq, Hkv, D):
    """Scores so large that a rounding of one is worth more than any weight: every
    result stays finite."""
    c = _case(63 + N, 2, N, Hq, Hkv, D, 32, [500, 130], shifts=(32, 0))
    c["q"] *= 3e4
    exp = _expect(c)
    assert np.isfinite(exp[0]).all() and np.abs(exp[1]).max() > 2.0 ** 40
    _close(_attend(c), exp, D)


@pytest.mark.parametrize("B,N,Hq,Hkv,D", [(350, 15, 8, 2, 128), (200, 60, 1, 1, 128), (60, 140, 4, 2, 64), (33, 300, 2, 1, 128), (9, 1024, 2, 2, 64)])
@pytest.mark.parametrize("top", [1, 200])
def test_attend_many_triples_with_little_behind_them(B, N, Hq, Hkv, D, top):
    """A multiprocessor's share holds several (sequence, head, row tile) triples, many
    of them with fresh entries alone, and begins anywhere within one."""
    lengths = np.random.default_rng(B).integers(0, top, B)
    c = _case(62, B, N, Hq, Hkv, D, 32, lengths)
    if N > 500:   # (the reference of a few sequences is enough)
        rows = [0, B // 2, B - 1]
        part = dict(c, q=c["q"][rows], k=c["k"][rows], v=c["v"][rows], see=c["see"][rows], table=c["table"][rows], lengths=c["lengths"][rows])
        _close([x[rows] for x in _attend(c)], _expect(part), D)
    else:
        _close(_attend(c), _expect(c), D)


def test_attend_queries_that_are_not_finite():
    c = _case(8, 1, 3, 4, 2, 64, 32, [40])
    c["q"][0, 1, 1, 3], c["q"][0, 2, 2, 0] = float("nan"), float("inf")
    out, lse = (f64(x) for x in _attend(c))
    bad = np.zeros((1, 3, 4), bool)
    bad[0, 1, 1] = bad[0, 2, 2] = True
    np.testing.assert_array_equal(np.isnan(lse), bad)
    np.testing.assert_array_equal(np.isnan(out).all(-1), bad)
    exp = _expect(c)
    ok = ~bad
    _close([torch.from_numpy(out[ok]), torch.from_numpy(lse[ok])], [x[ok] for x in exp], 64)


def test_attend_nan_in_a_cached_entry():
    c = _case(10, 2, 2, 2, 1, 128, 32, [100, 100])
    s = int(c["table"][0, 1]) * 32 + 7             # token 39 of sequence 0: one group of its value
    c["cache"][s // 32, 0, 0, 34 * 128 + 7 * 8 + 2] = 0x7f
    out, lse = (f64(x) for x in _attend(c))
    assert np.isnan(out[0, :, :, 32:48]).all() and np.isfinite(out[0, :, :, 48:]).all() and np.isfinite(out[0, :, :, :32]).all()
    assert np.isfinite(lse).all() and np.isfinite(out[1]).all()


@pytest.mark.parametrize("N,Hq", [(1, 2), (3, 64), (60, 16)])
def test_attend_bad_pages_and_lengths(N, Hq):
    """NaN for the sequences concerned, nothing for the others; pages that no
    token needs may hold anything."""
    c = _case(11, 6, N, Hq, 2, 64, 32, [90, 90, 90, 90, 33, 0])
    exp = _expect(c)
    c["table"][0, 1] = c["pages"]
    c["table"][1, 2] = -1
    c["table"][4, 2], c["table"][5, :] = 10 ** 9, -7   # not needed
    lengths = c["lengths"].copy()
    lengths[2], lengths[3] = -1, c["W"] * 32 + 1
    c["lengths"] = lengths
    got = _attend(c)
    assert np.isnan(f64(got[0])[:4]).all() and np.isnan(f64(got[1])[:4]).all()
    _close(got, exp, 64, rows=slice(4, 6))


def test_attend_scale_and_given_outputs():
    c = _case(12, 2, 5, 4, 4, 64, 32, [60, 61], shifts=(1, 4))
    for scale in (0.0, -0.3, 2.0):
        out = torch.full((2, 5, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((2, 5, 4), 7.0, device=DEV)
        got = _attend(c, scale=scale, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        _close(got, _expect(c, scale), 64)


def test_attend_same_result_every_time_and_on_other_streams():
    c = _case(13, 3, 9, 8, 2, 128, 64, [700, 3, 150], tree=True)
    a = _attend(c)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = _attend(c, stream=s)
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_attend_captured_and_replayed_with_other_lengths():
    c = _case(14, 2, 4, 8, 2, 64, 32, [200, 150])
    q, k, v = (c[x].to(DEV) for x in ("q", "k", "v"))
    cache, table, lengths = torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"])
    ws = sv.workspace(sv.spec_attend_workspace_bytes(2, 4, 8, 2, 64), DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 4, 8, device=DEV)

    def call():
        sv.spec_attend_q4(q, cache, table, lengths, k_new=k, v_new=v, out=out, lse=lse, workspace_buf=ws)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in ([200, 150], [1, 199], [0, 33]):
        lengths.copy_(i32(new))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        # behind a shorter length the cache holds ordinary tokens: they must not count
        _close((out, lse), _expect(c, lengths=np.array(new)), 64)


def test_attend_cache_beyond_32_bits():
    """Pages past 4 GiB of cache."""
    D, Hkv, P = 128, 8, 128
    pages = (1 << 32) // (Hkv * P * 144) + 40
    big = torch.zeros((pages, Hkv, P // 32, 36 * D), dtype=torch.uint8, device=DEV)
    c = _case(15, 2, 2, 16, Hkv, D, P, [300, 200])
    at = {int(p): pages - 1 - 3 * i for i, p in enumerate(np.unique(c["table"]))}
    for p, x in at.items():
        big[x] = torch.from_numpy(c["cache"][p]).to(DEV)
    table = np.vectorize(at.get)(c["table"])
    got = sv.spec_attend_q4(c["q"].to(DEV), big, i32(table), i32(c["lengths"]), k_new=c["k"].to(DEV), v_new=c["v"].to(DEV))
    _close(got, _expect(c), D)
    # the same for the way in
    new = torch.zeros_like(big)
    k = torch.randn(5, Hkv, D, device=DEV, dtype=torch.bfloat16)
    slots = np.array([pages * P - 1, pages * P - 200, 5, pages * P - 64, 77])
    sv.spec_kv_store_q4(k, k, i32(slots), new)
    small = sv.q4_cache(5, Hkv, P, D, DEV)
    sv.spec_kv_store_q4(k, k, i32(np.array([4 * P + P - 1, 3 * P + 56, 5, 4 * P + 64, 77])), small)
    assert torch.equal(new[pages - 1], small[4]) and torch.equal(new[pages - 2], small[3]) and torch.equal(new[0], small[0])
    assert int(new[1: pages - 2].count_nonzero()) == 0


def test_two_calls_at_once_with_their_own_workspaces():
    cs = [_case(20 + i, 2, 6, 8, 2, 128, 32, [500, 300]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[_attend(c, stream=s) for c, s in zip(cs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for c, g in zip(cs, pair):
            _close(g, _expect(c), 128)


# --- logit adjustments ------------------------------------------------------------
def _adjust_case(seed, B, R, V, dtype, H, M=0, tree=False, mask=False):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((B, R, V)) * 3).to(dtype)
    c = dict(rng=rng, logits=x, history=rng.integers(-2, V + 2, (B, H)), hist_len=rng.integers(0, H + 3, B), nodes=rng.integers(0, V, (B, R)),
             rep=1 + rng.random(B).astype(np.float32), freq=rng.random(B).astype(np.float32), pres=-rng.random(B).astype(np.float32))
    c["hist_len"][0] = H
    c["prompt_len"] = rng.integers(0, H + 1, B)
    c["nodes"][:, 1::3] = c["nodes"][:, :1]        # the same proposal again
    c["nodes"][0, -1] = -1
    c["see"] = np.broadcast_to(np.tril(np.ones((R, R), bool), -1), (B, R, R))
    c["masks"] = c["bias_tokens"] = c["bias_values"] = c["allowed"] = None
    if tree:
        par = np.array([[-1] + [int(rng.integers(0, i)) for i in range(1, R)] for _ in range(B)])
        m, _ = sv.spec_tree_mask(i32(par))
        c["masks"] = m
        c["see"] = ref.mask_bits(m.cpu().numpy(), R)
        c["see"][:, :, 0] = False
    if M:
        c["bias_tokens"] = rng.integers(0, V, (B, M))
        c["bias_tokens"][:, M // 2] = c["bias_tokens"][:, 0]     # the same token twice
        c["bias_tokens"][0, -1] = -1
        c["bias_tokens"][-1, -1] = V
        c["bias_values"] = rng.standard_normal((B, M)).astype(np.float32)
    if mask:
        c["words"] = rng.integers(0, 2 ** 32, (B, R, -(-V // 32)), dtype=np.uint64).astype(np.uint32)
        c["words"][0, 0] = 0                       # nothing allowed
        c["words"][-1, -1] = 2 ** 32 - 1
        c["allowed"] = ref.mask_bits(c["words"], V)
    return c


def _adjust(c, x=None, out=None, **kw):
    a = dict(history=i32(c["history"]), prompt_lengths=i32(c["prompt_len"]), history_lengths=i32(c["hist_len"]), repetition=f32(c["rep"]),
             frequency=f32(c["freq"]), presence=f32(c["pres"]), node_tokens=i32(c["nodes"]), masks=c["masks"])
    if c["bias_tokens"] is not None:
        a |= dict(bias_tokens=i32(c["bias_tokens"]), bias_values=f32(c["bias_values"]))
    if c["allowed"] is not None:
        a |= dict(allowed=i32(c["words"].view(np.int32)))
    a.update(kw)
    return sv.spec_adjust_logits(c["logits"].to(DEV) if x is None else x, out=out, **a)


def _adjust_expect(c, **kw):
    a = dict(history=c["history"], prompt_len=c["prompt_len"], hist_len=c["hist_len"], rep=c["rep"], freq=c["freq"], pres=c["pres"],
             nodes=c["nodes"], see=c["see"], bias_tokens=c["bias_tokens"], bias_values=c["bias_values"], allowed=c["allowed"])
    a.update(kw)
    return ref.adjust(f64(c["logits"]), **a)


def _adjust_close(got, exp, dtype):
    e, size = exp
    g = f64(got)
    np.testing.assert_array_equal(np.isnan(g), np.isnan(e))
    np.testing.assert_array_equal(g == -np.inf, e == -np.inf)
    tol = 6 * 2.0 ** -24 * size + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) * np.abs(e)
    fin = np.isfinite(e)
    assert (np.abs(g - e)[fin] <= tol[fin]).all(), np.max((np.abs(g - e) / np.maximum(tol, 1e-30))[fin])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,R,V,H,M", [(1, 1, 1, 1, 0), (2, 6, 1000, 50, 8), (3, 2, 999, 300, 0), (1, 33, 4096, 20, 40), (2, 5, 20011, 700, 5),
                                       (4, 6, 32000, 100, 64), (9, 1, 17, 40, 30)])
@pytest.mark.parametrize("tree,mask", [(False, False), (True, True), (False, True)])
def test_adjust_matches_reference(dtype, B, R, V, H, M, tree, mask):
    c = _adjust_case(B * R + V, B, R, V, dtype, H, M, tree, mask)
    exp = _adjust_expect(c)
    got = _adjust(c)
    _adjust_close(got, exp, dtype)
    x = c["logits"].to(DEV)
    assert _adjust(c, x, out=x) is x               # in place
    assert torch.equal(x.view(torch.int16 if dtype is torch.bfloat16 else I32), got.view(torch.int16 if dtype is torch.bfloat16 else I32))


def test_adjust_each_part_alone():
    c = _adjust_case(1, 2, 4, 300, torch.float32, 30, 6, False, True)
    none = dict(history=None, prompt_lengths=None, history_lengths=None, repetition=None, frequency=None, presence=None, node_tokens=None,
                bias_tokens=None, bias_values=None, allowed=None)
    off = dict(history=None, prompt_len=None, hist_len=None, rep=None, freq=None, pres=None, nodes=None, bias_tokens=None, bias_values=None, allowed=None)
    x = c["logits"].to(DEV)
    assert torch.equal(_adjust(c, **none), x)
    full = dict(history=i32(c["history"]), history_lengths=i32(c["hist_len"]))
    # without prompt lengths the whole history counts as generated
    _adjust_close(_adjust(c, **{**none, **full, "frequency": f32(c["freq"])}),
                  _adjust_expect(c, **{**off, "history": c["history"], "hist_len": c["hist_len"], "freq": c["freq"]}), torch.float32)
    _adjust_close(_adjust(c, **{**none, "node_tokens": i32(c["nodes"]), "presence": f32(c["pres"])}),
                  _adjust_expect(c, **{**off, "nodes": c["nodes"], "pres": c["pres"]}), torch.float32)
    _adjust_close(_adjust(c, **{**none, "bias_tokens": i32(c["bias_tokens"]), "bias_values": f32(c["bias_values"])}),
                  _adjust_expect(c, **{**off, "bias_tokens": c["bias_tokens"], "bias_values": c["bias_values"]}), torch.float32)
    _adjust_close(_adjust(c, **{**none, "allowed": i32(c["words"].view(np.int32))}), _adjust_expect(c, **{**off, "allowed": c["allowed"]}),
                  torch.float32)


def test_adjust_special_logits():
    """-inf, +inf, NaN and the type's lowest value pass through the rules."""
    c = _adjust_case(2, 1, 3, 64, torch.bfloat16, 64, 4, False, True)
    c["history"] = np.arange(64).reshape(1, 64)
    c["logits"][0, :, 3], c["logits"][0, :, 5], c["logits"][0, :, 7] = float("-inf"), float("inf"), float("nan")
    c["logits"][0, :, 9] = torch.finfo(torch.bfloat16).min
    c["rep"][:] = 1.0
    exp = _adjust_expect(c)
    _adjust_close(_adjust(c), exp, torch.bfloat16)


def test_adjust_unaligned_base():
    c = _adjust_case(4, 2, 3, 1024, torch.bfloat16, 40, 5, False, True)
    raw = torch.empty(2 * 3 * 1024 + 1, dtype=torch.bfloat16, device=DEV)
    x = raw[1:].view(2, 3, 1024)
    x.copy_(c["logits"])
    _adjust_close(_adjust(c, x), _adjust_expect(c), torch.bfloat16)


# --- together ----------------------------------------------------------------------
def test_one_speculative_step_after_another():
    """Admission of ragged prompts, then steps of map -> attention -> logits ->
    adjustments -> greedy verification -> commit, against the references with the
    library's own integers in between; at the end every sequence is released."""
    rng = np.random.default_rng(77)
    B, K, Hkv, G, D, P, V = 5, 3, 2, 2, 64, 32, 512
    F, W = 40, 6
    prompts = np.array([33, 1, 64, 90, 31])
    cache = sv.q4_cache(F, Hkv, P, D, DEV)
    table, ring = i32(np.full((B, W), -1)), i32(rng.permutation(F))
    state, held, lengths = i32([7, F]), i32(np.zeros(B)), i32(np.zeros(B))
    T = int(prompts.sum()) + 6
    k, v = _kv(rng, T, Hkv, D) * 0.2, _kv(rng, T, Hkv, D) * 0.2
    off, slots, pos, held, state, st = sv.spec_page_map(lengths, i32(prompts), held, ring, state, table, P, T)
    assert not st.any() and (slots[prompts.sum():] == -1).all()
    sv.spec_kv_store_q4(k.to(DEV), v.to(DEV), slots, cache)
    lengths = i32(prompts)
    head = torch.randn(G * Hkv * D, V, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    history = np.zeros((B, 200), np.int64)
    hist_len = np.ones(B, np.int64)
    for step in range(4):
        q, kn, vn = bf(rng.standard_normal((B, K + 1, G * Hkv, D))), _kv(rng, B, K + 1, Hkv, D) * 0.2, _kv(rng, B, K + 1, Hkv, D) * 0.2
        off, slots, pos, held, state, st = sv.spec_page_map(lengths, i32(np.full(B, K + 1)), held, ring, state, table, P, B * (K + 1))
        assert not st.any()
        out, lse = sv.spec_attend_q4(q.to(DEV), cache, table, lengths, k_new=kn.to(DEV), v_new=vn.to(DEV))
        see = np.broadcast_to(np.tril(np.ones((K + 1, K + 1), bool)), (B, K + 1, K + 1))
        exp = ref.attend(f64(q), cache.cpu().numpy(), table.cpu().numpy(), lengths.cpu().numpy(), f64(kn), f64(vn), see, D ** -0.5, 0, 0)
        _close((out, lse), exp, D)
        logits = (out.double().cpu().reshape(B, K + 1, -1) @ head).to(torch.float32).to(DEV)
        drafts = rng.integers(0, V, (B, K))
        best = logits.argmax(-1).cpu().numpy()
        drafts[:, 0] = best[:, 0]                       # the first draft is often right
        adj = sv.spec_adjust_logits(logits, history=i32(history), history_lengths=i32(hist_len), frequency=f32(np.full(B, 0.01)),
                                    node_tokens=i32(drafts))
        e, size = ref.adjust(f64(logits), history, None, hist_len, None, np.full(B, np.float32(0.01)), None, drafts,
                             np.broadcast_to(np.tril(np.ones((K + 1, K), bool), -1), (B, K + 1, K)), None, None, None)
        _adjust_close(adj, (e, size), torch.float32)
        tokens, n = sv.spec_verify_greedy(adj, i32(drafts))
        new = sv.spec_kv_commit_q4(cache, table, lengths, kn.to(DEV), vn.to(DEV), n + 1)
        np.testing.assert_array_equal(new.cpu().numpy(), (lengths + n + 1).cpu().numpy())
        for b in range(B):
            got = tokens[b, : int(n[b]) + 1].cpu().numpy()
            history[b, hist_len[b]: hist_len[b] + len(got)] = got
            hist_len[b] += len(got)
        lengths = new
    _, _, _, held, state, st = sv.spec_page_map(lengths, i32(np.full(B, -1)), held, ring, state, table, P, 0)
    assert not st.any() and not held.any() and int(state[1]) == F
    assert sorted(ring.cpu().tolist()) == list(range(F))


def test_binding_refuses_what_does_not_fit():
    c = _case(30, 1, 2, 4, 2, 64, 32, [40])
    q, cache, table, lengths = c["q"].to(DEV), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"])
    k = c["k"].to(DEV)
    with pytest.raises(ValueError, match="contiguous"):
        sv.spec_attend_q4(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, lengths)
    with pytest.raises(TypeError):
        sv.spec_attend_q4(q.float(), cache, table, lengths)
    with pytest.raises(sv.SpecError):
        sv.spec_attend_q4(q, cache, table, lengths, k_new=k)                  # no v_new: refused by the library
    with pytest.raises(ValueError, match="shape"):
        sv.spec_attend_q4(q, cache, table, lengths, k_new=k[:, :1].contiguous(), v_new=k)
    with pytest.raises(ValueError, match="must be on"):
        sv.spec_attend_q4(q, cache, table.cpu(), lengths)
    with pytest.raises(sv.SpecError):
        sv.spec_attend_q4(q, cache, table, lengths, workspace_buf=sv.workspace(64, DEV))
    with pytest.raises(ValueError, match="shape"):
        sv.spec_kv_store_q4(k[0], k[0], i32([1]), cache)
    with pytest.raises(TypeError):
        sv.spec_page_map(lengths.long(), lengths, lengths, lengths, lengths, table, 32, 4)
