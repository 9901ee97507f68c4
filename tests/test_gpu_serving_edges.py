"""Edges of the serving steps on the GPU: infinite scores, entries at the ends of
their types' ranges, the largest batches, waits that run out.

Tolerances are those of test_gpu_serving.py (derived there); where a score is an
infinity, the expected values come from the same reference with that node left out,
which is what a weight of zero means."""
import time

import numpy as np
import pytest
import torch

import serving_ref as ref
import speculative_decoding_verification_52_gb300 as sv
import test_gpu_serving as base
from test_gpu_serving import DEV, _attend, _case, _close, _expect, bf, f32, f64, i32

pytestmark = pytest.mark.gpu
# rows of a kv head below and above each kernel's row tiles
ROWS = [(1, 2, 1, 128), (6, 8, 2, 64)] + base.TILES


@pytest.mark.parametrize("shift", [-32, -9, 32])
def test_store_of_the_largest_values(shift):
    """Finite values whose quotient by 2^shift is beyond fp32: the scale is the largest
    one, not a NaN."""
    rng = np.random.default_rng(5)
    T, D = 64, 64
    k = bf(rng.standard_normal((T, 1, D)) * np.exp2(rng.integers(80, 127, (T, 1, 1))))
    k[3, 0, 17] = float("inf")
    k[5, 0, 40] = float("nan")
    k[7, 0, :] = torch.finfo(torch.bfloat16).max
    v = bf(rng.standard_normal((T, 1, D)) * np.exp2(rng.integers(-126, 127, (T, 1, D))))
    assert torch.isfinite(v).all()
    exp = np.zeros((2, 1, 1, 36 * D), np.uint8)
    for t in range(T):
        ref.q4_put(exp, t, 0, f64(k[t, 0]), f64(v[t, 0]), shift, shift)
    c = sv.q4_cache(2, 1, 32, D, DEV)
    sv.spec_kv_store_q4(k.to(DEV), v.to(DEV), i32(np.arange(T)), c, k_shift=shift, v_shift=shift)
    np.testing.assert_array_equal(c.cpu().numpy(), exp)
    c.zero_()
    new = sv.spec_kv_commit_q4(c, i32([[0, 1]]), i32([0]), k.view(1, T, 1, D).to(DEV), v.view(1, T, 1, D).to(DEV), i32([T]), k_shift=shift, v_shift=shift)
    assert new.tolist() == [T]
    np.testing.assert_array_equal(c.cpu().numpy(), exp)


@pytest.mark.parametrize("N", [49, 65])
def test_attend_batches_next_to_the_shared_memory_limit(N):
    """The prefix sums of a batch lie in shared memory beside the buffers: every batch
    up to the largest is taken."""
    D, P = 128, 32
    rng = np.random.default_rng(N)
    for B in [*range(2560, 2920, 24), 2703, 2704, 2767, 2768, 2799, 2800, 2863, 2864, 4096]:
        lengths = rng.integers(0, 4, B)
        q = torch.randn(B, N, 1, D, device=DEV, dtype=torch.bfloat16)
        k, v = (torch.randn(B, N, 1, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        pages = base._cache(rng, 8, 1, P, D)
        table = rng.integers(0, 8, (B, 1))
        got = sv.spec_attend_q4(q, torch.from_numpy(pages).to(DEV), i32(table), i32(lengths), k_new=k, v_new=v)
        rows = [0, B // 2, B - 1]
        see = np.broadcast_to(np.tril(np.ones((N, N), bool)), (3, N, N))
        exp = ref.attend(f64(q[rows]), pages, table[rows], lengths[rows], f64(k[rows]), f64(v[rows]), see, D ** -0.5, 0, 0)
        _close([x[rows] for x in got], exp, D)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS)
@pytest.mark.parametrize("every", [False, True])
def test_attend_scores_of_minus_infinity(N, Hq, Hkv, D, every):
    """A key with an infinity of the other sign than the queries' element gives every
    row that sees it a score of -inf, which weighs nothing: the first node's (all that
    row 0 sees of the fresh entries), or every node's."""
    c = _case(70 + N, 3, N, Hq, Hkv, D, 32, [0, 300, 33], shifts=(1, -1))
    c["q"][..., 5] = c["q"][..., 5].abs() + 0.5
    see = c["see"].copy()
    see[:, :, slice(None) if every else 0] = False
    exp = _expect(dict(c, see=see))
    c["k"][:, slice(None) if every else 0, :, 5] = float("-inf")
    assert (exp[1][0, 0] == -np.inf).all() and np.isfinite(exp[1][1:]).all()
    _close(_attend(c), exp, D)


def _stalled(seed, B, N, Hq, Hkv, D, fresh, ctas):
    """Calls in which a CTA waits for an arrival that never comes: what it works on is NaN,
    everything else has the bits of an ordinary call, and so has the next call."""
    rng = np.random.default_rng(seed)
    lengths, pages = rng.integers(1500, 2500, B), 64
    cache = torch.from_numpy(base._cache(rng, pages, Hkv, 32, D)).to(DEV)
    table, lens = i32(rng.integers(0, pages, (B, 80))), i32(lengths)
    q = torch.randn(B, N, Hq, D, device=DEV, dtype=torch.bfloat16)
    new = {x: torch.randn(B, N, Hkv, D, device=DEV, dtype=torch.bfloat16) for x in ("k_new", "v_new")} if fresh else {}
    out, lse = sv.spec_attend_q4(q, cache, table, lens, **new)
    assert torch.isfinite(lse).all()
    for cta in (*ctas, 100000):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        o, l = sv.spec_debug_attend_stall(q, cache, table, lens, cta, 2000, **new)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5
        void = torch.isnan(l)
        assert void.any().item() == (cta < 100000) and not void.all()
        assert torch.equal(torch.isnan(o), void[..., None].expand_as(o))
        assert torch.equal(l[~void], lse[~void]) and torch.equal(o[~void], out[~void])
        a = sv.spec_attend_q4(q, cache, table, lens, **new)
        assert torch.equal(a[0], out) and torch.equal(a[1], lse)


@pytest.mark.parametrize("B,N,Hq,Hkv,D", [(60, 13, 4, 1, 128), (40, 16, 16, 2, 128), (40, 65, 4, 2, 64), (30, 130, 2, 2, 128)])
@pytest.mark.parametrize("fresh", [False, True])
def test_attend_wait_that_runs_out_with_many_rows(B, N, Hq, Hkv, D, fresh):
    _stalled(B, B, N, Hq, Hkv, D, fresh, (0, 1, 77, 151))


@pytest.mark.parametrize("B,N,Hq,Hkv,D", [(120, 1, 16, 2, 128), (120, 6, 8, 2, 128), (100, 5, 16, 2, 128), (120, 3, 8, 2, 64), (60, 16, 16, 4, 64)])
@pytest.mark.parametrize("fresh", [False, True])
def test_attend_wait_that_runs_out_with_few_rows(B, N, Hq, Hkv, D, fresh):
    _stalled(B, B, N, Hq, Hkv, D, fresh, (0, 1, 200, 303))


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS)
@pytest.mark.parametrize("length", [0, 70])
def test_attend_queries_with_infinities(N, Hq, Hkv, D, length):
    """A query with an infinity has scores of -inf and +inf: all -inf is no weight at
    all, one +inf is NaN."""
    c = _case(74 + N, 2, N, Hq, Hkv, D, 32, [length, length], shifts=(0, 0))
    blk = c["cache"]
    blk[..., 5 // 2: 16 * D: D // 2] = (blk[..., 5 // 2: 16 * D: D // 2] & 0x0f) | 0x20   # element 5 of every key: +1 (times its scale)
    c["k"][..., 5] = 1.0
    exp = [x.copy() for x in _expect(c)]
    c["q"][0, N - 1, 0, 5], c["q"][1, N - 1, Hq - 1, 5] = float("-inf"), float("inf")
    sc = ref.q4_split(blk, D)[2].astype(int)
    assert (sc[..., 0] > 0).all()
    exp[0][0, N - 1, 0], exp[1][0, N - 1, 0] = 0, -np.inf
    exp[0][1, N - 1, Hq - 1], exp[1][1, N - 1, Hq - 1] = np.nan, np.nan
    _close(_attend(c), exp, D)


@pytest.mark.parametrize("N", [1, 20, 64])
def test_attend_largest_queries_against_keys_of_zero(N):
    """Keys of zero score 0 whatever the queries and the shift."""
    q = torch.full((1, N, 4, 128), 2.0 ** 126, dtype=torch.bfloat16, device=DEV)
    out, lse = sv.spec_attend_q4(q, sv.q4_cache(2, 1, 32, 128, DEV), i32([[0, 1]]), i32([40]), k_shift=32)
    assert not out.any()
    np.testing.assert_allclose(f64(lse), np.log(40.0), rtol=0, atol=2.0 ** -20 * 5)


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS[1:])
def test_attend_large_finite_keys_at_small_shifts(N, Hq, Hkv, D):
    """Scores far beyond the cache's, and within fp32: the node with the largest takes
    all of the weight."""
    c = _case(71 + N, 2, N, Hq, Hkv, D, 32, [40, 0], shifts=(-32, 0))
    c["k"][:, 2] *= 2.0 ** 100
    out, lse = (f64(x) for x in _attend(c))
    assert np.isfinite(lse).all() and np.isfinite(out).all()
    G = Hq // Hkv
    k, v, q = (f64(c[x]) for x in ("k", "v", "q"))
    z = np.einsum("bnid,bid->bni", q, np.repeat(k[:, 2], G, 1)) * D ** -0.5
    assert (np.abs(z) > 2.0 ** 60).all()
    wins = (z > 0) & (np.arange(N) >= 2)[None, :, None]
    want = np.broadcast_to(np.repeat(v[:, 2], G, 1)[:, None], out.shape)
    assert wins.any() and (np.abs(out - want) <= 2.0 ** -8 * np.abs(want))[wins].all()


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS[1:])
@pytest.mark.parametrize("shifts,ks,vs", [((0, 0), -20, -20), ((0, 0), -60, -45), ((32, 32), 0, 0), ((-32, -32), 8, 8), ((32, -32), 20, -10)])
def test_attend_fresh_entries_far_from_the_caches_unit(N, Hq, Hkv, D, shifts, ks, vs):
    """Fresh entries are bf16 whatever the shifts: keys of 2^ks (the queries make up
    for it, so that the scores are ordinary ones) and values of 2^vs, in units of
    2^shift; nothing is cached."""
    c = _case(72 + N, 2, N, Hq, Hkv, D, 32, [0, 0], shifts=shifts)
    c["k"] *= 2.0 ** ks
    c["q"] *= 2.0 ** -ks
    c["v"] *= 2.0 ** vs
    _close(_attend(c), _expect(c), D)


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS[1:])
def test_attend_fresh_entries_of_every_size_together(N, Hq, Hkv, D):
    """Nodes and columns of sizes between 2^-60 and 2^20 beside each other and beside
    cached tokens."""
    c = _case(73 + N, 3, N, Hq, Hkv, D, 32, [0, 70, 5], tree=True, shifts=(3, -4))
    rng = c["rng"]
    for x in ("k", "v"):
        c[x] = (c[x].double() * torch.from_numpy(np.exp2(rng.integers(-60, 3, (3, N, Hkv, 1)) + rng.integers(-12, 13, (3, N, Hkv, D))))).to(torch.bfloat16)
    _close(_attend(c), _expect(c), D)


def test_first_argument_by_name():
    """Every argument of the serving calls can be given by its name."""
    c = _case(75, 1, 2, 4, 2, 64, 32, [40])
    q, cache, table, lengths = c["q"].to(DEV), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"])
    a, b = sv.spec_attend_q4(q, cache, table, lengths), sv.spec_attend_q4(q=q, cache=cache, block_table=table, lengths=lengths)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = torch.randn(1, 2, 40, device=DEV)
    assert torch.equal(sv.spec_adjust_logits(logits=x), x)


def test_adjust_repetition_penalties_of_every_size():
    """logit / repetition takes two roundings (of the reciprocal and of the product),
    2^-24 each: 2^-23 (1 + 2^-25) of the quotient at most.  A negative logit's product
    takes one."""
    rng = np.random.default_rng(6)
    rep = np.array([1.1, 1.3, 2.0 ** -126, 2.0 ** 126, 7.0, 0.3], np.float32)
    B, V = len(rep), 4099
    x = (rng.standard_normal((B, 1, V)) * np.array([3, 3, 1e-12, 1e12, 3, 3])[:, None, None]).astype(np.float32)
    x = np.where((rep > 2)[:, None, None] | (rep < 0.1)[:, None, None], np.abs(x), x)
    got = sv.spec_adjust_logits(f32(x), history=i32(np.broadcast_to(np.arange(V), (B, V))), history_lengths=i32(np.full(B, V)),
                                prompt_lengths=i32(np.full(B, V)), repetition=f32(rep)).cpu().numpy()
    r = rep[:, None, None].astype(np.float64)
    exp = np.where(x > 0, x / r, x * r)
    assert (np.abs(got - exp) <= 2.0 ** -23 * (1 + 2.0 ** -25) * np.abs(exp)).all()


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attend_scales_with_every_row_tile(N, Hq, Hkv, D, scale):
    """A negative scale, a large one, and none, over cached and fresh entries."""
    c = _case(77 + N, 3, N, Hq, Hkv, D, 32, [150, 0, 33], tree=True, shifts=(1, -2))
    _close(_attend(c, scale=scale), _expect(c, scale), D)


@pytest.mark.parametrize("N,Hq,Hkv,D", ROWS[1:])
def test_attend_cached_tokens_alone_with_every_row_tile(N, Hq, Hkv, D):
    """Without fresh entries; queries of one size and of very different ones."""
    c = _case(78 + N, 4, N, Hq, Hkv, D, 32, [300, 0, 129, 1], fresh=False, shifts=(2, -3))
    c["q"][2:] *= torch.from_numpy(np.exp2(c["rng"].integers(-14, 3, (2, N, Hq, 1)))).to(torch.bfloat16)
    exp = _expect(c)
    assert (exp[1][1] == -np.inf).all()
    _close(_attend(c), exp, D)


@pytest.mark.parametrize("N,Hq,D", [(1, 8, 128), (2, 8, 128), (6, 4, 128), (8, 4, 64)])
def test_attend_largest_batch_of_few_rows(N, Hq, D):
    rng = np.random.default_rng(N)
    B, P, pages = 4096, 32, 16
    lengths, table = rng.integers(0, 90, B), rng.integers(0, pages, (B, 3))
    cache = base._cache(rng, pages, 1, P, D)
    q = torch.randn(B, N, Hq, D, device=DEV, dtype=torch.bfloat16)
    k, v = (torch.randn(B, N, 1, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    got = sv.spec_attend_q4(q, torch.from_numpy(cache).to(DEV), i32(table), i32(lengths), k_new=k, v_new=v)
    rows = [0, 1, 2047, B - 1]
    see = np.broadcast_to(np.tril(np.ones((N, N), bool)), (4, N, N))
    exp = ref.attend(f64(q[rows]), cache, table[rows], lengths[rows], f64(k[rows]), f64(v[rows]), see, D ** -0.5, 0, 0)
    _close([x[rows] for x in got], exp, D)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()


def test_attend_captured_with_many_rows_and_a_shared_workspace():
    """Two captured calls, of many rows and of few, that use one workspace in turn."""
    cs = [_case(79, 2, 40, 16, 2, 128, 32, [300, 150]), _case(80, 3, 2, 16, 2, 64, 32, [100, 300, 7])]
    ws = sv.workspace(max(sv.spec_attend_workspace_bytes(*c["q"].shape[:3], 2, c["D"]) for c in cs), DEV)
    calls = []
    for c in cs:
        q, k, v = (c[x].to(DEV) for x in ("q", "k", "v"))
        cache, table, lengths = torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"])
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)

        def call(q=q, k=k, v=v, cache=cache, table=table, lengths=lengths, out=out, lse=lse):
            sv.spec_attend_q4(q, cache, table, lengths, k_new=k, v_new=v, out=out, lse=lse, workspace_buf=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        calls.append((c, g, lengths, out, lse, call))   # (call keeps the tensors that the graph reads)
    for news in ([[300, 150], [100, 300, 7]], [[1, 0], [0, 33, 290]]):
        for (c, g, lengths, out, lse, _), new in zip(calls, news):
            lengths.copy_(i32(new))
            out.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for (c, g, lengths, out, lse, _), new in zip(calls, news):
            _close((out, lse), _expect(c, lengths=np.array(new)), c["D"])
