"""The steps after a verification on the GPU against plain 64-bit implementations
(after_ref.py).

Tolerances.  Integers, codes, scales and what is moved are compared exactly.
Log probabilities: a thread adds at most about 100 partial sums of a row, 2^-24 each, to
which come the exponentials (2^-22), the tree of threads and the rounding of log2(e) / T,
2^-24 of z = (l - max) / T * log2(e), whose mean under the weights is below log2 V + H: the
sum of the weights and that of the weights times z are each off by eps = 2^-17 of
themselves at most.  The given token's z has two roundings and the result two more:
  |d logprob| <= eps + 2^-21 (1 + |logprob| + log S),   log S: of sum e^(z - max).
The references lie up to 2^8 below the largest weight, so that exponents z' of up to 8
(log2) are among the terms e z', whose sizes then add up to at most |sum e z'| + 16 sum e,
and |sum e z'| / sum e <= (H + log S) / ln 2 + 8:
  |d entropy| <= eps (2 + 2 (H + log S) + 24 ln 2).
Weights: each term e^(s - lse) is off by what its exponent is: a product of D elements in
fp32, D 2^-23 scale sum |q k| (the tensor core may truncate), q in f16 at 2^-32 of the
row's largest element and more (taken with 2^-9 D 2^-23), the roundings of s and lse in
the log2 domain, 2^-22 (|s| + |lse|), and 2^-20 for the exponential and the sum's
steps; n G terms are added, 2^-24 each; the product with the decay is off by 2^-22."""
import numpy as np
import pytest
import torch

import after_ref as ref
import serving_ref as sref
import speculative_decoding_verification_52_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int64).to(I32).to(DEV)


def f32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.float32).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


# --- log probabilities --------------------------------------------------------
def _check_logprobs(logits, tokens, T, path, n, **kw):
    got = sv.spec_token_logprobs(logits, i32(tokens), T, path=None if path is None else i32(path), top_n=n, **kw)
    _compare_logprobs(got, ref.logprobs(f64(logits), tokens, T, path, n))
    return got


def _compare_logprobs(got, exp):
    lp, ent, rank, top, val = (f64(x) for x in got)
    elp, eent, erank, etop, eval_, log_s = exp
    np.testing.assert_array_equal(rank, erank)
    np.testing.assert_array_equal(top, etop)
    eps = 2.0 ** -17
    for g, e, tol in ((lp, elp, eps + 2.0 ** -21 * (1 + np.abs(elp) + log_s)), (ent, eent, eps * (2 + 2 * (eent + log_s) + 17)),
                      (val, eval_, eps + 2.0 ** -21 * (1 + np.abs(eval_) + log_s[..., None]))):
        np.testing.assert_array_equal(np.isnan(g), np.isnan(e))
        np.testing.assert_array_equal(np.isinf(g), np.isinf(e))
        fine = np.isfinite(e)
        assert (np.abs(g[fine] - e[fine]) <= tol[fine]).all(), np.max(np.abs(g[fine] - e[fine]) / tol[fine])


def _logits(rng, B, R, V, dtype, sigma=2.5):
    return torch.from_numpy(rng.standard_normal((B, R, V)) * sigma).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,M,V,n", [(1, 1, 1, 1), (3, 2, 2, 3), (2, 3, 7, 20), (2, 2, 8, 8), (5, 3, 9, 0), (4, 2, 33, 32), (300, 5, 250, 5),
                                     (9, 7, 2048, 20), (3, 3, 4096, 32), (3, 2, 4097, 9), (3, 2, 8200, 20), (40, 2, 16391, 1),
                                     (2, 3, 32003, 8), (1, 1, 128256, 5), (1, 2, 151936, 32), (2, 1, 128256, 0)])
def test_logprobs(B, M, V, n, dtype):
    rng = np.random.default_rng(V + n)
    x = _logits(rng, B, M + 1, V, dtype)
    tokens = rng.integers(0, V, (B, M))
    best = x.argmax(-1).cpu().numpy()
    tokens[0, 0] = best[0, 0]
    tokens[B - 1, M - 1] = -1
    for T in (1.0, 0.7):
        _check_logprobs(x, tokens, T, None, n)


@pytest.mark.parametrize("B", [200, 700])
def test_logprobs_of_many_rows(B):
    """More rows than CTAs at a time: one CTA a row, and clusters of a few."""
    rng = np.random.default_rng(B)
    x = _logits(rng, B, 1, 20000, torch.bfloat16)
    _check_logprobs(x, rng.integers(-1, 20000, (B, 1)), 0.9, None, 5)


@pytest.mark.parametrize("V,rows", [(4096, 1300), (16384, 4900), (1030, 3)])
@pytest.mark.parametrize("n", [5, 32])
def test_logprobs_of_a_warp_a_row(V, rows, n):
    """Short rows, or many of them: a warp each."""
    rng = np.random.default_rng(V + n)
    x = torch.randn(rows, 1, V, generator=torch.Generator(device=DEV).manual_seed(V), device=DEV) * 2
    x = x.to(torch.bfloat16)
    tokens = rng.integers(0, V, (rows, 1))
    some = np.unique(np.concatenate([[0, rows - 1], rng.integers(0, rows, 40)]))
    got = sv.spec_token_logprobs(x, i32(tokens), 0.8, top_n=n)
    _compare_logprobs([t[some] for t in got], ref.logprobs(f64(x[some]), tokens[some], 0.8, None, n))


@pytest.mark.parametrize("V", [1000, 9001])
def test_logprobs_of_tree_paths(V):
    rng = np.random.default_rng(V)
    B, N, M = 6, 9, 4
    x = _logits(rng, B, N, V, torch.bfloat16)
    path = rng.integers(0, N, (B, M))            # one column more than it takes
    tokens = rng.integers(0, V, (B, M))
    tokens[1, 2:] = -1
    path[1, 1:] = -1
    path[2, 0], path[3, 1] = N, -7
    tokens[4, 1] = V
    got = _check_logprobs(x, tokens, 1.3, path, 4)
    assert torch.isnan(got[0][2, 1]) and torch.isnan(got[0][3, 2]) and torch.isnan(got[0][4, 1])
    one = _check_logprobs(x, tokens[:, :1], 1.3, path[:, :1], 4)
    assert torch.equal(one[0][:, 0], got[0][:, 0])


def test_logprobs_after_verification():
    """out_tokens and out_path as they come."""
    rng = np.random.default_rng(4)
    B, V, parents = 5, 700, [-1, 0, 0, 1, 1, 2, 3]
    x = _logits(rng, B, 7, V, torch.float32)
    best = x.argmax(-1).cpu().numpy()
    nodes = rng.integers(0, V, (B, 7))
    nodes[:, 1], nodes[:3, 3], nodes[0, 6] = best[:, 0], best[:3, 1], best[0, 3]
    tokens, n, path = sv.spec_verify_tree_greedy(x, i32(parents), i32(nodes), 3)
    got = sv.spec_token_logprobs(x, tokens, path=path, top_n=1)
    _compare_logprobs(got, ref.logprobs(f64(x), tokens.cpu().numpy(), 1.0, path.cpu().numpy(), 1))
    there = tokens >= 0
    assert n.tolist()[0] == 3 and torch.equal(got[2][there], torch.ones_like(got[2][there])) and torch.equal(got[3][..., 0], torch.where(there, tokens, -1))


@pytest.mark.parametrize("V", [3000, 30011])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_of_odd_rows(V, dtype):
    """Equal logits, few different ones, rising and falling rows (a rising one fills the
    list of candidates), masks by -inf and by the type's lowest value, fewer allowed
    tokens than alternatives, allowed tokens at one end only, zeros of both signs."""
    rng = np.random.default_rng(V)
    low = torch.finfo(dtype).min
    rows = [np.zeros(V), rng.integers(0, 3, V) * 0.5, np.linspace(-5, 5, V), np.linspace(5, -5, V)]
    for keep, value in ((5, -np.inf), (5, low), (40, low)):
        r = np.full(V, value)
        at = rng.permutation(V)[:keep]
        r[at] = rng.standard_normal(keep)
        rows.append(r)
    for part in (slice(0, 700), slice(V - 900, V), slice(V // 2, V // 2 + 50)):
        r = np.full(V, -np.inf)
        r[part] = np.linspace(0, 3, len(r[part]))
        rows.append(r)
    r = rng.standard_normal(V) * 1e-3
    r[rng.random(V) < 0.5] = -0.0
    rows += [r, np.where(rng.random(V) < 0.5, 0.0, -0.0), np.full(V, -7.25), np.where(np.arange(V) == V - 1, 3.0, 2.0)]
    one = np.full(V, low)
    one[17] = 4.0
    rows.append(one)
    x = torch.from_numpy(np.stack(rows)[None]).to(dtype).to(DEV)
    M = len(rows)
    for tokens in (rng.integers(0, V, (1, M)), np.full((1, M), 17), np.full((1, M), V - 1), np.zeros((1, M), np.int64)):
        for n in (20, 3):
            _check_logprobs(x, tokens, 1.0, None, n)


def test_logprobs_of_invalid_rows_and_the_largest_logits():
    rng = np.random.default_rng(6)
    V = 9000
    rows = rng.standard_normal((9, V))
    rows[0, 5], rows[1, V - 1], rows[2], rows[3, 3000], rows[4, 0] = np.nan, np.inf, -np.inf, 2.0 ** 100, np.nan
    rows[5] = -(2.0 ** 100)
    rows[6, 77], rows[7, 88] = 1e30, 100.0
    rows[8] = -1e30
    x = torch.from_numpy(rows[None]).to(torch.float32).to(DEV)
    for tok in (88, 0):
        got = _check_logprobs(x, np.full((1, 9), tok), 1.0, None, 3)
        assert torch.isnan(got[0][0, :6]).all() and (got[2][0, :6] == -1).all() and (got[3][0, :6] == -1).all()
        assert torch.isfinite(got[1][0, 6:]).all()
    # a row without a token is not looked at
    tokens = np.full((1, 9), 3)
    tokens[0, :6] = -1
    got = _check_logprobs(x, tokens, 0.01, None, 2)
    assert (got[0][0, :6] == 0).all() and (got[1][0, :6] == 0).all() and (got[4][0, :6] == float("-inf")).all()


@pytest.mark.parametrize("T", [1e-4, 0.05, 30.0, 1e6])
def test_logprobs_temperatures(T):
    """At 1e-4 the exponents reach 10^5, of which only those near the largest count."""
    rng = np.random.default_rng(8)
    x = _logits(rng, 2, 2, 12345, torch.float32, 1.0)
    tokens = x.argmax(-1).cpu().numpy()
    _check_logprobs(x, tokens, T, None, 1)
    if T > 0.01:
        _check_logprobs(x, rng.integers(0, 12345, (2, 2)), T, None, 6)


def test_logprobs_unaligned_base_given_outputs_and_streams():
    rng = np.random.default_rng(9)
    B, M, V = 3, 2, 10007
    for dtype in (torch.bfloat16, torch.float32):
        raw = torch.empty(B * M * V + 3, dtype=dtype, device=DEV)
        for off in (1, 3):
            x = raw[off: off + B * M * V].view(B, M, V)
            x.copy_(_logits(rng, B, M, V, dtype))
            _check_logprobs(x, rng.integers(0, V, (B, M)), 1.0, None, 7)
    tokens = rng.integers(0, V, (B, M))
    outs = dict(logprobs=torch.zeros(B, M, device=DEV), entropy=torch.zeros(B, M, device=DEV), ranks=torch.zeros(B, M, dtype=I32, device=DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _check_logprobs(x, tokens, 1.0, None, 2, stream=s, **outs)
    assert got[0] is outs["logprobs"] and got[2] is outs["ranks"]


def test_logprobs_repeat_exactly_and_in_a_graph():
    rng = np.random.default_rng(10)
    x, tokens = _logits(rng, 20, 4, 50000, torch.bfloat16), i32(rng.integers(0, 50000, (20, 4)))
    first = sv.spec_token_logprobs(x, tokens, top_n=20)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, sv.spec_token_logprobs(x, tokens, top_n=20)))
    outs = [torch.zeros_like(t) for t in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_token_logprobs(x, tokens, top_n=20, logprobs=outs[0], entropy=outs[1], ranks=outs[2], top_tokens=outs[3], top_logprobs=outs[4])
    x.copy_(_logits(rng, 20, 4, 50000, torch.bfloat16))
    g.replay()
    _compare_logprobs(outs, ref.logprobs(f64(x), tokens.cpu().numpy(), 1.0, None, 20))


# --- weights -------------------------------------------------------------------
def _cache(rng, pages, Hkv, P, D):
    """Blocks with codes and scales as quantised entries have them (all codes; scales 2^-3 to 2)."""
    c = rng.integers(0, 256, (pages, Hkv, P // 32, 36 * D)).astype(np.uint8)
    c[..., 32 * D:] = rng.integers(0x20, 0x41, c[..., 32 * D:].shape)
    return c


def _table(rng, lengths, P, pages, extra=0):
    need = [-(-max(0, int(n)) // P) for n in lengths]
    W = max(1, max(need)) + extra
    ids = rng.permutation(pages)
    assert sum(need) <= pages
    t, at = np.full((len(lengths), W), -1), 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at: at + n]
        at += n
    return t


def _weigh_case(seed, B, N, G, Hkv, D, P, lengths, tree=False, count=None, extra=0):
    rng = np.random.default_rng(seed)
    W = min(N, 6) if tree else N
    lengths = np.asarray(lengths)
    pages = int(sum(-(-(int(n) + W) // P) for n in lengths)) + 2
    c = dict(rng=rng, B=B, N=N, D=D, P=P, lengths=lengths, scale=D ** -0.5, shift=-1, first=rng.integers(0, 1000, B), decay=0.9)
    c["cache"], c["table"] = _cache(rng, pages, Hkv, P, D), _table(rng, lengths + W, P, pages, extra)
    c["q"] = torch.from_numpy(rng.standard_normal((B, N, Hkv * G, D)) * 0.4).to(torch.bfloat16)
    c["lse"] = np.float32(rng.standard_normal((B, N, Hkv * G)) + 4)
    c["weights"], c["pos"] = np.float32(np.exp(rng.standard_normal((pages, Hkv, P)))), rng.integers(0, 999, (pages, Hkv, P))
    c["path"] = np.sort(rng.permuted(np.tile(np.arange(N), (B, 1)), axis=1)[:, :W], axis=1) if tree else None
    c["count"] = rng.integers(0, W + 1, B) if count is None else count
    return c


def _run_weigh(c, inplace=False, **kw):
    w, pos = f32(c["weights"]), i32(c["pos"])
    new = w if inplace else torch.full_like(w, 123.0)
    before = f64(new)
    opt = lambda x, f: None if x is None else f(x)  # noqa: E731
    args = dict(count=opt(c["count"], i32), path=opt(c["path"], i32), positions=pos, first_positions=opt(c["first"], i32),
                new_weights=None if inplace else new, scale=c["scale"], decay=c["decay"], k_shift=c["shift"])
    got = sv.spec_kv_weigh_q4(c["q"].to(DEV), f32(c["lse"]), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"]), w, **{**args, **kw})
    assert got.data_ptr() == new.data_ptr()
    new_w, new_p, tol = ref.weigh(f64(c["q"]), c["lse"], c["cache"], c["table"], c["lengths"], c["weights"], c["pos"], c["count"], c["path"],
                                  c["first"], c["scale"], c["decay"], c["shift"], before)
    d = np.abs(f64(got) - new_w)
    np.testing.assert_array_equal(pos.cpu().numpy(), new_p)
    assert (d <= tol).all(), (np.nanmax(d / np.maximum(tol, 1e-30)), np.argwhere(~(d <= tol))[:5])
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,G,Hkv,P,lengths,tree", [
    (1, 1, 1, 1, 32, [0], False), (1, 1, 4, 2, 32, [31], False), (2, 2, 1, 3, 64, [32, 777], False), (3, 6, 4, 2, 32, [0, 100, 63], False),
    (4, 5, 3, 1, 96, [1, 200, 95, 96], False), (2, 4, 8, 2, 64, [130, 5], False), (2, 9, 4, 1, 32, [64, 300], False),
    (3, 40, 2, 2, 64, [10, 500, 64], True), (1, 70, 4, 1, 128, [129], False), (2, 64, 7, 1, 32, [33, 1], True), (1, 200, 1, 2, 64, [600], False),
    (1, 3, 64, 1, 32, [50], False)])
def test_weigh(B, N, G, Hkv, P, lengths, tree, D):
    c = _weigh_case(B * 100 + N, B, N, G, Hkv, D, P, lengths, tree)
    _run_weigh(c)
    c["count"] = None
    _run_weigh(c, inplace=True)


def test_weigh_ragged_batch():
    rng = np.random.default_rng(0)
    lengths = rng.integers(0, 400, 37)
    c = _weigh_case(11, 37, 6, 2, 2, 64, 32, lengths, extra=50)
    c["first"] = None
    _run_weigh(c)
    c["decay"] = 0.0
    _run_weigh(c, inplace=True)


def test_weigh_chunk_over_long_context():
    _run_weigh(_weigh_case(12, 1, 300, 4, 1, 64, 64, [2500], count=np.array([300])))
    _run_weigh(_weigh_case(13, 1, 257, 2, 1, 128, 32, [1000], count=np.array([257])))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", [(2, 64), (1, 2)])
def test_weigh_of_very_long_sequences(N, G, D):
    """34 million tokens, of which three pages lie in the cache: a token's distance times the
    query heads of its kv head passes 32 bits."""
    c, W = _weigh_case(19, 1, N, G, 1, D, 2048, [5000], count=np.array([N])), 16602
    table = np.full((1, W), -1)
    table[0, 0], table[0, -2:] = c["table"][0, 0], c["table"][0, 1:3]
    c["table"], c["lengths"] = table, c["lengths"] + (W - 3) * 2048
    assert c["lengths"][0] * 64 >= 2 ** 31
    _run_weigh(c)


def test_weigh_requests_that_are_refused_or_ask_nothing():
    """Bad lengths, counts and paths leave a sequence as it is; the others are served.  A
    count of 0 lets the weights decay.  Pages outside the cache are passed over."""
    c = _weigh_case(14, 9, 12, 2, 2, 64, 32, [70] * 9, tree=True)
    W = c["path"].shape[1]
    c["count"][:] = W
    c["count"][0], c["count"][1], c["count"][2] = -1, W + 1, 0
    c["lengths"][3], c["lengths"][4] = -5, 10000
    c["path"][5, 2], c["path"][6, 0] = 12, -1
    c["table"][7, 1], c["table"][8, 0] = -1, len(c["weights"])
    _run_weigh(c)
    _run_weigh(c, inplace=True)


def test_weigh_rows_that_add_nothing():
    """Rows without a finite lse; NaN keys among the fresh tokens, which only rows without
    a finite lse see; infinite and NaN queries of rows that do not count."""
    c = _weigh_case(15, 2, 8, 2, 2, 128, 32, [100, 40])
    c["count"] = np.array([8, 3])
    c["lse"][0, 2], c["lse"][0, 3, 1], c["lse"][1, 1] = -np.inf, np.inf, np.nan
    c["lse"][0, 5:] = np.nan
    c["q"][0, 2], c["q"][1, 4:] = float("nan"), float("inf")
    for row in (105, 106):
        page = c["table"][0, row // 32]
        c["cache"][page, :, 0, 32 * 128 + (row % 32) * 8: 32 * 128 + (row % 32) * 8 + 8] = 0x7f
    w = _run_weigh(c)
    assert torch.isfinite(w).all()


def test_weigh_extreme_queries_and_shifts():
    for shift, size in ((20, 1e-7), (-20, 1e6), (0, 1.0)):
        c = _weigh_case(16, 2, 3, 2, 1, 64, 32, [90, 45])
        c["shift"] = shift
        c["q"] = (c["q"].double() * size).to(torch.bfloat16)
        _run_weigh(c)
    c = _weigh_case(17, 1, 2, 2, 1, 64, 32, [90])
    c["scale"] = -0.3
    _run_weigh(c)
    c["scale"] = 0.0
    _run_weigh(c)


def test_weigh_repeats_exactly_and_in_a_graph():
    c = _weigh_case(18, 4, 6, 4, 2, 128, 64, [300, 20, 1000, 0])
    w = f32(c["weights"])
    args = (c["q"].to(DEV), f32(c["lse"]), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"]))
    count = i32(c["count"])
    outs = [torch.zeros_like(w) for _ in range(3)]
    for o in outs[:2]:
        sv.spec_kv_weigh_q4(*args, w, count=count, new_weights=o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_kv_weigh_q4(*args, w, count=count, new_weights=outs[2])
    outs[2].zero_()
    g.replay()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,G,Hkv,lengths", [(3, 40, 3, 2, [0, 300, 129]), (1, 130, 5, 1, [127]), (2, 33, 64, 1, [1, 200]), (5, 64, 8, 1, [128, 256, 1000, 31, 500]),
                                               (1, 1024, 1, 2, [100]), (2, 13, 7, 3, [640, 65])])
def test_weigh_of_many_rows(B, N, G, Hkv, lengths, D):
    """The tensor cores' kernel: query heads that do and do not divide its tile of rows,
    rows that end inside one, tokens that see only the last rows, several sequences."""
    c = _weigh_case(1000 + B * N + G, B, N, G, Hkv, D, 32, lengths, extra=3)
    _run_weigh(c)
    c["count"] = np.maximum(c["count"], 1)
    c["count"][0] = N
    _run_weigh(c, inplace=True)


@pytest.mark.parametrize("D", [64, 128])
def test_weigh_of_many_rows_that_add_nothing(D):
    """As for few rows: NaN keys, NaN and infinite queries, rows without a finite lse, in
    tiles with others; requests that are refused, counts of 0, pages outside the cache."""
    c = _weigh_case(2000, 7, 150, 2, 2, D, 64, [200, 100, 70, 70, 70, 70, 300])
    c["count"] = np.array([150, 90, 0, -1, 151, 150, 149])
    c["lse"][0, 100:] = np.nan
    c["lse"][0, 7], c["lse"][1, 3, 1], c["lse"][6, 0] = -np.inf, np.inf, np.nan
    c["q"][0, 7], c["q"][0, 101:], c["q"][1, 90:], c["q"][6, 0] = float("nan"), float("inf"), float("nan"), float("-inf")
    for row in (300, 310):   # of sequence 0: behind 200 old ones, seen by rows from 100 on
        page = c["table"][0, row // 64]
        at = 32 * D + (row % 32) * (D // 16)
        c["cache"][page, :, row % 64 // 32, at: at + D // 16] = 0x7f
    c["lengths"][5] = 10 ** 6
    c["table"][6, 2] = len(c["weights"]) + 5
    w = _run_weigh(c)
    assert torch.isfinite(w).all()


@pytest.mark.parametrize("N", [1, 100])
def test_weigh_of_the_largest_batch(N):
    rng = np.random.default_rng(N)
    B = 4096
    c = _weigh_case(21, B, N, 1, 1, 64, 32, rng.integers(0, 40, B), count=(rng.random(B) < 0.1) * rng.integers(0, min(N, 40) + 1, B))
    _run_weigh(c)


def test_weigh_and_logprobs_on_two_streams():
    """Calls that overlap share nothing."""
    cases = [_weigh_case(30 + i, 3, n, 4, 2, 128, 64, [700, 20, 1500], count=np.array([n] * 3)) for i, n in enumerate((4, 60))]
    ins = [(c["q"].to(DEV), f32(c["lse"]), torch.from_numpy(c["cache"]).to(DEV), i32(c["table"]), i32(c["lengths"]), f32(c["weights"])) for c in cases]
    x = _logits(np.random.default_rng(1), 4, 2, 40000, torch.bfloat16)
    tokens = i32(np.random.default_rng(2).integers(0, 40000, (4, 2)))
    alone = [sv.spec_kv_weigh_q4(*t, new_weights=torch.zeros_like(t[5])) for t in ins]
    lp = sv.spec_token_logprobs(x, tokens, top_n=9)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(t[5]) for t in ins] for _ in range(5)]
    got = []
    for o in outs:
        for i, t in enumerate(ins):
            sv.spec_kv_weigh_q4(*t, new_weights=o[i], stream=streams[i])
        got.append(sv.spec_token_logprobs(x, tokens, top_n=9, stream=streams[2]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, alone))
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, lp))


def test_weigh_is_what_attention_gave():
    """With spec_attend_q4's lse a row's weights add up to its query heads' number."""
    rng = np.random.default_rng(19)
    B, Hkv, G, D, P, L = 3, 2, 4, 128, 64, 500
    cache = torch.from_numpy(_cache(rng, 3 * 8, Hkv, P, D)).to(DEV)
    table, lengths = i32(_table(rng, [L] * B, P, 24)), i32([L] * B)
    q = torch.from_numpy(rng.standard_normal((B, 1, Hkv * G, D)) * 0.5).to(torch.bfloat16).to(DEV)
    _, lse = sv.spec_attend_q4(q, cache, table, lengths)
    w = sv.spec_kv_weigh_q4(q, lse, cache, table, lengths - 1, torch.zeros(24, Hkv, P, device=DEV))
    got = w[table.long()].double().sum((1, 3)).cpu().numpy()
    assert np.abs(got - G).max() < G * 2.0 ** -9


# --- plan ---------------------------------------------------------------------------
def _plan(weights, positions, table, lengths, budgets, nxt, sinks, recent, most):
    B, Hkv = len(lengths), weights.shape[1]
    moves = torch.full((B, Hkv, most, 2), -9, dtype=I32, device=DEV)
    exp = ref.evict_plan(np.float32(weights), positions, table, lengths, budgets, nxt, sinks, recent, moves.cpu().numpy())
    got = sv.spec_kv_evict_plan(f32(weights), i32(positions), i32(table), i32(lengths), i32(budgets), i32(nxt), sinks=sinks, recent=recent, moves=moves)
    for name, g, e in zip(("counts", "lengths", "moves"), (got[1], got[2], got[0]), (exp[1], exp[2], exp[0])):
        np.testing.assert_array_equal(g.cpu().numpy(), e, err_msg=name)
    return exp


def _plan_case(seed, Hkv, P, lengths, extra=0):
    rng = np.random.default_rng(seed)
    pages = int(sum(-(-int(n) // P) for n in lengths)) + 2
    table = _table(rng, lengths, P, pages, extra)
    weights = np.exp(2 * rng.standard_normal((pages, Hkv, P)))
    weights[rng.random(weights.shape) < 0.05] = 0.0
    positions = np.zeros((pages, Hkv, P), np.int64)
    nxt = np.asarray(lengths) + 20
    for b, n in enumerate(lengths):
        t = np.arange(n)
        for h in range(Hkv):
            positions[table[b, t // P], h, t % P] = rng.permutation(n + 20)[:n]
    return rng, weights, positions, table, nxt


@pytest.mark.parametrize("Hkv,P,lengths,budget,sinks,recent", [
    (1, 32, [1], 0, 0, 0), (2, 32, [5], 4, 1, 1), (2, 64, [33, 64, 65, 0], 32, 2, 4), (3, 32, [300, 17, 256], 100, 0, 0),
    (8, 64, [2054] * 5, 2048, 4, 64), (1, 128, [20000], 4096, 4, 256), (2, 32, [5000, 2500], 2500, 0, 3000), (8, 32, [700] * 40, 699, 4, 32),
    (1, 32, [70000], 300, 4, 100), (4, 96, [9000, 8000], 7000, 0, 0)])
def test_plan(Hkv, P, lengths, budget, sinks, recent):
    rng, w, pos, table, nxt = _plan_case(len(lengths) + budget, Hkv, P, lengths)
    most = max(1, max(min(budget, n - budget) for n in lengths))
    _plan(w, pos, table, lengths, [budget] * len(lengths), nxt, sinks, recent, most)


@pytest.mark.parametrize("n,C", [(3000, "many heads"), (12000, "one head")])
def test_plan_of_equal_weights(n, C):
    """All equal, three values, equal ones across the parts of a cluster; -0 and 0; negative ones."""
    Hkv = 2 if C == "one head" else 320
    rng, w, pos, table, nxt = _plan_case(n, Hkv, 64, [n])
    for kind in range(4):
        x = [np.ones_like(w), rng.integers(0, 3, w.shape) * 1.0, np.where(rng.random(w.shape) < 0.5, 0.0, -0.0), -w][kind]
        _plan(x, pos, table, [n], [n // 3], nxt, 2, 5, n)
    _plan(np.zeros_like(w), pos, table, [n], [n // 2], nxt, 0, n, n)           # nearly all protected


def test_plan_of_no_numbers():
    rng, w, pos, table, nxt = _plan_case(3, 2, 32, [500, 400])
    w[rng.random(w.shape) < 0.3] = np.nan
    w[rng.random(w.shape) < 0.1] = np.inf
    w[rng.random(w.shape) < 0.1] = -np.inf
    for budget in (10, 250, 390):
        _plan(w, pos, table, [500, 400], [budget] * 2, nxt, 3, 7, 300)


def test_plan_of_extreme_positions():
    """Positions, next positions and ranges at the ends of 32 bits."""
    rng, w, pos, table, nxt = _plan_case(7, 2, 32, [500, 400])
    ends = np.array([-2 ** 31, -2 ** 31 + 2, -1, 0, 3, 2 ** 31 - 1])
    pos = np.where(rng.random(pos.shape) < 0.3, ends[rng.integers(0, 6, pos.shape)], pos)
    for nxt in ([2 ** 31 - 1, 420], [-2 ** 31, 0], [100, -2 ** 31]):
        for sinks, recent in ((4, 0), (0, 64), (2 ** 31 - 1, 0), (4, 2 ** 31 - 1)):
            for budget in (250, 390):
                _plan(w, pos, table, [500, 400], [budget] * 2, np.array(nxt), sinks, recent, 300)


def test_plan_long_tables_and_keys_that_do_not_fit():
    """Short sequences in wide tables (clusters with idle CTAs), and a part of a sequence
    that is longer than its CTA's keys in shared memory."""
    rng, w, pos, table, nxt = _plan_case(4, 2, 32, [40, 1, 3000], extra=2000)
    _plan(w, pos, table, [40, 1, 3000], [30, 0, 1000], nxt, 1, 2, 1000)
    rng, w, pos, table, nxt = _plan_case(5, 310, 64, [9000])
    _plan(w, pos, table, [9000], [500], nxt, 1, 2, 500)
    rng, w, pos, table, nxt = _plan_case(6, 1, 128, [90000])
    _plan(np.round(w, 1), pos, table, [90000], [45000], nxt, 0, 0, 45000)


@pytest.mark.parametrize("pairs", [1, 2, 613, 1217])
def test_plan_of_few_tokens_to_drop(pairs):
    """A step's drops: 1 to 33 of them (a warp a head looks for up to 32), with several heads
    a CTA, some of which have nothing to drop or are refused, equal weights among them that
    run its list over, and more protected tokens than the budget."""
    lengths = [0, 1, 33, 200, 260, 300, 301, 333, 97] if pairs > 2 else [300]
    Hkv = max(1, pairs // len(lengths))
    rng, w, pos, table, nxt = _plan_case(pairs, Hkv, 32, lengths, extra=4)
    lengths = np.array(lengths)
    for drop in (1, 2, 5, 31, 32, 33):
        _plan(w, pos, table, lengths, np.maximum(lengths - drop, 0), nxt, 1, 4, 40)
        _plan(np.where(w < 1, 0.0, w), pos, table, lengths, np.maximum(lengths - drop, 0), nxt, 0, 0, 40)
    _plan(w, pos, table, lengths, np.maximum(lengths - 20, 0), nxt, 250, 0, 40)
    if pairs > 2:
        table[5, 2], table[3, 6] = -1, len(w)
        budgets = lengths - rng.integers(-3, 12, len(lengths))
        exp = _plan(w, pos, table, lengths, budgets, nxt, 2, 8, 12)
        assert (exp[2] == -1).any()
    one = np.full_like(w, 2.0)
    one[rng.random(w.shape) < 0.03] = 1.0
    _plan(one, pos, table, lengths, np.maximum(lengths - 7, 0), nxt, 0, 0, 40)


def test_plan_refusals_per_sequence():
    lengths = [100, 100, 100, 100, 100, 100, 100, 64]
    rng, w, pos, table, nxt = _plan_case(7, 2, 32, lengths)
    table[1, 2], table[2, 0], table[6, 3] = -1, len(w), 1000
    bad = np.array(lengths)
    bad[3], bad[4] = -1, 100000
    budgets = np.array([60, 60, 60, 60, 60, -1, 100, 10])
    exp = _plan(w, pos, table, bad, budgets, nxt, 0, 0, 40)
    assert exp[2].tolist() == [60, -1, -1, -1, -1, 100, 100, 10]
    exp = _plan(w, pos, table, bad, budgets, nxt, 0, 0, 39)        # 40 moves may be needed, and there is room for 39
    assert exp[2].tolist() == [-1, -1, -1, -1, -1, 100, 100, 10]
    exp = _plan(w, pos, table, bad, budgets, np.array([-2 ** 31] * 8), 2 ** 31 - 1, 2 ** 31 - 1, 40)   # everything protected


# --- moves ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hkv,P,most", [(1, 1, 32, 1), (3, 2, 64, 50), (40, 8, 32, 6), (2, 3, 128, 700)])
def test_move(B, Hkv, P, most, D):
    rng = np.random.default_rng(B * 7 + most)
    pages = -(-2 * B * most // P) + 1
    cache = rng.integers(0, 256, (pages, Hkv, P // 32, 36 * D)).astype(np.uint8)
    moves = np.stack([rng.permutation(pages * P)[: 2 * B * most].reshape(B, most, 2) for _ in range(Hkv)], 1)
    counts = rng.integers(0, most + 1, (B, Hkv))
    counts[0, 0] = most
    w, pos = np.float32(rng.standard_normal((pages, Hkv, P))), rng.integers(0, 999, (pages, Hkv, P))
    for has_w, has_p in ((True, True), (False, True), (True, False), (False, False)):
        t, tw, tp = torch.from_numpy(cache).to(DEV), f32(w) if has_w else None, i32(pos) if has_p else None
        sv.spec_kv_move_q4(t, i32(moves), i32(counts), weights=tw, positions=tp)
        ec, ew, ep = ref.move(cache, w, pos, moves, counts)
        np.testing.assert_array_equal(t.cpu().numpy(), ec)
        if has_w:
            np.testing.assert_array_equal(tw.cpu().numpy(), ew)
        if has_p:
            np.testing.assert_array_equal(tp.cpu().numpy(), ep)


def test_move_leaves_out_bad_slots_and_counts():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (3, 2, 1, 36 * 64)).astype(np.uint8)
    moves = np.array([[[[1, 2], [96, 3], [-1, 4], [5, 96], [6, -2], [2 ** 31 - 1, 7]], [[9, 9], [10, 11], [40, 41], [90, 12], [0, 95], [13, 14]]]])
    for counts in ([[6, 6]], [[-3, 100]], [[0, 2]]):
        t = torch.from_numpy(cache).to(DEV)
        sv.spec_kv_move_q4(t, i32(moves), i32(counts))
        np.testing.assert_array_equal(t.cpu().numpy(), ref.move(cache, None, None, moves, np.array(counts))[0])


# --- pages ----------------------------------------------------------------------------
@pytest.mark.parametrize("B,P,W", [(1, 32, 4), (7, 16, 10), (513, 32, 6), (1300, 64, 3), (20, 1, 900)])
def test_trim(B, P, W):
    rng = np.random.default_rng(B + P)
    held = rng.integers(0, W + 1, B)
    tokens = rng.integers(0, W * P + 1, B)
    F = int(held.sum()) + 5
    table = np.full((B, W), -1)
    ids = rng.permutation(F)
    at = 0
    for b in range(B):
        table[b, : held[b]] = ids[at: at + held[b]]
        at += held[b]
    ring, state = rng.integers(0, F, F), np.array([int(rng.integers(0, F)), F - at])
    if B > 5:
        tokens[1], held[2], held[3] = -4, -1, W + 1
    for st in (state, np.array([state[0], F]), np.array([state[0], F - 3]), np.array([F, 1]), np.array([0, -1])):
        t_ring = i32(ring)
        got = sv.spec_page_trim(i32(tokens), i32(held), t_ring, i32(st), i32(table), P)
        for name, g, e in zip(("held", "state", "status", "ring"), [*got, t_ring], ref.page_trim(tokens, held, ring, st, table, P)):
            np.testing.assert_array_equal(g.cpu().numpy(), e, err_msg=name)


def test_trim_of_no_sequences():
    z = torch.zeros(0, dtype=I32, device=DEV)
    held, state, status = sv.spec_page_trim(z, z, i32([1, 2, 3]), i32([2, 1]), torch.zeros(0, 4, dtype=I32, device=DEV), 32)
    assert state.tolist() == [2, 1] and held.numel() == status.numel() == 0


# --- together ---------------------------------------------------------------------------
def test_steps_of_a_loop_that_keeps_to_a_budget():
    """Prompts, then steps of page map -> attention -> verification -> log probabilities ->
    commit -> weights -> plan -> moves -> trim, each against its reference with the library's own
    results in between; every head ends up with the same tokens' entries as its positions say, and
    every page comes back."""
    rng = np.random.default_rng(5)
    B, K, Hkv, G, D, P, V, budget = 4, 3, 2, 2, 64, 32, 300, 64
    F, W = 60, 8
    prompts = np.array([150, 40, 64, 200])
    cache = sv.q4_cache(F, Hkv, P, D, DEV)
    weights, positions = torch.full((F, Hkv, P), 1e9, device=DEV), torch.full((F, Hkv, P), -1, dtype=I32, device=DEV)
    table, ring = i32(np.full((B, W), -1)), i32(rng.permutation(F))
    state, held, lengths = i32([50, F]), i32(np.zeros(B)), i32(np.zeros(B))
    entries = {}   # (sequence, position) -> key and value of all heads
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s) * 0.3).to(torch.bfloat16)  # noqa: E731
    nxt = np.zeros(B, np.int64)

    def commit(q, lse, k, v, count):
        nonlocal lengths, held, state
        n = count.cpu().numpy()
        for b in range(B):
            for j in range(n[b]):
                entries[b, nxt[b] + j] = k[b, j], v[b, j]
        new = sv.spec_kv_commit_q4(cache, table, lengths, k.to(DEV), v.to(DEV), count)
        assert (new >= 0).all()
        before, pos_before = weights.cpu().numpy(), positions.cpu().numpy()
        sv.spec_kv_weigh_q4(q, lse, cache, table, lengths, weights, count=count, positions=positions, first_positions=i32(nxt), decay=0.95)
        ew, ep, tol = ref.weigh(f64(q), lse.cpu().numpy(), cache.cpu().numpy(), table.cpu().numpy(), lengths.cpu().numpy(), before, pos_before, n,
                                None, nxt, D ** -0.5, float(np.float32(0.95)), 0, before.astype(np.float64))
        assert (np.abs(f64(weights) - ew) <= tol).all()
        np.testing.assert_array_equal(positions.cpu().numpy(), ep)
        nxt[:] += n
        # down to the budget
        args = (weights.cpu().numpy(), positions.cpu().numpy(), table.cpu().numpy(), new.cpu().numpy())
        moves = torch.full((B, Hkv, 64, 2), -1, dtype=I32, device=DEV)
        exp = ref.evict_plan(*args, np.full(B, budget), nxt, 2, 8, moves.cpu().numpy())
        _, counts, cut = sv.spec_kv_evict_plan(weights, positions, table, new, i32(np.full(B, budget)), i32(nxt), sinks=2, recent=8, moves=moves)
        for g, e in zip((moves, counts, cut), exp):
            np.testing.assert_array_equal(g.cpu().numpy(), e)
        sv.spec_kv_move_q4(cache, moves, counts, weights=weights, positions=positions)
        held, state, st = sv.spec_page_trim(cut, held, ring, state, table, P)
        assert not st.any()
        lengths = cut

    def look():
        """Every entry is its position's, positions are distinct, sinks and recent ones are there."""
        c, t, p = cache.cpu().numpy(), table.cpu().numpy(), positions.cpu().numpy()
        for b in range(B):
            n = int(lengths[b])
            i = np.arange(n)
            slot = t[b, i // P].astype(np.int64) * P + i % P
            for h in range(Hkv):
                at = p[slot // P, h, slot % P]
                assert len(set(at)) == n and at.min() >= 0 and at.max() < nxt[b]
                assert {0, 1} <= set(at) and set(range(nxt[b] - min(8, n), nxt[b])) <= set(at)
                for s, a in list(zip(slot, at))[:: 7]:
                    one = np.zeros((1, Hkv, 1, 36 * D), np.uint8)
                    k, v = entries[b, a]
                    sref.q4_put(one, 0, h, f64(k[h]), f64(v[h]), 0, 0)
                    for x, y in zip(sref.q4_split(one[0, h, 0], D), sref.q4_split(c[s // P, h, s % P // 32], D)):
                        np.testing.assert_array_equal(x[0], y[s % 32])

    # the prompts, as one chunk that the batch pads
    N = int(prompts.max())
    q, k, v = bf(B, N, Hkv * G, D).to(DEV), bf(B, N, Hkv, D), bf(B, N, Hkv, D)
    *_, held, state, st = sv.spec_page_map(lengths, i32(prompts), held, ring, state, table, P, int(prompts.sum()))
    assert not st.any()
    _, lse = sv.spec_attend_q4(q, cache, table, lengths, k_new=k.to(DEV), v_new=v.to(DEV))
    commit(q, lse, k, v, i32(prompts))
    look()
    head = torch.randn(G * Hkv * D, V, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    for step in range(4):
        q, k, v = bf(B, K + 1, Hkv * G, D).to(DEV), bf(B, K + 1, Hkv, D), bf(B, K + 1, Hkv, D)
        *_, held, state, st = sv.spec_page_map(lengths, i32(np.full(B, K + 1)), held, ring, state, table, P, B * (K + 1))
        assert not st.any()
        out, lse = sv.spec_attend_q4(q, cache, table, lengths, k_new=k.to(DEV), v_new=v.to(DEV))
        logits = (out.double().cpu().reshape(B, K + 1, -1) @ head).to(torch.float32).to(DEV)
        drafts = rng.integers(0, V, (B, K))
        best = logits.argmax(-1).cpu().numpy()
        drafts[:, 0], drafts[:2, 1] = best[:, 0], best[:2, 1]
        tokens, n = sv.spec_verify_greedy(logits, i32(drafts))
        got = _check_logprobs(logits, tokens.cpu().numpy(), 1.0, None, 2)
        assert torch.equal(got[3][..., 0], tokens)
        commit(q, lse, k, v, n + 1)
        look()
    assert lengths.tolist() == np.minimum(nxt, budget).tolist()
    *_, held, state, st = sv.spec_page_map(lengths, i32(np.full(B, -1)), held, ring, state, table, P, 0)
    assert int(state[1]) == F and sorted(ring.cpu().tolist()) == list(range(F))


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros(2, 3, 10, device=DEV)
    with pytest.raises(TypeError):
        sv.spec_token_logprobs(x, torch.zeros(2, 3, dtype=torch.int64, device=DEV))
    with pytest.raises(sv.SpecError):
        sv.spec_token_logprobs(x, i32(np.zeros((2, 4))))
    with pytest.raises(ValueError, match="dimensions"):
        sv.spec_token_logprobs(x, i32(np.zeros((2, 3))), path=i32([0, 1]))
    with pytest.raises(ValueError, match="shape"):
        sv.spec_token_logprobs(x, i32(np.zeros((2, 3))), entropy=torch.zeros(2, 2, device=DEV))
    w, z = torch.zeros(4, 1, 32, device=DEV), i32([0])
    with pytest.raises(ValueError, match="max_moves"):
        sv.spec_kv_evict_plan(w, w.to(I32), i32([[0]]), z, z, z)
    with pytest.raises(ValueError, match="contiguous"):
        sv.spec_kv_evict_plan(w.expand(4, 2, 32), w.to(I32), i32([[0]]), z, z, z, max_moves=3)
    cache = sv.q4_cache(4, 1, 32, 64, DEV)
    with pytest.raises(ValueError, match="shape"):
        sv.spec_kv_move_q4(cache, i32(np.zeros((1, 2, 3, 2))), i32([[0]]))
    with pytest.raises(ValueError, match="shape"):
        sv.spec_kv_weigh_q4(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 1, 1, device=DEV), cache, i32([[0]]), z, w[:2])
    with pytest.raises(ValueError, match="must be on"):
        sv.spec_page_trim(z, z.cpu(), z, i32([0, 0]), i32([[0]]), 32)
