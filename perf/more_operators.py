"""What the steps after a verification cost: their cases, plain forms and definitions in 64 bits.

The operators: log probabilities, ranks, entropies and top alternatives of the tokens that a verification
emitted (spec_token_logprobs); the weight that the committed rows gave to each cached token, added up from
step to step (spec_kv_weigh_q4); which tokens of a head leave the cache by it (spec_kv_evict_plan); the
entries that fill their places (spec_kv_move_q4); and the pages that are free then (spec_page_trim).

The cache is [pages, kv heads, page_tokens / 32, 36 * D] bytes.  A block of 32 tokens holds, in this
order, the tokens' key codes (D / 2 bytes each, element 2i in the low half of byte i), their value
codes, their key scales (D / 16 e4m3 bytes each) and their value scales; an element is
e2m1(code) * e4m3(scale of its 16 elements) * 2^shift.  Weights (f32) and positions (int32) are
[pages, kv heads, page_tokens].
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FAR = 2.0 ** 100   # a logit of this size or more counts as an infinity


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's next token, five alternatives: latency counts
        {"name": "logprobs_one", "kind": "logprobs", "B": 1, "M": 1, "V": 128256, "dtype": "bf16", "T": 1.0, "top": 5, "tree": 0, "mask": False},
        # the headline batch: what chains of K = 5 drafts emitted, 20 alternatives each
        {"name": "logprobs_step", "kind": "logprobs", "B": 256, "M": 6, "V": 128256, "dtype": "bf16", "T": 0.7, "top": 20, "tree": 0, "mask": False},
        # f32 logits of trees of 64 nodes under a grammar, rows that no 16-byte vector divides
        {"name": "logprobs_tree", "kind": "logprobs", "B": 64, "M": 5, "V": 32003, "dtype": "f32", "T": 1.0, "top": 8, "tree": 64, "mask": True},
        # plain decoding of one short request
        {"name": "weigh_token", "kind": "weigh", "B": 1, "N": 1, "G": 4, "Hkv": 8, "D": 128, "P": 32, "ctx": 777, "form": "chain", "decay": 1.0, "shift": 0},
        # the headline batch: the accepted tokens of chains of K = 5 drafts
        {"name": "weigh_chain", "kind": "weigh", "B": 256, "N": 6, "G": 4, "Hkv": 8, "D": 128, "P": 64, "ctx": 2048, "form": "chain", "decay": 0.99, "shift": 0},
        # a prompt's next 1024 tokens behind 8k cached ones
        {"name": "weigh_chunk", "kind": "weigh", "B": 2, "N": 1024, "G": 8, "Hkv": 2, "D": 64, "P": 64, "ctx": 8192, "form": "chunk", "decay": 1.0, "shift": 0},
        # one step of 256 sequences that are held at 2,048 tokens
        {"name": "plan_step", "kind": "plan", "B": 256, "Hkv": 8, "P": 64, "budget": 2048, "ctx": 2048, "spread": False, "sinks": 4, "recent": 64},
        # prompts of 8k to 57k tokens cut down to 4,096
        {"name": "plan_prompts", "kind": "plan", "B": 8, "Hkv": 8, "P": 128, "budget": 4096, "ctx": 32768, "spread": True, "sinks": 4, "recent": 256},
        # what the step's plan moves (one layer)
        {"name": "move_step", "kind": "move", "B": 256, "Hkv": 8, "D": 128, "P": 64, "budget": 2048, "ctx": 2048, "spread": False},
        # what the prompts' plan moves (one layer)
        {"name": "move_prompts", "kind": "move", "B": 8, "Hkv": 8, "D": 128, "P": 128, "budget": 4096, "ctx": 32768, "spread": True},
        # a step after which some of 256 sequences need a page less
        {"name": "trim_step", "kind": "trim", "B": 256, "P": 32, "budget": 2048, "ctx": 2048, "spread": False},
        # the pages of 64 prompts of 4k to 28k tokens cut down to 2,048
        {"name": "trim_prompts", "kind": "trim", "B": 64, "P": 32, "budget": 2048, "ctx": 16384, "spread": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs", "logprobs", "weigh", "weigh", "weigh", "plan", "plan", "move", "trim"])
    if kind == "logprobs":
        V, tree = rng.choice([128256, 151936, 32000, _log(rng, 100, 128000)]), rng.choice([0, 0, rng.randint(2, 64)])
        M, dtype = rng.randint(1, min(8, tree)) if tree else rng.randint(1, 32), rng.choice(["bf16", "f32"])
        B = max(1, min(_log(rng, 1, 256), 360_000_000 // (V * (tree or M) * (2 if dtype == "bf16" else 4))))
        return {"kind": kind, "B": B, "M": M, "V": V, "dtype": dtype, "T": rng.choice([0.6, 0.7, 1.0, 1.3]),
                "top": rng.choice([0, 1, 5, 20, rng.randint(0, 32)]), "tree": tree, "mask": rng.random() < 0.3}
    if kind == "weigh":
        form = rng.choice(["chain", "chain", "tree", "chunk"])
        N = {"chain": rng.randint(1, 16), "tree": _log(rng, 8, 256), "chunk": _log(rng, 32, 1024)}[form]
        c = {"kind": kind, "B": _log(rng, 1, 256), "N": N, "G": rng.choice([1, 2, 3, 4, 8]), "Hkv": rng.choice([1, 2, 4, 8]),
             "D": rng.choice([64, 128]), "P": rng.choice([32, 64, 128]), "ctx": _log(rng, 1, 65536), "form": form,
             "decay": rng.choice([1.0, 0.99, 0.9]), "shift": rng.randint(-2, 2)}
        top = work({"kind": kind, "B": 2, "N": 1024, "G": 8, "Hkv": 2, "D": 64, "P": 64, "ctx": 8192, "form": "chunk"})["flops"]
        while (work(c)["flops"] > top or work(c)["bytes"] > 3e8) and c["ctx"] > 1:
            c["ctx"] = c["ctx"] * 2 // 3
        while (work(c)["flops"] > top or work(c)["bytes"] > 3e8) and c["B"] > 1:
            c["B"] = c["B"] * 2 // 3
        return c
    budget = _log(rng, 16, 8192)
    spread = rng.random() < 0.5
    ctx = _log(rng, 1, 65536) if spread else budget
    c = {"kind": kind, "B": max(1, min(_log(rng, 1, 256), 600_000 // ctx)), "P": rng.choice([32, 64, 128]), "budget": budget, "ctx": ctx, "spread": spread}
    if kind == "trim":
        return c
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    if kind == "move":
        return {**c, "D": rng.choice([64, 128])}
    return {**c, "sinks": rng.choice([0, 4]), "recent": rng.choice([0, min(64, budget // 2), budget // 4])}


def _ragged(mean, B):
    """B lengths around `mean`, from a quarter to seven quarters of it; the same ones for every seed."""
    if B == 1:
        return [max(1, mean)]
    return [max(1, int(mean * (0.25 + 1.5 * i / (B - 1)))) for i in range(B)]


def _accepted(B, N):
    """How many of N rows of B chains count (alpha = 0.75), the same ones for every seed."""
    got = []
    for i in range(B):
        u, n = (i + 0.5) / B, 0
        while n < N and u < 0.75 ** (n + 1):
            n += 1
        got.append(n)
    return got


def _emitted(c):
    """Tokens that a verification emitted for each sequence: the accepted drafts and one more."""
    return [n + 1 for n in _accepted(c["B"], c["M"] - 1)]


def _committed(c):
    """Rows that were committed for each sequence: all of a chunk, else the root and what was accepted."""
    if c["form"] == "chunk":
        return [c["N"]] * c["B"]
    return [n + 1 for n in _accepted(c["B"], _path_width(c) - 1)]


def _path_width(c):
    return min(c["N"], 8) if c["form"] == "tree" else c["N"]


def _evict_lengths(c):
    """Cached tokens of each sequence: its budget and up to 6 more in the steady state, a prompt's otherwise."""
    return _ragged(c["ctx"], c["B"]) if c["spread"] else [c["ctx"] + i % 7 for i in range(c["B"])]


def _most_moves(c):
    return max([1] + [min(c["budget"], n - c["budget"]) for n in _evict_lengths(c)])


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output written once."""
    c, kind = case, case["kind"]
    if kind == "logprobs":
        rows, e = sum(_emitted(c)), 2 if c["dtype"] == "bf16" else 4
        places = c["B"] * c["M"]
        # an exponential, a sum and a product by an element
        return {"bytes": rows * c["V"] * e + places * (4 + 12 + 8 * c["top"] + (4 if c["tree"] else 0)), "flops": 4 * rows * c["V"]}
    if kind == "weigh":
        D, Hkv, G = c["D"], c["Hkv"], c["G"]
        old, new = _ragged(c["ctx"], c["B"]), _committed(c)
        cached = sum(old) + sum(new)
        pairs = sum(L * n + n * (n + 1) // 2 for L, n in zip(old, new))
        data = cached * Hkv * (9 * D // 16 + 8) + sum(new) * Hkv * (G * (2 * D + 4) + 4) + 4 * cached // c["P"]
        return {"bytes": data, "flops": (2 * D + 4) * Hkv * G * pairs}
    lens = _evict_lengths(c)
    over = [max(0, n - c["budget"]) for n in lens]
    if kind == "trim":
        pages = sum(-(-n // c["P"]) - -(-min(n, c["budget"]) // c["P"]) for n in lens)
        return {"bytes": 8 * pages + 16 * c["B"], "flops": 0}
    # a share of budget / n of the tokens stays, wherever they are: so many of those past the budget move
    moves = sum(int(x * c["budget"] / n) for x, n in zip(over, lens)) * c["Hkv"]
    if kind == "plan":
        read = sum(n for n, x in zip(lens, over) if x) * c["Hkv"]
        return {"bytes": 8 * read + 8 * moves + 4 * c["B"] * (c["Hkv"] + 4), "flops": 0}
    return {"bytes": moves * (8 + 2 * (9 * c["D"] // 8 + 8)), "flops": 0}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(g, lengths, P):
    """A block table over shuffled pages for the sequences' tokens, and the number of pages."""
    need = (lengths.long() + P - 1) // P
    wide = max(1, int(need.max()))
    pages = int(need.sum()) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    first = torch.cumsum(need, 0) - need
    at = first[:, None] + torch.arange(wide, device=DEV)[None]
    have = torch.arange(wide, device=DEV)[None] < need[:, None]
    return torch.where(have, ids[at.clamp(max=pages - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), pages


def _entry_blocks(g, blocks, D, shift):
    """Blocks of the cache: keys as trained models have them (a few channels of larger size), quantised."""
    some = min(blocks, 8192)
    half = []
    for _ in range(2):
        wide = torch.where(_rand(g, D) < 0.06, 4.0, 1.0)
        x = (_randn(g, some, 32, D) * wide).unflatten(-1, (-1, 16))
        sc = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        y = x / sc.float().clamp(min=2.0 ** -9)[..., None]
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        code = (torch.bucketize(y.abs().contiguous(), edges) + 8 * (y < 0)).flatten(-2).to(torch.uint8)
        half.append((code[..., ::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)))
    one = torch.cat([half[0][0].flatten(1), half[1][0].flatten(1), half[0][1].flatten(1), half[1][1].flatten(1)], 1)
    return one.repeat(-(-blocks // some), 1)[:blocks]


def _prepare_logprobs(c, g):
    B, M, V, R = c["B"], c["M"], c["V"], c["tree"] or c["M"]
    s = {"case": c, "logits": (_randn(g, B, R, V) * 2.5).to(DTYPES[c["dtype"]]), "path": None}
    if c["mask"]:  # half of the sequences may take one token in 64
        tight = (torch.arange(B, device=DEV) % 2 == 0)[:, None, None] & (_rand(g, B, 1, V) > 1 / 64)
        tight[..., 0] = False
        s["logits"].masked_fill_(tight, -math.inf)
    emitted = _i32(_emitted(c))[torch.randperm(B, generator=g, device=DEV)]
    row = torch.arange(M, device=DEV).expand(B, M)
    if c["tree"]:
        nodes = torch.sort(torch.rand(B, R - 1, generator=g, device=DEV).argsort(-1)[:, : M - 1] + 1, -1).values if M > 1 else row[:, :0]
        s["path"] = torch.where(torch.arange(M - 1, device=DEV) < emitted[:, None] - 1, nodes, -1).int().contiguous() if M > 1 else None
        row = torch.cat([row[:, :1], nodes], 1)
    tokens = torch.empty(B, M, dtype=torch.int32, device=DEV)
    for b in range(B):  # drawn from the rows' own distributions
        x = s["logits"][b, row[b]].float() / c["T"]
        tokens[b] = (x - torch.log(-torch.log(_rand(g, M, V).clamp(1e-9, 1 - 1e-7)))).argmax(-1)
    s["tokens"] = torch.where(torch.arange(M, device=DEV) < emitted[:, None], tokens, -1)
    return s


def _prepare_weigh(c, g):
    B, N, G, Hkv, D, P = (c[k] for k in ("B", "N", "G", "Hkv", "D", "P"))
    s = {"case": c, "scale": D ** -0.5}
    mix = torch.randperm(B, generator=g, device=DEV)
    s["lengths"], new = _i32(_ragged(c["ctx"], B))[mix], _i32(_committed(c))
    s["count"] = None if c["form"] == "chunk" else new[torch.randperm(B, generator=g, device=DEV)]
    s["table"], pages = _tables(g, s["lengths"] + _path_width(c), P)
    s["cache"] = _entry_blocks(g, pages * Hkv * (P // 32), D, c["shift"]).view(pages, Hkv, P // 32, 36 * D)
    s["path"] = None
    if c["form"] == "tree":
        W = _path_width(c)
        nodes = torch.sort(torch.rand(B, N - 1, generator=g, device=DEV).argsort(-1)[:, : W - 1] + 1, -1).values
        s["path"] = torch.cat([torch.zeros(B, 1, dtype=torch.long, device=DEV), nodes], 1).int().contiguous()
    s["q"] = (_randn(g, B, N, Hkv * G, D) * 1.5).to(torch.bfloat16)
    s["lse"] = torch.zeros(B, N, Hkv * G, device=DEV)
    score, see, rows = _scores(s)
    lse = torch.logsumexp(score.masked_fill_(~see, -math.inf), -1).view(B, Hkv, -1, G).permute(0, 2, 1, 3).reshape(B, -1, Hkv * G)
    s["lse"].scatter_(1, rows[..., None].expand(-1, -1, Hkv * G), torch.where(torch.isfinite(lse), lse, 0.0))
    del score, see
    s["weights"] = torch.exp(_randn(g, pages, Hkv, P))
    s["new_weights"] = torch.zeros(pages, Hkv, P, device=DEV)
    s["positions"] = torch.randint(0, 1 << 20, (pages, Hkv, P), generator=g, device=DEV, dtype=torch.int32)
    s["first"] = s["lengths"] + torch.randint(0, 1000, (B,), generator=g, device=DEV, dtype=torch.int32)
    return s


def _prepare_evict(c, g):
    """What a cache looks like that has been cut before: the tokens' positions lie in no order."""
    B, Hkv, P = c["B"], c["Hkv"], c["P"]
    lens = _evict_lengths(c)
    s = {"case": c, "lengths": _i32(lens)[torch.randperm(B, generator=g, device=DEV)]}
    s["table"], pages = _tables(g, s["lengths"], P)
    s["budgets"] = torch.full((B,), c["budget"], dtype=torch.int32, device=DEV)
    wide = s["table"].shape[1] * P
    past = max(1, max(lens) // 8)
    s["next"] = s["lengths"] + past
    s["weights"] = torch.exp(2.0 * _randn(g, pages, Hkv, P)) * (_rand(g, pages, Hkv, P) > 0.02)
    s["positions"] = torch.zeros(pages, Hkv, P, dtype=torch.int32, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        i = torch.arange(n, device=DEV)
        page, at = s["table"][b, i // P].long(), i % P
        pos = _rand(g, Hkv, n + past).argsort(-1)[:, :n].int()
        s["positions"][page[None], torch.arange(Hkv, device=DEV)[:, None], at[None]] = pos
    s["moves"] = torch.full((B, Hkv, _most_moves(c), 2), -1, dtype=torch.int32, device=DEV)
    s["wide"] = wide
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)
    c, kind = case, case["kind"]
    if kind == "logprobs":
        return _prepare_logprobs(c, g)
    if kind == "weigh":
        return _prepare_weigh(c, g)
    if kind == "plan":
        return _prepare_evict(c, g)
    if kind == "move":
        s = _prepare_evict({**c, "sinks": 0, "recent": 0}, g)
        s["counts"] = _plain_plan(s)["counts"]
        pages, Hkv, P = s["weights"].shape
        s["cache"] = _entry_blocks(g, pages * Hkv * (P // 32), c["D"], 0).view(pages, Hkv, P // 32, 36 * c["D"])
        return s
    B, P = c["B"], c["P"]
    lens = _i32(_evict_lengths(c))[torch.randperm(B, generator=g, device=DEV)]
    s = {"case": c, "tokens": lens.clamp(max=c["budget"]), "held": ((lens + P - 1) // P).int()}
    s["table"], pages = _tables(g, lens, P)
    used = int(s["held"].sum())
    s["ring"] = torch.randint(0, pages, (pages,), generator=g, device=DEV, dtype=torch.int32)
    s["ring_state"] = _i32([pages // 3, pages - used])
    return s


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if own:
        return _OWN[kind](s)
    return _PLAIN[kind](s)


def _own_logprobs(s):
    import speculative_decoding_verification_52_gb300 as sv
    c = s["case"]
    lp, entropy, ranks, top_tokens, top_lp = sv.spec_token_logprobs(s["logits"], s["tokens"], c["T"], path=s["path"], top_n=c["top"])
    return {"logprobs": lp, "entropy": entropy, "ranks": ranks, "top_tokens": top_tokens, "top_logprobs": top_lp}


def _own_weigh(s):
    import speculative_decoding_verification_52_gb300 as sv
    c = s["case"]
    sv.spec_kv_weigh_q4(s["q"], s["lse"], s["cache"], s["table"], s["lengths"], s["weights"], count=s["count"], path=s["path"],
                        positions=s["positions"], first_positions=s["first"], new_weights=s["new_weights"], scale=s["scale"],
                        decay=c["decay"], k_shift=c["shift"])
    return {"weights": s["new_weights"], "positions": s["positions"]}


def _own_plan(s):
    import speculative_decoding_verification_52_gb300 as sv
    c = s["case"]
    moves, counts, lengths = sv.spec_kv_evict_plan(s["weights"], s["positions"], s["table"], s["lengths"], s["budgets"], s["next"],
                                                   sinks=c["sinks"], recent=c["recent"], moves=s["moves"])
    return {"moves": moves, "counts": counts, "lengths": lengths}


def _own_move(s):
    import speculative_decoding_verification_52_gb300 as sv
    sv.spec_kv_move_q4(s["cache"], s["moves"], s["counts"], weights=s["weights"], positions=s["positions"])
    return {**_cache_parts(s["cache"], s["case"]["D"]), "weights": s["weights"], "positions": s["positions"]}


def _own_trim(s):
    import speculative_decoding_verification_52_gb300 as sv
    held, state, status = sv.spec_page_trim(s["tokens"], s["held"], s["ring"], s["ring_state"], s["table"], s["case"]["P"])
    return {"held": held, "ring_state": state, "status": status, "ring": s["ring"]}


_OWN = {"logprobs": _own_logprobs, "weigh": _own_weigh, "plan": _own_plan, "move": _own_move, "trim": _own_trim}


def _cache_parts(cache, D):
    return {"codes": cache[..., : 32 * D], "scales": cache[..., 32 * D:].view(torch.float8_e4m3fn)}


def _ordered(x):
    """Integers that compare as the f32 values x do."""
    i = (x + 0.0).view(torch.int32).long()
    return torch.where(i < 0, -(i & 0x7fffffff) - 1, i)


def _plain_logprobs(s):
    c = s["case"]
    B, M, V, n = c["B"], c["M"], c["V"], c["top"]
    tokens, x = s["tokens"].long(), s["logits"]
    if s["path"] is not None:
        rows = torch.cat([torch.zeros(B, 1, dtype=torch.long, device=DEV), s["path"].long()], 1)
        x = torch.gather(x, 1, rows.clamp(min=0)[..., None].expand(-1, -1, V))
    elif c["tree"]:
        x = x[:, :1]
    x = x.float()
    x = torch.where(x <= -FAR, -math.inf, x)
    there = tokens >= 0
    at = tokens.clamp(min=0)[..., None]
    xt = torch.gather(x, 2, at)
    z = x / c["T"]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    entropy = torch.log(total).squeeze(-1) - torch.where(e > 0, e * (z - top), 0.0).sum(-1) / total.squeeze(-1)
    del e
    logprobs = (xt / c["T"] - lse).squeeze(-1)
    v = torch.arange(V, device=DEV)
    ranks = 1 + ((x > xt) | ((x == xt) & (v < at))).sum(-1)
    best = torch.topk(_ordered(x) * 2 ** 32 + (2 ** 32 - 1 - v), min(n, V), -1).values
    top_tokens = 2 ** 32 - 1 - (best & (2 ** 32 - 1))
    top_lp = torch.gather(z, 2, top_tokens) - lse
    found = torch.isfinite(top_lp) & there[..., None]
    top_tokens = torch.where(found, top_tokens, -1)
    top_lp = torch.where(found, top_lp, -math.inf)
    more = n - top_tokens.shape[-1]
    if more:
        top_tokens, top_lp = torch.nn.functional.pad(top_tokens, (0, more), value=-1), torch.nn.functional.pad(top_lp, (0, more), value=-math.inf)
    return {"logprobs": torch.where(there, logprobs, 0.0), "entropy": torch.where(there, entropy, 0.0),
            "ranks": torch.where(there, ranks, 0).int(), "top_tokens": top_tokens.int(), "top_logprobs": top_lp}


def _values(codes, scales, shift):
    """f32 values of codes [..., D / 2] under scales [..., D / 16]."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (both & 7).float()
    mag = torch.where(m < 5, m * 0.5, torch.where(m < 6, 3.0, torch.where(m < 7, 4.0, 6.0)))
    mag = torch.where(both >= 8, -mag, mag)
    sc = scales.view(torch.float8_e4m3fn).float() * 2.0 ** shift
    return (mag.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2)


def _scores(s):
    """Scores [B, Hkv, rows * G, tokens] of the rows that may be committed, which of them count, and the rows' nodes."""
    c = s["case"]
    B, N, G, Hkv, D = (c[k] for k in ("B", "N", "G", "Hkv", "D"))
    blocks = s["cache"][s["table"].long().clamp(min=0)].permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, Hkv, blocks, 36 D]
    codes, scales = blocks[..., : 16 * D].unflatten(-1, (32, -1)).flatten(2, 3), blocks[..., 32 * D: 34 * D].unflatten(-1, (32, -1)).flatten(2, 3)
    rows = (torch.arange(N, device=DEV).expand(B, N) if s["path"] is None else s["path"]).long()
    n = rows.shape[1]
    q = torch.gather(s["q"], 1, rows[:, :, None, None].expand(-1, -1, Hkv * G, D)).float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D) * s["scale"]
    score = q @ _values(codes, scales, c["shift"]).transpose(-1, -2)
    i = torch.arange(n, device=DEV)
    count = torch.full((B,), n, device=DEV) if s["count"] is None else s["count"].long()
    see = (torch.arange(score.shape[-1], device=DEV) <= s["lengths"].long()[:, None, None] + i[:, None]) & (i < count[:, None])[..., None]
    return score, see[:, None].repeat_interleave(G, 2), rows


def _plain_weigh(s):
    c = s["case"]
    B, G, Hkv, P = c["B"], c["G"], c["Hkv"], c["P"]
    score, see, rows = _scores(s)
    n, L = rows.shape[1], score.shape[-1]
    lse = torch.gather(s["lse"], 1, rows[..., None].expand(-1, -1, Hkv * G)).view(B, n, Hkv, G).permute(0, 2, 1, 3).reshape(B, Hkv, n * G, 1)
    given = torch.where(see, torch.exp(score - lse), 0.0).sum(2)
    del score, see
    at = torch.arange(L, device=DEV)
    old = s["lengths"].long()[:, None]
    count = torch.full((B,), n, device=DEV) if s["count"] is None else s["count"].long()
    page = s["table"].long()[:, at // P]
    before = s["weights"][page.clamp(min=0)[:, None], torch.arange(Hkv, device=DEV)[:, None], at % P]
    got = torch.where((at < old)[:, None], c["decay"] * before, 0.0) + given
    b, i = torch.nonzero(at < old + count[:, None], as_tuple=True)
    heads = torch.arange(Hkv, device=DEV)
    s["new_weights"][page[b, i][:, None], heads, (i % P)[:, None]] = got[b, :, i]
    fresh = i >= old[b, 0]
    b, i = b[fresh], i[fresh]
    s["positions"][page[b, i][:, None], heads, (i % P)[:, None]] = (s["first"].long()[b] + i - old[b, 0]).int()[:, None]
    return {"weights": s["new_weights"], "positions": s["positions"]}


def _plain_plan(s):
    c = s["case"]
    B, Hkv, P, wide = c["B"], c["Hkv"], c["P"], s["wide"]
    sinks, recent = c.get("sinks", 0), c.get("recent", 0)
    at = torch.arange(wide, device=DEV)
    slot = s["table"].long()[:, at // P] * P + at % P
    where = (slot.clamp(min=0) // P)[:, None], torch.arange(Hkv, device=DEV)[:, None], at % P
    have = (at < s["lengths"][:, None])[:, None]
    pos = s["positions"][where]
    safe = (pos < sinks) | (pos >= s["next"][:, None, None] - recent)
    key = torch.where(safe, 2 ** 40, _ordered(s["weights"][where]))
    key = torch.where(have, key, -2 ** 40)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    keep_n = torch.minimum(s["lengths"], s["budgets"]).long()[:, None, None]
    kept = torch.zeros(B, Hkv, wide, dtype=torch.bool, device=DEV).scatter_(2, order, (at < keep_n).expand(B, Hkv, wide))
    hole, mover = ~kept & (at < keep_n), kept & (at >= keep_n)
    for part, mark in ((1, hole), (0, mover)):
        b, h, i = torch.nonzero(mark, as_tuple=True)
        s["moves"][b, h, (torch.cumsum(mark.long(), -1) - 1)[b, h, i], part] = slot[b, i].int()
    return {"moves": s["moves"], "counts": hole.sum(-1).int(), "lengths": keep_n.flatten().int()}


def _plain_move(s):
    c = s["case"]
    D, P = c["D"], c["P"]
    there = torch.arange(s["moves"].shape[2], device=DEV) < s["counts"][..., None]
    b, h, i = torch.nonzero(there, as_tuple=True)
    src, dst = s["moves"][b, h, i].long().unbind(-1)
    starts, widths = (0, 16 * D, 32 * D, 34 * D), (D // 2, D // 2, D // 16, D // 16)
    col = torch.cat([torch.arange(w, device=DEV) + a for a, w in zip(starts, widths)])
    each = torch.cat([torch.full((w,), w, device=DEV) for w in widths])
    byte = lambda slot: ((slot // P)[:, None], h[:, None], (slot % P // 32)[:, None], col + (slot % 32)[:, None] * each)  # noqa: E731
    s["cache"][byte(dst)] = s["cache"][byte(src)]
    for name in ("weights", "positions"):
        s[name][dst // P, h, dst % P] = s[name][src // P, h, src % P]
    return {**_cache_parts(s["cache"], D), "weights": s["weights"], "positions": s["positions"]}


def _plain_trim(s):
    P, ring = s["case"]["P"], s["ring"]
    held, need = s["held"].long(), (s["tokens"].long() + P - 1) // P
    head, free = s["ring_state"].long()
    given = (held - need).clamp(min=0)
    first = torch.cumsum(given, 0) - given
    entry = torch.arange(s["table"].shape[1], device=DEV)
    b, e = torch.nonzero((entry >= need[:, None]) & (entry < held[:, None]), as_tuple=True)
    ring[(head + free + first[b] + e - need[b]) % ring.numel()] = s["table"][b, e]
    return {"held": torch.minimum(held, need).int(), "ring_state": torch.stack([head, free + given.sum()]).int(),
            "status": torch.zeros_like(s["held"]), "ring": ring}


_PLAIN = {"logprobs": _plain_logprobs, "weigh": _plain_weigh, "plan": _plain_plan, "move": _plain_move, "trim": _plain_trim}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def _e4m3_table():
    """The 256 values of e4m3 (1 sign, 4 exponent bits of bias 7, 3 of mantissa; 0x7f and 0xff are NaN)."""
    t = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t.append((-1.0 if b & 128 else 1.0) * (math.nan if b & 127 == 127 else v))
    return torch.tensor(t, dtype=torch.float64, device=DEV)


def _exact_logprobs(c, s):
    B, M, n = c["B"], c["M"], c["top"]
    lp, entropy = (torch.zeros(B, M, dtype=torch.float64, device=DEV) for _ in range(2))
    best = torch.full((B, M, n), -math.inf, dtype=torch.float64, device=DEV)
    for b, tokens in enumerate(s["tokens"].tolist()):
        rows = list(range(M)) if not c["tree"] else [0] + (s["path"][b].tolist() if M > 1 else [])
        m = sum(t >= 0 for t in tokens)
        p = torch.log_softmax(s["logits"][b, rows[:m]].double() / c["T"], -1)
        lp[b, :m] = p[torch.arange(m, device=DEV), _i32(tokens[:m]).long()]
        entropy[b, :m] = -(p.exp() * p.masked_fill(p == -math.inf, 0.0)).sum(-1)
        wide = min(n, c["V"])
        best[b, :m, :wide] = p.topk(wide, -1).values
    return {"logprobs": lp, "entropy": entropy, "ranks": None, "top_tokens": None, "top_logprobs": best}


def _exact_weigh(c, s):
    N, G, Hkv, D, P = (c[k] for k in ("N", "G", "Hkv", "D", "P"))
    half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    half, e4m3 = torch.cat([half, -half]), _e4m3_table()
    got = s["new_weights"].double()
    counts = [_path_width(c)] * c["B"] if s["count"] is None else s["count"].tolist()
    for b, (old, n) in enumerate(zip(s["lengths"].tolist(), counts)):
        nodes = list(range(n)) if s["path"] is None else s["path"][b, :n].tolist()
        L = old + n
        ids = s["table"][b, : -(-L // P)].long()
        page = s["cache"][ids].transpose(0, 1).reshape(Hkv, -1, 36 * D)
        code = page[..., : 16 * D].reshape(Hkv, -1, D // 2)
        sc = e4m3[page[..., 32 * D: 34 * D].reshape(Hkv, -1, D // 16).int()].repeat_interleave(16, -1) * 2.0 ** c["shift"]
        k = (torch.stack([half[(code & 15).int()], half[(code >> 4).int()]], -1).flatten(-2) * sc)[:, :L]
        t = torch.arange(L, device=DEV)
        slot = ids[t // P] * P + t % P
        for h in range(Hkv):
            w = s["weights"][slot // P, h, slot % P].double() * c["decay"]
            w[old:] = 0.0
            z = torch.einsum("ngd,ld->ngl", s["q"][b, nodes, h * G:(h + 1) * G].double(), k[h]) * s["scale"]
            z -= s["lse"][b, nodes, h * G:(h + 1) * G].double()[..., None]
            late = t > old + torch.arange(n, device=DEV)[:, None]
            w += z.masked_fill_(late[:, None], -math.inf).exp_().sum((0, 1))
            got[slot // P, h, slot % P] = w
    return {"weights": got, "positions": None}


def exact(case, seed):
    c, kind = case, case["kind"]
    if kind in ("plan", "trim"):   # whole numbers alone
        return None
    s = prepare(case, seed)
    if kind == "logprobs":
        return _exact_logprobs(c, s)
    if kind == "weigh":
        return _exact_weigh(c, s)
    # what a move carries, value by value
    D, P, Hkv = c["D"], c["P"], c["Hkv"]
    flat = _e4m3_table()[s["cache"][..., 32 * D:].long()].view(*s["cache"].shape[:3], 2, 32, D // 16)
    weights = s["weights"].double()
    for b, counts in enumerate(s["counts"].tolist()):
        for h in range(Hkv):
            src, dst = s["moves"][b, h, : counts[h]].long().T
            flat[dst // P, h, dst % P // 32, :, dst % 32] = flat[src // P, h, src % P // 32, :, src % 32]
            weights[dst // P, h, dst % P] = weights[src // P, h, src % P]
    return {"codes": None, "scales": flat.flatten(3), "weights": weights, "positions": None}
