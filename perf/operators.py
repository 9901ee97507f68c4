"""What the serving operators around verification cost: their cases, plain forms and definitions in 64 bits.

The operators: block tables and slot maps of a paged cache (spec_page_map), the two ways into a
cache held in 4 bits (spec_kv_store_q4 for packed prompts, spec_kv_commit_q4 for accepted drafts),
the verification attention over that cache (spec_attend_q4), and penalties, biases and grammar masks
on the logits that are verified (spec_adjust_logits).

The cache is [pages, kv heads, page_tokens / 32, 36 * D] bytes.  A block of 32 tokens holds, in this
order, the tokens' key codes (D / 2 bytes each, element 2i in the low half of byte i), their value
codes, their key scales (D / 16 e4m3 bytes each) and their value scales; an element is
e2m1(code) * e4m3(scale of its 16 elements) * 2^shift.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # the page bookkeeping of one speculative step: 256 sequences, K = 5 drafts and the bonus token
        {"name": "map_step", "kind": "map", "B": 256, "tokens": 6, "P": 32, "ctx": 2048},
        # admission of 64 prompts of 0.5k to 16k tokens at once
        {"name": "map_prompts", "kind": "map", "B": 64, "tokens": 8192, "P": 64, "ctx": 0},
        # the keys and values of packed prompts enter the cache (one layer)
        {"name": "store_prompts", "kind": "store", "T": 32001, "B": 13, "Hkv": 8, "D": 128, "P": 64, "shift": 0},
        # the accepted drafts of one step (B = 256, K = 5) enter the cache (one layer)
        {"name": "commit_step", "kind": "commit", "B": 256, "N": 6, "Hkv": 8, "D": 128, "P": 32, "ctx": 512, "shift": -2},
        # plain decoding of one short request: latency counts
        {"name": "attend_token", "kind": "attend", "B": 1, "N": 1, "G": 4, "Hkv": 8, "D": 128, "P": 32, "ctx": 777, "tree": False, "shift": 0},
        # the headline batch: chains of K = 5 drafts behind the last token
        {"name": "attend_chain", "kind": "attend", "B": 256, "N": 6, "G": 4, "Hkv": 8, "D": 128, "P": 64, "ctx": 2048, "tree": False, "shift": 0},
        # few requests with long contexts, one token each
        {"name": "attend_long", "kind": "attend", "B": 4, "N": 1, "G": 8, "Hkv": 8, "D": 128, "P": 128, "ctx": 65536, "tree": False, "shift": -1},
        # candidate trees of 64 nodes
        {"name": "attend_tree", "kind": "attend", "B": 32, "N": 64, "G": 4, "Hkv": 8, "D": 128, "P": 64, "ctx": 4096, "tree": True, "shift": 0},
        # a prompt's next 1024 tokens behind 8k cached ones
        {"name": "attend_chunk", "kind": "attend", "B": 2, "N": 1024, "G": 8, "Hkv": 2, "D": 64, "P": 64, "ctx": 8192, "tree": False, "shift": 0},
        # one request, chain of 5 drafts, penalties only
        {"name": "adjust_one", "kind": "adjust", "B": 1, "R": 6, "V": 128256, "dtype": "bf16", "hist": 1500, "tree": False, "bias": 0, "mask": False},
        # the headline batch, everything on
        {"name": "adjust_chain", "kind": "adjust", "B": 256, "R": 6, "V": 128256, "dtype": "bf16", "hist": 2048, "tree": False, "bias": 64, "mask": True},
        # f32 logits of trees over a vocabulary whose rows no 16-byte vector divides
        {"name": "adjust_tree", "kind": "adjust", "B": 16, "R": 64, "V": 32003, "dtype": "f32", "hist": 4096, "tree": True, "bias": 300, "mask": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["map", "store", "commit", "attend", "attend", "attend", "adjust", "adjust"])
    if kind == "map":
        B = _log(rng, 1, 1024)
        return {"kind": kind, "B": B, "tokens": min(_log(rng, 1, 8192), max(1, 500000 // B)), "P": rng.choice([16, 32, 64, 128]),
                "ctx": rng.choice([0, _log(rng, 1, 4096)])}
    heads = {"Hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128]), "P": rng.choice([32, 64, 128])}
    if kind == "store":
        T = _log(rng, 1, 32000)
        return {"kind": kind, "T": T, "B": min(T, rng.randint(1, 32)), **heads, "shift": rng.randint(-4, 4)}
    if kind == "commit":
        return {"kind": kind, "B": _log(rng, 1, 256), "N": rng.randint(1, 32), **heads, "ctx": _log(rng, 1, 512), "shift": rng.randint(-4, 4)}
    if kind == "attend":
        B, N, G, ctx = _log(rng, 1, 256), _log(rng, 1, 1024), rng.choice([1, 2, 4, 8]), _log(rng, 1, 65536)
        c = {"kind": kind, "B": B, "N": N, "G": G, **heads, "ctx": ctx, "tree": rng.random() < 0.4, "shift": rng.randint(-2, 2)}
        top = work({"kind": "attend", "B": 32, "N": 64, "G": 4, "Hkv": 8, "D": 128, "P": 64, "ctx": 4096, "tree": True})["flops"]
        while (work(c)["flops"] > top or work(c)["bytes"] > 3e8) and c["ctx"] > 1:
            c["ctx"] = c["ctx"] * 2 // 3
        while (work(c)["flops"] > top or work(c)["bytes"] > 3e8) and c["B"] > 1:
            c["B"] = c["B"] * 2 // 3
        return c
    V, R = rng.choice([128256, 151936, 32000, _log(rng, 100, 128000)]), rng.randint(1, 64)
    B = max(1, min(_log(rng, 1, 256), 180_000_000 // (V * R)))
    return {"kind": kind, "B": B, "R": R, "V": V, "dtype": rng.choice(["bf16", "f32"]), "hist": _log(rng, 1, 8192),
            "tree": rng.random() < 0.4, "bias": rng.choice([0, rng.randint(1, 512)]), "mask": rng.random() < 0.6}


def _ragged(mean, B):
    """B lengths around `mean`, from a quarter to seven quarters of it; the same ones for every seed."""
    if B == 1:
        return [max(1, mean)]
    return [max(1, int(mean * (0.25 + 1.5 * i / (B - 1)))) for i in range(B)]


def _accepted(B, N):
    """Accepted counts of B chains of N - 1 drafts and the bonus' row (alpha = 0.75), the same ones for every seed."""
    got = []
    for i in range(B):
        u, n = (i + 0.5) / B, 0
        while n < N and u < 0.75 ** (n + 1):
            n += 1
        got.append(n)
    return got


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output written once."""
    c, kind = case, case["kind"]
    if kind == "map":
        T = sum(_ragged(c["tokens"], c["B"]))
        # a slot and a position a token, a taken page read and written, seven numbers a sequence
        return {"bytes": 8 * T + 8 * (T // c["P"] + c["B"]) + 28 * c["B"], "flops": 0}
    if kind in ("store", "commit"):
        T = c["T"] if kind == "store" else sum(_accepted(c["B"], c["N"]))
        return {"bytes": T * c["Hkv"] * (4 * c["D"] + 9 * c["D"] // 8) + 4 * T + 12 * c["B"], "flops": 0}
    if kind == "attend":
        B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
        cached, rows = sum(_ragged(c["ctx"], B)), N * c["G"]
        seen = N * min(N, 5) if c["tree"] else N * (N + 1) // 2
        data = cached * Hkv * 9 * D // 8 + B * N * Hkv * D * 4 + B * rows * Hkv * (4 * D + 4)
        data += 4 * cached // c["P"] + (B * N * 4 * -(-N // 32) if c["tree"] else 0)
        return {"bytes": data, "flops": 4 * D * Hkv * (cached * rows + B * c["G"] * seen)}
    B, R, V, e = c["B"], c["R"], c["V"], 2 if c["dtype"] == "bf16" else 4
    read = B * R * V * e
    if c["mask"]:  # half of the sequences allow one token in 64, the others all but one in 64
        read = read // 2 + B * R * 4 * -(-V // 32)
    return {"bytes": read + B * R * V * e + 4 * sum(_ragged(c["hist"], B)) + 8 * B * c["bias"], "flops": 0}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _shuffled(g, values):
    t = torch.tensor(values, dtype=torch.int32, device=DEV)
    return t[torch.randperm(len(values), generator=g, device=DEV)]


def _entries(g, *shape):
    """Keys or values: normal, with a few channels of larger size as trained models have them."""
    wide = torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.06, 4.0, 1.0)
    return (_randn(g, *shape) * wide).to(torch.bfloat16)


def _tables(g, lengths, P, extra):
    """A block table over shuffled pages with room for `extra` more tokens a sequence, and the number of pages."""
    need = (lengths.long() + extra + P - 1) // P
    wide = int(need.max())
    pages = int(need.sum()) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    first = torch.cumsum(need, 0) - need
    at = first[:, None] + torch.arange(wide, device=DEV)[None]
    have = torch.arange(wide, device=DEV)[None] < need[:, None]
    return torch.where(have, ids[at.clamp(max=pages - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), pages


def _tree(g, B, N):
    """Ancestor words of B random trees, node i's parent among the 8 before it, [B, N, ceil(N / 32)] int32."""
    see = torch.zeros(B, N, N, dtype=torch.bool, device=DEV)
    see[:, 0, 0] = True
    back = torch.randint(1, 9, (B, N), generator=g, device=DEV)
    rows = torch.arange(B, device=DEV)
    for i in range(1, N):
        see[:, i] = see[rows, (i - back[:, i]).clamp(min=0)]
        see[:, i, i] = True
    words = -(-N // 32)
    bits = torch.zeros(B, N, words * 32, dtype=torch.int64, device=DEV)
    bits[:, :, :N] = see.long()
    w = (bits.view(B, N, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    return (w - ((w >> 31) << 32)).int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)
    c, kind = case, case["kind"]
    s = {"case": c}
    if kind == "map":
        B, P = c["B"], c["P"]
        s["count"] = _shuffled(g, _ragged(c["tokens"], B))
        s["lengths"] = _shuffled(g, _ragged(c["ctx"], B)) if c["ctx"] else torch.zeros(B, dtype=torch.int32, device=DEV)
        s["T"] = sum(_ragged(c["tokens"], B)) + 5
        held = (s["lengths"] + P - 1) // P
        wide = int(((s["lengths"] + s["count"]).max() + P - 1) // P)
        total = int(held.sum()) + s["T"] // P + B + 7
        ids = torch.randperm(total, generator=g, device=DEV).int()
        first = torch.cumsum(held, 0) - held
        at = (first[:, None] + torch.arange(wide, device=DEV)).clamp(max=total - 1)
        s["table"] = torch.where(torch.arange(wide, device=DEV) < held[:, None], ids[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
        used = int(held.sum())
        s["held"], s["ring"] = held.int(), torch.roll(ids, total // 3).contiguous()
        s["ring_state"] = torch.tensor([(used + total // 3) % total, total - used], dtype=torch.int32, device=DEV)
        if B > 8:  # one request in 32 has ended: its pages go back
            s["count"] = torch.where(torch.rand(B, generator=g, device=DEV) < 1 / 32, torch.full_like(s["count"], -1), s["count"])
        return s
    if kind in ("store", "commit"):
        Hkv, D, P = c["Hkv"], c["D"], c["P"]
        if kind == "store":
            T = c["T"]
            pages = -(-T // P) + c["B"] + 2
            cut = sorted({int(x) for x in torch.randint(0, T + 1, (c["B"] - 1,), generator=g, device=DEV).tolist()} | {0, T})
            lengths = torch.tensor([b - a for a, b in zip(cut, cut[1:])], dtype=torch.int32, device=DEV)
            table, pages = _tables(g, lengths, P, 0)
            start = torch.repeat_interleave(torch.tensor(cut[:-1], device=DEV), lengths)
            seq = torch.repeat_interleave(torch.arange(len(lengths), device=DEV), lengths)
            pos = torch.arange(T, device=DEV) - start
            s["slots"] = (table[seq, pos // P].long() * P + pos % P).int()
            shape = (T, Hkv, D)
        else:
            B, N = c["B"], c["N"]
            s["lengths"] = _shuffled(g, _ragged(c["ctx"], B))
            s["table"], pages = _tables(g, s["lengths"], P, N)
            s["count"] = _shuffled(g, _accepted(B, N))
            s["new_lengths"] = torch.empty_like(s["lengths"])
            shape = (B, N, Hkv, D)
        s["k"], s["v"] = (_entries(g, *shape) * 2.0 ** c["shift"] for _ in range(2))
        s["cache"] = torch.randint(0, 100, (pages, Hkv, P // 32, 36 * D), generator=g, device=DEV, dtype=torch.uint8)
        return s
    if kind == "attend":
        B, N, G, Hkv, D, P = (c[k] for k in ("B", "N", "G", "Hkv", "D", "P"))
        s["lengths"] = _shuffled(g, _ragged(c["ctx"], B))
        s["table"], pages = _tables(g, s["lengths"], P, N)
        blocks = pages * Hkv * (P // 32)
        some = min(blocks, 8192)
        kv = [_q4(_entries(g, some, 32, D), c["shift"]) for _ in range(2)]
        one = torch.cat([kv[0][0].flatten(1), kv[1][0].flatten(1), kv[0][1].flatten(1), kv[1][1].flatten(1)], 1)
        s["cache"] = one.repeat(-(-blocks // some), 1)[:blocks].view(pages, Hkv, P // 32, 36 * D).contiguous()
        s["q"] = (_randn(g, B, N, G * Hkv, D) * 1.5).to(torch.bfloat16)
        s["k_new"], s["v_new"] = _entries(g, B, N, Hkv, D), _entries(g, B, N, Hkv, D)
        s["masks"] = _tree(g, B, N) if c["tree"] else None
        s["scale"] = D ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, N, G * Hkv, device=DEV)
        s["ws"] = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
        return s
    B, R, V, dt = c["B"], c["R"], c["V"], DTYPES[c["dtype"]]
    s["logits"] = (_randn(g, B, R, V) * 2.5).to(dt)
    s["out"] = torch.empty_like(s["logits"])
    s["hist_len"] = _shuffled(g, _ragged(c["hist"], B))
    s["prompt_len"] = (s["hist_len"] * torch.rand(B, generator=g, device=DEV)).int()
    wide = int(s["hist_len"].max())
    s["history"] = (V * torch.rand(B, wide, generator=g, device=DEV) ** 3).int().clamp(max=V - 1)  # some tokens are frequent
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=DEV)
    s["frequency"] = 0.5 * torch.rand(B, generator=g, device=DEV)
    s["presence"] = 0.5 * torch.rand(B, generator=g, device=DEV)
    s["nodes"] = (V * torch.rand(B, R, generator=g, device=DEV) ** 3).int().clamp(max=V - 1)
    s["masks"] = _tree(g, B, R) if c["tree"] else None
    s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
    if c["bias"]:
        M = min(c["bias"], V)
        first = _ints(g, 0, V, B, 1)
        s["bias_tokens"] = ((first + torch.arange(M, device=DEV) * max(1, V // M)) % V).int()
        s["bias_values"] = _randn(g, B, M) * 3
    if c["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (6, B, R, -(-V // 32)), generator=g, device=DEV, dtype=torch.int64).int()
        tight, loose = words[0], words[0]
        for w in words[1:]:
            tight, loose = tight & w, loose | w
        half = torch.randperm(B, generator=g, device=DEV) < B // 2
        s["allowed"] = torch.where(half[:, None, None], tight, loose).contiguous()
    return s


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    kind = s["case"]["kind"]
    if own:
        return _OWN[kind](s)
    return _PLAIN[kind](s)


def _own_map(s):
    import speculative_decoding_verification_52_gb300 as sv
    offsets, slots, positions, held, ring_state, status = sv.spec_page_map(
        s["lengths"], s["count"], s["held"], s["ring"], s["ring_state"], s["table"], s["case"]["P"], s["T"])
    return {"offsets": offsets, "slots": slots, "positions": positions, "held": held, "ring_state": ring_state,
            "status": status, "table": s["table"], "ring": s["ring"]}


def _cache_parts(cache, D):
    return {"codes": cache[..., : 32 * D], "scales": cache[..., 32 * D:].view(torch.float8_e4m3fn)}


def _own_store(s):
    import speculative_decoding_verification_52_gb300 as sv
    c = s["case"]
    sv.spec_kv_store_q4(s["k"], s["v"], s["slots"], s["cache"], k_shift=c["shift"], v_shift=c["shift"])
    return _cache_parts(s["cache"], c["D"])


def _own_commit(s):
    import speculative_decoding_verification_52_gb300 as sv
    c = s["case"]
    sv.spec_kv_commit_q4(s["cache"], s["table"], s["lengths"], s["k"], s["v"], s["count"], k_shift=c["shift"],
                         v_shift=c["shift"], new_lengths=s["new_lengths"])
    return {**_cache_parts(s["cache"], c["D"]), "new_lengths": s["new_lengths"]}


def _own_attend(s):
    import speculative_decoding_verification_52_gb300 as sv
    sh = s["case"]["shift"]
    return sv.spec_attend_q4(s["q"], s["cache"], s["table"], s["lengths"], k_new=s["k_new"], v_new=s["v_new"], masks=s["masks"],
                             scale=s["scale"], k_shift=sh, v_shift=sh, out=s["out"], lse=s["lse"], workspace_buf=s["ws"])


def _own_adjust(s):
    import speculative_decoding_verification_52_gb300 as sv
    return sv.spec_adjust_logits(
        s["logits"], out=s["out"], history=s["history"], prompt_lengths=s["prompt_len"], history_lengths=s["hist_len"],
        repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], node_tokens=s["nodes"], masks=s["masks"],
        bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], allowed=s["allowed"])


_OWN = {"map": _own_map, "store": _own_store, "commit": _own_commit, "attend": _own_attend, "adjust": _own_adjust}


def _plain_map(s):
    P, T, F = s["case"]["P"], s["T"], s["ring"].numel()
    n, L, held, table = s["count"].long(), s["lengths"].long(), s["held"].long(), s["table"]
    head, avail = s["ring_state"].long()
    wide = table.shape[1]
    places = n.clamp(min=0)
    ends = torch.cumsum(places, 0)
    ok = (L >= 0) & (held >= 0) & (held <= wide) & ((n < 0) | ((L + n <= wide * P) & (ends <= T)))
    take = torch.where(ok & (n >= 0), ((L + n + P - 1) // P - held).clamp(min=0), 0)
    put = torch.where(ok & (n < 0), held, 0)
    taken, given = torch.cumsum(take, 0), torch.cumsum(put, 0)
    short = ((take > 0) & (taken > avail)) | ((put > 0) & (avail + given > F))
    good = ok & ~short
    status = torch.where(ok, torch.where(short, -3, 0), -1).int()
    take, put = torch.where(short, 0, take), torch.where(short, 0, put)
    j = torch.arange(wide, device=DEV)
    new = (j >= held[:, None]) & (j < (held + take)[:, None])
    at = (head + (taken - take)[:, None] + j - held[:, None]) % F
    after = torch.where(new, s["ring"][at], table)
    back = torch.where(j < put[:, None], (head + avail + (given - put)[:, None] + j) % F, F)
    ring = torch.cat([s["ring"], s["ring"][:1]]).scatter(0, back.flatten(), table.flatten())[:F]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(ends, t, right=True)
    live = seq < n.numel()
    seq = seq.clamp(max=n.numel() - 1)
    pos = L[seq] + t - (ends - places)[seq]
    live = live & good[seq]
    page = after[seq, (pos // P).clamp(0, wide - 1)].long()
    live_page = live & (page >= 0) & (page < F)
    slots = torch.where(live_page, page * P + pos % P, -1).int()
    moved, released = take.sum(), put.sum()
    return {"offsets": torch.cat([ends.new_zeros(1), ends]).clamp(max=T).int(), "slots": slots,
            "positions": torch.where(live, pos, -1).int(),
            "held": torch.where(good & (n < 0), 0, held + take).int(),
            "ring_state": torch.stack([(head + moved) % F, avail - moved + released]).int(),
            "status": status, "table": after, "ring": ring}


def _e2m1(y):
    """The code of the e2m1 value nearest to y (to the even one between two), saturating at 6."""
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int()
            + (a > 5.0).int())
    return code + 8 * torch.signbit(y).int()


def _q4(x, shift):
    """Codes [..., D / 2] and scales [..., D / 16] (bytes) of x [..., D]."""
    y = x.float() * 2.0 ** -shift
    grp = y.unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(grp).all(-1)
    top = torch.where(bad, 0.0, grp.abs().amax(-1))
    scale = (top / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    div = scale.float()[..., None]
    code = _e2m1(torch.where((div > 0) & ~bad[..., None], grp / torch.where(div > 0, div, 1.0), 0.0)).flatten(-2)
    code = torch.where((div > 0).expand_as(grp).flatten(-2), code, 0)
    byte = torch.where(bad, torch.full_like(top, 127, dtype=torch.uint8), scale.view(torch.uint8))
    return (code[..., ::2] | (code[..., 1::2] << 4)).to(torch.uint8), byte


def _put(cache, slots, k, v, P, D, k_shift, v_shift):
    """The cache with entry i of k and v [T, Hkv, D] at slots[i]; a negative slot takes none."""
    pages, Hkv = cache.shape[:2]
    got = torch.cat([cache, cache[:1]])  # a page more takes what goes nowhere
    slots = torch.where(slots >= 0, slots.long(), pages * P)
    page, row = slots // P, slots % P
    at = 0
    for codes_or_scales in (0, 1):
        for x, sh in ((k, k_shift), (v, v_shift)):
            part = _q4(x, sh)[codes_or_scales]
            wide = part.shape[-1]
            col = at + (row % 32)[:, None] * wide + torch.arange(wide, device=DEV)
            got[page[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None], (row // 32)[:, None, None], col[:, None, :]] = part
            at += 32 * wide
    return got[:pages]


def _plain_store(s):
    c = s["case"]
    return _cache_parts(_put(s["cache"], s["slots"], s["k"], s["v"], c["P"], c["D"], c["shift"], c["shift"]), c["D"])


def _plain_commit(s):
    c = s["case"]
    P, N, L, n = c["P"], c["N"], s["lengths"].long(), s["count"].long()
    j = torch.arange(N, device=DEV)
    pos = L[:, None] + j
    slots = torch.where(j < n[:, None], torch.gather(s["table"].long(), 1, (pos // P).clamp(max=s["table"].shape[1] - 1)) * P + pos % P, -1)
    got = _put(s["cache"], slots.flatten(), s["k"].flatten(0, 1), s["v"].flatten(0, 1), P, c["D"], c["shift"], c["shift"])
    return {**_cache_parts(got, c["D"]), "new_lengths": (L + n.clamp(min=0)).int()}


def _values(codes, scales, shift):
    """f32 values of codes [..., D / 2] under scales [..., D / 16]."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (both & 7).float()
    mag = torch.where(m < 5, m * 0.5, torch.where(m < 6, 3.0, torch.where(m < 7, 4.0, 6.0)))
    mag = torch.where(both >= 8, -mag, mag)
    sc = scales.view(torch.float8_e4m3fn).float() * 2.0 ** shift
    return (mag.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2)


def _bits(words, n):
    return ((words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1).flatten(-2)[..., :n].bool()


def _plain_attend(s):
    c = s["case"]
    B, N, G, Hkv, D, P, sh = (c[k] for k in ("B", "N", "G", "Hkv", "D", "P", "shift"))
    pages = s["cache"][s["table"].long().clamp(min=0)]                      # [B, pages, Hkv, P / 32, 36 D]
    pages = pages.permute(0, 2, 1, 3, 4).flatten(2, 3)                      # [B, Hkv, blocks, 36 D]
    part = torch.split(pages, [16 * D, 16 * D, 2 * D, 2 * D], -1)
    part = [x.unflatten(-1, (32, -1)).flatten(2, 3) for x in part]          # [B, Hkv, L, ...]
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) * s["scale"]
    k_new, v_new = (s[x].float().permute(0, 2, 1, 3) for x in ("k_new", "v_new"))
    k = torch.cat([_values(part[0], part[2], sh), k_new], 2)
    score = q @ k.transpose(-1, -2)
    del k
    L = part[0].shape[2]
    node = _bits(s["masks"], N) if c["tree"] else torch.ones(N, N, dtype=torch.bool, device=DEV).tril().expand(B, N, N)
    node = node[:, None, :, None].expand(B, 1, N, G, N).reshape(B, 1, N * G, N)
    old = (torch.arange(L, device=DEV) < s["lengths"][:, None])[:, None, None]
    see = torch.cat([old.expand(B, 1, N * G, L), node], -1)
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.cat([torch.where(old.squeeze(2)[..., None], _values(part[1], part[3], sh), 0.0), v_new], 2)
    out = (p @ v) / total
    back = lambda x: x.view(B, Hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, -1)  # noqa: E731
    return back(out).to(torch.bfloat16), back(top + torch.log(total)).squeeze(-1)


def _plain_adjust(s):
    c = s["case"]
    B, R, V = c["B"], c["R"], c["V"]
    x = s["logits"].float()
    at = torch.arange(s["history"].shape[1], device=DEV)
    have = at < s["hist_len"][:, None]
    made = have & (at >= s["prompt_len"][:, None])
    seen = torch.zeros(B, V, device=DEV).scatter_add(1, s["history"].long(), have.float())
    count = torch.zeros(B, V, device=DEV).scatter_add(1, s["history"].long(), made.float())
    j = torch.arange(R, device=DEV)
    before = _bits(s["masks"], R) & (j > 0) if c["tree"] else (j[None] < j[:, None]).expand(B, R, R)
    drafts = torch.zeros(B, R, V, device=DEV).scatter_add(2, s["nodes"].long()[:, None].expand(B, R, R), before.float())
    count = count[:, None] + drafts
    seen = (seen[:, None] + drafts) > 0
    wide = lambda t: t[:, None, None]  # noqa: E731
    x = torch.where(seen, torch.where(x > 0, x / wide(s["repetition"]), x * wide(s["repetition"])), x)
    x = x - (wide(s["frequency"]) * count + torch.where(count > 0, wide(s["presence"]), 0.0))
    if s["bias_tokens"] is not None:
        x = x + torch.zeros(B, V, device=DEV).scatter_add(1, s["bias_tokens"].long(), s["bias_values"])[:, None]
    if s["allowed"] is not None:
        x = torch.where(_bits(s["allowed"], V), x, -math.inf)
    return x.to(s["logits"].dtype)


_PLAIN = {"map": _plain_map, "store": _plain_store, "commit": _plain_commit, "attend": _plain_attend, "adjust": _plain_adjust}


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


def _exact_scales(x, shift):
    """The e4m3 values of the groups' scales of x [..., D], by the nearest of all of them."""
    grid = _e4m3_table()[:127]
    top = (x.double().unflatten(-1, (-1, 16)).abs().amax(-1) * 2.0 ** -shift / 6.0).contiguous()
    hi = torch.searchsorted(grid, top).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - top, top - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])


def exact(case, seed):
    c, kind = case, case["kind"]
    if kind == "map":
        return None
    s = prepare(case, seed)
    if kind in ("store", "commit"):
        D, P = c["D"], c["P"]
        got = _e4m3_table()[s["cache"][..., 32 * D:].long()]
        if kind == "store":
            rows, slots = (s["k"], s["v"]), s["slots"].long()
        else:
            at = [(b, j) for b, n in enumerate(s["count"].tolist()) for j in range(n)]
            b, j = (torch.tensor([x[i] for x in at], device=DEV, dtype=torch.long) for i in range(2))
            pos = s["lengths"].long()[b] + j
            slots = s["table"].long()[b, pos // P] * P + pos % P
            rows = (s["k"][b, j], s["v"][b, j])
        for half, x in enumerate(rows):
            if not len(slots):
                break
            wide = D // 16
            col = 32 * wide * half + (slots % 32)[:, None] * wide + torch.arange(wide, device=DEV)
            got[(slots // P)[:, None, None], torch.arange(c["Hkv"], device=DEV)[None, :, None], (slots % P // 32)[:, None, None], col[:, None]] = \
                _exact_scales(x, c["shift"])
        out = {"codes": None, "scales": got}
        return {**out, "new_lengths": None} if kind == "commit" else out
    if kind == "attend":
        B, N, G, Hkv, D, P = (c[k] for k in ("B", "N", "G", "Hkv", "D", "P"))
        half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        half, e4m3 = torch.cat([half, -half]), _e4m3_table()
        out = torch.zeros(B, N, Hkv * G, D, dtype=torch.float64, device=DEV)
        lse = torch.zeros(B, N, Hkv * G, dtype=torch.float64, device=DEV)
        causal = torch.arange(N, device=DEV)
        for b, n in enumerate(s["lengths"].tolist()):
            page = s["cache"][s["table"][b, : -(-n // P)].long()].transpose(0, 1).reshape(Hkv, -1, 36 * D)
            code = page[..., : 32 * D].reshape(Hkv, -1, 2, 32, D // 2)
            sc = e4m3[page[..., 32 * D:].reshape(Hkv, -1, 2, 32, D // 16).int()].repeat_interleave(16, -1) * 2.0 ** c["shift"]
            val = torch.stack([half[(code & 15).int()], half[(code >> 4).int()]], -1).flatten(-2) * sc
            k, v = (val[:, :, i].reshape(Hkv, -1, D)[:, :n] for i in range(2))
            k = torch.cat([k, s["k_new"][b].double().transpose(0, 1)], 1)
            v = torch.cat([v, s["v_new"][b].double().transpose(0, 1)], 1)
            if c["tree"]:
                see = (s["masks"][b].long()[:, causal // 32] >> (causal % 32)) & 1 == 1
            else:
                see = causal[None] <= causal[:, None]
            see = torch.cat([torch.ones(N, n, dtype=torch.bool, device=DEV), see], 1)
            for h in range(Hkv):
                q = s["q"][b, :, h * G:(h + 1) * G].double()
                z = torch.einsum("ngd,ld->ngl", q, k[h]) * s["scale"]
                z = z.masked_fill(~see[:, None], -math.inf)
                lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[b, :, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(z, -1), v[h])
        return out, lse
    B, R, V = c["B"], c["R"], c["V"]
    got = s["logits"].double()
    lens, prompts = s["hist_len"].tolist(), s["prompt_len"].tolist()
    node = torch.arange(R, device=DEV)
    for b in range(B):
        words = s["history"][b, : lens[b]].long()
        count = torch.bincount(words[prompts[b]:], minlength=V)
        seen = torch.bincount(words, minlength=V)
        r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        if c["tree"]:
            path = ((s["masks"][b].long()[:, node // 32] >> (node % 32)) & 1 == 1) & (node > 0)
        else:
            path = node[None] < node[:, None]
        more = torch.zeros(R, V, dtype=torch.int64, device=DEV)
        more.index_add_(1, s["nodes"][b].long(), path.long())
        x, n = got[b], count + more
        x = torch.where(seen + more > 0, torch.where(x > 0, x / r, x * r), x) - f * n - p * (n > 0)
        if s["bias_tokens"] is not None:
            x.index_add_(1, s["bias_tokens"][b].long(), s["bias_values"][b].double().expand(R, -1))
        if s["allowed"] is not None:
            v = torch.arange(V, device=DEV)
            x = x.masked_fill((s["allowed"][b].long()[:, v // 32] >> (v % 32)) & 1 == 0, -math.inf)
        got[b] = x
    return got
