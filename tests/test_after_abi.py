"""The steps after a verification on the host (no GPU needed): what the entry points refuse
before touching the device, and the tests' own references pinned by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

import after_ref as ref
import serving_ref as sref
from speculative_decoding_verification_52_gb300 import binding as B
from speculative_decoding_verification_52_gb300 import build as build_mod
from test_serving_abi import _call

BAD, UNSUP, OK = B.SPEC_ERR_INVALID_ARG, B.SPEC_ERR_UNSUPPORTED, B.SPEC_OK


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


LP = dict(p_logits=16, dtype=B.SPEC_BF16, p_tokens=32, p_path=48, T=1.0, B=2, R=6, V=100, M=4, W=3, n=5, p_lp=64, p_ent=80, p_ranks=96,
          p_tt=112, p_tl=128)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(R=0), BAD), (dict(V=0), BAD), (dict(M=0), BAD), (dict(n=-1), BAD), (dict(n=33), UNSUP), (dict(dtype=5), BAD),
    (dict(T=0.0), BAD), (dict(T=-1.0), BAD), (dict(T=float("nan")), BAD), (dict(T=float("inf")), BAD), (dict(T=5e-5), UNSUP),
    (dict(W=2), BAD), (dict(p_path=0, M=7), BAD), (dict(V=(1 << 30) + 1), UNSUP), (dict(B=1 << 20, M=1 << 12, R=1 << 12, W=1 << 12), UNSUP),
    (dict(p_logits=0), BAD), (dict(p_tokens=0), BAD), (dict(p_lp=0), BAD), (dict(p_tt=0), BAD), (dict(p_tl=0), BAD), (dict(p_logits=17), BAD),
    (dict(dtype=B.SPEC_F32, p_logits=18), BAD), (dict(B=0, p_logits=0, p_lp=0), OK),
])
def test_logprobs_refusals(L, kw, status):
    assert _call(L.spec_token_logprobs, LP, **kw) == status
    assert status == OK or B.last_error()


WG = dict(p_q=16, p_lse=32, p_path=48, p_count=64, p_cache=80, p_table=96, p_len=112, p_first=128, B=2, N=6, W=4, Hq=8, Hkv=2, D=128, P=32,
          pages=9, maxp=4, ks=0, scale=0.1, decay=0.9, p_w=144, p_new=144, p_pos=176)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(N=0), BAD), (dict(N=1025), BAD), (dict(W=0), BAD), (dict(W=1025), UNSUP), (dict(Hq=7), BAD), (dict(Hq=0), BAD),
    (dict(Hkv=0), BAD), (dict(D=96), UNSUP), (dict(P=48), BAD), (dict(P=0), BAD), (dict(pages=0), BAD), (dict(maxp=0), BAD),
    (dict(Hq=130), UNSUP), (dict(B=4097), UNSUP), (dict(ks=33), BAD), (dict(scale=float("inf")), BAD), (dict(decay=float("nan")), BAD),
    (dict(pages=1 << 26), UNSUP), (dict(maxp=1 << 26), UNSUP), (dict(p_q=0), BAD), (dict(p_lse=0), BAD), (dict(p_cache=0), BAD),
    (dict(p_table=0), BAD), (dict(p_len=0), BAD), (dict(p_w=0), BAD), (dict(p_new=0), BAD), (dict(p_q=24), BAD), (dict(p_cache=88), BAD),
    (dict(B=0, p_q=0, p_new=0), OK), (dict(Hkv=1 << 14, Hq=1 << 14, P=1 << 10, pages=1 << 20), UNSUP),
])
def test_weigh_refusals(L, kw, status):
    assert _call(L.spec_kv_weigh_q4, WG, **kw) == status


PLAN = dict(p_w=16, p_pos=32, p_table=48, p_len=64, p_budget=80, p_next=96, B=2, Hkv=2, P=32, pages=9, maxp=4, sinks=1, recent=2, most=8,
            p_moves=112, p_counts=128, p_new=144)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(Hkv=0), BAD), (dict(P=40), BAD), (dict(pages=0), BAD), (dict(maxp=0), BAD), (dict(sinks=-1), BAD),
    (dict(recent=-1), BAD), (dict(most=0), BAD), (dict(maxp=1 << 26), UNSUP), (dict(pages=1 << 26), UNSUP), (dict(p_w=0), BAD),
    (dict(p_pos=0), BAD), (dict(p_table=0), BAD), (dict(p_len=0), BAD), (dict(p_budget=0), BAD), (dict(p_next=0), BAD), (dict(p_moves=0), BAD),
    (dict(p_counts=0), BAD), (dict(p_new=0), BAD), (dict(p_new=64), BAD), (dict(p_moves=116), BAD), (dict(B=0, p_w=0), OK),
    (dict(Hkv=1 << 14, P=1 << 10, pages=1 << 20), UNSUP),
])
def test_plan_refusals(L, kw, status):
    assert _call(L.spec_kv_evict_plan, PLAN, **kw) == status


MOVE = dict(p_cache=16, p_w=32, p_pos=48, p_moves=64, p_counts=80, B=2, Hkv=2, D=64, P=32, pages=9, most=8)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(Hkv=0), BAD), (dict(D=32), UNSUP), (dict(P=31), BAD), (dict(pages=0), BAD), (dict(most=0), BAD),
    (dict(pages=1 << 26), UNSUP), (dict(p_cache=0), BAD), (dict(p_moves=0), BAD), (dict(p_counts=0), BAD), (dict(p_cache=24), BAD),
    (dict(p_moves=68), BAD), (dict(B=0, p_cache=0), OK),
])
def test_move_refusals(L, kw, status):
    assert _call(L.spec_kv_move_q4, MOVE, **kw) == status


TRIM = dict(p_tokens=16, p_held=32, p_ring=48, p_state=64, p_table=80, B=2, F=100, P=32, W=8, p_new=96, p_new_state=112, p_status=128)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(F=0), BAD), (dict(P=0), BAD), (dict(W=0), BAD), (dict(F=1 << 27), UNSUP), (dict(W=1 << 27), UNSUP),
    (dict(p_tokens=0), BAD), (dict(p_held=0), BAD), (dict(p_ring=0), BAD), (dict(p_state=0), BAD), (dict(p_table=0), BAD), (dict(p_new=0), BAD),
    (dict(p_new_state=0), BAD), (dict(p_status=0), BAD), (dict(p_new=32), BAD), (dict(p_new_state=64), BAD), (dict(B=0, p_ring=0), BAD),
])
def test_trim_refusals(L, kw, status):
    assert _call(L.spec_page_trim, TRIM, **kw) == status


def test_binding_checks_tensors():
    import speculative_decoding_verification_52_gb300 as sv
    z = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sv.spec_token_logprobs(torch.zeros(1, 1, 8), z.view(1, 2)), lambda: sv.spec_page_trim(z, z, z, z, z.view(1, 2), 32),
                 lambda: sv.spec_kv_evict_plan(torch.zeros(1, 1, 32), z, z, z, z, z, max_moves=4),
                 lambda: sv.spec_kv_move_q4(sv.q4_cache(1, 1, 32, 64, "cpu"), z, z),
                 lambda: sv.spec_kv_weigh_q4(torch.zeros(1, 1, 1, 64), z, sv.q4_cache(1, 1, 32, 64, "cpu"), z, z, z)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# --- the references ---------------------------------------------------------
def test_reference_logprobs_by_hand():
    row = np.log(np.array([1.0, 2.0, 4.0, 1.0]))          # p = 1/8, 1/4, 1/2, 1/8
    lp, ent, rank, top, val, _ = ref.logprobs_row(row, 3, 1.0, 3)
    assert abs(lp - math.log(1 / 8)) < 1e-12 and rank == 4 and top.tolist() == [2, 1, 0]
    assert abs(ent - (0.5 * math.log(2) + 0.25 * math.log(4) + 0.25 * math.log(8))) < 1e-12
    assert np.abs(val - np.log([0.5, 0.25, 0.125])).max() < 1e-12
    # half the temperature squares the odds: 1, 4, 16, 1
    assert abs(ref.logprobs_row(row, 1, 0.5, 0)[0] - math.log(4 / 22)) < 1e-12
    # masked ones have no probability and are no alternatives, but stand in the order
    lp, ent, rank, top, val, _ = ref.logprobs_row(np.array([0.0, -np.inf, -3e38, 0.0]), 2, 1.0, 3)
    assert lp == -np.inf and rank == 4 and top.tolist() == [0, 3, -1] and abs(ent - math.log(2)) < 1e-12 and val[2] == -np.inf
    for bad in ([np.nan, 1.0], [np.inf, 0.0], [-np.inf, -np.inf], [2.0 ** 100, 0.0]):
        assert np.isnan(ref.logprobs_row(np.array(bad), 0, 1.0, 1)[0])
    assert np.isnan(ref.logprobs_row(np.zeros(3), 3, 1.0, 1)[0])


def test_reference_weigh_by_hand():
    """One head, two committed rows behind two cached tokens: keys of zero score 0, so that
    a row gives e^-lse to each token it sees."""
    cache, D, P = np.zeros((2, 1, 1, 36 * 64), np.uint8), 64, 32
    w = np.zeros((2, 1, P))
    w[1, 0, :4] = [1, 2, 99, 99]
    pos = np.full((2, 1, P), 7)
    q, lse = np.ones((1, 3, 1, D)), np.log(np.array([2.0, 5.0, 4.0])).reshape(1, 3, 1)
    new, p, _ = ref.weigh(q, lse, cache, np.array([[1]]), np.array([2]), w, pos, np.array([2]), np.array([[0, 2]]), np.array([50]), 1.0, 0.5, 0,
                          w)
    # rows 0 (1/2 to tokens 0..2) and 2 (1/4 to tokens 0..3)
    assert np.allclose(new[1, 0, :5], [0.5 + 0.75, 1 + 0.75, 0.75, 0.25, 0]) and p[1, 0, 1:5].tolist() == [7, 50, 51, 7]
    assert (new[0] == 0).all()


def test_reference_plan_by_hand():
    w = np.zeros((2, 1, 32))
    w[1, 0, :6] = [5, 1, np.nan, 3, 3, 9]
    pos = np.zeros((2, 1, 32), int)
    pos[1, 0, :6] = [10, 11, 12, 13, 0, 15]
    moves = np.full((1, 1, 4, 2), -1)
    m, c, n = ref.evict_plan(w, pos, np.array([[1]]), np.array([6]), np.array([3]), np.array([16]), 0, 0, moves)
    assert n[0] == 3
    # the largest are 9, 5 and, of the two 3s, the lower place: 5, 0 and 3 stay; 1 and 2 become free
    assert c[0, 0] == 2 and m[0, 0].tolist() == [[32 + 3, 32 + 1], [32 + 5, 32 + 2], [-1, -1], [-1, -1]]
    # position 0 is a sink, 15 recent: places 4 and 5 stay, and the 5
    m, c, n = ref.evict_plan(w, pos, np.array([[1]]), np.array([6]), np.array([3]), np.array([16]), 1, 1, moves)
    assert c[0, 0] == 2 and m[0, 0, :2].tolist() == [[32 + 4, 32 + 1], [32 + 5, 32 + 2]]
    assert ref.evict_plan(w, pos, np.array([[1]]), np.array([6]), np.array([3]), np.array([16]), 0, 0, moves[:, :, :2])[2][0] == -1
    assert ref.evict_plan(w, pos, np.array([[2]]), np.array([6]), np.array([3]), np.array([16]), 0, 0, moves)[2][0] == -1
    assert ref.evict_plan(w, pos, np.array([[2]]), np.array([6]), np.array([6]), np.array([16]), 0, 0, moves)[2][0] == 6


def test_reference_move_and_trim_by_hand():
    rng = np.random.default_rng(0)
    cache = rng.integers(0, 100, (2, 1, 1, 36 * 64)).astype(np.uint8)
    got, w, p = ref.move(cache, np.arange(64.0).reshape(2, 1, 32), None, np.array([[[[40, 3], [99, 4], [1, 2]]]]), np.array([[2]]))
    for a, b in zip(sref.q4_split(got, 64), sref.q4_split(cache, 64)):
        assert (a[0, 0, 0, 3] == b[1, 0, 0, 8]).all() and (a[0, 0, 0, 2] == b[0, 0, 0, 2]).all()
    assert w[0, 0, 3] == 40 and w[0, 0, 4] == 4 and p is None and (got != cache).any()
    held, state, status, ring = ref.page_trim(np.array([33, 5, 64]), np.array([4, 1, 3]), np.arange(8), np.array([6, 3]),
                                              np.array([[10, 11, 12, 13], [14, -1, -1, -1], [15, 16, 17, -1]]), 32)
    # free ids at 6, 7, 0; 12, 13 and 17 follow at 1, 2, 3
    assert held.tolist() == [2, 1, 2] and state.tolist() == [6, 6] and not status.any() and ring.tolist() == [0, 12, 13, 17, 4, 5, 6, 7]
