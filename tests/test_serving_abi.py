"""The serving entry points on the host (no GPU needed): what they refuse before
touching the device, their sizes, and the tests' own references pinned by hand."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as ref
from speculative_decoding_verification_52_gb300 import binding as B
from speculative_decoding_verification_52_gb300 import build as build_mod

P = ctypes.c_void_p
BAD, UNSUP, WS = B.SPEC_ERR_INVALID_ARG, B.SPEC_ERR_UNSUPPORTED, B.SPEC_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def _call(f, args, **kw):
    a = {**args, **kw}
    assert set(a) == set(args)
    return f(*[P(x) if isinstance(x, int) and k.startswith("p_") and x else (None if k.startswith("p_") else x) for k, x in a.items()], None)


MAP = dict(p_lengths=16, p_count=32, p_held=48, p_ring=64, p_ring_state=80, p_table=96, B=2, F=100, P=32, W=8, T=64,
           p_offsets=112, p_slots=128, p_positions=144, p_new_held=160, p_new_state=176, p_status=192)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(F=0), BAD), (dict(P=0), BAD), (dict(W=0), BAD), (dict(T=-1), BAD),
    (dict(p_lengths=0), BAD), (dict(p_count=0), BAD), (dict(p_held=0), BAD), (dict(p_ring=0), BAD), (dict(p_ring_state=0), BAD),
    (dict(p_table=0), BAD), (dict(p_offsets=0), BAD), (dict(p_slots=0), BAD), (dict(p_positions=0), BAD), (dict(p_status=0), BAD),
    (dict(p_new_held=48), BAD), (dict(p_new_state=80), BAD),
    (dict(F=1 << 27, P=32), UNSUP), (dict(W=1 << 27, P=32), UNSUP), (dict(B=0, p_offsets=0), BAD), (dict(B=0, p_slots=0), BAD),
])
def test_page_map_refusals(L, kw, status):
    assert _call(L.spec_page_map, MAP, **kw) == status
    assert B.last_error()


STORE = dict(p_k=16, p_v=32, p_slots=48, T=4, Hkv=2, D=128, P=64, pages=5, ks=0, vs=0, p_cache=64)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), UNSUP), (dict(D=256), UNSUP), (dict(P=48), BAD), (dict(P=0), BAD), (dict(Hkv=0), BAD), (dict(pages=0), BAD),
    (dict(T=-1), BAD), (dict(ks=33), BAD), (dict(vs=-33), BAD), (dict(p_k=0), BAD), (dict(p_slots=0), BAD),
    (dict(p_cache=0), BAD), (dict(p_k=24), BAD), (dict(p_cache=72), BAD), (dict(pages=1 << 26, P=64), UNSUP), (dict(T=0, p_k=0), B.SPEC_OK),
])
def test_store_refusals(L, kw, status):
    assert _call(L.spec_kv_store_q4, STORE, **kw) == status


COMMIT = dict(p_cache=16, p_table=32, p_lengths=48, p_k=64, p_v=80, p_path=96, p_count=112, B=2, N=6, W=6, Hkv=2, D=64, P=32,
              pages=9, maxp=4, ks=0, vs=0, p_new=128)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(N=0), BAD), (dict(W=0), BAD), (dict(D=80), UNSUP), (dict(P=33), BAD), (dict(maxp=0), BAD),
    (dict(p_new=48), BAD), (dict(p_new=0), BAD), (dict(p_cache=0), BAD), (dict(p_count=0), BAD), (dict(p_v=84), BAD),
    (dict(ks=40), BAD), (dict(maxp=1 << 27), UNSUP), (dict(B=0, p_cache=0), B.SPEC_OK),
])
def test_commit_refusals(L, kw, status):
    assert _call(L.spec_kv_commit_q4, COMMIT, **kw) == status


ATT = dict(p_q=16, p_kn=32, p_vn=48, p_masks=64, p_cache=80, p_table=96, p_len=112, B=2, N=6, Hq=8, Hkv=2, D=128, P=32, pages=9, maxp=4,
           ks=0, vs=0, scale=0.1, p_out=128, p_lse=144, p_ws=256, wsb=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(N=0), BAD), (dict(N=1025), BAD), (dict(Hq=7), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(D=32), UNSUP),
    (dict(P=16), BAD), (dict(Hq=130, Hkv=2), UNSUP), (dict(B=5000), UNSUP), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(p_kn=0), BAD), (dict(p_vn=0), BAD), (dict(p_kn=0, p_vn=0), BAD),
    (dict(p_q=0), BAD), (dict(p_q=24), BAD), (dict(p_out=0), BAD), (dict(p_out=130), BAD), (dict(p_cache=81), BAD),
    (dict(p_ws=0), WS), (dict(wsb=100), WS), (dict(p_ws=264), WS), (dict(ks=-50), BAD),
    (dict(B=0, p_q=0, p_ws=0, wsb=0), B.SPEC_OK),
])
def test_attend_refusals(L, kw, status):
    assert _call(L.spec_attend_q4, ATT, **kw) == status


ADJ = dict(p_logits=16, dtype=B.SPEC_BF16, p_hist=32, p_plen=48, p_hlen=64, p_rep=80, p_freq=96, p_pres=112, p_nodes=128, p_masks=0,
           p_bt=144, p_bv=160, p_allowed=176, B=2, R=6, V=100, H=20, Nt=5, M=3, p_out=192)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(R=0), BAD), (dict(R=1025), BAD), (dict(V=0), BAD), (dict(H=-1), BAD), (dict(M=-1), BAD), (dict(Nt=1025), BAD),
    (dict(dtype=7), BAD), (dict(p_hlen=0), BAD), (dict(Nt=4), BAD), (dict(p_masks=208), BAD), (dict(p_bv=0), BAD), (dict(p_bt=0), BAD),
    (dict(p_logits=0), BAD), (dict(p_out=0), BAD), (dict(p_logits=17), BAD), (dict(V=(1 << 30) + 1), UNSUP),
    (dict(B=0, p_logits=0, p_out=0), B.SPEC_OK),
])
def test_adjust_refusals(L, kw, status):
    assert _call(L.spec_adjust_logits, ADJ, **kw) == status


def test_sizes(L):
    assert [L.spec_q4_block_bytes(d) for d in (64, 128, 96, 0)] == [2304, 4608, 0, 0]
    assert L.spec_attend_workspace_bytes(1, 1, 32, 8, 128) > 0
    for bad in [(-1, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 1025, 8, 8, 64), (1, 1, 7, 2, 64), (1, 1, 8, 8, 80), (5000, 1, 8, 8, 64), (1, 1, 65, 1, 64)]:
        assert L.spec_attend_workspace_bytes(*bad) == 0


def test_binding_checks_tensors():
    """The binding refuses host tensors before any C call."""
    import speculative_decoding_verification_52_gb300 as sv
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_page_map(z, z, z, z, z, z.view(1, 2), 32, 4)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_adjust_logits(torch.zeros(1, 1, 8))
    with pytest.raises(ValueError, match="multiple of 32"):
        sv.q4_cache(1, 1, 40, 64, "cpu")


# --- the references ---------------------------------------------------------
def test_reference_quantiser_by_hand():
    x = np.zeros(16)
    x[:7] = [6, -3, 1.25, 0.25, 0.75, 5.0, -0.2]
    code, sb = ref.q4_quantise(x, 0)
    assert ref.E4M3[sb[0]] == 1.0
    # 1.25 lies between 1 (code 2) and 1.5 (3): even; 0.25 -> 0; 0.75 -> 1 (code 2); 5 -> 4 (code 6); -0.2 -> -0 (8)
    assert code[:7].tolist() == [7, 8 + 5, 2, 0, 2, 6, 8]
    x[3] = np.nan
    code, sb = ref.q4_quantise(x, 0)
    assert sb[0] == 0x7f and not code.any()
    code, sb = ref.q4_quantise(np.full(16, 1e6), 0)      # the scale saturates at 448, the code at 6
    assert ref.E4M3[sb[0]] == 448 and (code == 7).all()
    code, sb = ref.q4_quantise(np.full(16, 1e-5), 0)
    assert sb[0] == 0 and not code.any()
    assert ref.q4_quantise(np.full(16, 1e6), 10)[1][0] == ref.q4_quantise(np.full(16, 1e6 / 1024), 0)[1][0]


def test_reference_cache_round_trip():
    rng = np.random.default_rng(0)
    cache = np.zeros((3, 2, 2, 36 * 64), np.uint8)
    k, v = rng.standard_normal((2, 64))
    ref.q4_put(cache, 2 * 64 + 37, 1, k, v, 1, -1)
    kk, vv = (ref.q4_read(cache, np.array([2 * 64 + 37]), 1, s, i)[0] for i, s in enumerate((1, -1)))
    # a step of e2m1 is at most a third of the group's largest element's sixth, twice over
    for a, b in ((k, kk), (v, vv)):
        top = np.abs(a).reshape(-1, 16).max(-1).repeat(16)
        assert (np.abs(a - b) <= top * (1 / 6 + 1 / 16) + 1e-12).all()


def test_reference_page_map_by_hand():
    ring = np.array([5, 6, 7, 0, 1, 2, 3, 4])
    table = np.array([[3, -1, -1], [-1, -1, -1], [4, 2, -1]])
    off, slots, pos, held, state, status, tab, rng = ref.page_map(
        np.array([3, 0, 8]), np.array([2, 6, -1]), np.array([1, 0, 2]), ring, np.array([6, 5]), table, 4, 9)
    # ring from position 6: 3, 4, 5, 6, 7
    assert off.tolist() == [0, 2, 8, 8] and status.tolist() == [0, 0, 0]
    assert tab[0].tolist() == [3, 3, -1] and tab[1].tolist() == [4, 5, -1]
    assert slots.tolist() == [15, 12, 16, 17, 18, 19, 20, 21, -1]
    assert held.tolist() == [2, 2, 0] and state.tolist() == [1, 4]
    assert rng[3:5].tolist() == [4, 2]


@pytest.mark.parametrize("kw,status", [(dict(cta=-1), BAD), (dict(us=99), BAD), (dict(us=1000001), BAD), (dict(N=0), BAD), (dict(D=96), UNSUP),
                                       (dict(p_ws=0), WS), (dict(B=0, p_q=0, p_ws=0, wsb=0), B.SPEC_OK)])
def test_attend_stall_hook_refusals(L, kw, status):
    at = list(ATT).index("p_out")
    args = dict(list(ATT.items())[:at] + [("cta", 0), ("us", 2000)] + list(ATT.items())[at:])
    assert _call(L.spec_debug_attend_stall, args, **kw) == status


def test_binding_takes_every_argument_by_name():
    """Named or not, the first argument is looked at in the same way; none is an error
    of the call."""
    import speculative_decoding_verification_52_gb300 as sv
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_page_map(lengths=z, count=z, held=z, ring=z, ring_state=z, block_table=z.view(1, 2), page_tokens=32, max_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_adjust_logits(logits=torch.zeros(1, 1, 8))
    with pytest.raises(TypeError, match="logits"):
        sv.spec_adjust_logits()
