"""Thin Python binding of the C ABI in include/spec_verify.h.

Argument marshalling only: torch tensors are checked for device, dtype and
layout, outputs and the caller-side workspace are allocated with torch when
not supplied, and the C entry points of libspecverify.so are called with raw
pointers and the current CUDA stream.  Every step of the verification runs in
the library's CUDA kernels; there is no fallback of any kind -- if the library
is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "spec_verify.h")

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA, SPEC_ERR_WORKSPACE = range(5)
SPEC_F32, SPEC_BF16 = 0, 1
SPEC_DRAFT_LOGITS, SPEC_DRAFT_PROBS = 0, 1
SPEC_MAX_K = 31
SPEC_MAX_TREE_NODES = 1024

_lock = threading.Lock()
_lib = None


class SpecError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {status_string(status)}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libspecverify.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            L.spec_workspace_bytes.argtypes = [I, I, I]
            L.spec_workspace_bytes.restype = Z
            L.spec_tree_workspace_bytes.argtypes = [I, I, I]
            L.spec_tree_workspace_bytes.restype = Z
            L.spec_verify_sample.argtypes = [P, I, P, I, I, P, P, F, I, I, I, P, P, P, Z, P]
            L.spec_verify_sample.restype = I
            L.spec_verify_sample_noalloc.argtypes = [P, I, P, I, I, P, P, F, I, I, I, P, P, P]
            L.spec_verify_sample_noalloc.restype = I
            L.spec_verify_greedy.argtypes = [P, I, P, I, I, I, P, P, P, Z, P]
            L.spec_verify_greedy.restype = I
            L.spec_verify_tree_greedy.argtypes = [P, I, P, P, I, I, I, I, P, P, P, P, Z, P]
            L.spec_verify_tree_greedy.restype = I
            L.spec_debug_residual.argtypes = [P, I, P, I, I, P, P, F, I, I, I, I, I, P, P, P, P, P, Z, P]
            L.spec_debug_residual.restype = I
            L.spec_debug_stall.argtypes = [P, I, P, I, I, P, P, F, I, I, I, I, ctypes.c_uint, P, P, P, Z, P]
            L.spec_debug_stall.restype = I
            L.spec_tree_mask.argtypes = [P, I, I, P, P, P]
            L.spec_tree_mask.restype = I
            L.spec_kv_commit.argtypes = [P, P, P, P, P, I, I, I, I, Z, P, P]
            L.spec_kv_commit.restype = I
            L.spec_row_stats.argtypes = [P, I, P, I, I, F, I, I, I, P, P, P, P]
            L.spec_row_stats.restype = I
            L.spec_tree_draft.argtypes = [P, I, P, I, I, I, I, F, P, P, P]
            L.spec_tree_draft.restype = I
            L.spec_q4_block_bytes.argtypes = [I]
            L.spec_q4_block_bytes.restype = Z
            L.spec_page_map.argtypes = [P] * 6 + [I] * 5 + [P] * 7
            L.spec_page_map.restype = I
            L.spec_kv_store_q4.argtypes = [P] * 3 + [I] * 7 + [P] * 2
            L.spec_kv_store_q4.restype = I
            L.spec_kv_commit_q4.argtypes = [P] * 7 + [I] * 10 + [P] * 2
            L.spec_kv_commit_q4.restype = I
            L.spec_attend_workspace_bytes.argtypes = [I] * 5
            L.spec_attend_workspace_bytes.restype = Z
            L.spec_attend_q4.argtypes = [P] * 7 + [I] * 10 + [F, P, P, P, Z, P]
            L.spec_attend_q4.restype = I
            L.spec_debug_attend_stall.argtypes = [P] * 7 + [I] * 10 + [F, I, ctypes.c_uint, P, P, P, Z, P]
            L.spec_debug_attend_stall.restype = I
            L.spec_adjust_logits.argtypes = [P, I] + [P] * 11 + [I] * 6 + [P] * 2
            L.spec_adjust_logits.restype = I
            L.spec_token_logprobs.argtypes = [P, I, P, P, F] + [I] * 6 + [P] * 6
            L.spec_token_logprobs.restype = I
            L.spec_kv_weigh_q4.argtypes = [P] * 8 + [I] * 10 + [F] * 2 + [P] * 4
            L.spec_kv_weigh_q4.restype = I
            L.spec_kv_evict_plan.argtypes = [P] * 6 + [I] * 8 + [P] * 4
            L.spec_kv_evict_plan.restype = I
            L.spec_kv_move_q4.argtypes = [P] * 5 + [I] * 6 + [P]
            L.spec_kv_move_q4.restype = I
            L.spec_page_trim.argtypes = [P] * 5 + [I] * 4 + [P] * 4
            L.spec_page_trim.restype = I
            L.spec_profile_begin.argtypes = [I]
            L.spec_profile_begin.restype = I
            L.spec_profile_end.argtypes = [P, P, P]
            L.spec_profile_end.restype = I
            L.spec_status_string.argtypes = [I]
            L.spec_status_string.restype = ctypes.c_char_p
            L.spec_last_error.argtypes = []
            L.spec_last_error.restype = ctypes.c_char_p
            _lib = L
    return _lib


def declared_functions() -> list[str]:
    """Names of the functions include/spec_verify.h declares."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(spec_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().spec_status_string(int(status)).decode()


def last_error() -> str:
    return lib().spec_last_error().decode()


def _check(fn: str, status: int):
    if status != SPEC_OK:
        raise SpecError(fn, status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def spec_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(lib().spec_workspace_bytes(B, K, V))


def spec_tree_workspace_bytes(B: int, N: int, V: int) -> int:
    return int(lib().spec_tree_workspace_bytes(B, N, V))


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _outputs(B, W, device, out_tokens, num_accepted):
    if out_tokens is None:
        out_tokens = torch.empty((B, W), dtype=torch.int32, device=device)
    if num_accepted is None:
        num_accepted = torch.empty((B,), dtype=torch.int32, device=device)
    _dev(out_tokens, "out_tokens")
    _dev(num_accepted, "num_accepted")
    return out_tokens, num_accepted


def spec_verify_sample(target_logits, draft, draft_tokens, uniforms, temperature, *,
                       draft_kind: str = "logits", out_tokens=None, num_accepted=None,
                       workspace_buf=None, stream=None):
    """Sampling-mode verification.  target_logits [B,K+1,V] (bf16/f32),
    draft [B,K,V] (logits: bf16/f32; probs: f32), draft_tokens [B,K] int32,
    uniforms [B,K+1,2] f32.  Returns (out_tokens [B,K+1], num_accepted [B])."""
    _dev(target_logits, "target_logits")
    B, W, V = target_logits.shape
    K = W - 1
    kind = SPEC_DRAFT_PROBS if draft_kind == "probs" else SPEC_DRAFT_LOGITS
    for t, n in ((draft, "draft"), (draft_tokens, "draft_tokens"), (uniforms, "uniforms")):
        if t is not None:
            _dev(t, n)
    ddt = _dtype_code(draft) if draft is not None else SPEC_F32
    out_tokens, num_accepted = _outputs(B, W, target_logits.device, out_tokens, num_accepted)
    if workspace_buf is None:
        workspace_buf = workspace(spec_workspace_bytes(B, K, V), target_logits.device)
    st = lib().spec_verify_sample(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), ddt, kind,
                                  _ptr(draft_tokens), _ptr(uniforms), float(temperature), B, K, V,
                                  _ptr(out_tokens), _ptr(num_accepted), _ptr(workspace_buf),
                                  workspace_buf.numel(), _stream(stream))
    _check("spec_verify_sample", st)
    return out_tokens, num_accepted


def spec_verify_sample_noalloc(target_logits, draft, draft_tokens, uniforms, temperature, *,
                               draft_kind: str = "logits", out_tokens=None, num_accepted=None, stream=None):
    """spec_verify_sample with the library's fixed scratch instead of a
    workspace.  Pass out_tokens / num_accepted to keep the call free of any
    allocation (otherwise they are allocated here)."""
    _dev(target_logits, "target_logits")
    B, W, V = target_logits.shape
    K = W - 1
    kind = SPEC_DRAFT_PROBS if draft_kind == "probs" else SPEC_DRAFT_LOGITS
    for t, n in ((draft, "draft"), (draft_tokens, "draft_tokens"), (uniforms, "uniforms")):
        if t is not None:
            _dev(t, n)
    ddt = _dtype_code(draft) if draft is not None else SPEC_F32
    out_tokens, num_accepted = _outputs(B, W, target_logits.device, out_tokens, num_accepted)
    st = lib().spec_verify_sample_noalloc(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), ddt, kind,
                                          _ptr(draft_tokens), _ptr(uniforms), float(temperature), B, K, V,
                                          _ptr(out_tokens), _ptr(num_accepted), _stream(stream))
    _check("spec_verify_sample_noalloc", st)
    return out_tokens, num_accepted


def spec_verify_greedy(target_logits, draft_tokens, *, out_tokens=None, num_accepted=None,
                       workspace_buf=None, stream=None):
    """Greedy verification.  Returns (out_tokens [B,K+1], num_accepted [B])."""
    _dev(target_logits, "target_logits")
    B, W, V = target_logits.shape
    K = W - 1
    if draft_tokens is not None:
        _dev(draft_tokens, "draft_tokens")
    out_tokens, num_accepted = _outputs(B, W, target_logits.device, out_tokens, num_accepted)
    if workspace_buf is None:
        workspace_buf = workspace(spec_workspace_bytes(B, K, V), target_logits.device)
    st = lib().spec_verify_greedy(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft_tokens), B, K, V,
                                  _ptr(out_tokens), _ptr(num_accepted), _ptr(workspace_buf),
                                  workspace_buf.numel(), _stream(stream))
    _check("spec_verify_greedy", st)
    return out_tokens, num_accepted


def spec_verify_tree_greedy(target_logits, parents, node_tokens, max_depth: int, *, with_path: bool = True,
                            out_tokens=None, num_accepted=None, out_path=None, workspace_buf=None,
                            stream=None):
    """Greedy tree verification.  target_logits [B,N,V], parents [N] int32,
    node_tokens [B,N] int32.  Returns (out_tokens, num_accepted, out_path|None)."""
    _dev(target_logits, "target_logits")
    _dev(parents, "parents")
    _dev(node_tokens, "node_tokens")
    B, N, V = target_logits.shape
    W = max_depth + 1
    out_tokens, num_accepted = _outputs(B, W, target_logits.device, out_tokens, num_accepted)
    if with_path and out_path is None:
        out_path = torch.empty((B, W), dtype=torch.int32, device=target_logits.device)
    if workspace_buf is None:
        workspace_buf = workspace(spec_tree_workspace_bytes(B, N, V), target_logits.device)
    st = lib().spec_verify_tree_greedy(_ptr(target_logits), _dtype_code(target_logits), _ptr(parents),
                                       _ptr(node_tokens), B, N, V, int(max_depth), _ptr(out_tokens),
                                       _ptr(num_accepted), _ptr(out_path), _ptr(workspace_buf),
                                       workspace_buf.numel(), _stream(stream))
    _check("spec_verify_tree_greedy", st)
    return out_tokens, num_accepted, out_path


def spec_debug_residual(target_logits, draft, draft_tokens, uniforms, temperature, debug_b: int, debug_t: int,
                        *, draft_kind: str = "logits", stream=None):
    """The device's normalised replacement distribution at (debug_b, debug_t).
    Returns (row [V] f32, mass [1] f32, out_tokens, num_accepted)."""
    _dev(target_logits, "target_logits")
    B, W, V = target_logits.shape
    K = W - 1
    dev = target_logits.device
    row = torch.full((V,), float("nan"), dtype=torch.float32, device=dev)
    mass = torch.zeros((1,), dtype=torch.float32, device=dev)
    out_tokens, num_accepted = _outputs(B, W, dev, None, None)
    ws = workspace(spec_workspace_bytes(B, K, V), dev)
    kind = SPEC_DRAFT_PROBS if draft_kind == "probs" else SPEC_DRAFT_LOGITS
    ddt = _dtype_code(draft) if draft is not None else SPEC_F32
    st = lib().spec_debug_residual(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), ddt, kind,
                                   _ptr(draft_tokens), _ptr(uniforms), float(temperature), B, K, V, int(debug_b),
                                   int(debug_t), _ptr(row), _ptr(mass), _ptr(out_tokens), _ptr(num_accepted),
                                   _ptr(ws), ws.numel(), _stream(stream))
    _check("spec_debug_residual", st)
    return row, mass, out_tokens, num_accepted


def spec_debug_stall(target_logits, draft, draft_tokens, uniforms, temperature, stall_b: int, timeout_us: int, *,
                     stream=None):
    """Test hook: spec_verify_sample with short wait limits while one
    sequence's scan waits for a unit that never comes.  Returns
    (out_tokens, num_accepted); every sequence should read -2."""
    _dev(target_logits, "target_logits")
    B, W, V = target_logits.shape
    K = W - 1
    out_tokens, num_accepted = _outputs(B, W, target_logits.device, None, None)
    ws = workspace(spec_workspace_bytes(B, K, V), target_logits.device)
    st = lib().spec_debug_stall(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), _dtype_code(draft),
                                SPEC_DRAFT_LOGITS, _ptr(draft_tokens), _ptr(uniforms), float(temperature), B, K, V,
                                int(stall_b), int(timeout_us), _ptr(out_tokens), _ptr(num_accepted), _ptr(ws),
                                ws.numel(), _stream(stream))
    _check("spec_debug_stall", st)
    return out_tokens, num_accepted


def spec_tree_mask(parents, *, masks=None, status=None, stream=None):
    """Ancestor masks.  parents [B, N] (or [N]) int32 on the device.  Returns
    (masks [B, N, ceil(N/32)] int32 holding the uint32 bit words, status [B])."""
    _dev(parents, "parents")
    par = parents if parents.dim() == 2 else parents.unsqueeze(0)
    par = par.contiguous()
    B, N = par.shape
    NW = (N + 31) // 32
    if masks is None:
        masks = torch.empty((B, N, NW), dtype=torch.int32, device=par.device)
    if status is None:
        status = torch.empty((B,), dtype=torch.int32, device=par.device)
    st = lib().spec_tree_mask(_ptr(par), B, N, _ptr(masks), _ptr(status), _stream(stream))
    _check("spec_tree_mask", st)
    return masks, status


def spec_kv_commit(cache, lengths, scratch, count, *, path=None, new_lengths=None, stream=None):
    """Append the selected scratch entries to the cache in place.  cache
    [B, Lmax, ...], scratch [B, N, ...] (same trailing shape and dtype),
    lengths / count [B] int32, path [B, W] int32 or None.  Returns new_lengths."""
    for t, n in ((cache, "cache"), (lengths, "lengths"), (scratch, "scratch"), (count, "count")):
        _dev(t, n)
    B, Lmax = cache.shape[:2]
    N = scratch.shape[1]
    E = cache[0, 0].numel() * cache.element_size() if Lmax else scratch[0, 0].numel() * scratch.element_size()
    W = 0
    if path is not None:
        _dev(path, "path")
        W = path.shape[1]
    if new_lengths is None:
        new_lengths = torch.empty((B,), dtype=torch.int32, device=cache.device)
    st = lib().spec_kv_commit(_ptr(cache), _ptr(lengths), _ptr(scratch), _ptr(path), _ptr(count), B, Lmax, N, W, E,
                              _ptr(new_lengths), _stream(stream))
    _check("spec_kv_commit", st)
    return new_lengths


def spec_row_stats(target_logits, draft, temperature, *, draft_kind: str = "logits", alpha=None, kl=None,
                   tv=None, stream=None):
    """Per-position acceptance statistics.  target_logits [B,K+1,V] (bf16/f32),
    draft [B,K,V] (logits: bf16/f32; probs: f32).  Returns (alpha, kl, tv), each
    [B,K] f32: sum min(p,q), KL(q||p), TV(p,q)."""
    _dev(target_logits, "target_logits")
    _dev(draft, "draft")
    B, W, V = target_logits.shape
    K = W - 1
    kind = SPEC_DRAFT_PROBS if draft_kind == "probs" else SPEC_DRAFT_LOGITS
    outs = []
    for o, n in ((alpha, "alpha"), (kl, "kl"), (tv, "tv")):
        if o is None:
            o = torch.empty((B, K), dtype=torch.float32, device=target_logits.device)
        _dev(o, n)
        outs.append(o)
    st = lib().spec_row_stats(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), _dtype_code(draft), kind,
                              float(temperature), B, K, V, _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]),
                              _stream(stream))
    _check("spec_row_stats", st)
    return tuple(outs)


def spec_tree_draft(draft_logits, parents, temperature, max_children: int, *, node_tokens=None, node_logq=None,
                    stream=None):
    """Top-k tree drafting.  draft_logits [B,N,V] (bf16/f32), parents [N] int32.
    Returns (node_tokens [B,N] int32, node_logq [B,N] f32)."""
    _dev(draft_logits, "draft_logits")
    _dev(parents, "parents")
    B, N, V = draft_logits.shape
    if node_tokens is None:
        node_tokens = torch.empty((B, N), dtype=torch.int32, device=draft_logits.device)
    if node_logq is None:
        node_logq = torch.empty((B, N), dtype=torch.float32, device=draft_logits.device)
    _dev(node_tokens, "node_tokens")
    _dev(node_logq, "node_logq")
    st = lib().spec_tree_draft(_ptr(draft_logits), _dtype_code(draft_logits), _ptr(parents), B, N, V,
                               int(max_children), float(temperature), _ptr(node_tokens), _ptr(node_logq),
                               _stream(stream))
    _check("spec_tree_draft", st)
    return node_tokens, node_logq


# ---------------------------------------------------------------------------
# serving steps around verification
#
# These check every tensor's type and shape (the C side gets bare pointers), run
# with the tensors' device current, and allocate outputs that are not supplied on
# the stream that the call uses.
# ---------------------------------------------------------------------------
def _take(t, name: str, dtype, shape, dev: int):
    """A tensor argument's address, after a look at its type, shape, device and
    layout; None for an argument that is None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _serve(fn):
    """Runs a serving call on its tensors' device (its first argument's) and the given
    stream: fn gets the device's index and the stream's handle."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if not args and name not in kw:
            raise TypeError(f"{fn.__name__}() missing argument: '{name}'")
        first = args[0] if args else kw[name]
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError(f"{fn.__name__}: tensors must be CUDA tensors")
        dev = first.get_device()
        if stream is None and dev == torch._C._cuda_getDevice():
            return fn(*args, dev=dev, stream=torch._C._cuda_getCurrentRawStream(dev), **kw)
        if stream is not None and stream.device.index != dev:
            raise ValueError(f"{fn.__name__}: the stream is on {stream.device}, the tensors on cuda:{dev}")
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return fn(*args, dev=dev, stream=torch._C._cuda_getCurrentRawStream(dev), **kw)
    return call


def _cols(t, rows, name):
    """Shape [rows, any] of a two-dimensional argument."""
    if t is None:
        return None
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(t.shape)}")
    return (rows, t.shape[1])


def spec_q4_block_bytes(D: int) -> int:
    """Bytes of a block of 32 tokens of one kv head (36 * D); 0 if D is not 64 or 128."""
    return int(lib().spec_q4_block_bytes(D))


def spec_attend_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().spec_attend_workspace_bytes(B, N, Hq, Hkv, D))


def q4_cache(num_pages: int, Hkv: int, page_tokens: int, D: int, device) -> torch.Tensor:
    """An empty 4-bit cache [num_pages, Hkv, page_tokens / 32, 36 * D] (bytes)."""
    if page_tokens % 32 or D not in (64, 128):
        raise ValueError("page_tokens must be a multiple of 32 and D 64 or 128")
    return torch.zeros((num_pages, Hkv, page_tokens // 32, 36 * D), dtype=torch.uint8, device=device)


def _q4_shape(cache, name="cache"):
    """(pages, Hkv, page_tokens, D) of a cache tensor."""
    if cache.dim() != 4 or cache.shape[3] % 36:
        raise ValueError(f"{name} must be [pages, Hkv, page_tokens / 32, 36 * D], got {tuple(cache.shape)}")
    return cache.shape[0], cache.shape[1], 32 * cache.shape[2], cache.shape[3] // 36


@_serve
def spec_page_map(lengths, count, held, ring, ring_state, block_table, page_tokens: int, max_tokens: int, *,
                  offsets=None, slots=None, positions=None, new_held=None, new_ring_state=None, status=None,
                  dev=None, stream=None):
    """Block tables and slot maps from the requests' lengths.  lengths, count, held
    [B] int32; ring [F], ring_state [2], block_table [B, W] int32 (ring and table
    updated in place).  Returns (offsets [B+1], slots [max_tokens], positions
    [max_tokens], new_held [B], new_ring_state [2], status [B]), all int32; those
    not supplied are parts of one allocation."""
    i32, B = torch.int32, lengths.numel()
    one, given = (B,), (slots, positions, offsets, new_held, status, new_ring_state)
    sizes = (max_tokens, max_tokens, B + 1, B, B, 2)
    if all(t is None for t in given):
        pad = -max_tokens % 4   # slots and positions start at 16-byte borders
        new = torch.empty(2 * (max_tokens + pad) + 3 * B + 3, dtype=i32, device=lengths.device)
        at = new.data_ptr()
        slots, _, positions, _, offsets, new_held, status, new_ring_state = new.split_with_sizes(
            (max_tokens, pad, max_tokens, pad, B + 1, B, B, 2))
        rest = at + 8 * (max_tokens + pad)
        to = (at, at + 4 * (max_tokens + pad), rest, rest + 4 * (B + 1), rest + 4 * (2 * B + 1), rest + 4 * (3 * B + 1))
    else:
        slots, positions, offsets, new_held, status, new_ring_state = out = tuple(
            torch.empty(n, dtype=i32, device=lengths.device) if t is None else t for t, n in zip(given, sizes))
        to = tuple(_take(t, name, i32, (n,), dev) for t, name, n in zip(
            out, ("slots", "positions", "offsets", "new_held", "status", "new_ring_state"), sizes))
    table = _cols(block_table, B, "block_table")
    st = (_lib or lib()).spec_page_map(
        _take(lengths, "lengths", i32, one, dev), _take(count, "count", i32, one, dev), _take(held, "held", i32, one, dev),
        _take(ring, "ring", i32, (ring.numel(),), dev), _take(ring_state, "ring_state", i32, (2,), dev),
        _take(block_table, "block_table", i32, table, dev), B, ring.numel(), page_tokens, table[1], max_tokens,
        to[2], to[0], to[1], to[3], to[5], to[4], stream)
    if st:
        _check("spec_page_map", st)
    return offsets, slots, positions, new_held, new_ring_state, status


@_serve
def spec_kv_store_q4(k, v, slots, cache, *, k_shift: int = 0, v_shift: int = 0, dev=None, stream=None):
    """Entries t of k and v [T, Hkv, D] bf16 into the 4-bit cache at slots[t]
    ([T] int32; a slot outside the cache is skipped).  Returns the cache."""
    pages, Hkv, P, D = _q4_shape(cache)
    T = k.shape[0]
    st = (_lib or lib()).spec_kv_store_q4(
        _take(k, "k", torch.bfloat16, (T, Hkv, D), dev), _take(v, "v", torch.bfloat16, (T, Hkv, D), dev),
        _take(slots, "slots", torch.int32, (T,), dev), T, Hkv, D, P, pages, k_shift, v_shift,
        _take(cache, "cache", torch.uint8, cache.shape, dev), stream)
    if st:
        _check("spec_kv_store_q4", st)
    return cache


@_serve
def spec_kv_commit_q4(cache, block_table, lengths, k, v, count, *, path=None, new_lengths=None, k_shift: int = 0,
                      v_shift: int = 0, dev=None, stream=None):
    """Appends accepted entries of k and v [B, N, Hkv, D] bf16 to the paged 4-bit
    cache behind lengths [B]: entries path[b, :count[b]] ([B, W] int32), or the
    first count[b] without a path.  block_table [B, pages].  Returns new_lengths."""
    pages, Hkv, P, D = _q4_shape(cache)
    i32, bf = torch.int32, torch.bfloat16
    if k.dim() != 4:
        raise ValueError(f"k must be [B, N, Hkv, D], got {tuple(k.shape)}")
    B, N = k.shape[0], k.shape[1]
    if new_lengths is None:
        new_lengths = torch.empty((B,), dtype=i32, device=cache.device)
    table, way = _cols(block_table, B, "block_table"), _cols(path, B, "path")
    st = (_lib or lib()).spec_kv_commit_q4(
        _take(cache, "cache", torch.uint8, cache.shape, dev), _take(block_table, "block_table", i32, table, dev),
        _take(lengths, "lengths", i32, (B,), dev), _take(k, "k", bf, (B, N, Hkv, D), dev), _take(v, "v", bf, (B, N, Hkv, D), dev),
        _take(path, "path", i32, way, dev), _take(count, "count", i32, (B,), dev), B, N, 0 if path is None else way[1], Hkv, D,
        P, pages, table[1], k_shift, v_shift, _take(new_lengths, "new_lengths", i32, (B,), dev), stream)
    if st:
        _check("spec_kv_commit_q4", st)
    return new_lengths


@_serve
def spec_attend_q4(q, cache, block_table, lengths, *, k_new=None, v_new=None, masks=None, scale=None, k_shift: int = 0,
                   v_shift: int = 0, out=None, lse=None, workspace_buf=None, dev=None, stream=None):
    """Attention of N nodes per sequence over the paged 4-bit cache and the nodes'
    own entries.  q [B, N, Hq, D], k_new / v_new [B, N, Hkv, D] bf16 (or neither),
    masks [B, N, ceil(N/32)] int32 (spec_tree_mask's; None: a chain), block_table
    [B, pages], lengths [B] int32; scale defaults to 1 / sqrt(D).  Returns (out
    [B, N, Hq, D] bf16, lse [B, N, Hq] f32)."""
    pages, Hkv, P, D = _q4_shape(cache)
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    if q.dim() != 4:
        raise ValueError(f"q must be [B, N, Hq, D], got {tuple(q.shape)}")
    B, N, Hq = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = torch.empty((B, N, Hq, D), dtype=bf, device=q.device)
    if lse is None:
        lse = torch.empty((B, N, Hq), dtype=f32, device=q.device)
    if workspace_buf is None:
        workspace_buf = workspace(spec_attend_workspace_bytes(B, N, Hq, Hkv, D), q.device)
    table = _cols(block_table, B, "block_table")
    st = (_lib or lib()).spec_attend_q4(
        _take(q, "q", bf, (B, N, Hq, D), dev), _take(k_new, "k_new", bf, (B, N, Hkv, D), dev),
        _take(v_new, "v_new", bf, (B, N, Hkv, D), dev), _take(masks, "masks", i32, (B, N, (N + 31) // 32), dev),
        _take(cache, "cache", torch.uint8, cache.shape, dev), _take(block_table, "block_table", i32, table, dev),
        _take(lengths, "lengths", i32, (B,), dev), B, N, Hq, Hkv, D, P, pages, table[1], k_shift, v_shift,
        D ** -0.5 if scale is None else scale, _take(out, "out", bf, (B, N, Hq, D), dev), _take(lse, "lse", f32, (B, N, Hq), dev),
        _take(workspace_buf, "workspace_buf", torch.uint8, (workspace_buf.numel(),), dev), workspace_buf.numel(), stream)
    if st:
        _check("spec_attend_q4", st)
    return out, lse


@_serve
def spec_debug_attend_stall(q, cache, block_table, lengths, stall_cta: int, timeout_us: int, *, k_new=None, v_new=None,
                            dev=None, stream=None):
    """Test hook: spec_attend_q4 with short wait limits while CTA stall_cta waits for an
    arrival that never comes.  Returns (out, lse); what waits for it is NaN."""
    pages, Hkv, P, D = _q4_shape(cache)
    B, N, Hq = q.shape[0], q.shape[1], q.shape[2]
    i32, bf = torch.int32, torch.bfloat16
    out = torch.empty_like(q)
    lse = torch.empty((B, N, Hq), dtype=torch.float32, device=q.device)
    ws = workspace(spec_attend_workspace_bytes(B, N, Hq, Hkv, D), q.device)
    table = _cols(block_table, B, "block_table")
    st = lib().spec_debug_attend_stall(
        _take(q, "q", bf, (B, N, Hq, D), dev), _take(k_new, "k_new", bf, (B, N, Hkv, D), dev),
        _take(v_new, "v_new", bf, (B, N, Hkv, D), dev), None, _take(cache, "cache", torch.uint8, cache.shape, dev),
        _take(block_table, "block_table", i32, table, dev), _take(lengths, "lengths", i32, (B,), dev), B, N, Hq, Hkv, D, P,
        pages, table[1], 0, 0, D ** -0.5, int(stall_cta), int(timeout_us), out.data_ptr(), lse.data_ptr(), ws.data_ptr(),
        ws.numel(), stream)
    _check("spec_debug_attend_stall", st)
    return out, lse


@_serve
def spec_adjust_logits(logits, *, out=None, history=None, prompt_lengths=None, history_lengths=None, repetition=None,
                       frequency=None, presence=None, node_tokens=None, masks=None, bias_tokens=None,
                       bias_values=None, allowed=None, dev=None, stream=None):
    """Penalties, biases and grammar masks on logits [B, R, V] (bf16/f32).  history
    [B, H] int32 with prompt_lengths and history_lengths [B]; repetition,
    frequency, presence [B] f32; node_tokens [B, Nt] int32 (row r sees the first r
    of them, or with masks [B, R, ceil(R/32)] int32 the row's ancestors);
    bias_tokens / bias_values [B, M]; allowed [B, R, ceil(V/32)] int32 bit words.
    out may be logits.  Returns out."""
    if logits.dim() != 3:
        raise ValueError(f"logits must be [B, R, V], got {tuple(logits.shape)}")
    B, R, V = logits.shape
    i32, f32, one, shape, dt = torch.int32, torch.float32, (B,), (B, R, V), logits.dtype
    code = _dtype_code(logits)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=logits.device)
    past, nodes, biased = _cols(history, B, "history"), _cols(node_tokens, B, "node_tokens"), _cols(bias_tokens, B, "bias_tokens")
    st = (_lib or lib()).spec_adjust_logits(
        _take(logits, "logits", dt, shape, dev), code, _take(history, "history", i32, past, dev),
        _take(prompt_lengths, "prompt_lengths", i32, one, dev), _take(history_lengths, "history_lengths", i32, one, dev),
        _take(repetition, "repetition", f32, one, dev), _take(frequency, "frequency", f32, one, dev),
        _take(presence, "presence", f32, one, dev), _take(node_tokens, "node_tokens", i32, nodes, dev),
        _take(masks, "masks", i32, (B, R, (R + 31) // 32), dev), _take(bias_tokens, "bias_tokens", i32, biased, dev),
        _take(bias_values, "bias_values", f32, biased or _cols(bias_values, B, "bias_values"), dev),
        _take(allowed, "allowed", i32, (B, R, (V + 31) // 32), dev), B, R, V, past[1] if past else 0,
        nodes[1] if nodes else 0, biased[1] if biased else 0, _take(out, "out", dt, shape, dev), stream)
    if st:
        _check("spec_adjust_logits", st)
    return out


# ---------------------------------------------------------------------------
# steps after a verification
# ---------------------------------------------------------------------------
@_serve
def spec_token_logprobs(logits, tokens, temperature: float = 1.0, *, path=None, top_n: int = 0, logprobs=None, entropy=None,
                        ranks=None, top_tokens=None, top_logprobs=None, dev=None, stream=None):
    """Log probabilities of tokens [B, M] int32 (negative: none) under logits [B, R, V]
    (bf16/f32) at a temperature; token m belongs to row m, or with path [B, W] int32
    (out_path) to row 0 (m = 0) or path[b, m - 1].  Returns (logprobs, entropy [B, M] f32,
    ranks [B, M] int32, top_tokens int32, top_logprobs f32 [B, M, top_n])."""
    if logits.dim() != 3 or tokens.dim() != 2:
        raise ValueError(f"logits must be [B, R, V] and tokens [B, M], got {tuple(logits.shape)} and {tuple(tokens.shape)}")
    B, R, V = logits.shape
    M = tokens.shape[1]
    i32, f32, two, three = torch.int32, torch.float32, (B, M), (B, M, top_n)
    if logprobs is entropy is ranks is top_tokens is top_logprobs is None:   # (allocations are cheaper than views of one)
        on = logits.device
        logprobs, entropy = torch.empty(two, dtype=f32, device=on), torch.empty(two, dtype=f32, device=on)
        ranks, top_tokens = torch.empty(two, dtype=i32, device=on), torch.empty(three, dtype=i32, device=on)
        top_logprobs = torch.empty(three, dtype=f32, device=on)
        to = (logprobs.data_ptr(), entropy.data_ptr(), ranks.data_ptr(), top_tokens.data_ptr(), top_logprobs.data_ptr())
    else:
        logprobs, entropy, ranks, top_tokens, top_logprobs = out = tuple(
            torch.empty(shape, dtype=dt, device=logits.device) if t is None else t for t, shape, dt in (
                (logprobs, two, f32), (entropy, two, f32), (ranks, two, i32), (top_tokens, three, i32), (top_logprobs, three, f32)))
        to = tuple(_take(t, name, dt, shape, dev) for t, name, dt, shape in zip(
            out, ("logprobs", "entropy", "ranks", "top_tokens", "top_logprobs"), (f32, f32, i32, i32, f32), (two, two, two, three, three)))
    way = _cols(path, B, "path")
    st = (_lib or lib()).spec_token_logprobs(
        _take(logits, "logits", logits.dtype, (B, R, V), dev), _dtype_code(logits), _take(tokens, "tokens", i32, two, dev),
        _take(path, "path", i32, way, dev), temperature, B, R, V, M, way[1] if way else 0, top_n, *to, stream)
    if st:
        _check("spec_token_logprobs", st)
    return logprobs, entropy, ranks, top_tokens, top_logprobs


@_serve
def spec_kv_weigh_q4(q, lse, cache, block_table, lengths, weights, *, count=None, path=None, positions=None,
                     first_positions=None, new_weights=None, scale=None, decay: float = 1.0, k_shift: int = 0, dev=None, stream=None):
    """Adds to weights [pages, Hkv, page_tokens] f32 what the committed rows of q [B, N, Hq,
    D] bf16 with lse [B, N, Hq] f32 gave to each cached token: rows path[b, :count[b]], or
    the first count[b] (None: all); lengths [B] before the commit.  Marks the committed
    tokens in positions (int32, weights' shape).  In place unless new_weights is given;
    returns it."""
    pages, Hkv, P, D = _q4_shape(cache)
    i32, f32 = torch.int32, torch.float32
    if q.dim() != 4:
        raise ValueError(f"q must be [B, N, Hq, D], got {tuple(q.shape)}")
    B, N, Hq = q.shape[0], q.shape[1], q.shape[2]
    if new_weights is None:
        new_weights = weights
    one, slots = (B,), (pages, Hkv, P)
    table, way = _cols(block_table, B, "block_table"), _cols(path, B, "path")
    st = (_lib or lib()).spec_kv_weigh_q4(
        _take(q, "q", torch.bfloat16, (B, N, Hq, D), dev), _take(lse, "lse", f32, (B, N, Hq), dev), _take(path, "path", i32, way, dev),
        _take(count, "count", i32, one, dev), _take(cache, "cache", torch.uint8, cache.shape, dev),
        _take(block_table, "block_table", i32, table, dev), _take(lengths, "lengths", i32, one, dev),
        _take(first_positions, "first_positions", i32, one, dev), B, N, way[1] if way else 0, Hq, Hkv, D, P, pages, table[1],
        k_shift, D ** -0.5 if scale is None else scale, decay, _take(weights, "weights", f32, slots, dev),
        _take(new_weights, "new_weights", f32, slots, dev), _take(positions, "positions", i32, slots, dev), stream)
    if st:
        _check("spec_kv_weigh_q4", st)
    return new_weights


@_serve
def spec_kv_evict_plan(weights, positions, block_table, lengths, budgets, next_positions, *, sinks: int = 0, recent: int = 0,
                       max_moves=None, moves=None, move_counts=None, new_lengths=None, dev=None, stream=None):
    """Which tokens each kv head keeps when sequences are cut to budgets [B], and the moves
    that fill the places below.  weights f32 and positions int32 [pages, Hkv, page_tokens],
    lengths, next_positions [B] int32; room for max_moves a head (or moves' own).
    Returns (moves [B, Hkv, max_moves, 2], move_counts [B, Hkv], new_lengths [B]) int32."""
    if weights.dim() != 3:
        raise ValueError(f"weights must be [pages, Hkv, page_tokens], got {tuple(weights.shape)}")
    (pages, Hkv, P), B, i32 = weights.shape, lengths.numel(), torch.int32
    if moves is not None:
        if moves.dim() != 4 or max_moves not in (None, moves.shape[2]):
            raise ValueError(f"moves must be [B, Hkv, max_moves, 2], got {tuple(moves.shape)} with max_moves={max_moves}")
        max_moves = moves.shape[2]
    elif max_moves is None:
        raise ValueError("spec_kv_evict_plan: max_moves or moves is needed")
    else:
        moves = torch.empty((B, Hkv, max_moves, 2), dtype=i32, device=weights.device)
    one, slots, table = (B,), (pages, Hkv, P), _cols(block_table, B, "block_table")
    if move_counts is None:
        move_counts = torch.empty((B, Hkv), dtype=i32, device=weights.device)
    if new_lengths is None:
        new_lengths = torch.empty(one, dtype=i32, device=weights.device)
    st = (_lib or lib()).spec_kv_evict_plan(
        _take(weights, "weights", torch.float32, slots, dev), _take(positions, "positions", i32, slots, dev),
        _take(block_table, "block_table", i32, table, dev), _take(lengths, "lengths", i32, one, dev),
        _take(budgets, "budgets", i32, one, dev), _take(next_positions, "next_positions", i32, one, dev), B, Hkv, P, pages,
        table[1], sinks, recent, max_moves, _take(moves, "moves", i32, (B, Hkv, max_moves, 2), dev),
        _take(move_counts, "move_counts", i32, (B, Hkv), dev), _take(new_lengths, "new_lengths", i32, one, dev), stream)
    if st:
        _check("spec_kv_evict_plan", st)
    return moves, move_counts, new_lengths


@_serve
def spec_kv_move_q4(cache, moves, move_counts, *, weights=None, positions=None, dev=None, stream=None):
    """A plan's moves [B, Hkv, max_moves, 2] int32 (the first move_counts[b, h] of each head)
    in the 4-bit cache and, given, in weights f32 and positions int32 [pages, Hkv,
    page_tokens].  Returns the cache."""
    pages, Hkv, P, D = _q4_shape(cache)
    if moves.dim() != 4:
        raise ValueError(f"moves must be [B, Hkv, max_moves, 2], got {tuple(moves.shape)}")
    B, most, i32, slots = moves.shape[0], moves.shape[2], torch.int32, (pages, Hkv, P)
    st = (_lib or lib()).spec_kv_move_q4(
        _take(cache, "cache", torch.uint8, cache.shape, dev), _take(weights, "weights", torch.float32, slots, dev),
        _take(positions, "positions", i32, slots, dev), _take(moves, "moves", i32, (B, Hkv, most, 2), dev),
        _take(move_counts, "move_counts", i32, (B, Hkv), dev), B, Hkv, D, P, pages, most, stream)
    if st:
        _check("spec_kv_move_q4", st)
    return cache


@_serve
def spec_page_trim(tokens, held, ring, ring_state, block_table, page_tokens: int, *, new_held=None, new_ring_state=None,
                   status=None, dev=None, stream=None):
    """Gives the pages that tokens [B] int32 do not need back to spec_page_map's ring
    (updated in place).  Returns (new_held [B], new_ring_state [2], status [B]) int32."""
    i32, B = torch.int32, tokens.numel()
    if new_held is new_ring_state is status is None:
        on = tokens.device
        new_held, new_ring_state, status = (torch.empty(B, dtype=i32, device=on), torch.empty(2, dtype=i32, device=on),
                                            torch.empty(B, dtype=i32, device=on))
        to = (new_held.data_ptr(), new_ring_state.data_ptr(), status.data_ptr())
    else:
        new_held, new_ring_state, status = out = tuple(
            torch.empty(n, dtype=i32, device=tokens.device) if t is None else t for t, n in ((new_held, B), (new_ring_state, 2), (status, B)))
        to = tuple(_take(t, name, i32, (n,), dev) for t, name, n in zip(out, ("new_held", "new_ring_state", "status"), (B, 2, B)))
    one, table = (B,), _cols(block_table, B, "block_table")
    st = (_lib or lib()).spec_page_trim(
        _take(tokens, "tokens", i32, one, dev), _take(held, "held", i32, one, dev), _take(ring, "ring", i32, (ring.numel(),), dev),
        _take(ring_state, "ring_state", i32, (2,), dev), _take(block_table, "block_table", i32, table, dev), B, ring.numel(),
        page_tokens, table[1], *to, stream)
    if st:
        _check("spec_page_trim", st)
    return new_held, new_ring_state, status


def spec_profile_begin(max_calls: int):
    _check("spec_profile_begin", lib().spec_profile_begin(int(max_calls)))


def spec_profile_end():
    """(sweep_ms_total, finish_ms_total, calls) over the recorded calls."""
    a, b, n = ctypes.c_float(), ctypes.c_float(), ctypes.c_int()
    _check("spec_profile_end", lib().spec_profile_end(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n)))
    return a.value, b.value, n.value
