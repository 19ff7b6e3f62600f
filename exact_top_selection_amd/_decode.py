"""The operators around the selection in a sparse decode step (C ABI:
``include/ets_decode.h``).

* :func:`rope`            -- rotary positions of queries and keys;
* :func:`cache_write`,
  :func:`cache_read`      -- the 8-bit cache: e4m3 codes [S, H, D] with one
  power-of-two scale byte for each 32 values, value = code * 2^(byte - 127);
* :func:`index_scores`    -- the indexer scores that ``topk_paged`` ranks;
* :func:`attend_selected`,
  :func:`attend_paged`    -- attention over selected slots, or over whole
  sequences, with a tree of drafted tokens in either form.

Like the rest of the binding this module only checks and marshals arguments;
every value is computed in the HIP kernels on torch's current stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad as _forward

from . import _check, _load, _on, _require, _rows, _same_device, _stream, _vec

CACHE_BLOCK = 32
MAX_ROPE_DIM, MAX_HEAD_DIM, MAX_INDEX_DIM, MAX_INDEX_HEADS, MAX_TREE = 4096, 576, 256, 128, 64
MAX_LENGTH = 0x7FFFF000  # positions of a sequence, slots of a list
_INT32 = 0x7FFFFFFF      # sizes are 32-bit numbers in the C ABI, which ctypes would cut silently
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUTS = {"interleaved": 0, "half": 1}

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class _AttendArgs(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "T", "Hq", "Hkv", "D", "Dv", "dtype", "K", "L", "page_size")]
                + [("S", _i64), ("q", _vp), ("q_b", _i64), ("q_t", _i64), ("q_h", _i64)]
                + [(n, t) for c in "kv" for n, t in ((c + "_codes", _vp), (c + "_s", _i64), (c + "_h", _i64),
                                                     (c + "_scales", _vp), (c + "s_s", _i64), (c + "s_h", _i64))]
                + [("slots", _vp), ("slots_b", _i64), ("slots_t", _i64), ("page_table", _vp), ("pt_b", _i64),
                   ("seq_lens", _vp), ("tree_slots", _vp), ("tree_b", _i64), ("tree_mask", _vp), ("mask_b", _i64),
                   ("out", _vp), ("lse", _vp)])


_typed = False


def _lib():
    global _typed
    lib = _load()
    if not _typed:
        lib.ets_rope.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _i32, _i32, _i32,
                                 ctypes.c_double, _i32, _i32, _vp]
        lib.ets_cache_write.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _i64,
                                        _i32, _vp]
        lib.ets_cache_read.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp]
        lib.ets_index_scores.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i64, _vp,
                                         _i64, _i64, _vp, _i64, _vp, _i32, _i32, _vp, _i64, _i32, _vp]
        lib.ets_attend_workspace_size.argtypes = [ctypes.POINTER(_AttendArgs), ctypes.POINTER(_sz)]
        lib.ets_attend.argtypes = [ctypes.POINTER(_AttendArgs), _vp, _sz, _vp]
        for fn in (lib.ets_rope, lib.ets_cache_write, lib.ets_cache_read, lib.ets_index_scores,
                   lib.ets_attend_workspace_size, lib.ets_attend):
            fn.restype = _i32
        _typed = True
    return lib


def _floats(t: torch.Tensor, name: str, dim: int, types: str = "bf16, fp16 or fp32") -> int:
    """Checks a floating tensor whose innermost dimension is contiguous; its type's number."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    kind = _DTYPES.get(t.dtype)
    if kind is None or (kind == 2 and "fp32" not in types):
        raise TypeError("%s must be %s, got %s" % (name, types, t.dtype))
    if t.ndim != dim:
        raise ValueError("%s must be %d-D, got shape %s" % (name, dim, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be on a HIP device, got %s" % (name, t.device))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    return kind


def _vector(t: torch.Tensor, name: str, n: int, index: int) -> int:
    """Address of a contiguous int32 [n] on device `index`: one test where all is well, the binding's messages where not."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == (n,) and t.get_device() == index
            and (n < 2 or t.stride(0) == 1)):
        _vec(t, name, n)
        _same_device(index, (t, name))
    return t.data_ptr()


def _run(index: int, what: str, fn, *args) -> None:
    """fn(*args, current stream of device `index`) with that device current; raises on a status."""
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _stream(index))
    if st:
        _check(st, what)


def _no_grad(t: torch.Tensor, name: str, what: str, instead: str = "call it under torch.no_grad()") -> None:
    """Refuses a tensor whose gradient or tangent the call would drop."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s records no gradient: detach %s, or %s" % (what, name, instead))
    if _forward._current_level >= 0 and _forward.unpack_dual(t).tangent is not None:
        raise ValueError("%s has no forward-mode derivative: take the primal of %s" % (what, name))


def _cache(codes: torch.Tensor, scales: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """Checks a cache; (S, H, D)."""
    if not isinstance(codes, torch.Tensor) or not isinstance(scales, torch.Tensor):
        raise TypeError("%scodes and %sscales must be torch.Tensors" % (name, name))
    if codes.dtype is not torch.float8_e4m3fn and codes.dtype is not torch.uint8:
        raise TypeError("%scodes must be torch.float8_e4m3fn (or its bytes as uint8), got %s" % (name, codes.dtype))
    if codes.ndim != 3:
        raise ValueError("%scodes must be 3-D [S, H, D], got shape %s" % (name, tuple(codes.shape)))
    if not codes.is_cuda:
        raise ValueError("%scodes must be on a HIP device, got %s" % (name, codes.device))
    _require(scales, name + "scales", torch.uint8, 3)
    S, H, D = codes.shape
    if D < CACHE_BLOCK or D % CACHE_BLOCK:
        raise ValueError("%scodes must have a multiple of %d channels, got %d" % (name, CACHE_BLOCK, D))
    if H < 1 or S > _INT32 or H * D > 1 << 28:
        raise ValueError("%scodes must have at least one head, at most 2^28 values a slot and fewer than 2^31 slots" % name)
    if scales.shape != (S, H, D // CACHE_BLOCK):
        raise ValueError("%sscales must have shape %s, got %s" % (name, (S, H, D // CACHE_BLOCK), tuple(scales.shape)))
    if codes.stride(2) != 1 or (D > CACHE_BLOCK and scales.stride(2) != 1):
        raise ValueError("%scodes and %sscales must be contiguous in their last dimension" % (name, name))
    return S, H, D


def _overlaps(t: torch.Tensor) -> bool:
    """Whether two rows of a 3-D tensor to be written could be the same memory."""
    (n, h, d), (sn, sh, _) = t.shape, t.stride()
    if n <= 1 or h <= 1:
        return (n > 1 and sn < d) or (h > 1 and sh < d)
    return sh < d or sn < d or (sn < (h - 1) * sh + d and sh < (n - 1) * sn + d)


def rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, layout: str = "interleaved", offset: int = 0,
         scale: float = 1.0, inverse: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotates channels [offset, offset + R) of ``x`` [N, H, D], R = 2 * len(inv_freq), and copies the others.

    Pair i of token n turns by ``positions[n] * inv_freq[i]`` (int32 [N]; float64 [R / 2], radians a position) and is
    multiplied by ``scale``.  Pairs are channels (2i, 2i + 1) for layout "interleaved", (i, R / 2 + i) for "half".
    Frequencies that were stretched for long contexts, and the factor that goes with them, come in ``inv_freq`` and
    ``scale``.  ``inverse`` turns the other way and multiplies by the same scale: the transposed map, which is the
    gradient's (the gradient of ``rope(x, ...)`` is ``rope(grad, ..., inverse=True)``; no autograd graph is built).
    ``x`` is bf16, fp16 or fp32; ``out`` may be ``x``.
    """
    kind = _floats(x, "x", 3)
    _no_grad(x, "x", "rope", "take its gradient as rope(grad, ..., inverse=True)")
    N, H, D = x.shape
    strides = x.stride()
    index = x.get_device()
    at = _vector(positions, "positions", N, index)
    if not (isinstance(inv_freq, torch.Tensor) and inv_freq.dtype is torch.float64 and inv_freq.ndim == 1
            and inv_freq.get_device() == index):
        _require(inv_freq, "inv_freq", torch.float64, 1)
        _same_device(index, (inv_freq, "inv_freq"))
    _no_grad(inv_freq, "inv_freq", "rope")
    R = 2 * inv_freq.shape[0]
    if R > 2 and inv_freq.stride(0) != 1:
        raise ValueError("inv_freq must be contiguous")
    pairs = _LAYOUTS.get(layout)
    if pairs is None:
        raise ValueError("layout must be 'interleaved' or 'half', got %r" % (layout,))
    if D < 1 or D > MAX_ROPE_DIM or H > _INT32:
        raise ValueError("x must have 1 to %d channels and at most %d heads, got %d and %d" % (MAX_ROPE_DIM, _INT32, D, H))
    if offset < 0 or offset + R > D:
        raise ValueError("channels [%d, %d) do not lie inside the %d of x" % (offset, offset + R, D))
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        to_n, to_h = H * D, D
    else:
        _floats(out, "out", 3)
        _no_grad(out, "out", "rope")
        if out.shape != x.shape or out.dtype is not x.dtype or out.get_device() != index:
            raise ValueError("out must have the shape, type and device of x")
        if _overlaps(out):
            raise ValueError("rows of out must not overlap")
        if out.data_ptr() == x.data_ptr() and out.stride() != strides:
            raise ValueError("out may be x itself, or memory apart from it")
        to_n, to_h, _ = out.stride()
    _run(index, "ets_rope", _lib().ets_rope, x.data_ptr(), strides[0], strides[1], out.data_ptr(), to_n, to_h, N, H, D, at,
         inv_freq.data_ptr(), R, offset, pairs, scale, 1 if inverse else 0, kind)
    return out


def cache_write(x: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor) -> None:
    """Quantises rows ``x`` [N, H, D] (bf16, fp16 or fp32) into slots ``slots`` (int32 [N]) of a cache.

    ``codes`` float8_e4m3fn [S, H, D], ``scales`` uint8 [S, H, D / 32].  A block of 32 values gets the smallest power of
    two that keeps it within +-448.  Slots outside [0, S) are skipped; the others of one call must differ.
    """
    kind = _floats(x, "x", 3)
    _no_grad(x, "x", "cache_write")
    S, H, D = _cache(codes, scales, "")
    N = x.shape[0]
    if x.shape[1] != H or x.shape[2] != D:
        raise ValueError("x must have shape [N, %d, %d], got %s" % (H, D, tuple(x.shape)))
    index = x.get_device()
    at = _vector(slots, "slots", N, index)
    _same_device(index, (codes, "codes"), (scales, "scales"))
    if _overlaps(codes) or _overlaps(scales):
        raise ValueError("rows of codes and scales must not overlap")
    from_n, from_h, _ = x.stride()
    codes_s, codes_h, _ = codes.stride()
    scales_s, scales_h, _ = scales.stride()
    _run(index, "ets_cache_write", _lib().ets_cache_write, x.data_ptr(), from_n, from_h, N, H, D, at, codes.data_ptr(), codes_s,
         codes_h, scales.data_ptr(), scales_s, scales_h, S, kind)


def cache_read(codes: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of the cache's rows ``slots`` (int32 [N]) as [N, H, D] of ``dtype``; zeros for slots outside [0, S)."""
    S, H, D = _cache(codes, scales, "")
    index = codes.get_device()
    if not isinstance(slots, torch.Tensor) or slots.ndim != 1:
        _require(slots, "slots", torch.int32, 1)
    N = slots.shape[0]
    at = _vector(slots, "slots", N, index)
    _same_device(index, (scales, "scales"))
    kind = _DTYPES.get(dtype)
    if kind is None:
        raise TypeError("dtype must be torch.bfloat16, torch.float16 or torch.float32, got %s" % (dtype,))
    if out is None:
        out = codes.new_empty((N, H, D), dtype=dtype)
    elif out.dtype is not dtype or out.shape != (N, H, D) or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be contiguous %s [%d, %d, %d] on cuda:%d" % (dtype, N, H, D, index))
    else:
        _no_grad(out, "out", "cache_read")
    codes_s, codes_h, _ = codes.stride()
    scales_s, scales_h, _ = scales.stride()
    _run(index, "ets_cache_read", _lib().ets_cache_read, codes.data_ptr(), codes_s, codes_h, scales.data_ptr(), scales_s,
         scales_h, S, at, N, H, D, out.data_ptr(), kind)
    return out


def _pages(page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int, L: int, B: int) -> None:
    _require(page_table, "page_table", torch.int32, 2)
    _vec(seq_lens, "seq_lens", B)
    if page_table.shape[0] != B:
        raise ValueError("page_table must have %d rows, got %d" % (B, page_table.shape[0]))
    if not 1 <= page_size <= _INT32 or not 0 <= L <= MAX_LENGTH:
        raise ValueError("page_size must be 1 to %d and L 0 to %d, got %s and %s" % (_INT32, MAX_LENGTH, page_size, L))
    if page_table.shape[1] * page_size < L:
        raise ValueError("page_table has %d pages of %d, fewer than L = %d positions"
                         % (page_table.shape[1], page_size, L))


def index_scores(q: torch.Tensor, weights: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int, L: int,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Indexer scores, float32 [B * T, L], row b * T + t: the rows that the selection ranks.

    Score of position p: sum over h of weights[b, t, h] * max(0, q[b, t, h] . key), the key being the cache's row at slot
    page_table[b, p // page_size] * page_size + p % page_size; -inf from min(seq_lens[b], L) on.  ``q`` is bf16 or fp16
    [B, T, H, D], ``weights`` float32 [B, T, H], the cache [S, 1, D].
    """
    kind = _floats(q, "q", 4, "bf16 or fp16")
    _no_grad(q, "q", "index_scores")
    B, T, H, D = q.shape
    index = q.get_device()
    _require(weights, "weights", torch.float32, 3)
    _no_grad(weights, "weights", "index_scores")
    if weights.shape != (B, T, H):
        raise ValueError("weights must have shape %s, got %s" % ((B, T, H), tuple(weights.shape)))
    if H > 1 and weights.stride(2) != 1:
        raise ValueError("weights must be contiguous in its last dimension")
    S, heads, Dk = _cache(codes, scales, "")
    if heads != 1 or Dk != D:
        raise ValueError("codes must have shape [S, 1, %d], got %s" % (D, tuple(codes.shape)))
    if D > MAX_INDEX_DIM or not 1 <= H <= MAX_INDEX_HEADS:
        raise ValueError("q must have 1 to %d heads of at most %d channels" % (MAX_INDEX_HEADS, MAX_INDEX_DIM))
    if B > 65535 or T > _INT32:
        raise ValueError("q must have at most 65535 sequences and %d tokens, got %d and %d" % (_INT32, B, T))
    _pages(page_table, seq_lens, page_size, L, B)
    _same_device(index, (weights, "weights"), (codes, "codes"), (scales, "scales"), (page_table, "page_table"),
                 (seq_lens, "seq_lens"))
    if out is None:
        out = torch.empty((B * T, L), dtype=torch.float32, device=q.device)
    else:
        _require(out, "out", torch.float32, 2)
        _no_grad(out, "out", "index_scores")
        if out.shape != (B * T, L) or out.get_device() != index:
            raise ValueError("out must be float32 [%d, %d] on cuda:%d" % (B * T, L, index))
        if B * T > 1 and out.stride(0) < L:
            raise ValueError("rows of out must not overlap")
    q_b, q_t, q_h, _ = q.stride()
    w_b, w_t, _ = weights.stride()
    _run(index, "ets_index_scores", _lib().ets_index_scores, q.data_ptr(), q_b, q_t, q_h, weights.data_ptr(), w_b, w_t, B, T,
         H, D, codes.data_ptr(), codes.stride(0), scales.data_ptr(), scales.stride(0), S, page_table.data_ptr(),
         _rows(page_table, "page_table"), seq_lens.data_ptr(), page_size, L, out.data_ptr(), _rows(out, "out"), kind)
    return out


def _attend(what, q, k_codes, k_scales, v_codes, v_scales, tree_slots, tree_mask, workspace, slots=None, page_table=None,
            seq_lens=None, page_size=1, L=0):
    kind = _floats(q, "q", 4, "bf16 or fp16")
    _no_grad(q, "q", what)
    B, T, Hq, D = q.shape
    index = q.get_device()
    S, Hkv, Dk = _cache(k_codes, k_scales, "k_")
    Sv, Hv, Dv = _cache(v_codes, v_scales, "v_")
    if Dk != D:
        raise ValueError("k_codes must have %d channels like q, got %d" % (D, Dk))
    if Sv != S or Hv != Hkv:
        raise ValueError("v_codes must have the slots and heads of k_codes %s, got %s" % ((S, Hkv), (Sv, Hv)))
    if D > MAX_HEAD_DIM or Dv > MAX_HEAD_DIM:
        raise ValueError("heads may have at most %d channels" % MAX_HEAD_DIM)
    if B * T * Hq > _INT32:
        raise ValueError("q must have at most %d rows, got %d" % (_INT32, B * T * Hq))
    if Hq < 1 or Hq % Hkv:
        raise ValueError("q must have a multiple of the cache's %d heads, got %d" % (Hkv, Hq))
    _same_device(index, (k_codes, "k_codes"), (k_scales, "k_scales"), (v_codes, "v_codes"), (v_scales, "v_scales"),
                 (slots, "slots"), (page_table, "page_table"), (seq_lens, "seq_lens"), (tree_slots, "tree_slots"),
                 (tree_mask, "tree_mask"))
    if (tree_slots is None) != (tree_mask is None):
        raise ValueError("tree_slots and tree_mask go together")
    if tree_slots is not None:
        _require(tree_slots, "tree_slots", torch.int32, 2)
        _require(tree_mask, "tree_mask", torch.int64, 2)
        if T > MAX_TREE:
            raise ValueError("a tree has at most %d tokens, got %d" % (MAX_TREE, T))
        if tree_slots.shape != (B, T) or tree_mask.shape != (B, T):
            raise ValueError("tree_slots and tree_mask must have shape %s" % ((B, T),))
    out = q.new_empty((B, T, Hq, Dv))
    lse = q.new_empty((B, T, Hq), dtype=torch.float32)
    sel, sel_b, sel_t, K, table, pt_b, lens = None, 0, 0, 0, None, 0, None
    if slots is not None:
        # an empty list is a list: its address stands for the form of the call
        sel, K, (sel_b, sel_t, _) = slots.data_ptr() or q.data_ptr(), slots.shape[2], slots.stride()
    else:
        table, pt_b, lens = page_table.data_ptr(), _rows(page_table, "page_table"), seq_lens.data_ptr()
    tree, tree_b, mask, mask_b = None, 0, None, 0
    if tree_slots is not None:
        tree, tree_b = tree_slots.data_ptr(), _rows(tree_slots, "tree_slots")
        mask, mask_b = tree_mask.data_ptr(), _rows(tree_mask, "tree_mask")
    args = ctypes.byref(_AttendArgs(
        B, T, Hq, Hkv, D, Dv, kind, K, L, page_size, S, q.data_ptr(), *q.stride()[:3],
        k_codes.data_ptr(), *k_codes.stride()[:2], k_scales.data_ptr(), *k_scales.stride()[:2],
        v_codes.data_ptr(), *v_codes.stride()[:2], v_scales.data_ptr(), *v_scales.stride()[:2],
        sel, sel_b, sel_t, table, pt_b, lens, tree, tree_b, mask, mask_b, out.data_ptr(), lse.data_ptr()))
    lib = _lib()
    need = _sz(0)
    if torch._C._cuda_getDevice() == index:
        st = lib.ets_attend_workspace_size(args, ctypes.byref(need))
    else:
        st = _on(index, lib.ets_attend_workspace_size, args, ctypes.byref(need))
    if st:
        _check(st, what)
    nbytes = need.value
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous torch.Tensor on a HIP device")
        _same_device(index, (workspace, "workspace"))
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace must hold at least %d bytes" % nbytes)
    elif nbytes:
        # torch's allocator orders it on this stream, and keeps it for a graph that is being captured
        workspace = q.new_empty(nbytes, dtype=torch.uint8)
    _run(index, what, lib.ets_attend, args, workspace.data_ptr() if nbytes else None, nbytes)
    return out, lse


def attend_selected(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                    v_scales: torch.Tensor, slots: torch.Tensor, tree_slots: Optional[torch.Tensor] = None,
                    tree_mask: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of each token over its own selected cache slots: (out [B, T, Hq, Dv] of q's type, lse float32 [B, T, Hq]).

    ``q`` bf16 or fp16 [B, T, Hq, D]; caches [S, Hkv, D] and [S, Hkv, Dv], Hq a multiple of Hkv (for one shared latent
    head, v_codes and v_scales are the first channels of k_codes and k_scales); ``slots`` int32 [B, T, K] in any order,
    as ``topk_paged`` makes them: entries outside [0, S), the -1 padding among them, are not seen.  Scores are scaled by
    D^-1/2.  Drafted tokens: token t of sequence b also sees ``tree_slots[b, j]`` (int32 [B, T]) for each bit j that is
    set in ``tree_mask[b, t]`` (int64 [B, T]).  A token that sees nothing has out 0 and lse -inf.
    """
    _require(slots, "slots", torch.int32, 3)
    if not isinstance(q, torch.Tensor) or q.ndim != 4 or slots.shape[:2] != q.shape[:2]:
        raise ValueError("slots must have shape [B, T, K] like q [B, T, Hq, D], got %s" % (tuple(slots.shape),))
    if slots.shape[2] > MAX_LENGTH:
        raise ValueError("slots must have at most %d entries a token, got %d" % (MAX_LENGTH, slots.shape[2]))
    if slots.shape[2] > 1 and slots.stride(2) != 1:
        raise ValueError("slots must be contiguous in its last dimension")
    return _attend("ets_attend (selected)", q, k_codes, k_scales, v_codes, v_scales, tree_slots, tree_mask, workspace,
                   slots=slots)


def attend_paged(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int, L: int,
                 tree_slots: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of each token over all of its sequence's first min(seq_lens[b], L) positions, found through the page
    table as ``topk_paged`` finds them, and over the drafted tokens that it sees; see :func:`attend_selected`."""
    if not isinstance(q, torch.Tensor) or q.ndim != 4:
        raise ValueError("q must be a 4-D tensor [B, T, Hq, D]")
    _pages(page_table, seq_lens, page_size, L, q.shape[0])
    return _attend("ets_attend (paged)", q, k_codes, k_scales, v_codes, v_scales, tree_slots, tree_mask, workspace,
                   page_table=page_table, seq_lens=seq_lens, page_size=page_size, L=L)
