"""The operators of a speculative decode step over a pool of cache pages (C ABI: ``include/ets_speculate.h``).

* :func:`block_write`,
  :func:`block_keep`     -- the writes of a block cache: e4m3 codes [S, H, D] with one power-of-two scale byte for N slots
  and a head, [S / N, H], value = code * 2^(byte - 127);
* :func:`attend_blocks`  -- attention over it: single tokens, trees of drafted tokens, pieces of prompts;
* :func:`verify_drafts`  -- which drafted tokens stand, and the next one;
* :func:`pages_copy`, :func:`pages_extend`, :func:`pages_free`, :func:`pages_fork`,
  :func:`pages_compact`  -- the pages of a pool, whose counts and tables stay on the device.

Like the rest of the binding this module only checks and marshals arguments; every value is computed in the HIP kernels
on torch's current stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import _check, _load, _on, _require, _rows, _same_device
from ._decode import _INT32, CACHE_BLOCK, MAX_LENGTH, MAX_TREE, _floats, _no_grad, _overlaps, _run, _vector

MAX_BLOCK_DIM, MAX_BUFFERS, MAX_PAGES = 256, 64, 1 << 26

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class _BlocksArgs(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("B", "T", "Hq", "Hkv", "D", "Dv", "dtype", "block", "L", "page_size")]
                + [("S", _i64), ("q", _vp), ("q_b", _i64), ("q_t", _i64), ("q_h", _i64)]
                + [(n, t) for c in "kv" for n, t in ((c + "_codes", _vp), (c + "_s", _i64), (c + "_h", _i64),
                                                     (c + "_scales", _vp), (c + "s_s", _i64), (c + "s_h", _i64))]
                + [("page_table", _vp), ("pt_b", _i64), ("seq_lens", _vp), ("first", _vp), ("tree_mask", _vp),
                   ("mask_b", _i64), ("out", _vp), ("lse", _vp)])


class _PageBuffer(ctypes.Structure):
    _fields_ = [("data", _vp), ("page_bytes", _i64)]


_typed = False


def _lib():
    global _typed
    lib = _load()
    if not _typed:
        lib.ets_block_write.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _i64,
                                        _i32, _vp, _i64, _i32, _i32, _vp, _vp, _i32, _vp]
        lib.ets_block_keep.argtypes = [_i32, _i32, _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _i32,
                                       _i32, _vp, _vp, _i64, _vp, _vp]
        lib.ets_attend_blocks_workspace_size.argtypes = [ctypes.POINTER(_BlocksArgs), ctypes.POINTER(_sz)]
        lib.ets_attend_blocks.argtypes = [ctypes.POINTER(_BlocksArgs), _vp, _sz, _vp]
        lib.ets_verify_workspace_size.argtypes = [_i32, _i32, _i32, ctypes.POINTER(_sz)]
        lib.ets_verify_drafts.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _i64, _vp, _i64,
                                          _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp]
        buffers = ctypes.POINTER(_PageBuffer)
        lib.ets_pages_workspace_size.argtypes = [_i64, _i64, ctypes.POINTER(_sz)]
        lib.ets_pages_copy.argtypes = [buffers, _i32, _i64, _vp, _vp, _i64, _vp]
        lib.ets_pages_extend.argtypes = [_vp, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _sz, _vp]
        lib.ets_pages_free.argtypes = [_vp, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp]
        lib.ets_pages_fork.argtypes = [_vp, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _i64, _i32, _vp, buffers,
                                       _i32, _vp, _sz, _vp]
        lib.ets_pages_compact.argtypes = [_vp, _i64, _vp, _i64, _i32, _i32, _vp, buffers, _i32, _vp, _sz, _vp]
        for fn in (lib.ets_block_write, lib.ets_block_keep, lib.ets_attend_blocks_workspace_size, lib.ets_attend_blocks,
                   lib.ets_verify_workspace_size, lib.ets_verify_drafts, lib.ets_pages_workspace_size, lib.ets_pages_copy,
                   lib.ets_pages_extend, lib.ets_pages_free, lib.ets_pages_fork, lib.ets_pages_compact):
            fn.restype = _i32
        _typed = True
    return lib


def _block_cache(codes: torch.Tensor, scales: torch.Tensor, name: str, page_size: int) -> Tuple[int, int, int, int]:
    """Checks a block cache; (S, H, D, slots of a block)."""
    if not isinstance(codes, torch.Tensor) or not isinstance(scales, torch.Tensor):
        raise TypeError("%scodes and %sscales must be torch.Tensors" % (name, name))
    if codes.dtype is not torch.float8_e4m3fn and codes.dtype is not torch.uint8:
        raise TypeError("%scodes must be torch.float8_e4m3fn (or its bytes as uint8), got %s" % (name, codes.dtype))
    if codes.ndim != 3:
        raise ValueError("%scodes must be 3-D [S, H, D], got shape %s" % (name, tuple(codes.shape)))
    if not codes.is_cuda:
        raise ValueError("%scodes must be on a HIP device, got %s" % (name, codes.device))
    _require(scales, name + "scales", torch.uint8, 2)
    S, H, D = codes.shape
    if D < CACHE_BLOCK or D % CACHE_BLOCK or D > MAX_BLOCK_DIM:
        raise ValueError("%scodes must have a multiple of %d channels, at most %d, got %d" % (name, CACHE_BLOCK, MAX_BLOCK_DIM, D))
    if H < 1 or S > _INT32 or H * D > 1 << 28:
        raise ValueError("%scodes must have at least one head, at most 2^28 values a slot and fewer than 2^31 slots" % name)
    if not 1 <= page_size <= _INT32:
        raise ValueError("page_size must be 1 to %d, got %s" % (_INT32, page_size))
    blocks = scales.shape[0]
    if scales.shape[1] != H or (S == 0) != (blocks == 0) or (blocks and S % blocks):
        raise ValueError("%sscales must have shape [S / N, H] for blocks of N slots of codes %s, got %s"
                         % (name, tuple(codes.shape), tuple(scales.shape)))
    block = S // blocks if blocks else 1
    if page_size % block:
        raise ValueError("pages of %d slots must be whole blocks of %sscales' %d" % (page_size, name, block))
    if codes.stride(2) != 1:
        raise ValueError("%scodes must be contiguous in its last dimension" % name)
    return S, H, D, block


def _rows_overlap(t: torch.Tensor) -> bool:
    """Whether two elements of a 2-D tensor to be written could be the same memory."""
    (n, h), (sn, sh) = t.shape, t.stride()
    if n <= 1 or h <= 1:
        return (n > 1 and sn < 1) or (h > 1 and sh < 1)
    return sn < 1 or sh < 1 or (sn <= (h - 1) * sh and sh <= (n - 1) * sn)


def _table(page_table: torch.Tensor, B: int, page_size: int) -> int:
    _require(page_table, "page_table", torch.int32, 2)
    if page_table.shape[0] != B:
        raise ValueError("page_table must have %d rows, got %d" % (B, page_table.shape[0]))
    pages = page_table.shape[1]
    if pages * page_size > MAX_LENGTH:
        raise ValueError("page_table must have room for at most %d positions, got %d pages of %d" % (MAX_LENGTH, pages, page_size))
    return _rows(page_table, "page_table")


def _write_checks(codes, scales, page_table, first, counts, page_size, B, index):
    S, H, D, block = _block_cache(codes, scales, "", page_size)
    if codes.get_device() != index:
        raise ValueError("codes must be on cuda:%d" % index)
    if _overlaps(codes) or _rows_overlap(scales):
        raise ValueError("rows of codes and scales must not overlap")
    pt_b = _table(page_table, B, page_size)
    _same_device(index, (scales, "scales"), (page_table, "page_table"))
    return S, H, D, block, pt_b, _vector(first, "first", B, index), _vector(counts, "counts", B, index)


def block_write(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, first: torch.Tensor,
                counts: torch.Tensor, page_size: int) -> None:
    """Quantises rows ``x`` [B, T, H, D] (bf16, fp16 or fp32) into a block cache: row t of sequence b, t < counts[b], to position
    first[b] + t (int32 [B] both), found through ``page_table`` (int32 [B, pages]).

    ``codes`` float8_e4m3fn [S, H, D], ``scales`` uint8 [S / N, H]; N slots make a block, and whole blocks a page.  A block
    and head gets the smallest power of two that keeps its new rows within +-448, and no smaller one than it has where rows
    of earlier positions stay in it: their codes are rounded to a larger one.  Rows of the block behind the new ones keep
    their bytes and are taken for nothing.  Positions without a page are skipped; the pages that one call writes belong to
    one sequence each.
    """
    kind = _floats(x, "x", 4)
    _no_grad(x, "x", "block_write")
    B, T = x.shape[:2]
    index = x.get_device()
    S, H, D, block, pt_b, at, many = _write_checks(codes, scales, page_table, first, counts, page_size, B, index)
    if x.shape[2] != H or x.shape[3] != D:
        raise ValueError("x must have shape [B, T, %d, %d], got %s" % (H, D, tuple(x.shape)))
    if T > _INT32 or B * H > _INT32:
        raise ValueError("x must have at most %d tokens, and sequences times heads, got %s" % (_INT32, tuple(x.shape)))
    _run(index, "ets_block_write", _lib().ets_block_write, x.data_ptr(), *x.stride()[:3], B, T, H, D, codes.data_ptr(),
         *codes.stride()[:2], scales.data_ptr(), *scales.stride(), S, block, page_table.data_ptr(), pt_b, page_table.shape[1],
         page_size, at, many, kind)


def block_keep(codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor, first: torch.Tensor, path: torch.Tensor,
               counts: torch.Tensor, page_size: int) -> None:
    """Moves the rows of a line of drafted tokens to the front: row first[b] + path[b, i] to first[b] + i, i < counts[b].

    ``path`` (int32 [B, T], T at most 64) and ``counts`` as :func:`verify_drafts` returns them.  All rows are read before any
    is written, and written as :func:`block_write` writes their values; rows at the start whose place does not change stay.
    An entry of ``path`` outside [0, T), or without a page, leaves a row of zeros.
    """
    if not isinstance(path, torch.Tensor):
        raise TypeError("path must be a torch.Tensor")
    _require(path, "path", torch.int32, 2)
    B, T = path.shape
    index = path.get_device()
    if T > MAX_TREE:
        raise ValueError("path must have at most %d entries a sequence, got %d" % (MAX_TREE, T))
    S, H, D, block, pt_b, at, many = _write_checks(codes, scales, page_table, first, counts, page_size, B, index)
    if B * H > _INT32:
        raise ValueError("path must have at most %d sequences times heads" % _INT32)
    _run(index, "ets_block_keep", _lib().ets_block_keep, B, T, H, D, codes.data_ptr(), *codes.stride()[:2], scales.data_ptr(),
         *scales.stride(), S, block, page_table.data_ptr(), pt_b, page_table.shape[1], page_size, at, path.data_ptr(),
         _rows(path, "path"), many)


@functools.lru_cache(maxsize=256)
def _bytes(what, index, size, *args):
    """Bytes of workspace that `size` asks for on a device: a function of the sizes in `args` alone."""
    need = _sz(0)
    sizes = (ctypes.byref(_BlocksArgs(*args)),) if what == "ets_attend_blocks" else args
    st = _on(index, getattr(_lib(), size), *sizes, ctypes.byref(need))
    if st:
        _check(st, what)
    return need.value


def _space(what, index, like, workspace, size, *args):
    """(address, bytes) of the workspace that `size` asks for, and what keeps it alive."""
    nbytes = _bytes(what, index, size, *args)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous torch.Tensor on a HIP device")
        _same_device(index, (workspace, "workspace"))
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace must hold at least %d bytes" % nbytes)
    elif nbytes:
        # torch's allocator orders it on this stream, and keeps it for a graph that is being captured
        workspace = like.new_empty(nbytes, dtype=torch.uint8)
    return workspace.data_ptr() if nbytes else None, nbytes, workspace


def attend_blocks(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                  page_table: torch.Tensor, seq_lens: torch.Tensor, page_size: int, L: int, first: Optional[torch.Tensor] = None,
                  tree_mask: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention over a block cache: (out [B, T, Hq, Dv] of q's type, lse float32 [B, T, Hq]).

    ``q`` bf16 or fp16 [B, T, Hq, D]; caches [S, Hkv, D] and [S, Hkv, Dv] (up to 256 channels) with blocks of one size, Hq a
    multiple of Hkv.  Each token sees positions p < min(seq_lens[b], L) of its sequence, all of them without ``first``
    (int32 [B]).  With it, token t stands at position first[b] + t and sees p <= first[b] + t; with ``tree_mask`` (int64
    [B, T], T at most 64) it sees p < first[b], and first[b] + j for each set bit j < T.  A token whose own position is not
    below the length is padding.  Scores are scaled by D^-1/2.  A token that sees nothing has out 0 and lse -inf.
    """
    kind = _floats(q, "q", 4, "bf16 or fp16")
    _no_grad(q, "q", "attend_blocks")
    B, T, Hq, D = q.shape
    index = q.get_device()
    S, Hkv, Dk, block = _block_cache(k_codes, k_scales, "k_", page_size)
    Sv, Hv, Dv, block_v = _block_cache(v_codes, v_scales, "v_", page_size)
    if Dk != D:
        raise ValueError("k_codes must have %d channels like q, got %d" % (D, Dk))
    if Sv != S or Hv != Hkv or block_v != block:
        raise ValueError("v_codes must have the slots, heads and blocks of k_codes %s, got %s" % ((S, Hkv, block), (Sv, Hv, block_v)))
    if B * T * Hq > _INT32:
        raise ValueError("q must have at most %d rows, got %d" % (_INT32, B * T * Hq))
    if Hq < 1 or Hq % Hkv:
        raise ValueError("q must have a multiple of the cache's %d heads, got %d" % (Hkv, Hq))
    pt_b = _table(page_table, B, page_size)
    if not 0 <= L <= MAX_LENGTH or page_table.shape[1] * page_size < L:
        raise ValueError("L must be 0 to the %d pages of %d of page_table, got %s" % (page_table.shape[1], page_size, L))
    lens = _vector(seq_lens, "seq_lens", B, index)
    start = None if first is None else _vector(first, "first", B, index)
    _same_device(index, (k_codes, "k_codes"), (k_scales, "k_scales"), (v_codes, "v_codes"), (v_scales, "v_scales"),
                 (page_table, "page_table"), (tree_mask, "tree_mask"))
    mask, mask_b = None, 0
    if tree_mask is not None:
        _require(tree_mask, "tree_mask", torch.int64, 2)
        if first is None:
            raise ValueError("tree_mask needs first")
        if T > MAX_TREE:
            raise ValueError("a tree has at most %d tokens, got %d" % (MAX_TREE, T))
        if tree_mask.shape != (B, T):
            raise ValueError("tree_mask must have shape %s" % ((B, T),))
        mask, mask_b = tree_mask.data_ptr(), _rows(tree_mask, "tree_mask")
    out = q.new_empty((B, T, Hq, Dv))
    lse = q.new_empty((B, T, Hq), dtype=torch.float32)
    q_b, q_t, q_h, _ = q.stride()
    k_s, k_h, _ = k_codes.stride()
    v_s, v_h, _ = v_codes.stride()
    args = ctypes.byref(_BlocksArgs(
        B, T, Hq, Hkv, D, Dv, kind, block, L, page_size, S, q.data_ptr(), q_b, q_t, q_h,
        k_codes.data_ptr(), k_s, k_h, k_scales.data_ptr(), *k_scales.stride(),
        v_codes.data_ptr(), v_s, v_h, v_scales.data_ptr(), *v_scales.stride(),
        page_table.data_ptr(), pt_b, lens, start, mask, mask_b, out.data_ptr(), lse.data_ptr()))
    at, nbytes, kept = _space("ets_attend_blocks", index, q, workspace, "ets_attend_blocks_workspace_size", B, T, Hq, Hkv, D, Dv, kind, block, L, page_size, S)
    _run(index, "ets_attend_blocks", _lib().ets_attend_blocks, args, at, nbytes)
    return out, lse


def verify_drafts(probs: torch.Tensor, tokens: torch.Tensor, uniform: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                  tree_mask: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Which drafted tokens stand, and the next one: (tokens int32 [B, T], path int32 [B, T], counts int32 [B]).

    ``tokens`` int32 [B, T], T at most 64: node 0 is the last token that stands already, the others were drafted; node t
    hangs on the highest bit below t of ``tree_mask[b, t]`` (int64 [B, T], as for attention), or on t - 1 without a mask.
    ``lens`` (int32 [B]): nodes of a sequence, T without it.  ``probs`` [B, T, V] (bf16, fp16 or fp32): the target's
    distribution after each node.  ``uniform`` float32 [B, T] in [0, 1): the random number of each node's test, the first for
    the last draw.

    From node 0 on, a child with token x is taken if u * q(x) < p(x), with ``draft_probs`` [B, T - 1, V] the distributions
    that tokens 1 .. of a chain (no mask) were drawn from; without them (tokens that are no samples), if u * rest < p(x),
    where rest is 1 less the p of the children refused before it.  Where no child is taken the last token is drawn: from
    max(p - q, 0) if one was refused, without draft_probs from p less the refused tokens, else from p; the lowest v whose
    running sum passes u_0 times the total.  Everything is computed in 64 bits.

    Row b of the result has counts[b] tokens (the drafted ones that stand and the drawn one) and nodes (0 and those of the
    drafted ones), then -1: ``path`` and ``counts`` are what :func:`block_keep` takes.  counts is 0 where lens is.
    """
    kind = _floats(probs, "probs", 3)
    _no_grad(probs, "probs", "verify_drafts")
    B, T, V = probs.shape
    index = probs.get_device()
    if not 1 <= T <= MAX_TREE:
        raise ValueError("probs must have 1 to %d nodes a sequence, got %d" % (MAX_TREE, T))
    if not 1 <= V <= _INT32 - 4096 or -(-V // 4096) * B > _INT32:
        raise ValueError("probs must have 1 to %d tokens, and at most 2^31 - 1 pieces of 4096 of them, got %d for %d sequences"
                         % (_INT32 - 4096, V, B))
    _require(tokens, "tokens", torch.int32, 2)
    _require(uniform, "uniform", torch.float32, 2)
    _no_grad(uniform, "uniform", "verify_drafts")
    if tokens.shape != (B, T) or uniform.shape != (B, T):
        raise ValueError("tokens and uniform must have shape %s" % ((B, T),))
    _same_device(index, (tokens, "tokens"), (uniform, "uniform"), (draft_probs, "draft_probs"), (tree_mask, "tree_mask"))
    draft, q_b, q_t, mask, mask_b = None, 0, 0, None, 0
    if draft_probs is not None:
        if tree_mask is not None:
            raise ValueError("draft_probs go with chains: a tree's tokens are taken for no samples")
        if _floats(draft_probs, "draft_probs", 3) != kind or draft_probs.shape != (B, T - 1, V):
            raise ValueError("draft_probs must have shape %s and the type of probs" % ((B, T - 1, V),))
        _no_grad(draft_probs, "draft_probs", "verify_drafts")
        # of a chain of one node there are none: any address stands for the form of the call
        draft, (q_b, q_t, _) = draft_probs.data_ptr() or probs.data_ptr(), draft_probs.stride()
    if tree_mask is not None:
        _require(tree_mask, "tree_mask", torch.int64, 2)
        if tree_mask.shape != (B, T):
            raise ValueError("tree_mask must have shape %s" % ((B, T),))
        mask, mask_b = tree_mask.data_ptr(), _rows(tree_mask, "tree_mask")
    many = None if lens is None else _vector(lens, "lens", B, index)
    out = probs.new_empty((2, B, T), dtype=torch.int32)
    counts = probs.new_empty((B,), dtype=torch.int32)
    lib = _lib()
    at, nbytes, kept = _space("ets_verify_drafts", index, probs, workspace, "ets_verify_workspace_size", B, T, V)
    _run(index, "ets_verify_drafts", lib.ets_verify_drafts, probs.data_ptr(), *probs.stride()[:2], draft, q_b, q_t, B, T, V,
         tokens.data_ptr(), _rows(tokens, "tokens"), uniform.data_ptr(), _rows(uniform, "uniform"), mask, mask_b, many,
         out.data_ptr(), out.data_ptr() + 4 * B * T, counts.data_ptr(), kind, at, nbytes)
    return (*out.unbind(0), counts)


def _pool(refs: torch.Tensor, table: torch.Tensor, what: str) -> Tuple[int, int]:
    """Checks a pool's counts and its table; (P, device)."""
    _require(refs, "refs", torch.int32, 1)
    P = refs.shape[0]
    index = refs.get_device()
    if P > MAX_PAGES:
        raise ValueError("refs must have at most %d pages, got %d" % (MAX_PAGES, P))
    if P > 1 and refs.stride(0) != 1:
        raise ValueError("refs must be contiguous")
    _require(table, what, torch.int32, 2)
    _same_device(index, (table, what))
    if table.numel() > _INT32 - 4096:
        raise ValueError("%s must have at most %d entries" % (what, _INT32 - 4096))
    _written(table, what)
    return P, index


def _written(table: torch.Tensor, what: str) -> None:
    if table.shape[0] > 1 and table.stride(0) < table.shape[1]:
        raise ValueError("rows of %s must not overlap" % what)


def _near(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether an entry of one 2-D int32 tensor lies between the first and the last of the other."""
    def span(t):
        (n, m), (sn, sm) = t.shape, t.stride()
        return t.data_ptr(), t.data_ptr() + 4 * ((n - 1) * sn + (m - 1) * sm + 1)
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _buffers(buffers: Sequence[torch.Tensor], P: int, index: int):
    """A pool's buffers as the C ABI takes them: P pages of equal size each, one after another."""
    if isinstance(buffers, torch.Tensor) or len(buffers) > MAX_BUFFERS:
        raise TypeError("buffers must be a list of at most %d tensors" % MAX_BUFFERS)
    held = (_PageBuffer * max(1, len(buffers)))()
    for i, t in enumerate(buffers):
        if not isinstance(t, torch.Tensor):
            raise TypeError("buffers must be torch.Tensors")
        if t.get_device() != index:
            raise ValueError("buffers must be on cuda:%d" % index)
        if not t.is_contiguous() or t.ndim < 1 or (t.shape[0] % P if P else t.shape[0]):
            raise ValueError("buffers must be contiguous, with a first dimension that is a multiple of the %d pages, got %s"
                             % (P, tuple(t.shape)))
        _no_grad(t, "the buffers", "a move of pages")
        held[i].data, held[i].page_bytes = t.data_ptr(), t.numel() * t.element_size() // P if P else 0
    return held, len(buffers)


def pages_copy(buffers: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, pages: int) -> None:
    """Page dst[i] of every buffer becomes page src[i] (int32 [n] both).

    Each of up to 64 contiguous ``buffers`` holds ``pages`` pages one after another: its first dimension is a multiple of
    ``pages`` (slots, blocks).  Pairs with a number outside [0, pages) are skipped; the destinations of one call differ from
    each other and from its sources.
    """
    if not isinstance(src, torch.Tensor) or src.ndim != 1:
        _require(src, "src", torch.int32, 1)
    index, n = src.get_device(), src.shape[0]
    if not src.is_cuda:
        raise ValueError("src must be on a HIP device, got %s" % src.device)
    if not 0 <= pages <= MAX_PAGES:
        raise ValueError("pages must be 0 to %d, got %s" % (MAX_PAGES, pages))
    at, to = _vector(src, "src", n, index), _vector(dst, "dst", n, index)
    held, count = _buffers(buffers, pages, index)
    _run(index, "ets_pages_copy", _lib().ets_pages_copy, held, count, pages, at, to, n)


def pages_extend(refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, page_size: int,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gives row b of ``page_table`` (int32 [B, M]) pages for positions [0, lens[b]); how many it lacks, int32 [B].

    ``refs`` int32 [P] counts the table entries that hold each page (free: 0 or less).  Of the first ceil(lens[b] /
    page_size) entries, M at most, those that hold none (outside [0, P)) get the free pages, lowest first, in the order of
    rows and entries; where none is left they become -1.
    """
    P, index = _pool(refs, page_table, "page_table")
    B, M = page_table.shape
    need = _vector(lens, "lens", B, index)
    if not 1 <= page_size <= _INT32:
        raise ValueError("page_size must be 1 to %d, got %s" % (_INT32, page_size))
    lacking = refs.new_empty((B,))
    lib = _lib()
    at, nbytes, kept = _space("ets_pages_extend", index, refs, workspace, "ets_pages_workspace_size", P, B * M)
    _run(index, "ets_pages_extend", lib.ets_pages_extend, refs.data_ptr(), P, page_table.data_ptr(), _rows(page_table, "page_table"),
         B, M, need, page_size, lacking.data_ptr(), at, nbytes)
    return lacking


def pages_free(refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, page_size: int) -> None:
    """Row b of ``page_table`` keeps its pages for positions [0, lens[b]); its other entries become -1, and the pages they
    held lose one from ``refs``.  A length of 0 lets a whole sequence go."""
    P, index = _pool(refs, page_table, "page_table")
    B, M = page_table.shape
    keep = _vector(lens, "lens", B, index)
    if not 1 <= page_size <= _INT32:
        raise ValueError("page_size must be 1 to %d, got %s" % (_INT32, page_size))
    _run(index, "ets_pages_free", _lib().ets_pages_free, refs.data_ptr(), P, page_table.data_ptr(), _rows(page_table, "page_table"),
         B, M, keep, page_size)


def pages_fork(refs: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, page_size: int, parents: torch.Tensor,
               buffers: Sequence[torch.Tensor] = (), out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Branches of sequences: (their table rows, int32 [n, M], and whether each lacks its last page, int32 [n]).

    Row i shares the pages that the lens[b] positions of row b = parents[i] (int32 [n]) fill, which gain one in ``refs``
    each; a page that they fill in part is copied, in all ``buffers`` (as for :func:`pages_copy`), to a free one, lowest
    first in the order of i.  Other entries are -1; all are where parents[i] is outside [0, B).  ``out`` (int32 [n, any
    width]) may be rows of the same table, parents among them: all are read before any is written (from a copy of the table,
    where the two overlap).  What they held before is not let go.  A branch has the pages that its row of ``out`` has room
    for; those behind them are not shared, and are not counted as lacking.
    """
    P, index = _pool(refs, page_table, "page_table")
    B, M = page_table.shape
    have = _vector(lens, "lens", B, index)
    if not isinstance(parents, torch.Tensor) or parents.ndim != 1:
        _require(parents, "parents", torch.int32, 1)
    n = parents.shape[0]
    of = _vector(parents, "parents", n, index)
    if not 1 <= page_size <= _INT32:
        raise ValueError("page_size must be 1 to %d, got %s" % (_INT32, page_size))
    if out is None:
        out = page_table.new_empty((n, M))
    else:
        _require(out, "out", torch.int32, 2)
        _same_device(index, (out, "out"))
        if out.shape[0] != n or out.shape[1] > _INT32:
            raise ValueError("out must have %d rows, got %d" % (n, out.shape[0]))
        _written(out, "out")
        if _near(out, page_table):
            page_table = page_table.clone()
    lacking = refs.new_empty((n,))
    held, count = _buffers(buffers, P, index)
    lib = _lib()
    at, nbytes, kept = _space("ets_pages_fork", index, refs, workspace, "ets_pages_workspace_size", P, n)
    _run(index, "ets_pages_fork", lib.ets_pages_fork, refs.data_ptr(), P, page_table.data_ptr(), _rows(page_table, "page_table"), B, M,
         have, page_size, of, n, out.data_ptr(), _rows(out, "out"), out.shape[1], lacking.data_ptr(), held, count, at, nbytes)
    return out, lacking


def pages_compact(refs: torch.Tensor, page_table: torch.Tensor, buffers: Sequence[torch.Tensor] = (),
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Draws a pool together; each page's new number, int32 [P], -1 for free ones.

    Of the u pages in use, those numbered u or more move, lowest first, to the free ones under u, lowest first: in all
    ``buffers`` (as for :func:`pages_copy`), with their ``refs``, and in ``page_table``, whose entries that hold a free page
    become -1.
    """
    P, index = _pool(refs, page_table, "page_table")
    B, M = page_table.shape
    moved = refs.new_empty((P,))
    held, count = _buffers(buffers, P, index)
    lib = _lib()
    at, nbytes, kept = _space("ets_pages_compact", index, refs, workspace, "ets_pages_workspace_size", P, B * M)
    _run(index, "ets_pages_compact", lib.ets_pages_compact, refs.data_ptr(), P, page_table.data_ptr(),
         _rows(page_table, "page_table"), B, M, moved.data_ptr(), held, count, at, nbytes)
    return moved
