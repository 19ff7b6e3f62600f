"""CPU checks of the speculative step's C ABI: exports, the binding's constants, and refusals before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from tests import decode_reference as ref
from tests import speculate_reference as spec

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ets_speculate.h")
INVALID, WORKSPACE = 1, 3
F = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
SPACE = 1 << 40              # bytes that are enough


@pytest.fixture(scope="module")
def lib():
    import exact_top_selection_amd as ets
    from exact_top_selection_amd import _speculate
    if not os.path.exists(ets.library_path()):
        from exact_top_selection_amd import _build
        _build.build()
    return _speculate._lib()


def test_library_exports_every_declared_symbol(lib):
    names = re.findall(r"^ets_status (ets_\w+)\(", open(HEADER).read(), re.M)
    assert len(names) == 12
    for name in names:
        assert hasattr(lib, name), name


def test_header_compiles_as_c_and_matches_the_binding(tmp_path):
    from exact_top_selection_amd import _speculate
    text = open(HEADER).read()
    for name, value in (("ETS_MAX_BLOCK_DIM", _speculate.MAX_BLOCK_DIM), ("ETS_MAX_BUFFERS", _speculate.MAX_BUFFERS)):
        assert int(re.search(r"#define %s\s+(\d+)" % name, text).group(1)) == value, name
    for struct, cls in (("ets_attend_blocks_args", _speculate._BlocksArgs), ("ets_page_buffer", _speculate._PageBuffer)):
        fields = [n for n, _ in cls._fields_]
        src = tmp_path / "layout.c"
        src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ets_speculate.h"\nint main(void){\n'
                       + "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (struct, n) for n in fields)
                       + 'printf("%%zu\\n", sizeof(%s)); return 0; }\n' % struct)
        exe = str(tmp_path / "layout")
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
        assert got == [getattr(cls, n).offset for n in fields] + [ctypes.sizeof(cls)]


def _write(lib, B=2, T=3, H=2, D=64, S=32, block=4, pages=4, page=8, x=F, codes=F, scales=F, table=F, first=F, counts=F, dtype=0):
    return lib.ets_block_write(x, T * H * D, H * D, D, B, T, H, D, codes, H * D, D, scales, H, 1, S, block, table, pages, pages, page,
                               first, counts, dtype, None)


def _keep(lib, B=2, T=3, H=2, D=64, S=32, block=4, pages=4, page=8, codes=F, scales=F, table=F, first=F, path=F, counts=F):
    return lib.ets_block_keep(B, T, H, D, codes, H * D, D, scales, H, 1, S, block, table, pages, pages, page, first, path, T, counts,
                              None)


def test_write_refusals(lib):
    shared = [dict(B=-1), dict(T=-1), dict(H=0), dict(D=0), dict(D=48), dict(D=288), dict(S=-1), dict(S=1 << 31), dict(S=30),
              dict(block=0), dict(block=3), dict(page=0), dict(page=6), dict(pages=-1), dict(pages=1 << 30, page=8), dict(codes=None),
              dict(scales=None), dict(table=None), dict(first=None), dict(counts=None), dict(H=1 << 23), dict(B=1 << 28, H=8)]
    for bad in shared + [dict(x=None), dict(dtype=3), dict(dtype=-1)]:
        assert _write(lib, **bad) == INVALID, bad
    for bad in shared + [dict(path=None), dict(T=65)]:
        assert _keep(lib, **bad) == INVALID, bad
    assert _write(lib, B=0, x=None) == 0 and _write(lib, T=0, x=None) == 0 and _keep(lib, B=0, path=None) == 0


def test_attend_refusals(lib):
    from exact_top_selection_amd._speculate import _BlocksArgs
    need = ctypes.c_size_t(0)
    good = dict(B=2, T=2, Hq=4, Hkv=2, D=64, Dv=64, dtype=0, block=4, L=16, page_size=8, S=32)

    def status(**over):
        return lib.ets_attend_blocks_workspace_size(ctypes.byref(_BlocksArgs(**{**good, **over})), ctypes.byref(need))

    for bad in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=0), dict(D=48), dict(D=288), dict(Dv=40),
                dict(Dv=288), dict(dtype=2), dict(S=-1), dict(S=1 << 31), dict(S=30), dict(L=-1), dict(L=0x7FFFF001), dict(page_size=0),
                dict(block=0), dict(block=3), dict(tree_mask=0x1000), dict(tree_mask=0x1000, first=0x1000, T=65), dict(k_s=-1),
                dict(ks_s=1 << 32), dict(v_s=1 << 32), dict(vs_s=-1), dict(B=1 << 20, T=1 << 10)):
        assert status(**bad) == INVALID, bad
    assert lib.ets_attend_blocks_workspace_size(ctypes.byref(_BlocksArgs(**good)), None) == INVALID
    assert status(B=0) == 0 and need.value == 0
    assert lib.ets_attend_blocks(ctypes.byref(_BlocksArgs(**{**good, "T": 0})), None, 0, None) == 0
    assert lib.ets_attend_blocks(None, None, 0, None) == INVALID


def _verify(lib, B=2, T=3, V=100, probs=F, draft=None, tokens=F, uniform=F, mask=None, out=F, dtype=2, space=F, nbytes=SPACE):
    return lib.ets_verify_drafts(probs, T * V, V, draft, T * V, V, B, T, V, tokens, T, uniform, T, mask, T, None, out, out, out, dtype,
                                 space, nbytes, None)


def test_verify_refusals(lib):
    for bad in (dict(B=-1), dict(T=-1), dict(T=0), dict(T=65), dict(V=0), dict(V=0x7FFFFFFF), dict(dtype=3), dict(probs=None),
                dict(tokens=None), dict(uniform=None), dict(out=None), dict(draft=F, mask=F)):
        assert _verify(lib, **bad) == INVALID, bad
    for bad in (dict(space=None), dict(space=ctypes.c_void_p(0x1001)), dict(nbytes=8)):
        assert _verify(lib, **bad) == WORKSPACE, bad
    assert _verify(lib, B=0, probs=None) == 0
    need = ctypes.c_size_t(0)
    assert lib.ets_verify_workspace_size(2, 3, 100, None) == INVALID
    assert lib.ets_verify_workspace_size(2, 65, 100, ctypes.byref(need)) == INVALID


def test_pages_refusals(lib):
    from exact_top_selection_amd._speculate import _PageBuffer
    one = (_PageBuffer * 65)(*[_PageBuffer(0x1000, 64)] * 65)
    none = (_PageBuffer * 1)(_PageBuffer(None, 64))
    below = (_PageBuffer * 1)(_PageBuffer(0x1000, -1))
    copy = lambda b=one, c=1, P=8, s=F, d=F, n=2: lib.ets_pages_copy(b, c, P, s, d, n, None)  # noqa: E731
    for bad in (dict(c=-1), dict(c=65), dict(P=-1), dict(P=(1 << 26) + 1), dict(n=-1), dict(s=None), dict(d=None), dict(b=None),
                dict(b=none), dict(b=below), dict(n=1 << 40)):
        assert copy(**bad) == INVALID, bad
    assert copy(n=0, s=None, d=None) == 0 and copy(c=0, b=None) == 0

    extend = lambda r=F, P=8, t=F, B=2, M=4, n=F, page=8, k=F, w=F, wb=SPACE: lib.ets_pages_extend(r, P, t, M, B, M, n, page, k, w, wb, None)  # noqa: E731
    free = lambda r=F, P=8, t=F, B=2, M=4, n=F, page=8: lib.ets_pages_free(r, P, t, M, B, M, n, page, None)  # noqa: E731
    for bad in (dict(r=None), dict(P=-1), dict(P=(1 << 26) + 1), dict(t=None), dict(B=-1), dict(M=-1), dict(B=1 << 16, M=1 << 15),
                dict(n=None), dict(page=0)):
        assert extend(**bad) == INVALID and free(**bad) == INVALID, bad
    assert extend(k=None) == INVALID
    assert extend(w=None) == WORKSPACE and extend(wb=64) == WORKSPACE and extend(w=ctypes.c_void_p(0x1004)) == WORKSPACE
    assert extend(B=0) == 0 and free(B=0) == 0 and free(M=0) == 0

    def fork(r=F, P=8, t=F, B=2, M=4, n=F, page=8, parents=F, rows=3, out=F, k=F, b=one, c=1, w=F, wb=SPACE):
        return lib.ets_pages_fork(r, P, t, M, B, M, n, page, parents, rows, out, M, M, k, b, c, w, wb, None)

    for bad in (dict(r=None), dict(P=-1), dict(t=None), dict(n=None), dict(page=0), dict(parents=None), dict(rows=-1), dict(out=None),
                dict(k=None), dict(c=65), dict(b=none), dict(b=below)):
        assert fork(**bad) == INVALID, bad
    assert fork(w=None) == WORKSPACE and fork(rows=0) == 0

    def compact(r=F, P=8, t=F, B=2, M=4, moved=F, b=one, c=1, w=F, wb=SPACE):
        return lib.ets_pages_compact(r, P, t, M, B, M, moved, b, c, w, wb, None)

    for bad in (dict(r=None), dict(P=-1), dict(t=None), dict(B=-1), dict(M=-1), dict(moved=None), dict(c=-1), dict(b=none)):
        assert compact(**bad) == INVALID, bad
    assert compact(w=None) == WORKSPACE and compact(P=0, r=None, moved=None) == 0


def test_binding_refuses_host_tensors():
    import exact_top_selection_amd as ets
    codes, scales = torch.zeros(8, 1, 32, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)
    i, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32)
    q = torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16)
    for call in (lambda: ets.block_write(q, codes, scales, table, i, i, 4),
                 lambda: ets.block_keep(codes, scales, table, i, table, i, 4),
                 lambda: ets.attend_blocks(q, codes, scales, codes, scales, table, i, 4, 4),
                 lambda: ets.verify_drafts(q[:, 0], table.expand(2, 4), torch.zeros(2, 4)),
                 lambda: ets.pages_copy([codes], i, i, 2),
                 lambda: ets.pages_extend(i, table, i, 4),
                 lambda: ets.pages_free(i, table, i, 4),
                 lambda: ets.pages_fork(i, table, i, 4, i),
                 lambda: ets.pages_compact(i, table)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_reference_verification_follows_the_target():
    """The oracle's own rule: over a fine grid of random numbers, first tokens come as the target's distribution says."""
    p = torch.tensor([[0.5, 0.3, 0.2], [0.2, 0.2, 0.6]], dtype=torch.float64)
    q = torch.tensor([0.1, 0.6, 0.3], dtype=torch.float64)
    n = 60
    grid = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    counts = torch.zeros(3, dtype=torch.float64)
    for x in range(3):  # a drafted token, drawn from q
        for u in grid.tolist():
            first = torch.zeros(3, dtype=torch.float64)
            for last in grid.tolist():
                got = spec.verify(p[None], torch.tensor([[0, x]]), torch.tensor([[last, u]], dtype=torch.float64), draft=q[None, None])
                first[int(got[0][0, 0])] += 1 / n
            counts += q[x] * first / n
    # midpoints: the share under a border is off by half a cell at most, for a test and a draw of each token
    assert (counts - p[0]).abs().max() <= 2 / (2 * n)
    counts.zero_()
    mask = torch.tensor([[1, 3, 5, 1]])  # two drafted siblings, and one that has the first one's token again
    n = 24
    grid = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).tolist()
    for u1 in grid:
        for u2 in grid:
            for last in grid:
                got = spec.verify(p[[0, 1, 1, 1]][None], torch.tensor([[0, 2, 0, 2]]),
                                  torch.tensor([[last, u1, u2, 0.5]], dtype=torch.float64), mask=mask)
                counts[int(got[0][0, 0])] += 1 / n ** 3
    # midpoints: the share under a border is off by half a cell at most, for two tests and a draw
    assert (counts - p[0]).abs().max() <= 3 / (2 * n)


def test_reference_codes():
    codes, scales = torch.zeros(8, 1, 32, dtype=torch.uint8), torch.full((2, 1), 127, dtype=torch.uint8)
    x = torch.zeros(1, 3, 1, 32)
    x[0, 0, 0, 0], x[0, 1, 0, 0], x[0, 2, 0, 0] = 448, 2.0 ** -9, 900
    table = torch.tensor([[0, 1]])
    codes, scales = spec.block_write(x[:, :2], codes, scales, table, torch.tensor([0]), torch.tensor([2]), 4)
    assert scales[0, 0] == 127 and codes[0, 0, 0] == 126 and codes[1, 0, 0] == 1
    codes, scales = spec.block_write(x[:, 2:], codes, scales, table, torch.tensor([2]), torch.tensor([1]), 4)
    assert scales[0, 0] == 129 and codes[0, 0, 0] == 110 and codes[1, 0, 0] == 0 and scales[1, 0] == 127
    assert ref._CODES[110] * 4 == 448 and ref._CODES[codes[2, 0, 0].long()] * 4 == 896
