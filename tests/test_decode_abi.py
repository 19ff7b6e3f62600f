"""CPU checks of the decode operators' C ABI: exports, the binding's constants, and refusals before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ets_decode.h")
INVALID = 1
F = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    import exact_top_selection_amd as ets
    from exact_top_selection_amd import _decode
    if not os.path.exists(ets.library_path()):
        from exact_top_selection_amd import _build
        _build.build()
    return _decode._lib()


def test_library_exports_every_declared_symbol(lib):
    names = re.findall(r"^ets_status (ets_\w+)\(", open(HEADER).read(), re.M)
    assert len(names) == 6
    for name in names:
        assert hasattr(lib, name), name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "ets_decode.h"\nint main(void){ ets_attend_args a; return sizeof a ? ETS_OK : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o",
                    str(tmp_path / "use")], check=True)


def test_binding_matches_the_header(tmp_path):
    from exact_top_selection_amd import _decode
    text = open(HEADER).read()
    for name, value in (("ETS_MAX_ROPE_DIM", _decode.MAX_ROPE_DIM), ("ETS_MAX_HEAD_DIM", _decode.MAX_HEAD_DIM),
                        ("ETS_MAX_INDEX_DIM", _decode.MAX_INDEX_DIM), ("ETS_MAX_INDEX_HEADS", _decode.MAX_INDEX_HEADS),
                        ("ETS_MAX_TREE", _decode.MAX_TREE), ("ETS_BF16", 0), ("ETS_FP16", 1), ("ETS_FP32", 2)):
        assert int(re.search(r"#define %s\s+(\d+)" % name, text).group(1)) == value, name
    # the argument structure, field by field
    fields = [n for n, _ in _decode._AttendArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ets_decode.h"\nint main(void){\n'
                   + "".join('printf("%%zu\\n", offsetof(ets_attend_args, %s));\n' % n for n in fields)
                   + 'printf("%zu\\n", sizeof(ets_attend_args)); return 0; }\n')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.dirname(HEADER), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(_decode._AttendArgs, n).offset for n in fields] + [ctypes.sizeof(_decode._AttendArgs)]


def _rope(lib, N=4, H=2, D=64, R=32, offset=0, layout=0, dtype=0, x=F, pos=F, freq=F, out=F):
    return lib.ets_rope(x, H * D, D, out, H * D, D, N, H, D, pos, freq, R, offset, layout, 1.0, 0, dtype, None)


def test_rope_refusals(lib):
    for bad in (dict(N=-1), dict(H=-1), dict(D=0), dict(D=4097), dict(R=31), dict(R=-2), dict(offset=-1), dict(offset=33),
                dict(R=66), dict(layout=2), dict(dtype=3), dict(dtype=-1), dict(x=None), dict(pos=None), dict(freq=None),
                dict(out=None)):
        assert _rope(lib, **bad) == INVALID, bad
    assert _rope(lib, N=0, x=None, out=None) == 0


def _write(lib, N=4, H=2, D=64, S=8, x=F, slots=F, codes=F, scales=F, dtype=0):
    return lib.ets_cache_write(x, H * D, D, N, H, D, slots, codes, H * D, D, scales, H * D // 32, D // 32, S, dtype, None)


def _read(lib, N=4, H=2, D=64, S=8, out=F, slots=F, codes=F, scales=F, dtype=0):
    return lib.ets_cache_read(codes, H * D, D, scales, H * D // 32, D // 32, S, slots, N, H, D, out, dtype, None)


def test_cache_refusals(lib):
    for call, rows in ((_write, "x"), (_read, "out")):
        for bad in (dict(N=-1), dict(H=0), dict(D=0), dict(D=48), dict(S=-1), dict(dtype=3), {rows: None}, dict(slots=None),
                    dict(codes=None), dict(scales=None)):
            assert call(lib, **bad) == INVALID, (call, bad)
        assert call(lib, N=0, slots=None) == 0


def _scores(lib, B=2, T=1, H=4, D=64, S=8, page=4, L=8, stride=8, q=F, w=F, codes=F, scales=F, table=F, lens=F, out=F, dtype=0):
    return lib.ets_index_scores(q, T * H * D, H * D, D, w, T * H, H, B, T, H, D, codes, D, scales, D // 32, S, table, 2, lens,
                                page, L, out, stride, dtype, None)


def test_scores_refusals(lib):
    for bad in (dict(B=-1), dict(B=65536), dict(T=-1), dict(H=0), dict(H=129), dict(D=16), dict(D=288), dict(S=-1),
                dict(S=1 << 31), dict(page=0), dict(L=-1), dict(stride=7), dict(dtype=2), dict(q=None), dict(w=None),
                dict(codes=None), dict(scales=None), dict(table=None), dict(lens=None), dict(out=None)):
        assert _scores(lib, **bad) == INVALID, bad
    assert _scores(lib, B=0, q=None) == 0 and _scores(lib, T=0, q=None) == 0 and _scores(lib, L=0, q=None) == 0


def test_attend_refusals(lib):
    from exact_top_selection_amd._decode import _AttendArgs
    need = ctypes.c_size_t(0)
    good = dict(B=2, T=2, Hq=4, Hkv=2, D=64, Dv=64, dtype=0, K=8, L=8, page_size=4, S=16)

    def status(**over):
        return lib.ets_attend_workspace_size(ctypes.byref(_AttendArgs(**{**good, **over})), ctypes.byref(need))

    for bad in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=0), dict(D=48), dict(D=608), dict(Dv=40),
                dict(Dv=608), dict(dtype=2), dict(S=-1), dict(S=1 << 31), dict(L=-1), dict(page_size=0),
                dict(K=-1, slots=0x1000), dict(T=65, tree_slots=0x1000), dict(B=1 << 20, T=1 << 10, Hq=4)):
        assert status(**bad) == INVALID, bad
    assert lib.ets_attend_workspace_size(ctypes.byref(_AttendArgs(**good)), None) == INVALID
    assert status(B=0) == 0 and need.value == 0
    assert lib.ets_attend(ctypes.byref(_AttendArgs(**{**good, "T": 0})), None, 0, None) == 0
    assert lib.ets_attend(None, None, 0, None) == INVALID


def test_slot_strides_out_of_range(lib):
    """Strides from slot to slot are 32-bit numbers in the kernels: others are refused, not cut short."""
    from exact_top_selection_amd._decode import _AttendArgs
    need = ctypes.c_size_t(0)
    for bad in (-1, 1 << 32):
        for codes_s, scales_s in ((bad, 2), (64, bad)):
            assert lib.ets_index_scores(F, 256, 256, 64, F, 4, 4, 2, 1, 4, 64, F, codes_s, F, scales_s, 8, F, 2, F, 4, 8, F, 8, 0,
                                        None) == INVALID
        for name in ("k_s", "ks_s", "v_s", "vs_s"):
            args = _AttendArgs(B=2, T=2, Hq=4, Hkv=2, D=64, Dv=64, dtype=0, K=8, L=8, page_size=4, S=16, **{name: bad})
            assert lib.ets_attend_workspace_size(ctypes.byref(args), ctypes.byref(need)) == INVALID, name


def test_binding_refuses_host_tensors():
    import exact_top_selection_amd as ets
    x = torch.zeros(2, 1, 32)
    codes, scales = torch.zeros(4, 1, 32, dtype=torch.uint8), torch.zeros(4, 1, 1, dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 4, 32, dtype=torch.bfloat16)
    for call in (lambda: ets.rope(x, i, torch.zeros(4, dtype=torch.float64)),
                 lambda: ets.cache_write(x, i, codes, scales),
                 lambda: ets.cache_read(codes, scales, i),
                 lambda: ets.index_scores(q, torch.zeros(2, 1, 4), codes, scales, i.view(2, 1), i, 4, 4),
                 lambda: ets.attend_selected(q, codes, scales, codes, scales, i.view(2, 1, 1)),
                 lambda: ets.attend_paged(q, codes, scales, codes, scales, i.view(2, 1), i, 4, 4)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(TypeError):
        ets.rope(None, i, i)


def test_reference_quantiser():
    """The oracle's own codes: every value of the format is kept, and halves go to the even code."""
    from tests import decode_reference as ref
    size = ref._CODES[:127]
    x = torch.zeros(4, 1, 32, dtype=torch.float64)
    x[0, 0, 0], x[0, 0, 1:32] = 448, size[64:95]
    x[1, 0, 0], x[1, 0, 1] = 448, (size[100] + size[101]) / 2
    x[2, 0, 0] = 449
    codes, scales = ref.quantise(x)
    assert scales[:, 0, 0].tolist() == [127, 127, 128, 118]
    assert torch.equal(ref.values(codes, scales)[0], x[0])
    assert codes[1, 0, 1] == 100
    assert codes[2, 0, 0] == 118  # 224.5 to 224
