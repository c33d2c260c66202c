"""The C-ABI library of the paged 8-bit cache loads and exports every entry point
include/cmr_kv8.h declares, and rejects bad arguments on the host before touching a
GPU.  No call here reaches a kernel."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from vlm_decoder_positional_b200 import build as libbuild
from vlm_decoder_positional_b200 import cmr, kv8

HEADER = os.path.join(libbuild.INCLUDE, "cmr_kv8.h")
FAKE = 0x10000  # a 16-byte aligned address; never dereferenced
SEC = (ctypes.c_int32 * 3)(11, 11, 10)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return kv8.lib()


def declared():
    return re.findall(r"CMR_API\s+[\w\s\*]+?\b(cmr_\w+)\s*\(", open(HEADER).read())


def test_header_binding_and_library_agree(lib):
    names = set(declared())
    assert names == set(kv8.SIGNATURES) and len(names) == 11
    out = subprocess.run(["nm", "-D", "--defined-only", libbuild.KV8_LIB], check=True,
                         capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert {s for s in exported if "cmr" in s.lower()} == names
    for n in ("rotate_qk_kv8", "attend_kv8", "kv8_extend", "kv8_fork", "kv8_free", "kv8_compact"):
        assert n in pkg.__all__ and callable(getattr(pkg, n))


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "cmr_kv8.h"\nint main(void) { return CMR_DEVICE_BAD_SCALE == 16 ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", libbuild.INCLUDE,
                    "-fsyntax-only", str(src)], check=True)


def call_write(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, seqs=2, off=None, start=FAKE, amount=FAKE, n=10,
             L=1, hq=8, hk=2, D=256, theta=1e7, sec=SEC, rot=64, kp=FAKE, vp=FAKE, ks=FAKE,
             vs=FAKE, pages=4, P=64, table=FAKE, rows=2, cols=2, slot=None, status=None)
    a.update(kw)
    return lib.cmr_kv8_rotate_qk(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(n=-1), 1), (dict(n=2 ** 31), 1), (dict(seqs=-1), 1), (dict(seqs=0), 1), (dict(L=-1), 1),
    (dict(hq=-1), 1), (dict(hk=0), 1), (dict(D=96), 3), (dict(D=512), 3), (dict(P=48), 3),
    (dict(P=256), 3), (dict(P=0), 3), (dict(pages=0), 1), (dict(rows=0), 1), (dict(cols=0), 1),
    (dict(theta=0.0), 1), (dict(theta=float("nan")), 1), (dict(rot=24), 1), (dict(rot=0), 1),
    (dict(rot=128, D=64), 1), (dict(sec=(ctypes.c_int32 * 3)(12, 11, 10)), 1),
    (dict(sec=(ctypes.c_int32 * 3)(0, 20, 12)), 1), (dict(sec=None), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1), (dict(q=FAKE + 2), 1),
    (dict(kp=None), 1), (dict(vp=FAKE + 4), 1), (dict(ks=None), 1), (dict(vs=FAKE + 2), 1),
    (dict(table=None), 1), (dict(start=None), 1), (dict(amount=None), 1), (dict(slot=FAKE + 1), 1),
    (dict(cu=None, seqs=3), 1), (dict(hk=1 << 20, L=1 << 12), 3), (dict(hk=1 << 16), 3),
    (dict(pages=1 << 30, hk=4), 3), (dict(L=32768), 3), (dict(), 1),
])
def test_write_rejects_bad_arguments_on_the_host(lib, kw, want):
    # the last case is well formed but for its addresses, which no device has
    assert call_write(lib, **kw) == want, lib.cmr_kv8_last_error_message()
    assert lib.cmr_kv8_last_error_message() != b"no error"


def test_write_of_nothing_is_a_no_op(lib):
    assert call_write(lib, n=0, seqs=0, q=None, k=None, v=None) == 0
    assert call_write(lib, n=0, seqs=2) == 0
    assert call_write(lib, L=0) == 0


def call_attend(lib, **kw):
    a = dict(q=FAKE, out=FAKE + (1 << 20), cu=FAKE, seqs=2, off=None, n=10, L=1, hq=8, hk=2,
             D=256, scale=0.0625, kp=FAKE + (1 << 24), vp=FAKE + (1 << 25), ks=FAKE, vs=FAKE,
             pages=4, P=64, table=FAKE, rows=2, cols=2, slot=None, ws=FAKE, ws_bytes=1 << 30,
             status=None)
    a.update(kw)
    return lib.cmr_kv8_attend(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(n=-1), 1), (dict(seqs=0), 1), (dict(hq=7), 1), (dict(hq=0), 1), (dict(hq=258), 1),
    (dict(hk=0), 1), (dict(D=80), 3), (dict(P=17), 3), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(scale=1e300), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(out=FAKE), 1), (dict(out=FAKE + 16), 1), (dict(kp=FAKE + (1 << 20) + 64), 1),
    (dict(q=FAKE + 4), 1), (dict(kp=None), 1), (dict(vs=None), 1), (dict(pages=0), 1),
    (dict(table=None), 1), (dict(rows=0), 1), (dict(cols=1 << 25), 1), (dict(cu=None, seqs=4), 1),
    (dict(L=-1), 1), (dict(L=32768), 3), (dict(), 1),
])
def test_attend_rejects_bad_arguments_on_the_host(lib, kw, want):
    assert call_attend(lib, **kw) == want, lib.cmr_kv8_last_error_message()


def test_attend_of_nothing_is_a_no_op(lib):
    assert call_attend(lib, n=0, seqs=0) == 0
    assert call_attend(lib, L=0) == 0
    assert kv8.attend_kv8_workspace_bytes(0, 0, 1, 8, 2, 256) == 0
    assert kv8.attend_kv8_workspace_bytes(2, 10, 1, 8, 3, 256) == 0
    assert kv8.attend_kv8_workspace_bytes(2, 10, 1, 8, 2, 72) == 0


POOL = [FAKE, FAKE, FAKE, FAKE]


def call_extend(lib, **kw):
    a = dict(table=FAKE, rows=2, cols=2, refs=FAKE, pages=4, P=64, slots=FAKE, lens=FAKE, n=1,
             ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return lib.cmr_kv8_extend(*a.values(), None, None)


def call_fork(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, L=1, hk=2, D=256, pages=4, P=64, table=FAKE,
             rows=2, cols=2, refs=FAKE, src=FAKE, dst=FAKE, lens=FAKE, n=1, ws=FAKE,
             ws_bytes=1 << 20)
    a.update(kw)
    return lib.cmr_kv8_fork(*a.values(), None, None)


def call_free(lib, **kw):
    a = dict(table=FAKE, rows=2, cols=2, refs=FAKE, pages=4, slots=FAKE, n=1)
    a.update(kw)
    return lib.cmr_kv8_free(*a.values(), None, None)


def call_compact(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, L=1, hk=2, D=256, pages=4, P=64, table=FAKE,
             rows=2, cols=2, refs=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return lib.cmr_kv8_compact(*a.values(), None, None)


@pytest.mark.parametrize("call, bad", [
    (call_extend, [dict(table=None), dict(refs=None), dict(slots=None), dict(lens=None),
                   dict(n=-1), dict(pages=0), dict(rows=0), dict(cols=0), dict(P=65),
                   dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=8), dict()]),
    (call_fork, [dict(kp=None), dict(vp=FAKE + 8), dict(ks=None), dict(src=None), dict(dst=None),
                 dict(lens=None), dict(n=-2), dict(D=100), dict(P=8), dict(hk=0), dict(refs=None),
                 dict(ws_bytes=0), dict()]),
    (call_free, [dict(table=None), dict(refs=FAKE + 2), dict(slots=None), dict(n=-1),
                 dict(pages=0), dict()]),
    (call_compact, [dict(table=None), dict(refs=None), dict(kp=None), dict(pages=-1), dict(D=1),
                    dict(ws=None), dict(ws_bytes=4), dict()]),
])
def test_page_calls_reject_bad_arguments_on_the_host(lib, call, bad):
    for kw in bad:
        unsupported = kw.get("P") in (65, 8) or kw.get("D") in (100, 1)
        assert call(lib, **kw) == (3 if unsupported else 1), (kw, lib.cmr_kv8_last_error_message())


def test_page_calls_of_nothing_are_no_ops(lib):
    assert call_extend(lib, n=0, slots=None, lens=None) == 0
    assert call_fork(lib, n=0, src=None, dst=None, lens=None) == 0
    assert call_free(lib, n=0, slots=None) == 0
    assert kv8.kv8_pages_workspace_bytes(0, 4) == 0
    assert kv8.kv8_pages_workspace_bytes(2, 4, -1) == 0
    assert kv8.kv8_pages_workspace_bytes(2, 1000, 8) >= 4 * (1000 * 2 + 8 * 4)


def test_calls_by_words_are_the_calls(lib):
    for name, (number, words) in kv8._CALLS.items():
        args = kv8.SIGNATURES[name][1]
        kinds = "".join("d" if a is ctypes.c_double else "q" for a in args)
        plain = words.format.lstrip("=")
        spelled = "".join((c[-1] * int(c[:-1] or 1)) for c in re.findall(r"\d*[qd]", plain))
        assert spelled == kinds, name
        ok = words.pack(*[0.0 if k == "d" else 0 for k in kinds])
        assert lib.cmr_kv8_call(number, ok, len(kinds)) in (1, 3)      # zeros: refused
        assert lib.cmr_kv8_call(number, ok, len(kinds) - 1) == 1
        assert b"words" in lib.cmr_kv8_last_error_message()
    assert lib.cmr_kv8_call(6, b"", 0) == 1 and lib.cmr_kv8_call(-1, b"", 0) == 1
    assert lib.cmr_kv8_call(0, None, 28) == 1
    # a count that does not fit 32 bits is refused, not cut
    free = kv8._CALLS["cmr_kv8_free"][1]
    assert lib.cmr_kv8_call(4, free.pack(FAKE, 2, 2, FAKE, 4, FAKE, 1 << 32, 0, 0), 9) == 1
    assert b"negative n" in lib.cmr_kv8_last_error_message()


def test_python_refuses_what_is_not_on_a_gpu():
    f8 = torch.zeros(1, 2, 2, 64, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(1, 2, 2)
    x = torch.zeros(1, 2, 2, 256, dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        pkg.rotate_qk_kv8(None, x, x, v, v, f8, f8, s, s, t)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pkg.attend_kv8(x, f8, f8, s, s, t)
    with pytest.raises(TypeError, match="q must be torch.bfloat16"):
        pkg.attend_kv8(x.float(), f8, f8, s, s, t)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        pkg.attend_kv8(None, f8, f8, s, s, t)
    with pytest.raises(ValueError, match="page_table must be a CUDA tensor"):
        pkg.kv8_free(t, v, v)
    assert cmr.CMR_DEVICE_CACHE_RANGE == 2 and pkg.CMR_DEVICE_PAGES_FULL == 8
