"""cmr_kv8_rotate_qk refuses, on the host, a q that overlaps the k or v that it reads beside it, and
q, k and v that lie in the pages.  No call here reaches a kernel: the addresses are no device's."""
import ctypes

import pytest

from vlm_decoder_positional_b200 import build as libbuild
from vlm_decoder_positional_b200 import kv8

SEC = (ctypes.c_int32 * 3)(11, 11, 10)
N, L, HQ, HK, D, P, PAGES = 10, 2, 8, 2, 256, 64, 4
Q, KV, POOL = L * N * HQ * D * 2, L * N * HK * D * 2, L * PAGES * HK * P * D
AT = dict(q=1 << 20, k=2 << 20, v=3 << 20, kp=4 << 20, vp=5 << 20)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return kv8.lib()


def call(lib, hq=HQ, **kw):
    a = {**AT, **kw}
    return lib.cmr_kv8_rotate_qk(a["q"], a["k"], a["v"], 1 << 16, 2, None, 1 << 16, 1 << 16, N, L, hq,
                                 HK, D, 1e7, SEC, 64, a["kp"], a["vp"], 1 << 16, 1 << 16, PAGES, P,
                                 1 << 16, 2, 2, None, None, None), lib.cmr_kv8_last_error_message()


@pytest.mark.parametrize("name, at", [
    ("k", AT["q"]), ("v", AT["q"]), ("k", AT["q"] + Q - 16), ("v", AT["q"] - KV + 16),
    ("q", AT["kp"]), ("q", AT["vp"] + POOL - 16), ("k", AT["kp"] + 64), ("k", AT["vp"]),
    ("v", AT["kp"] - KV + 16), ("v", AT["vp"])])
def test_overlaps_are_refused(lib, name, at):
    status, message = call(lib, **{name: at})
    assert status == 1 and b"overlaps" in message


@pytest.mark.parametrize("kw", [
    {}, dict(k=AT["q"] + Q), dict(v=AT["q"] - KV), dict(v=AT["k"]), dict(k=AT["kp"] + POOL),
    dict(hq=0, q=None), dict(hq=0, q=AT["k"])])
def test_neighbours_and_shared_inputs_are_not(lib, kw):
    # refused as well, but as addresses of no device
    status, message = call(lib, **kw)
    assert status == 1 and b"not a CUDA pointer" in message
