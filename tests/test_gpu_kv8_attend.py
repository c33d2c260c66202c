"""GPU checks of the attention over the paged 8-bit cache against a 64-bit model, with
the tolerance that tests/kv8_model.py derives from the roundings."""
import numpy as np
import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from tests.kv8_model import Cache, assert_within, attend, i32

pytestmark = pytest.mark.gpu
NAN = 0x7F


def run(dev, lens, offs, L=1, hq=8, hk=2, D=256, P=64, scale=None, seed=0, step=False, slot=None,
        cache=None, change=None, tail=0, q_scale=1.0, want_status=0, kernel=None, **kw):
    g = torch.Generator(device=dev).manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1]) + tail
    spans = [(int(cu[b]), int(cu[b + 1]), int(offs[b])) for b in range(len(lens))]
    if cache is None:
        rows = len(lens) if slot is None else max(slot) + 1
        counts = [0] * rows
        for b, (lo, hi, off) in enumerate(spans):
            counts[b if slot is None else slot[b]] = max(0, -(-(off + hi - lo) // P))
        cache = Cache(dev, counts, L, hk, D, P, seed=seed)
    q = (q_scale * torch.randn((L, n, hq, D), generator=g, device=dev)).to(torch.bfloat16)
    if change is not None:
        change(q, cache)
    scale = D ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full_like(q, 7.0)
    got = pkg.attend_kv8(q, *cache.pool(), cache.table, cu_seqlens=None if step else i32(cu, dev),
                         pos_offset=i32(offs, dev), slot=None if slot is None else i32(slot, dev),
                         scale=scale, out=out, device_status=status, **kw)
    torch.cuda.synchronize()
    assert got is out and int(status.item()) == want_status
    if kernel is not None:
        assert pkg.last_attend_kernel() == kernel
    if tail:
        assert torch.equal(out[:, n - tail:], torch.full_like(out[:, n - tail:], 7.0))
    want, tol = attend(q[:, :n - tail], cache, spans, scale, slot)
    assert_within(out[:, :n - tail], want, tol)
    return out, q, cache


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_steps_of_mixed_depths(cuda_device, D, P):
    offs = [0, 1, 15, 16, 62, 63, 64, 65, 127, 128, 700, 1500, 3]
    run(cuda_device, [1] * 13, offs, D=D, P=P, step=True, seed=D + P, kernel="attend_rows_kernel")


@pytest.mark.parametrize("hq, hk", [(1, 1), (8, 8), (4, 1), (6, 2), (7, 1), (9, 1), (16, 1), (24, 2),
                                    (40, 2), (128, 1)])
def test_groups_of_heads(cuda_device, hq, hk):
    run(cuda_device, [1] * 3, [5, 200, 90], hq=hq, hk=hk, D=64, step=True)
    run(cuda_device, [3, 1, 40], [5, 200, 0], hq=hq, hk=hk, D=64)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_chunks_behind_contexts(cuda_device, D, P):
    run(cuda_device, [1, 100, 0, 33, 64, 250], [300, 0, 9, 127, 128, 1000], D=D, P=P, seed=D + P,
        kernel="attend_tiles_kernel")


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 600])
def test_prompts_of_odd_lengths(cuda_device, n):
    run(cuda_device, [n], [0], L=2)
    run(cuda_device, [n, 1, n], [0, 0, 1], hq=4, hk=4, D=64)


def test_short_chunks_by_rows(cuda_device):
    # few rows per sequence: the decode kernel, with 16 rows of several tokens
    run(cuda_device, [2, 4, 1, 3, 0], [100, 64, 5, 0, 9], hq=8, hk=2, kernel="attend_rows_kernel")
    run(cuda_device, [7, 1, 2], [100, 640, 63], hq=2, hk=1, D=128, P=32, kernel="attend_rows_kernel")


@pytest.mark.parametrize("L", [1, 3])
def test_more_sequences_than_are_split_evenly(cuda_device, L):
    rng = np.random.default_rng(0)
    run(cuda_device, [1] * 2100, rng.integers(0, 70, 2100), L=L, hq=2, hk=1, D=64, P=16, step=True)


@pytest.mark.parametrize("longest", [319, 320])   # with its token: 5 tiles of 64, and one more
def test_tables_of_a_few_pages(cuda_device, longest):
    run(cuda_device, [1] * 5, [longest, 0, 5, 63, 64], P=16, step=True, kernel="attend_rows_kernel")
    run(cuda_device, [2, 3, 1], [longest - 1, 60, 0], D=64, P=16, kernel="attend_rows_kernel")


def test_one_long_sequence(cuda_device):
    run(cuda_device, [1], [70000], hq=8, hk=2, D=128, P=128, step=True)
    run(cuda_device, [40], [20000], hq=8, hk=2, D=128, P=16)


@pytest.mark.parametrize("lens, offs, shape", [
    ([1] * 33 + [130], [200] * 33 + [30000], dict(D=64)),
    ([100] + [6] * 255, [9000] + [70] * 255, dict(D=64, hq=4)),
    ([100] + [6] * 256, [9000] + [70] * 256, dict(D=64, hq=4)),
    ([100] + [6] * 255, [9000] + [70] * 255, dict(D=64)),                    # as many as are planned
    ([100] + [6] * 256, [9000] + [70] * 256, dict(D=64)),                    # one more
    ([0, 40, 0, 0, 300, 7], [5, 4000, 70, 0, 0, 900], dict(L=5, hk=1, P=16)),  # 29 to a head
    ([60, 20], [3000, 100], dict(L=37, hq=2, hk=2, D=64)),                   # 2 to a head
    ([60, 20], [3000, 100], dict(L=38, hq=2, hk=2, D=64)),                   # 1: none is split
    ([128], [127], dict(hq=1, hk=1, D=128)),                                 # a row tile of two tiles
    ([2000], [0], dict(hq=2, hk=1, D=128))])
def test_items_cut_in_pieces(cuda_device, lens, offs, shape):
    # whatever the workspace holds before
    L, D, hq, hk = (shape.get(k, d) for k, d in (("L", 1), ("D", 256), ("hq", 8), ("hk", 2)))
    need = pkg.attend_kv8_workspace_bytes(len(lens), sum(lens), L, hq, hk, D)
    for fill in (0x7F, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda_device)
        run(cuda_device, lens, offs, kernel="attend_tiles_kernel", workspace=ws, **shape)


BOTH = "attend_rows_kernel, attend_tiles_kernel"


@pytest.mark.parametrize("D, P", [(64, 16), (128, 128), (256, 64)])
@pytest.mark.parametrize("lens, offs", [
    ([1] * 60 + [8, 9, 33], [50, 900, 3] * 20 + [700, 64, 4000]),     # 32, 36 and 132 rows
    ([33] + [1] * 40, [5000] + [0, 63, 64, 300] * 10),
    ([0, 2] * 16 + [16, 0], [100] * 34),
    ([1] * 300 + [200], [70] * 300 + [1000])])                        # more than are planned
def test_decode_steps_beside_a_chunk(cuda_device, lens, offs, D, P):
    need = pkg.attend_kv8_workspace_bytes(len(lens), sum(lens) + 5, 1, 8, 2, D)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device)
    a, q, c = run(cuda_device, lens, offs, D=D, P=P, kernel=BOTH, workspace=ws, tail=5)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]), cuda_device)
    b = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=cu, pos_offset=i32(offs, cuda_device))
    n = sum(lens)
    assert torch.equal(a[:, :n], b[:, :n])


def test_malformed_decode_steps_beside_a_chunk_are_flagged(cuda_device):
    dev = cuda_device
    c = Cache(dev, [4] * 40)
    q = torch.ones((1, 70, 8, 256), device=dev, dtype=torch.bfloat16)
    for cu in ([0, 75] + [70] * 39, [0, -1] + [70] * 39, list(range(20)) + [60, 30] + [70] * 19):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=i32(cu, dev), device_status=status)
        assert pkg.last_attend_kernel() == BOTH and int(status.item()) & 1


def test_a_step_of_a_large_group_cut_in_pieces(cuda_device):
    run(cuda_device, [1] * 3, [5, 9000, 300], hq=40, hk=1, D=128, step=True,
        kernel="attend_tiles_kernel")


def test_sequences_that_overlap_are_flagged(cuda_device):
    dev = cuda_device
    c = Cache(dev, [40] * 4)
    cu, offs = i32([0, 200, 100, 300, 0], dev), i32([2000] * 4, dev)
    q = torch.ones((1, 300, 8, 256), device=dev, dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=cu, pos_offset=offs, device_status=status)
    assert int(status.item()) == 1


def test_slots_and_rows_behind_the_last_sequence(cuda_device):
    run(cuda_device, [1, 1, 1], [40, 3, 200], slot=[5, 0, 3], step=True)
    run(cuda_device, [30, 1, 90], [40, 3, 0], slot=[1, 4, 0], tail=37)
    run(cuda_device, [3, 1], [40, 3], tail=2)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.5, 1e-30])
def test_softmax_scales(cuda_device, scale):
    run(cuda_device, [1, 1], [100, 17], scale=scale, step=True, D=64)
    run(cuda_device, [60, 9], [100, 17], scale=scale, D=64)


@pytest.mark.parametrize("lens, step", [([1, 1, 1], True), ([90, 40, 7], False)])
def test_pages_of_very_different_scales(cuda_device, lens, step):
    def change(q, c):
        e = torch.randint(-20, 21, c.vs.shape, device=q.device)
        c.vs.copy_(torch.exp2(e.float()))
        c.ks.copy_(torch.exp2(torch.randint(-12, -5, c.ks.shape, device=q.device).float()))
    run(cuda_device, lens, [300, 64, 1000], P=16, D=128, step=step, change=change)


@pytest.mark.parametrize("lens, step", [([1, 1], True), ([3, 2], False), ([150, 30], False)])
def test_what_nobody_sees_never_shows(cuda_device, lens, step):
    # NaN codes in every row behind a sequence's last token, in pages and in keys and values
    offs = [70, 33]

    def change(q, c):
        for b, (n, off) in enumerate(zip(lens, offs)):
            for x in (c.k, c.v):
                u = x.view(torch.uint8)
                last = off + n
                u[:, c.table[b, (last - 1) // c.P].long(), :, (last - 1) % c.P + 1:] = NAN
    run(cuda_device, lens, offs, step=step, change=change)


@pytest.mark.parametrize("lens, offs", [([3, 2], [70, 33]), ([150, 30], [0, 33]), ([130], [0])])
def test_a_nan_reaches_exactly_the_tokens_that_see_it(cuda_device, lens, offs):
    def change(q, c):
        for b, (n, off) in enumerate(zip(lens, offs)):
            at = off + n // 2                       # a value that later tokens see
            c.v.view(torch.uint8)[:, c.table[b, at // c.P].long(), 0, at % c.P, 17] = 0xFF
            c.v.view(torch.uint8)[:, c.table[b, at // c.P].long(), 1, at % c.P, 200] = NAN
            if n > 100:                             # a key, and a value all see
                at = off + n - 3
                c.k.view(torch.uint8)[:, c.table[b, at // c.P].long(), 0, at % c.P, 3] = NAN
                c.v.view(torch.uint8)[:, c.table[b, 0].long(), 1, 0, 5] = NAN
    out, _, _ = run(cuda_device, lens, offs, change=change)
    assert out.isnan().any() and not out.isnan().all()


@pytest.mark.parametrize("lens, step", [([1, 1], True), ([2, 1], False), ([80, 20], False)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row(cuda_device, lens, step, value):
    dev = cuda_device
    clean, q, c = run(dev, lens, [90, 10], step=step)
    q2 = q.clone()
    q2[0, 0, 1, 100] = value
    out = pkg.attend_kv8(q2, *c.pool(), c.table, pos_offset=i32([90, 10], dev),
                         cu_seqlens=None if step else i32(np.concatenate([[0], np.cumsum(lens)]), dev))
    assert out[0, 0, 1].isnan().all()
    out[0, 0, 1] = clean[0, 0, 1]
    assert torch.equal(out, clean)


def test_tokens_that_see_nothing_get_zeros(cuda_device):
    out, _, _ = run(cuda_device, [1, 1], [-1, 5], step=True)
    assert not out[0, 0].any()
    out, _, _ = run(cuda_device, [6, 50], [-3, -20])
    assert not out[0, :3].any() and not out[0, 6:26].any()
    out, _, _ = run(cuda_device, [60], [-100], hq=4, hk=4)
    assert not out.any()


@pytest.mark.parametrize("lens, step", [([1, 1], True), ([3, 1], False), ([100, 40], False)])
def test_missing_pages_and_bad_scales_are_as_if_not_there(cuda_device, lens, step):
    dev = cuda_device
    offs = [200, 90]
    for spoil, flag in ((lambda c, page: c.table.__setitem__((0, 1), -1), 2),
                        (lambda c, page: c.table.__setitem__((0, 1), c.pages), 2),
                        (lambda c, page: c.ks.__setitem__((0, page), 0.0), 16),
                        (lambda c, page: c.vs.__setitem__((0, page), float("nan")), 16),
                        (lambda c, page: c.vs.__setitem__((0, page), 2.0 ** 61), 16)):
        counts = [-(-(o + n) // 64) for o, n in zip(offs, lens)]
        c = Cache(dev, counts)
        page = int(c.table[0, 1])
        # the model: very low scores for the tokens of that page, by keys of their own
        g = torch.Generator(device=dev).manual_seed(0)
        q = torch.randn((1, sum(lens), 8, 256), generator=g, device=dev).to(torch.bfloat16)
        spoil(c, page)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        cu = i32(np.concatenate([[0], np.cumsum(lens)]), dev)
        out = pkg.attend_kv8(q, *c.pool(), c.table, pos_offset=i32(offs, dev),
                             cu_seqlens=None if step else cu, device_status=status)
        assert int(status.item()) == flag
        # the same sequence without that page: tokens 64 .. 127 taken out
        m = Cache(dev, counts)
        t = m.table.clone()
        t[0, 1:-1] = m.table[0, 2:]
        m.table = t
        want, tol = attend(q, m, [(0, lens[0], offs[0] - 64), (lens[0], sum(lens), offs[1])],
                           256 ** -0.5)
        seen_by_all = slice(0, sum(lens))
        assert_within(out[:, seen_by_all], want, tol)


def test_a_context_longer_than_the_table_is_cut(cuda_device):
    for lens, step in (([1], True), ([70], False)):
        c = Cache(cuda_device, [2])
        run(cuda_device, lens, [150], cache=c, step=step, want_status=2)


def test_slot_outside_the_table(cuda_device):
    dev = cuda_device
    c = Cache(dev, [2, 2])
    for n in (1, 40):
        q = torch.ones((1, 2 * n, 8, 256), device=dev, dtype=torch.bfloat16)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=i32([0, n, 2 * n], dev),
                             pos_offset=i32([3, 4], dev), slot=i32([7, 1], dev),
                             device_status=status)
        assert int(status.item()) == 2
        assert not out[:, :n].any() and out[:, n:].abs().sum() > 0


@pytest.mark.parametrize("n", [4, 200])
def test_malformed_cu_seqlens_are_flagged(cuda_device, n):
    dev = cuda_device
    c = Cache(dev, [4, 4])
    q = torch.ones((1, n, 8, 256), device=dev, dtype=torch.bfloat16)
    for cu in ([0, n + 5, n], [0, -1, n], [2, 1, n]):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=i32(cu, dev), device_status=status)
        assert int(status.item()) & 1


def test_the_same_call_gives_the_same_bits(cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(1)
    offs = rng.integers(0, 2000, 60)
    a, q, c = run(dev, [1] * 60, offs, step=True, D=128)
    for _ in range(5):
        b = pkg.attend_kv8(q, *c.pool(), c.table, pos_offset=i32(offs, dev))
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens, offs", [([280], [1000]), ([90, 1, 300], [0, 2000, 128]),
                                        ([1, 1], [3000, 90])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_slow_memory_changes_nothing(cuda_device, lens, offs, D):
    # with the caches full of something else the loads come late and in other orders
    dev = cuda_device
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    want, q, c = run(dev, lens, offs, D=D)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]), dev)
    for r in range(15):
        flush.fill_(r)
        torch.cuda.synchronize()
        out = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=cu, pos_offset=i32(offs, dev))
        assert torch.equal(out, want)


def test_pages_beyond_four_gigabytes(cuda_device):
    # codes whose byte offsets pass 32 bits: the last pages of a pool of 4.6 GB for K and as
    # much for V, written and read by each kernel
    dev = cuda_device
    pages, P, D, hk = 35000, 128, 256, 2
    c = Cache(dev, [1], 1, hk, D, 16)
    c.P, c.pages = P, pages
    c.k, c.v = (torch.empty((2, pages, hk, P, D), dtype=torch.uint8, device=dev)
                .view(torch.float8_e4m3fn) for _ in range(2))
    c.L = 2
    c.ks, c.vs = (torch.ones((2, pages, hk), device=dev) for _ in range(2))
    c.table = i32([[pages - 1, 3, pages - 2], [pages - 3, pages - 5, -1]], dev)
    g = torch.Generator(device=dev).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)
    text = i32([1 << 30] * 2, dev), i32([0, 0], dev)
    k, v = rand(2, 500, hk, D), rand(2, 500, hk, D)
    pkg.rotate_qk_kv8(None, k, v, *text, *c.pool(), c.table, cu_seqlens=i32([0, 300, 500], dev))
    run(dev, [300, 200], [0, 0], L=2, D=D, P=P, cache=c, kernel="attend_tiles_kernel")
    pkg.rotate_qk_kv8(None, k[:, :2].contiguous(), v[:, :2].contiguous(), *text, *c.pool(), c.table,
                      pos_offset=i32([300, 200], dev))
    run(dev, [1, 1], [300, 200], L=2, D=D, P=P, cache=c, step=True, kernel="attend_rows_kernel")
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    for p in c.table.flatten().tolist():
        if p >= 0:
            refs[p] = 1
    want = [c.values(w, 1, r, 1, n).clone() for w in "kv" for r, n in ((0, 301), (1, 201))]
    pkg.kv8_compact(*c.pool(), c.table, refs)
    assert int(c.table.max()) == 4
    got = [c.values(w, 1, r, 1, n) for w in "kv" for r, n in ((0, 301), (1, 201))]
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_sequences_of_one_token_with_cu_seqlens_are_a_step(cuda_device):
    offs = [300, 5, 64, 1000]
    a, q, c = run(cuda_device, [1] * 4, offs, step=True)
    b = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=i32([0, 1, 2, 3, 4], cuda_device),
                       pos_offset=i32(offs, cuda_device))
    assert torch.equal(a, b)


def test_empty_calls(cuda_device):
    dev = cuda_device
    c = Cache(dev, [1])
    q = torch.zeros((1, 0, 8, 256), device=dev, dtype=torch.bfloat16)
    assert pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=i32([0], dev)).shape == q.shape
    q3 = torch.ones((2, 8, 256), device=dev, dtype=torch.bfloat16)       # [N, H, D]
    assert pkg.attend_kv8(q3, *c.pool(), c.table, cu_seqlens=i32([0, 2], dev)).shape == q3.shape


def test_two_streams_with_workspaces_of_their_own(cuda_device):
    dev = cuda_device
    offs = [[5000, 100, 2500], [300, 4000, 64]]
    made, want, ws, streams = [], [], [], []
    for i in range(2):
        out, q, c = run(dev, [1] * 3, offs[i], step=True, seed=i, D=128)
        made.append((q, c))
        want.append(out)
        ws.append(torch.empty(pkg.attend_kv8_workspace_bytes(3, 3, 1, 8, 2, 128), dtype=torch.uint8,
                              device=dev))
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    outs = [[], []]
    for rep in range(20):
        for i in range(2):
            q, c = made[i]
            outs[i].append(pkg.attend_kv8(q, *c.pool(), c.table, pos_offset=i32(offs[i], dev),
                                          workspace=ws[i], stream=streams[i], out=torch.empty_like(q)))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


@pytest.mark.parametrize("lens, step", [([1, 1, 1], True), ([90, 40, 7], False)])
def test_captured_and_replayed(cuda_device, lens, step):
    # the first call of these shapes may well be the captured one
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(0)
    c = Cache(dev, [40, 40, 40], D=128)
    q = torch.randn((1, sum(lens), 8, 128), generator=g, device=dev).to(torch.bfloat16)
    cu = None if step else i32(np.concatenate([[0], np.cumsum(lens)]), dev)
    off = i32([1000, 0, 77], dev)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=cu, pos_offset=off, out=out)
    for o in ([1000, 0, 77], [5, 2000, 600], [0, 0, 0]):
        off.copy_(i32(o, dev))
        graph.replay()
        torch.cuda.synchronize()
        again = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=cu, pos_offset=off)
        assert torch.equal(out, again)


def test_refusals(cuda_device):
    dev = cuda_device
    c = Cache(dev, [2, 2], D=64)
    q = torch.ones((1, 2, 4, 64), device=dev, dtype=torch.bfloat16)
    ok = lambda **kw: pkg.attend_kv8(**{**dict(q=q, k_pages=c.k, v_pages=c.v, k_scales=c.ks,
                                               v_scales=c.vs, page_table=c.table), **kw})
    ok()
    need = pkg.attend_kv8_workspace_bytes(2, 2, 1, 4, 2, 64)
    for kw, err in [(dict(q=q.half()), TypeError), (dict(q=q[:, :, :3].contiguous()), pkg.Kv8Error),
                    (dict(out=q), pkg.Kv8Error), (dict(out=q.float()), TypeError),
                    (dict(out=torch.empty_like(q)[:, :1]), ValueError),
                    (dict(k_pages=c.k[..., :32].contiguous()), ValueError),
                    (dict(scale=float("nan")), pkg.Kv8Error),
                    (dict(workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev)), pkg.Kv8Error),
                    (dict(workspace=torch.empty(need, dtype=torch.uint8)), ValueError),
                    (dict(workspace=torch.empty(need + 8, dtype=torch.uint8, device=dev)[8:]),
                     pkg.Kv8Error),
                    (dict(pos_offset=i32([1], dev)), ValueError),
                    (dict(slot=i32([[0, 1]], dev)), ValueError),
                    (dict(page_table=c.table.long()), TypeError)]:
        with pytest.raises(err):
            ok(**kw)


def test_queries_beyond_four_gigabytes(cuda_device):
    # elements of Q, K, V and the result whose indices pass 31 bits: the last sequences of a
    # large call are what they are alone
    dev = cuda_device
    n, T, D, P, hk = 1 << 20, 512, 256, 128, 9
    B, pages = n // T, T // P
    g = torch.Generator(device=dev).manual_seed(3)
    text = lambda m: (i32([1 << 30] * m, dev), i32([0] * m, dev))
    cu = i32(np.arange(B + 1) * T, dev)
    k = torch.empty((1, n, hk, D), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    v = k.flip(1)
    table = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
    codes = lambda m: torch.zeros((1, m, hk, P, D), dtype=torch.uint8, device=dev).view(
        torch.float8_e4m3fn)
    pool = (codes(B * pages), codes(B * pages), *(torch.ones((1, B * pages, hk), device=dev)
                                                  for _ in range(2)))
    pkg.rotate_qk_kv8(None, k, v, *text(B), *pool, table, cu_seqlens=cu)
    few = (codes(pages), codes(pages), *(torch.ones((1, pages, hk), device=dev) for _ in range(2)))
    pkg.rotate_qk_kv8(None, k[:, -T:].contiguous(), v[:, -T:].contiguous(), *text(1), *few,
                      table[:1].contiguous(), cu_seqlens=i32([0, T], dev))
    for whole, alone in zip(pool, few):
        assert torch.equal(whole[:, -pages:].view(torch.uint8), alone.view(torch.uint8))
    q = k                                        # [1, n, 9, 256]: as many query heads
    out = pkg.attend_kv8(q, *pool, table, cu_seqlens=cu)
    assert pkg.last_attend_kernel() == "attend_tiles_kernel"
    want = pkg.attend_kv8(q[:, -T:].contiguous(), *pool, table[-1:].contiguous(),
                          cu_seqlens=i32([0, T], dev))
    # each is within half a step of bf16 and 2^-9 of the mean magnitude of the exact result
    mean = float(want.float().abs().max())
    assert float((out[:, -T:].float() - want.float()).abs().max()) <= (2 * 2 ** -8 + 2 * 2 ** -9) * \
        max(mean, float(v.float().abs().max()))
    # a step of as many sequences, all of which read one row
    slot = torch.full((n,), B - 1, dtype=torch.int32, device=dev)
    off = torch.full((n,), T - 1, dtype=torch.int32, device=dev)
    pkg.attend_kv8(q, *pool, table, pos_offset=off, slot=slot, out=out)
    assert pkg.last_attend_kernel() == "attend_rows_kernel"
    one = pkg.attend_kv8(q[:, -3000:].contiguous(), *pool, table, pos_offset=off[:3000].contiguous(),
                         slot=slot[:3000].contiguous())
    assert torch.equal(out[:, -3000:], one)


def test_sequences_without_tokens_leave_everything_as_it_was(cuda_device):
    dev = cuda_device
    c = Cache(dev, [1, 1])
    q = torch.ones((1, 70, 8, 256), device=dev, dtype=torch.bfloat16)
    out = torch.full_like(q, 7.0)
    for n in (70, 2):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.attend_kv8(q[:, :n].contiguous(), *c.pool(), c.table, cu_seqlens=i32([0, 0, 0], dev),
                       out=out[:, :n].contiguous() if n < 70 else out, device_status=status)
        assert int(status.item()) == 0
    assert torch.equal(out, torch.full_like(out, 7.0))
