"""GPU checks of the upkeep of the paged cache against a model on whole numbers, and of
all its calls together as a serving loop uses them."""
import numpy as np
import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from tests.kv8_model import Cache, Pages, assert_within, attend, i32
from vlm_decoder_positional_b200 import cmr

pytestmark = pytest.mark.gpu


class Both:
    """A cache on the GPU and its model, side by side."""

    def __init__(self, dev, rows, cols, pages, P=64, L=2, hk=2, D=64, seed=0):
        self.dev, self.P = dev, P
        self.c = Cache(dev, [], L, hk, D, P, spare=pages, seed=seed)
        self.c.table = torch.full((rows, cols), -1, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.m = Pages(self.c.table.cpu(), self.refs.cpu(), P)
        self.codes = [x.view(torch.uint8).clone() for x in (self.c.k, self.c.v)]
        self.scales = [x.clone() for x in (self.c.ks, self.c.vs)]

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.c.table.cpu().numpy(), self.m.t)
        assert np.array_equal(self.refs.cpu().numpy(), self.m.r)
        assert int(self.status.item()) == self.m.status
        for x, y in zip((self.c.k, self.c.v), self.codes):
            assert torch.equal(x.view(torch.uint8), y)
        for x, y in zip((self.c.ks, self.c.vs), self.scales):
            assert torch.equal(x, y)

    def extend(self, slots, lens):
        pkg.kv8_extend(self.c.table, self.refs, i32(slots, self.dev), i32(lens, self.dev), self.P,
                       device_status=self.status)
        self.m.extend(slots, lens)
        self.same()

    def free(self, slots):
        pkg.kv8_free(self.c.table, self.refs, i32(slots, self.dev), device_status=self.status)
        self.m.free(slots)
        self.same()

    def fork(self, src, dst, lens):
        pkg.kv8_fork(*self.c.pool(), self.c.table, self.refs, i32(src, self.dev),
                     i32(dst, self.dev), i32(lens, self.dev), device_status=self.status)
        for a, b, n in self.m.fork(src, dst, lens):
            for x in self.codes:
                x[:, b, :, :n] = x[:, a, :, :n]
            for x in self.scales:
                x[:, b] = x[:, a]
        self.same()

    def compact(self):
        pkg.kv8_compact(*self.c.pool(), self.c.table, self.refs, device_status=self.status)
        for a, b in self.m.compact():
            for x in self.codes + self.scales:
                x[:, b] = x[:, a]
        self.same()


def test_a_life_of_a_pool(cuda_device):
    b = Both(cuda_device, 8, 6, 40)
    b.extend([0, 3, 5], [64, 1, 200])
    b.extend([3, 0], [130, 64])
    b.fork([5, 5, 0], [1, 2, 7], [200, 64, 0])
    b.fork([1], [4], [130])
    b.free([5, 0])
    b.extend([6, 5], [300, 20])
    b.compact()
    b.free([1, 2, 3, 4, 5, 6, 7])
    b.compact()
    assert not b.m.status and not b.m.r.any()


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("P", [16, 128])
def test_random_lives(cuda_device, seed, P):
    rng = np.random.default_rng(seed)
    rows, cols, pages = 24, 12, 90
    b = Both(cuda_device, rows, cols, pages, P=P, L=1, hk=1, seed=seed)
    for _ in range(25):
        kind = rng.integers(0, 4)
        n = int(rng.integers(1, 9))
        slots = rng.integers(-1, rows + 1, n)          # some twice, some outside
        lens = rng.integers(-1, cols * P + 20, n)
        if kind == 0:
            b.extend(slots.tolist(), (lens // 3).tolist())
        elif kind == 1:
            b.free(slots.tolist())
        elif kind == 2:
            src = rng.integers(-1, rows + 1, n)
            held = [b.m.count(s) * P if 0 <= s < rows else 5 for s in src]
            b.fork(src.tolist(), slots.tolist(),
                   [int(rng.integers(-1, h + 3)) for h in held])
        else:
            b.compact()


def test_a_pool_that_runs_out(cuda_device):
    b = Both(cuda_device, 6, 8, 10)
    b.extend([0, 1, 2, 3], [64 * 4, 64 * 5, 64 * 2, 64])       # 2 and 3 find too few
    assert b.m.status == pkg.CMR_DEVICE_PAGES_FULL
    b.extend([3], [64])
    b.fork([0, 0, 1], [2, 4, 5], [70, 256, 80])                # no page for the tails
    b.free([0])
    b.fork([1, 1], [0, 2], [70, 100])


def test_the_same_row_twice_and_rows_outside(cuda_device):
    b = Both(cuda_device, 5, 4, 16)
    b.extend([1, 1, 2], [100, 200, 10])
    b.fork([1, 1, 2], [3, 3, 3], [100, 90, 10])
    b.fork([1, 1], [1, 2], [64, 64])                           # onto itself, onto a full row
    b.fork([4], [0], [1])                                      # of an empty row
    b.free([3, 3, 3, 9, -1])
    b.free([3])
    assert b.m.status == 2


def test_a_large_pool_and_many_entries(cuda_device):
    rng = np.random.default_rng(3)
    rows = 3000
    b = Both(cuda_device, rows, 40, 70001, P=16, L=1, hk=1, D=64)
    lens = rng.integers(0, 600, rows)
    b.extend(list(range(rows)), lens.tolist())
    gone = rng.permutation(rows)[:1500].tolist()
    b.free(gone)
    src = [s for s in range(rows) if s not in set(gone)]
    b.fork(src, gone[:len(src)], [int(lens[s]) for s in src])
    b.free(src[::2])
    b.compact()


def test_compaction_of_nothing_and_of_a_full_pool(cuda_device):
    b = Both(cuda_device, 2, 8, 8)
    b.compact()
    b.extend([0, 1], [64 * 4, 64 * 4])
    b.compact()
    b.free([0])
    b.compact()
    assert b.m.r.tolist() == [1] * 4 + [0] * 4


def test_a_freed_page_that_is_free_already_is_flagged(cuda_device):
    b = Both(cuda_device, 3, 4, 8)
    b.extend([0], [128])
    b.refs.zero_()
    pkg.kv8_free(b.c.table, b.refs, i32([0], b.dev), device_status=b.status)
    assert int(b.status.item()) == 2 and not b.refs.any() and (b.c.table == -1).all()


def test_refusals(cuda_device):
    dev = cuda_device
    b = Both(dev, 3, 4, 8)
    one = i32([0], dev)
    with pytest.raises(pkg.Kv8Error):
        pkg.kv8_extend(b.c.table, b.refs, one, one, 48)
    with pytest.raises(ValueError):
        pkg.kv8_extend(b.c.table, b.refs, one, i32([1, 2], dev), 64)
    with pytest.raises(TypeError):
        pkg.kv8_free(b.c.table, b.refs.long(), one)
    with pytest.raises(ValueError):
        pkg.kv8_fork(*b.c.pool(), b.c.table, b.refs[:4], one, one, one)
    with pytest.raises(ValueError):
        pkg.kv8_compact(*b.c.pool(), b.c.table, b.refs.reshape(2, 4))
    with pytest.raises(pkg.Kv8Error):
        pkg.kv8_compact(*b.c.pool(), b.c.table, b.refs,
                        workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    none = i32([], dev)
    assert pkg.kv8_extend(b.c.table, b.refs, none, none, 64) is b.c.table
    pkg.kv8_free(b.c.table, b.refs, none)
    pkg.kv8_fork(*b.c.pool(), b.c.table, b.refs, none, none, none)
    b.same()


def test_captured_and_replayed(cuda_device):
    dev = cuda_device
    b = Both(dev, 6, 4, 24)
    slots, lens = i32([0, 1, 2], dev), i32([100, 64, 200], dev)
    dst, n = i32([3, 4], dev), i32([100, 130], dev)
    src = i32([0, 2], dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkg.kv8_extend(b.c.table, b.refs, slots, lens, 64)
        pkg.kv8_fork(*b.c.pool(), b.c.table, b.refs, src, dst, n)
        pkg.kv8_free(b.c.table, b.refs, slots)
        pkg.kv8_compact(*b.c.pool(), b.c.table, b.refs)
        pkg.kv8_free(b.c.table, b.refs, dst)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert not b.refs.any() and (b.c.table == -1).all()


def test_calls_follow_what_other_streams_and_libraries_enqueue(cuda_device):
    """Each call's first kernel may be placed before the work ahead of it ends, but must
    see all of it: long kernels of torch write every input just before, on the same
    stream, on another one behind an event, and inside a capture with such a join."""
    dev = cuda_device
    L, B, D, P = 1, 4, 64, 16
    g = torch.Generator(device=dev).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)
    b = Both(dev, B, 8, 40, P=P, L=L, hk=2, D=D)
    src = [rand(L, B, h, D) for h in (4, 2, 2)]
    off0, lens0 = i32([5, 30, 77, 0], dev), i32([6, 31, 78, 1], dev)
    slots = i32([0, 1, 2, 3], dev)
    start, amount = i32([cmr.TEXT_ONLY_START] * B, dev), i32([0] * B, dev)
    big = torch.ones(1 << 27, device=dev)
    held = [b.c.table, b.refs, b.c.ks, b.c.vs, b.c.k.view(torch.uint8), b.c.v.view(torch.uint8)]
    state = [x.clone() for x in held]

    def work(inputs, out):
        q, k, v, off, lens = inputs
        big.mul_(1.0)                                  # half a GB twice: about 0.2 ms
        for x, y in zip((q, k, v, off, lens), (*src, off0, lens0)):
            x.copy_(y)
        return q, k, v, off, lens

    def calls(inputs, out, side=None):
        if side is None:
            work(inputs, out)
        else:
            cur = torch.cuda.current_stream()
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                work(inputs, out)
            cur.wait_stream(side)
        q, k, v, off, lens = inputs
        pkg.kv8_extend(b.c.table, b.refs, slots, lens, P)
        pkg.rotate_qk_kv8(q, k, v, start, amount, *b.c.pool(), b.c.table, pos_offset=off)
        pkg.attend_kv8(q, *b.c.pool(), b.c.table, pos_offset=off, out=out)
        pkg.kv8_free(b.c.table, b.refs, slots)
        pkg.kv8_compact(*b.c.pool(), b.c.table, b.refs)

    def fresh():
        return [torch.zeros_like(x) for x in (*src, off0, lens0)], torch.zeros_like(src[0])

    def reset():
        for x, y in zip(held, state):
            x.copy_(y)
        torch.cuda.synchronize()

    reset()
    inputs, want = fresh()
    calls(inputs, want)
    torch.cuda.synchronize()
    assert want.abs().sum() > 0 and not b.refs.any()
    side = torch.cuda.Stream()
    for other in (None, side):
        for _ in range(4):
            reset()
            inputs, out = fresh()
            torch.cuda.synchronize()
            calls(inputs, out, other)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    inputs, out = fresh()
    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        calls(inputs, out, side)
    for _ in range(3):
        reset()
        for x in (*inputs, out):
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_serving_loop(cuda_device):
    """Prompts in, branches forked, tokens appended to each, some sequences leave, the pool
    is compacted, others come: at each point the attention equals the model's over the
    values that the cache holds, and those are the written ones within e4m3's rounding."""
    dev = cuda_device
    L, hq, hk, D, P = 2, 8, 2, 128, 32
    rows = 6
    b = Both(dev, rows, 12, 60, P=P, L=L, hk=hk, D=D)
    g = torch.Generator(device=dev).manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)
    kept = {}  # row: (K as the cache should hold it, V), [L, tokens, hk, D]
    text = lambda n: (i32([cmr.TEXT_ONLY_START] * n, dev), i32([0] * n, dev))

    def put(slots, lens):
        n = sum(lens)
        offs = [kept[s][0].shape[1] if s in kept else 0 for s in slots]
        pkg.kv8_extend(b.c.table, b.refs, i32(slots, dev),
                       i32([o + k for o, k in zip(offs, lens)], dev), P, device_status=b.status)
        q, k, v = rand(L, n, hq, D), rand(L, n, hk, D), rand(L, n, hk, D)
        cu = np.concatenate([[0], np.cumsum(lens)])
        spans = [(int(cu[i]), int(cu[i + 1]), offs[i]) for i in range(len(slots))]
        start, amount = text(len(slots))
        step = all(x == 1 for x in lens)
        kw = dict(cu_seqlens=None if step else i32(cu, dev), pos_offset=i32(offs, dev),
                  slot=i32(slots, dev), device_status=b.status)
        rk = k.clone()
        cmr.rotate_qk_shift(None, rk, start, amount, cu_seqlens=i32(cu, dev),
                            pos_offset=i32(offs, dev))
        pkg.rotate_qk_kv8(q, k, v, start, amount, *b.c.pool(), b.c.table, **kw)
        out = pkg.attend_kv8(q, *b.c.pool(), b.c.table, **kw)
        for i, s in enumerate(slots):
            new = (rk[:, cu[i]:cu[i + 1]], v[:, cu[i]:cu[i + 1]])
            kept[s] = new if s not in kept else tuple(
                torch.cat([x, y], dim=1) for x, y in zip(kept[s], new))
        want, tol = attend(q, b.c, spans, D ** -0.5, slots)
        assert_within(out, want, tol)
        assert int(b.status.item()) == 0
        check()

    def check():
        for s, (k, v) in kept.items():
            n = k.shape[1]
            for l in range(L):
                for h in range(hk):
                    for which, x in (("k", k), ("v", v)):
                        got = b.c.values(which, l, s, h, n)
                        x = x[l, :, h].double()
                        # half a step: 2^-4 relative, or half of 2^-9 of the largest scale
                        # there is for values of this size, and once more where a page's
                        # scale grew
                        top = 2.0 ** np.ceil(np.log2(float(x.abs().max()) / 448))
                        assert ((got - x).abs() <= x.abs() * 2.0 ** -4 + top * 2.0 ** -9).all()

    put([0, 2], [70, 45])
    put([0, 2], [1, 1])
    pkg.kv8_fork(*b.c.pool(), b.c.table, b.refs, i32([0, 0, 2], dev), i32([1, 3, 4], dev),
                 i32([71, 64, 46], dev), device_status=b.status)
    kept[1], kept[4] = kept[0], kept[2]
    kept[3] = tuple(x[:, :64] for x in kept[0])
    check()
    for _ in range(3):
        put([0, 1, 2, 3, 4], [1] * 5)
    pkg.kv8_free(b.c.table, b.refs, i32([0, 2], dev), device_status=b.status)
    del kept[0], kept[2]
    pkg.kv8_compact(*b.c.pool(), b.c.table, b.refs, device_status=b.status)
    live = int((b.refs > 0).sum())
    assert (b.refs[:live] > 0).all() and int(b.c.table.max()) < live
    check()
    put([0, 5, 1, 3], [90, 3, 20, 1])
    put([0, 1, 3, 4, 5], [1] * 5)
