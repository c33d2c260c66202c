"""GPU checks of the rotation that writes the paged 8-bit cache: the codes and scales
are those of the definition exactly, on the rotated K that cmr_rotate_qk_cache stores,
and Q is rotated bit for bit as there."""
import numpy as np
import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from tests.kv8_model import Cache, encode, i32, scale_exp
from vlm_decoder_positional_b200 import cmr

pytestmark = pytest.mark.gpu


def rand(shape, g, dev):
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


def state(spans, rng, dev):
    """(start, amount) of sequences of which half hold an image."""
    start, amount = [], []
    for lo, hi, off in spans:
        total = max(0, off) + hi - lo
        image = total > 67 and rng.random() < 0.6
        start.append(int(rng.integers(0, total - 67)) + 67 if image else cmr.TEXT_ONLY_START)
        amount.append(58 if image else 0)
    return i32(start, dev), i32(amount, dev)


def rotated(x, start, amount, spans, sections, rot):
    """x rotated by the bf16 kernels; tokens of no sequence left as they are."""
    out = x.clone()
    for b, (lo, hi, off) in enumerate(spans):
        if hi > lo:
            part = x[:, lo:hi].clone(memory_format=torch.contiguous_format)
            cu = i32([0, hi - lo], x.device)
            cmr.rotate_qk_shift(None, part, start[b:b + 1], amount[b:b + 1], cu_seqlens=cu,
                                pos_offset=i32([off], x.device), sections=sections, rot_dim=rot)
            out[:, lo:hi] = part
    return out


def expected(cache, which, x, spans, slot):
    """Codes (uint8) and scales after the write of rows x."""
    codes = (cache.k if which == "k" else cache.v).view(torch.uint8).clone()
    scales = (cache.ks if which == "k" else cache.vs).clone()
    P, table = cache.P, cache.table.cpu().numpy()
    flag = 0
    for b, (lo, hi, off) in enumerate(spans):
        row = b if slot is None else slot[b]
        if hi > lo and off < 0:
            flag |= 2
        p = max(off, 0)
        while p < off + hi - lo:
            end = min(off + hi - lo, (p // P + 1) * P)
            j, first = p // P, p % P
            inside = 0 <= row < table.shape[0] and j < table.shape[1]
            page = table[row, j] if inside else -1
            if not 0 <= page < cache.pages:
                flag |= 2
                p = end
                continue
            new = x[:, lo + p - off:lo + end - off]                     # [L, n, hk, D]
            for l in range(cache.L):
                for h in range(cache.hk):
                    y = new[l, :, h]
                    fin = y[torch.isfinite(y)]
                    e = scale_exp(float(fin.abs().max()) if fin.numel() else 0.0)
                    s, old = 2.0 ** e, float(scales[l, page, h])
                    if first:
                        if not 2.0 ** -60 <= old <= 2.0 ** 60:
                            flag |= 16
                        elif old >= s:
                            s = old
                        else:
                            held = codes[l, page, h, :first].view(torch.float8_e4m3fn).double()
                            codes[l, page, h, :first] = encode(held * old, s)
                    codes[l, page, h, first:first + end - p] = encode(y, s)
                    scales[l, page, h] = s
            p = end
    return codes, scales, flag


def check(dev, lens, offs, L=2, hq=4, hk=2, D=128, P=64, rot=64, sections=(11, 11, 10), seed=0,
          step=False, slot=None, max_pages=None, tail=0, change=None, stream=None, scales=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1]) + tail
    spans = [(int(cu[b]), int(cu[b + 1]), int(offs[b])) for b in range(len(lens))]
    rows = len(lens) if slot is None else max(slot) + 1
    counts = [0] * rows
    for b, (lo, hi, off) in enumerate(spans):
        r = b if slot is None else slot[b]
        if r >= 0:
            counts[r] = max(0, -(-(off + hi - lo) // P))
    if max_pages is not None:
        counts = [min(c, max_pages) for c in counts]
    cache = Cache(dev, counts, L, hk, D, P, seed=seed, max_pages=max_pages)
    if scales is not None:
        scales(cache)
    q, k, v = rand((L, n, hq, D), g, dev), rand((L, n, hk, D), g, dev), rand((L, n, hk, D), g, dev)
    if change is not None:
        change(k, v)
    start, amount = state(spans, rng, dev)
    want_q = rotated(q, start, amount, spans, sections, rot) if hq else q.clone()
    want_k = rotated(k, start, amount, spans, sections, rot)
    want = {w: expected(cache, w, x, spans, slot) for w, x in (("k", want_k), ("v", v))}
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kk, vv = k.clone(), v.clone()
    pkg.rotate_qk_kv8(q if hq else None, kk, vv, start, amount, *cache.pool(), cache.table,
                      cu_seqlens=None if step else i32(cu, dev), pos_offset=i32(offs, dev),
                      slot=None if slot is None else i32(slot, dev), sections=sections,
                      rot_dim=rot, device_status=status, stream=stream)
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(q, want_q) and same(kk, k) and same(vv, v)
    for w, codes, sc in (("k", cache.k, cache.ks), ("v", cache.v, cache.vs)):
        assert torch.equal(sc.view(torch.int32), want[w][1].view(torch.int32)), w
        assert torch.equal(codes.view(torch.uint8), want[w][0]), w
    assert int(status.item()) == want["k"][2] | want["v"][2]
    return cache


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_ragged_prompts_and_chunks(cuda_device, D, P):
    check(cuda_device, [1, 200, 0, 77, 128, 3, 300], [0, 0, 5, 64, 130, 255, 17], D=D, P=P, seed=D + P)


@pytest.mark.parametrize("hq, hk, rot, sections", [
    (8, 8, 64, (11, 11, 10)), (3, 1, 16, (4, 2, 2)), (0, 3, 64, (11, 11, 10)),
    (2, 2, 48, (8, 8, 8)), (16, 1, 128, (22, 21, 21)), (5, 5, 32, (16, 0, 0))])
def test_heads_and_rotated_dims(cuda_device, hq, hk, rot, sections):
    check(cuda_device, [90, 33], [11, 0], hq=hq, hk=hk, D=128, rot=rot, sections=sections, seed=hq)


def test_every_dim_rotated(cuda_device):
    check(cuda_device, [150, 1], [0, 127], D=256, P=128, rot=256, sections=(43, 43, 42))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 128])
def test_steps_append_and_grow_scales(cuda_device, D, P):
    offs = [0, 1, P - 1, P, 5 * P + 3, 2 * P - 1, 40]
    def grow(k, v):  # some tokens far above their page's scale, some far below
        k[:, 2], v[:, 3], k[:, 4], v[:, 5] = k[:, 2] * 64, v[:, 3] * 300, k[:, 4] / 1000, 0
    check(cuda_device, [1] * 7, offs, D=D, P=P, step=True, change=grow, seed=3)


def test_a_step_of_many_sequences_and_one_of_one(cuda_device):
    rng = np.random.default_rng(0)
    check(cuda_device, [1] * 130, rng.integers(0, 900, 130), L=6, hq=8, D=256, step=True)
    check(cuda_device, [1], [700], L=1, hq=8, D=256, step=True)


def test_growing_scales_of_chunks(cuda_device):
    def grow(k, v):
        k[:, :60] *= 100
        v[:, 70:] *= 1e6
    check(cuda_device, [60, 60], [40, 7], D=256, change=grow)


def test_values_at_the_ends_of_the_range(cuda_device):
    def extreme(k, v):
        k[0, 0], k[0, 1] = 3e38, -1e-38           # beyond 448 * 2^60, and far below 2^-60
        k[1] = 0
        v[0, :20, 0] = 448 * 2.0 ** 5              # exactly on the border of a scale
        v[0, :20, 1] = 450.0                       # just above it
        v[1] = 1e-30
    check(cuda_device, [20], [0], D=128, change=extreme)
    check(cuda_device, [1, 1], [0, 3], D=128, step=True,
          change=lambda k, v: (k.fill_(3e38), v.fill_(1e-38)))


@pytest.mark.parametrize("step", [False, True])
def test_what_is_not_finite_is_held_as_nan(cuda_device, step):
    def odd(k, v):
        k[0, 0, 0, 100] = float("inf")            # dims that are not rotated
        k[1, 1, 1, 90] = float("nan")
        v[0, 0, 1, 5] = -float("inf")
        v[1, 1, 0] = float("nan")                 # a whole row
    lens, offs = ([1, 1, 1], [3, 64, 130]) if step else ([40, 70], [3, 0])
    check(cuda_device, lens, offs, D=128, step=step, change=odd)


def test_rows_behind_the_last_sequence_are_left_alone(cuda_device):
    check(cuda_device, [30, 50], [0, 9], tail=45)


def test_slots_and_what_lies_outside_the_cache(cuda_device):
    dev = cuda_device
    check(dev, [70, 1, 40], [0, 100, 30], slot=[4, 0, 2])
    check(dev, [70, 1, 40], [0, 100, 30], slot=[1, -1, 3])                 # no such row
    check(dev, [200, 50], [0, 100], max_pages=2)                           # behind the table
    check(dev, [1, 1, 1], [200, 5, 127], max_pages=2, step=True)
    check(dev, [30, 1], [-10, -1])                                         # before the start
    check(dev, [1, 1], [-5, 3], step=True)

    def holes(cache):
        cache.table[0, 1], cache.table[1, 0] = -1, cache.pages
    check(dev, [200, 50], [0, 20], scales=holes)


@pytest.mark.parametrize("bad", [0.0, float("nan"), float("inf"), -1.0, 2.0 ** 70])
def test_a_held_page_with_a_bad_scale_is_flagged(cuda_device, bad):
    def spoil(cache):
        cache.ks.fill_(bad)
    check(cuda_device, [20], [10], scales=spoil)
    check(cuda_device, [1], [10], scales=spoil, step=True)


def test_malformed_cu_seqlens_set_the_status_and_touch_nothing_else(cuda_device):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(1)
    cache = Cache(dev, [2, 2], D=64)
    before = [x.clone() for x in cache.pool()]
    q, k, v = rand((1, 20, 2, 64), g, dev), rand((1, 20, 2, 64), g, dev), rand((1, 20, 2, 64), g, dev)
    s, a = i32([cmr.TEXT_ONLY_START] * 2, dev), i32([0, 0], dev)
    for cu in ([0, 25, 20], [0, -3, 20], [10, 5, 20]):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.rotate_qk_kv8(q, k, v, s, a, *cache.pool(), cache.table, cu_seqlens=i32(cu, dev),
                          device_status=status)
        assert int(status.item()) & 1
    # only rows of the table's own pages were written
    own = cache.table.unique().long()
    other = [i for i in range(cache.pages) if i not in own.tolist()]
    for x, y in zip(cache.pool(), before):
        assert torch.equal(x[:, other].float(), y[:, other].float())


def test_a_prompt_written_by_tokens_equals_one_written_at_once(cuda_device):
    # the scales agree, and codes differ at most where a value was rounded under a
    # smaller scale first: by one step of e4m3's smallest numbers
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(2)
    n, D = 40, 64
    k, v = rand((1, n, 2, D), g, dev), rand((1, n, 2, D), g, dev)
    k *= torch.linspace(0.01, 8, n, device=dev)[None, :, None, None].to(torch.bfloat16)
    s, a = i32([cmr.TEXT_ONLY_START], dev), i32([0], dev)
    one = Cache(dev, [1], D=D, seed=5)
    many = Cache(dev, [1], D=D, seed=5)
    pkg.rotate_qk_kv8(None, k, v, s, a, *one.pool(), one.table, cu_seqlens=i32([0, n], dev))
    for t in range(n):
        pkg.rotate_qk_kv8(None, k[:, t:t + 1].contiguous(), v[:, t:t + 1].contiguous(), s, a,
                          *many.pool(), many.table, pos_offset=i32([t], dev))
    page = int(one.table[0, 0])
    assert torch.equal(one.ks[:, page], many.ks[:, page])
    x, y = one.k[:, page, :, :n].double(), many.k[:, page, :, :n].double()
    # halving rounds each time only below 2^-6, by half a step of 2^-9; ten doublings of the
    # scale add at most twice half a step
    assert float((x - y).abs().max()) <= 2.0 ** -9
    assert torch.equal(x[x.abs() >= 2.0 ** -6], y[x.abs() >= 2.0 ** -6])


def test_on_another_stream_and_captured(cuda_device):
    dev = cuda_device
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(dev, [30, 40], [0, 9], stream=side)
    # a decode step captured once and replayed at moving positions
    g = torch.Generator(device=dev).manual_seed(3)
    B, D = 3, 64
    q, k, v = rand((2, B, 4, D), g, dev), rand((2, B, 2, D), g, dev), rand((2, B, 2, D), g, dev)
    q0 = q.clone()
    s, a = i32([cmr.TEXT_ONLY_START] * B, dev), i32([0] * B, dev)
    caches = [Cache(dev, [2] * B, 2, 2, D, seed=7) for _ in range(2)]
    off = i32([5, 63, 64], dev)
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pkg.rotate_qk_kv8(q, k, v, s, a, *caches[0].pool(), caches[0].table, pos_offset=off)
    for step in range(3):
        q.copy_(q0)
        graph.replay()
        pkg.rotate_qk_kv8(None, k, v, s, a, *caches[1].pool(), caches[1].table, pos_offset=off)
        off += 1
    torch.cuda.synchronize()
    for x, y in zip(caches[0].pool(), caches[1].pool()):
        assert torch.equal(x.float(), y.float())


def test_refusals(cuda_device):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(4)
    c = Cache(dev, [2, 2], D=64)
    q, k = rand((1, 2, 4, 64), g, dev), rand((1, 2, 2, 64), g, dev)
    s, a = i32([cmr.TEXT_ONLY_START] * 2, dev), i32([0, 0], dev)
    ok = lambda **kw: pkg.rotate_qk_kv8(**{**dict(
        q=q, k=k, v=k, start=s, amount=a, k_pages=c.k, v_pages=c.v, k_scales=c.ks, v_scales=c.vs,
        page_table=c.table, pos_offset=i32([0, 0], dev)), **kw})
    ok()
    for kw, err in [(dict(v=k[:, :, :1].contiguous()), ValueError), (dict(q=q.float()), TypeError),
                    (dict(k_pages=c.k.view(torch.uint8)), TypeError),
                    (dict(v_pages=c.v[:, :1].contiguous()), ValueError),
                    (dict(k_scales=c.ks.double()), TypeError), (dict(start=s[:1]), ValueError),
                    (dict(page_table=c.table[0]), ValueError),
                    (dict(page_table=c.table.t()), ValueError),
                    (dict(slot=i32([0], dev)), ValueError),
                    (dict(cu_seqlens=i32([0, 1, 1, 2], dev)), ValueError),
                    (dict(pos_offset=i32([0], dev)), ValueError), (dict(rot_dim=128), pkg.Kv8Error),
                    (dict(theta=-1.0), pkg.Kv8Error), (dict(sections=(32, 1, 0)), pkg.Kv8Error),
                    (dict(k=k.cpu()), ValueError), (dict(k=k[..., ::2]), ValueError)]:
        with pytest.raises(err):
            ok(**kw)
    cpu = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ok(device_status=cpu)
