"""What is measured of the paged 8-bit KV cache: the rotation that writes it, the attention that
reads it, and the upkeep of its pages.

The cache is a pool of pages of P tokens: codes in e4m3, k_pages / v_pages [L, pages, hk, P, D], and
one scale, a power of two, for each page and head, k_scales / v_scales [L, pages, hk].  A row of
page_table [rows, max_pages] lists the pages of one sequence in order (-1: none); page_refs [pages]
counts the rows that hold each page.  The decoder's own shape is 6 full-attention layers, 8 query and
2 key/value heads of 256 dims, of which the first 64 are rotated with sections [11, 11, 10] and theta
1e7.
"""
import math
import random

import torch

own = False

THETA = 1e7
SECTIONS = (11, 11, 10)
ROT = 64
TEXT_ONLY = 1 << 30
IMAGE_TOKENS = 67  # <image>, 64 rows, </image> and the line end
E4M3_TOP = 448.0


# ----------------------------------------------------------------------------- cases

def listed():
    shape = {"hq": 8, "hk": 2, "dim": 256, "page": 64}
    return [
        # one user's next token: all six layers written by one call
        dict(shape, name="write_step_1", op="write", layers=6, batch=1, ctx_lo=700, ctx_hi=700,
             new_lo=1, new_hi=1, sizes=1),
        # a full decode batch of users at different depths
        dict(shape, name="write_step_256", op="write", layers=6, batch=256, ctx_lo=64, ctx_hi=2048,
             new_lo=1, new_hi=1, sizes=2),
        # later turns of a chat: ragged chunks behind ragged contexts, pages that begin half full
        dict(shape, name="write_chunk_12", op="write", layers=6, batch=12, ctx_lo=1, ctx_hi=3000,
             new_lo=1, new_hi=900, sizes=3),
        # prompts of the engine's full context, written from the start
        dict(shape, name="write_prompt_8x4096", op="write", layers=6, batch=8, ctx_lo=0, ctx_hi=0,
             new_lo=4096, new_hi=4096, sizes=4),
        # one user's next token in one layer
        dict(shape, name="attend_step_1x700", op="attend", layers=1, batch=1, ctx_lo=700,
             ctx_hi=700, new_lo=1, new_hi=1, sizes=5),
        # a decode batch at the engine's full context
        dict(shape, name="attend_step_64x4095", op="attend", layers=1, batch=64, ctx_lo=4095,
             ctx_hi=4095, new_lo=1, new_hi=1, sizes=6),
        # a decode batch of very different depths
        dict(shape, name="attend_step_128_mixed", op="attend", layers=1, batch=128, ctx_lo=1,
             ctx_hi=8191, new_lo=1, new_hi=1, sizes=7),
        # one long document, one token at a time
        dict(shape, name="attend_step_1x262143", op="attend", layers=1, batch=1, ctx_lo=262143,
             ctx_hi=262143, new_lo=1, new_hi=1, sizes=8),
        # ragged chunks behind ragged contexts
        dict(shape, name="attend_chunk_8", op="attend", layers=1, batch=8, ctx_lo=1, ctx_hi=6000,
             new_lo=1, new_hi=700, sizes=9),
        # whole prompts
        dict(shape, name="attend_prompt_4x8192", op="attend", layers=1, batch=4, ctx_lo=0, ctx_hi=0,
             new_lo=8192, new_hi=8192, sizes=10),
        # a search step: the old branches are freed, each of 4 parents is forked into 8 new ones
        dict(shape, name="pages_fork_4x8", op="fork", layers=6, batch=4, children=8, ctx_lo=500,
             ctx_hi=3500, sizes=11),
        # a quarter of the users leave, the pool is compacted, as many new ones come
        dict(shape, name="pages_compact_64", op="compact", layers=6, batch=64, ctx_lo=2048,
             ctx_hi=2048, sizes=12),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = rng.choice([(8, 2), (8, 2), (8, 8), (4, 1), (6, 2), (16, 2)])
    case = {"hq": heads[0], "hk": heads[1], "dim": rng.choice([64, 128, 256, 256]),
            "page": rng.choice([16, 32, 64, 64, 128]), "sizes": rng.randrange(1 << 30)}
    kind = rng.choice(["write_step", "write_chunk", "attend_step", "attend_long", "attend_chunk",
                       "attend_prompt", "fork", "compact"])
    if kind.startswith("write"):
        case.update(op="write", layers=rng.choice([1, 6]))
        if kind == "write_step":
            case.update(batch=_spread(rng, 1, 256), ctx_lo=1, ctx_hi=_spread(rng, 64, 2048),
                        new_lo=1, new_hi=1)
        else:
            case.update(batch=_spread(rng, 1, 16), ctx_lo=rng.choice([0, 1]),
                        ctx_hi=rng.choice([1, _spread(rng, 16, 2048)]), new_lo=1,
                        new_hi=_spread(rng, 8, 2048))
    elif kind.startswith("attend"):
        case.update(op="attend", layers=1)
        if kind == "attend_step":
            case.update(batch=_spread(rng, 2, 128), ctx_lo=rng.choice([0, 1, 100]),
                        ctx_hi=_spread(rng, 128, 8191), new_lo=1, new_hi=1,
                        layers=rng.choice([1, 1, 2]))
        elif kind == "attend_long":
            ctx = _spread(rng, 8192, 200_000)
            case.update(batch=1, ctx_lo=ctx, ctx_hi=ctx, new_lo=1, new_hi=1)
        elif kind == "attend_chunk":
            case.update(batch=_spread(rng, 1, 12), ctx_lo=1, ctx_hi=_spread(rng, 16, 6000),
                        new_lo=1, new_hi=_spread(rng, 2, 900))
        else:
            new = _spread(rng, 256, 6000)
            case.update(batch=rng.choice([1, 2, 4]), ctx_lo=0, ctx_hi=0,
                        new_lo=rng.choice([1, new]), new_hi=new)
    elif kind == "fork":
        case.update(op="fork", layers=rng.choice([1, 6]), batch=_spread(rng, 1, 8),
                    children=_spread(rng, 1, 16), ctx_lo=1, ctx_hi=_spread(rng, 64, 4096))
    else:
        ctx = _spread(rng, 128, 2048)
        case.update(op="compact", layers=rng.choice([1, 6]), batch=rng.choice([8, 16, 32, 64]),
                    ctx_lo=rng.choice([1, ctx]), ctx_hi=ctx)
    return case


def _lens(case):
    """(tokens before the call, new tokens) of every sequence: by the case alone."""
    r = random.Random(case["sizes"])

    def one(lo, hi):
        if lo == hi:
            return lo
        return _spread(r, lo, hi) if lo > 0 else r.choice([0, _spread(r, 1, hi)])

    n = case["batch"]
    ctx = [one(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [one(case["new_lo"], case["new_hi"]) for _ in range(n)] if "new_lo" in case else [0] * n
    return ctx, new


def work(case):
    L, hq, hk, D, P = (case[k] for k in ("layers", "hq", "hk", "dim", "page"))
    ctx, new = _lens(case)
    N = sum(new)
    if case["op"] == "write":
        # Q's rotated dims read and written, K and V read, their codes written, the scales of
        # the touched pages, the state and the table
        pages = sum((c + n - 1) // P - c // P + 1 for c, n in zip(ctx, new) if n)
        moved = N * (hq * ROT * 2 * 2 + hk * D * 2 * (2 + 1)) + pages * (hk * 2 * 4)
        return {"bytes": L * moved + pages * 4 + len(ctx) * 16,
                "flops": L * N * (hq + hk) * ROT * 3}
    if case["op"] == "attend":
        seen = sum(c + n for c, n in zip(ctx, new))
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        pages = sum(-(-(c + n) // P) for c, n in zip(ctx, new))
        return {"bytes": L * (seen * hk * D * 2 + pages * hk * 2 * 4 + N * hq * D * 2 * 2)
                + pages * 4 + len(ctx) * 8, "flops": L * 4 * pairs * hq * D}
    if case["op"] == "fork":
        # the rows of each branch's own last page, read and written, and the shared pages' entries
        rows = case["children"] * sum(c % P for c in ctx)
        pages = case["children"] * sum(-(-c // P) for c in ctx)
        return {"bytes": L * rows * hk * D * 2 * 2 + pages * 4 * 6 + L * case["children"]
                * len(ctx) * hk * 16, "flops": 0}
    # compact: the pages of the sequences that left are refilled from the pool's end
    gone = case["batch"] // 4
    pages = [-(-c // P) for c in ctx]
    moved = min(sum(pages[:gone]), sum(pages[gone:2 * gone]))
    page = L * hk * (P * D + 4) * 2
    return {"bytes": 2 * moved * page + sum(pages) * 4 * 3, "flops": 0}


# ----------------------------------------------------------------------------- inputs

def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, within 2^-60 .. 2^60."""
    m, e = torch.frexp(amax)                      # amax = m * 2^e, 0.5 <= m < 1, 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-60, 60)
    e = torch.where(amax > 0, e, torch.full_like(e, -60))
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(x):
    return x.clamp(-E4M3_TOP, E4M3_TOP).to(torch.float8_e4m3fn)


def _pool(case, pages, g, dev):
    """A pool whose pages hold keys with a few strong channels, as the rotated dims have, and values."""
    L, hk, D, P = case["layers"], case["hk"], case["dim"], case["page"]
    channel = 1 + 4 * (torch.rand(D, generator=g, device=dev) > 0.95).float()
    made = []
    for weight in (channel, torch.ones(D, device=dev)):
        codes = torch.empty((L, pages, hk, P, D), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((L, pages, hk), dtype=torch.float32, device=dev)
        step = max(1, (1 << 25) // (hk * P * D))
        for lay in range(L):
            for lo in range(0, pages, step):
                hi = min(pages, lo + step)
                x = torch.randn((hi - lo, hk, P, D), generator=g, device=dev) * weight
                s = _pow2_scale(x.abs().amax(dim=(2, 3)))
                codes[lay, lo:hi] = _codes(x / s[..., None, None])
                scales[lay, lo:hi] = s
        made += [codes, scales]
    return {"k_pages": made[0], "k_scales": made[1], "v_pages": made[2], "v_scales": made[3]}


def _table(rows, max_pages, counts, order, dev):
    """page_table with counts[r] pages in row r, taken from `order` one after another."""
    t = torch.full((rows, max_pages), -1, dtype=torch.int32)
    at = 0
    for r, c in enumerate(counts):
        t[r, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    return t.to(dev)


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    L, hq, hk, D, P = (case[k] for k in ("layers", "hq", "hk", "dim", "page"))
    ctx, new = _lens(case)
    B = len(ctx)
    st = {"op": case["op"], "page": P}
    if case["op"] in ("write", "attend"):
        N = sum(new)
        counts = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        pages = sum(counts) + 3
        order = list(range(pages))
        r.shuffle(order)
        st.update(_pool(case, pages, g, dev))
        st["page_table"] = _table(B, max(counts) + 1, counts, order, dev)
        st["pos_offset"] = _i32(ctx, dev)
        step = all(n == 1 for n in new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu_seqlens"] = None if step else _i32(cu, dev)
        st["max_new"], st["max_seen"] = max(new), max(c + n for c, n in zip(ctx, new))
        channel = 1 + 4 * (torch.rand(D, generator=g, device=dev) > 0.95).float()
        st["q"] = torch.randn((L, N, hq, D), generator=g, device=dev).to(torch.bfloat16)
        if case["op"] == "write":
            st["k"] = (torch.randn((L, N, hk, D), generator=g, device=dev)
                       * channel).to(torch.bfloat16)
            st["v"] = torch.randn((L, N, hk, D), generator=g, device=dev).to(torch.bfloat16)
            # half of the sequences hold an image somewhere in what they will have been given
            start, amount = [], []
            for c, n in zip(ctx, new):
                image = r.random() < 0.5 and c + n > IMAGE_TOKENS
                o = r.randrange(c + n - IMAGE_TOKENS) if image else 0
                start.append(o + IMAGE_TOKENS if image else TEXT_ONLY)
                amount.append(58 if image else 0)
            st["start"], st["amount"] = _i32(start, dev), _i32(amount, dev)
        else:
            st["scale"] = 1 / math.sqrt(D)
        return st
    counts = [-(-c // P) for c in ctx]
    if case["op"] == "fork":
        F = B * case["children"]
        pages = sum(counts) + F + 5
        order = list(range(pages))
        r.shuffle(order)
        st.update(_pool(case, pages, g, dev))
        st["page_table"] = _table(B + F, max(counts) + 1, counts, order, dev)
        st["src"] = _i32([i % B for i in range(F)], dev)
        dst = list(range(B, B + F))
        r.shuffle(dst)
        st["dst"] = _i32(dst, dev)
        st["lens"] = _i32([ctx[i % B] for i in range(F)], dev)
    else:
        gone = B // 4
        pages = sum(counts) + sum(counts) // 8 + 1
        # the sequences that came last, the first quarter, hold the pool's end; the second quarter
        # leaves next: its pages lie among those of the rest
        rest = list(range(sum(counts[gone:])))
        r.shuffle(rest)
        order = list(range(sum(counts[gone:]), sum(counts))) + rest
        st.update(_pool(case, pages, g, dev))
        st["page_table"] = _table(B, max(counts) + 1, counts, order, dev)
        st["turn"] = [(_i32(list(range(gone, 2 * gone)), dev), _i32(ctx[gone:2 * gone], dev)),
                      (_i32(list(range(gone)), dev), _i32(ctx[:gone], dev))]
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[torch.tensor(order[:sum(counts)], dtype=torch.int64)] = 1
    st["page_refs"] = refs.to(dev)
    return st


# ----------------------------------------------------------------------------- plain forms

def _tokens(st, n):
    """(sequence, index within its new tokens) of each of n packed tokens."""
    t = torch.arange(n, device=st["q"].device)
    if st["cu_seqlens"] is None:
        return t, torch.zeros_like(t)
    cu = st["cu_seqlens"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _planes(p, start, amount):
    """The canvas table's three planes at absolute indices p."""
    o = start - amount - 9
    d = p - o
    k = d - 1
    row, col = o + k.div(8, rounding_mode="floor"), o + k.remainder(8)
    h = torch.where(d < 0, p, torch.where(d == 0, o - 1, torch.where(
        d <= 64, row, torch.where(d == 65, o + 8, o))))
    w = torch.where(d < 0, p, torch.where(d == 0, o - 1, torch.where(
        d <= 64, col, torch.where(d == 65, o + 8, o))))
    t = torch.where(d < 0, p, o)
    after = p >= start
    return torch.stack([torch.where(after, p - amount, x) for x in (t, h, w)])


def _rotated(x, cos, sin):
    """Head rows [L, N, H, D] in 32 bits, their first ROT dims turned by the tokens' angles."""
    x = x.float()
    F = ROT // 2
    a, b = x[..., :F], x[..., F:ROT]
    c, s = cos[None, :, None, :], sin[None, :, None, :]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., ROT:]], dim=-1)


def _plain_write(st):
    q, k, v = st["q"], st["k"], st["v"]
    L, n, hk, D = k.shape
    P = st["page"]
    b, i = _tokens(st, n)
    off = st["pos_offset"].long()
    p = off[b] + i
    planes = _planes(p, st["start"].long()[b], st["amount"].long()[b])
    j = torch.arange(ROT // 2, device=q.device)
    plane = torch.where((j % 3 == 1) & (j < 3 * SECTIONS[1]), 1,
                        torch.where((j % 3 == 2) & (j < 3 * SECTIONS[2]), 2, 0))
    angle = planes[plane].T.double() * THETA ** (-2.0 * j.double() / ROT)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q.copy_(_rotated(q, cos, sin))
    page = st["page_table"].long()[b, p // P]
    row = p % P
    first = st["page_table"].long().gather(1, (off // P)[:, None])[:, 0].clamp(min=0)
    kept = torch.arange(P, device=q.device)[None, :] < (off % P)[:, None]    # [B, P]
    # the cache holds the rotated key as the rotation gives it, in bf16: a scale then never hangs on
    # the last bit of a 32-bit angle
    new_rows = ((_rotated(k, cos, sin).to(torch.bfloat16).float(), "k"), (v.float(), "v"))
    fresh = torch.zeros(st["k_scales"].shape[1], dtype=torch.bool, device=q.device)
    fresh[page[row == 0]] = True
    touched = torch.zeros_like(fresh)
    touched[page] = True

    def put(x, which):
        codes, scales = st[which + "_pages"], st[which + "_scales"]
        amax = torch.zeros_like(scales).index_reduce_(1, page, x.abs().amax(dim=-1), "amax")
        s = _pow2_scale(amax)
        s = torch.where(fresh[None, :, None], s, torch.maximum(s, scales))
        s = torch.where(touched[None, :, None], s, scales)
        # rows that a page held before, under the page's new scale
        held = codes.view(torch.uint8)[:, first].view(torch.float8_e4m3fn)
        again = _codes(held.float() * (scales / s)[:, first][..., None, None])
        held = torch.where(kept[None, :, None, :, None], again.view(torch.uint8),
                           held.view(torch.uint8))
        codes.view(torch.uint8)[:, first] = held
        new = _codes(x / s[:, page][..., None])
        codes.view(torch.uint8)[:, page, :, row] = new.view(torch.uint8).transpose(0, 1)
        scales.copy_(s)

    put(*new_rows[0])
    put(*new_rows[1])


def _plain_attend(st):
    q = st["q"]
    L, n, hq, D = q.shape
    hk, P = st["k_pages"].shape[2], st["page"]
    G = hq // hk
    B = st["pos_offset"].numel()
    m = st["max_new"]
    M = -(-st["max_seen"] // P)
    b, i = _tokens(st, n)
    pages = st["page_table"][:, :M].long().clamp(min=0)

    def gathered(which):
        x = st[which + "_pages"].view(torch.uint8)[:, pages].view(torch.float8_e4m3fn).float()
        x = x * st[which + "_scales"][:, pages][..., None, None]              # [L, B, M, hk, P, D]
        return x.permute(0, 1, 3, 2, 4, 5).reshape(L, B, hk, M * P, D)

    rows = torch.zeros((L, B, m, hq, D), device=q.device)
    rows[:, b, i] = q.float()
    rows = rows.view(L, B, m, hk, G, D).permute(0, 1, 3, 2, 4, 5).reshape(L, B, hk, m * G, D)
    s = torch.matmul(rows, gathered("k").transpose(-1, -2)) * st["scale"]
    at = st["pos_offset"].long()[:, None] + torch.arange(m, device=q.device)  # [B, m]
    seen = torch.arange(M * P, device=q.device)[None, None] <= at[..., None]
    s.masked_fill_(~seen.repeat_interleave(G, dim=1)[None, :, None], float("-inf"))
    s -= s.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    s.exp_()
    o = torch.matmul(s, gathered("v")) / s.sum(dim=-1, keepdim=True)
    o = o.view(L, B, hk, m, G, D).permute(0, 1, 3, 2, 4, 5).reshape(L, B, m, hq, D)
    return o[:, b, i].to(torch.bfloat16)


def _plain_free(st, slots):
    rows = st["page_table"][slots.long()]
    held = rows[rows >= 0].long()
    st["page_refs"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    st["page_table"][slots.long()] = -1


def _lowest_free(st, count):
    return torch.nonzero(st["page_refs"] == 0)[:count, 0]


def _plain_extend(st, slots, lens):
    table, slots = st["page_table"], slots.long()
    have = (table[slots] >= 0).sum(dim=1)
    need = (-(-lens.long() // st["page"]) - have).clamp(min=0)
    row = torch.repeat_interleave(need)
    free = _lowest_free(st, row.numel())
    place = torch.arange(row.numel(), device=row.device) - (need.cumsum(0) - need)[row]
    table[slots[row], have[row] + place] = free.int()
    st["page_refs"][free] = 1


def _plain_fork(st):
    table, P = st["page_table"], st["page"]
    src, dst, lens = st["src"].long(), st["dst"].long(), st["lens"].long()
    whole, rest = lens // P, lens % P
    col = torch.arange(table.shape[1], device=table.device)[None]
    rows = torch.where(col < whole[:, None], table[src], -1)
    tail = torch.nonzero(rest > 0)[:, 0]
    free = _lowest_free(st, tail.numel())
    shared = rows[rows >= 0].long()
    st["page_refs"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    st["page_refs"][free] = 1
    rows[tail, whole[tail]] = free.int()
    last = table[src[tail], whole[tail]].long()
    table[dst] = rows
    kept = (torch.arange(P, device=table.device)[None] < rest[tail][:, None])[None, :, None, :, None]

    def move(which):
        codes = st[which + "_pages"].view(torch.uint8)
        codes[:, free] = torch.where(kept, codes[:, last], codes[:, free])
        st[which + "_scales"][:, free] = st[which + "_scales"][:, last]

    move("k")
    move("v")


def _plain_compact(st):
    refs, table = st["page_refs"], st["page_table"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    holes = torch.nonzero(~live & (at < count))[:, 0]
    moved = torch.nonzero(live & (at >= count))[:, 0]
    goes = at.clone()
    goes[moved] = holes

    def move(which):
        codes, scales = st[which + "_pages"].view(torch.uint8), st[which + "_scales"]
        codes[:, holes] = codes[:, moved]
        scales[:, holes] = scales[:, moved]

    move("k")
    move("v")
    refs[holes] = refs[moved]
    refs[moved] = 0
    table.copy_(torch.where(table >= 0, goes[table.long().clamp(min=0)].int(), table))


# ----------------------------------------------------------------------------- one pass

def run(state):
    st = state
    pool = ("k_pages", "v_pages", "k_scales", "v_scales")
    if own:
        import vlm_decoder_positional_b200 as cmr
        if st["op"] == "write":
            cmr.rotate_qk_kv8(st["q"], st["k"], st["v"], st["start"], st["amount"],
                              *(st[x] for x in pool), st["page_table"],
                              cu_seqlens=st["cu_seqlens"], pos_offset=st["pos_offset"])
        elif st["op"] == "attend":
            return cmr.attend_kv8(st["q"], *(st[x] for x in pool), st["page_table"],
                                  cu_seqlens=st["cu_seqlens"], pos_offset=st["pos_offset"],
                                  scale=st["scale"])
        elif st["op"] == "fork":
            cmr.kv8_free(st["page_table"], st["page_refs"], st["dst"])
            cmr.kv8_fork(*(st[x] for x in pool), st["page_table"], st["page_refs"], st["src"],
                         st["dst"], st["lens"])
        else:
            slots, lens = st["turn"][0]
            st["turn"].reverse()
            cmr.kv8_free(st["page_table"], st["page_refs"], slots)
            cmr.kv8_compact(*(st[x] for x in pool), st["page_table"], st["page_refs"])
            cmr.kv8_extend(st["page_table"], st["page_refs"], slots, lens, st["page"])
    elif st["op"] == "write":
        _plain_write(st)
    elif st["op"] == "attend":
        return _plain_attend(st)
    elif st["op"] == "fork":
        _plain_free(st, st["dst"])
        _plain_fork(st)
    else:
        slots, lens = st["turn"][0]
        st["turn"].reverse()
        _plain_free(st, slots)
        _plain_compact(st)
        _plain_extend(st, slots, lens)
    if st["op"] == "write":
        # the cache as it is held: e4m3 numbers, and beside them the powers of two they stand with
        return {x: st[x] for x in ("q",) + pool}
    # moved, not computed: the codes byte for byte
    return {"k_pages": st["k_pages"].view(torch.uint8), "v_pages": st["v_pages"].view(torch.uint8),
            "k_scales": st["k_scales"], "v_scales": st["v_scales"],
            "page_table": st["page_table"], "page_refs": st["page_refs"]}


# ----------------------------------------------------------------------------- in 64 bits

def _spans(st):
    n = st["q"].shape[1]
    cu = list(range(n + 1)) if st["cu_seqlens"] is None else st["cu_seqlens"].tolist()
    return list(zip(cu[:-1], cu[1:], st["pos_offset"].tolist()))


def _exact_write(st):
    dev, P, F = st["q"].device, st["page"], ROT // 2
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    starts, amounts = st["start"].tolist(), st["amount"].tolist()
    table = st["page_table"].tolist()
    freq = torch.tensor([THETA ** (-2 * j / ROT) for j in range(F)], dtype=torch.float64, device=dev)
    plane = torch.zeros(F, dtype=torch.int64, device=dev)
    for a in (1, 2):
        for m in range(SECTIONS[a]):
            plane[3 * m + a] = a
    coords = []
    for (lo, hi, off), s, a in zip(_spans(st), starts, amounts):
        o = s - a - 9
        for p in range(off, off + hi - lo):
            if p >= s:
                c = (p - a,) * 3
            elif p < o:
                c = (p,) * 3
            elif p == o:
                c = (o, o - 1, o - 1)
            elif p <= o + 64:
                c = (o, o + (p - o - 1) // 8, o + (p - o - 1) % 8)
            elif p == o + 65:
                c = (o, o + 8, o + 8)
            else:
                c = (o, o, o)
            coords.append(c)
    turn = torch.tensor(coords, dtype=torch.float64, device=dev)[:, plane] * freq
    unit = torch.polar(torch.ones_like(turn), turn)[None, :, None]
    for x in (q, k):
        z = torch.complex(x[..., :F], x[..., F:ROT]) * unit
        x[..., :F], x[..., F:ROT] = z.real, z.imag
    k = k.to(torch.bfloat16).double()             # by definition: the key as the rotation gives it
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        codes, scales = st[name + "_pages"].double(), st[name + "_scales"].double()
        for row, (lo, hi, off) in enumerate(_spans(st)):
            at = off
            while at < off + hi - lo:
                end = min(off + hi - lo, (at // P + 1) * P)
                page, first = table[row][at // P], at % P
                new = x[:, lo + at - off:lo + end - off].transpose(1, 2)      # [L, hk, rows, D]
                need = torch.exp2(torch.ceil(torch.log2(new.abs().amax(dim=(2, 3)) / 448)))
                s = torch.maximum(need, scales[:, page]) if first else need
                codes[:, page, :, :first] *= (scales[:, page] / s)[..., None, None]
                codes[:, page, :, first:first + end - at] = new / s[..., None, None]
                scales[:, page] = s
                at = end
        out[name + "_pages"], out[name + "_scales"] = codes, scales
    return {x: out[x] for x in ("q", "k_pages", "v_pages", "k_scales", "v_scales")}


def _exact_attend(st):
    q = st["q"].double()
    L, n, hq, D = q.shape
    hk, P = st["k_pages"].shape[2], st["page"]
    out = torch.zeros_like(q)
    for row, (lo, hi, off) in enumerate(_spans(st)):
        last = off + hi - lo
        if hi == lo:
            continue
        own_pages = st["page_table"][row, :-(-last // P)].long()
        for lay in range(L):
            for h in range(hk):
                kv = []
                for name in ("k", "v"):
                    c = st[name + "_pages"].view(torch.uint8)[lay, own_pages, h]
                    c = c.view(torch.float8_e4m3fn).double()
                    c = c * st[name + "_scales"][lay, own_pages, h].double()[:, None, None]
                    kv.append(c.reshape(-1, D)[:last])
                for g in range(hq // hk):
                    head = h * (hq // hk) + g
                    s = q[lay, lo:hi, head] @ kv[0].T * st["scale"]
                    s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu(off + 1), -math.inf)
                    out[lay, lo:hi, head] = torch.softmax(s, dim=-1) @ kv[1]
    return out


def exact(case, seed):
    if case["op"] not in ("write", "attend"):
        return None                               # bytes that are moved, and whole numbers
    st = prepare(case, seed)
    return _exact_write(st) if case["op"] == "write" else _exact_attend(st)
