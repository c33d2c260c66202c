"""GPU checks of the attention over the paged 8-bit cache where one token's weight is far above all
others' and its value is zero, so that the result is a sum of many small weights."""
import math

import numpy as np
import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from tests.kv8_model import Cache, assert_within, i32

pytestmark = pytest.mark.gpu

# The weights of each kernel in its products, relative to the row's largest: rounded by `half`
# of a weight's own size at most, or by `floor` where that is more.
#   decode: f16 (half a step 2^-11 of the number, or half of 2^-24), the largest weight at 2^13 or more
#   prompts: f16, then three terms of e5m2 (half a step 2^-9 together, or half of 2^-16), the
#            largest at 2^9 or more
ROWS = dict(half=2.0 ** -11, floor=2.0 ** -25 / 2 ** 13)
TILES = dict(half=2.0 ** -9 + 2.0 ** -11, floor=(2.0 ** -17 + 2.0 ** -25) / 2 ** 9)


def model(q, c, spans, scale, half, floor):
    """(out, tolerance) in 64 bits of causal attention over keys and values under scales of 1.

    The tolerance counts: the result's rounding to bf16 (2^-8 |o|); the weights' as above; the scores'
    (q by 2^-10 of s, max |q| > 224 s, in the prompt kernel; fp32 sums over D dims; exponents up to 64
    in fp32 and ex2's last two bits, together under 2^-17 of a weight); and the fp32 sums, 16 tokens
    at a time, by a last bit of the accumulator and one of the product at each.  What changes a weight
    enters twice, by it and by the sum of weights."""
    L, N, hq, D = q.shape
    G = hq // c.hk
    out = torch.zeros_like(q, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b, (lo, hi, off) in enumerate(spans):
        n = off + hi - lo
        at = torch.arange(off, n, device=q.device)
        unseen = torch.arange(n, device=q.device)[None] > at[:, None]
        for h in range(c.hk):
            k, v = (c.values(w, 0, b, h, n) for w in "kv")
            for g in range(G):
                x = q[0, lo:hi, h * G + g].double()
                s = (x @ k.T * scale).masked_fill(unseen, -math.inf)
                u = torch.exp(s - s.amax(-1, keepdim=True))
                sum_u = u.sum(-1, keepdim=True)
                o = (u @ v) / sum_u
                off_q = 2.0 ** -10 / 224 * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)
                off_s = D * 2.0 ** -23 * (x.abs() @ k.abs().T)
                change = 2 * abs(scale) * (off_q + off_s) + 2.0 ** -17
                lost = torch.minimum(u, torch.full_like(u, floor)) + u * (half + 2 * change)
                mean_change = ((u * change).sum(-1, keepdim=True) / sum_u)
                out[0, lo:hi, h * G + g] = o
                tol[0, lo:hi, h * G + g] = (lost @ v.abs()) / sum_u + o.abs() * (
                    2.0 ** -8 + 2 * mean_change + n / 16 * 2.0 ** -22) + 1e-30
    return out, tol


def check(dev, lens, offs, strong, margin, kernel, sizes, D=64, hq=8, hk=2, P=64, varied=False,
          step=False):
    g = torch.Generator(device=dev).manual_seed(int(margin * 10) + D)
    cu = np.concatenate([[0], np.cumsum(lens)])
    spans = [(int(cu[b]), int(cu[b + 1]), int(offs[b])) for b in range(len(lens))]
    c = Cache(dev, [-(-(o + n) // P) for o, n in zip(offs, lens)], 1, hk, D, P)
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)
    k, v = c.k.view(torch.uint8), c.v.view(torch.uint8)
    k.zero_()
    if varied:                                       # +-2^-6 in all dims but the first
        k[..., 1:] = 0x08 + 0x80 * torch.randint(0, 2, k[..., 1:].shape, generator=g, device=dev,
                                                 dtype=torch.uint8)
    v.copy_(torch.randint(0x38, 0x40, v.shape, generator=g, device=dev, dtype=torch.uint8))  # 1 .. 2
    for b in range(len(lens)):
        page, row = c.table[b, strong[b] // P].long(), strong[b] % P
        k[:, page, :, row] = 0
        k[:, page, :, row, 0] = 0x58                 # 16
        v[:, page, :, row] = 0
    q = torch.randn((1, sum(lens), hq, D), generator=g, device=dev).to(torch.bfloat16)
    q[..., 0] = 1.0
    scale = margin / 16                              # the strong token's score is the margin
    out = pkg.attend_kv8(q, *c.pool(), c.table, cu_seqlens=None if step else i32(cu, dev),
                         pos_offset=i32(offs, dev), scale=scale)
    assert pkg.last_attend_kernel() == kernel
    want, tol = model(q, c, spans, scale, **sizes)
    assert (want >= 0).all() and (want > 0).any()    # a row that sees the strong token alone: 0
    assert_within(out, want, tol)


MARGINS = [6, 10, 13, 14, 15, 16, 17, 17.4, 18, 20]


@pytest.mark.parametrize("varied", [False, True])
@pytest.mark.parametrize("margin", MARGINS)
def test_steps_behind_one_strong_token(cuda_device, margin, varied):
    check(cuda_device, [1, 1, 1], [49999, 700, 3000], [0, 100, 2999], margin, "attend_rows_kernel",
          ROWS, varied=varied, step=True)
    check(cuda_device, [1], [250000], [3], margin, "attend_rows_kernel", ROWS, D=128, hq=4, hk=1,
          P=128, varied=varied, step=True)


@pytest.mark.parametrize("margin", MARGINS)
def test_short_chunks_behind_one_strong_token(cuda_device, margin):
    check(cuda_device, [4, 3], [20000, 900], [0, 899], margin, "attend_rows_kernel", ROWS, D=256)


@pytest.mark.parametrize("varied", [False, True])
@pytest.mark.parametrize("margin", MARGINS)
def test_prompts_behind_one_strong_token(cuda_device, margin, varied):
    check(cuda_device, [1500], [0], [0], margin, "attend_tiles_kernel", TILES, hq=2, hk=1,
          varied=varied)
    check(cuda_device, [40, 130], [30000, 2000], [0, 1500], margin, "attend_tiles_kernel", TILES,
          D=256, varied=varied)
