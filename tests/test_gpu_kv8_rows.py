"""GPU checks of what the page calls take for a row's pages: the entries up to the first negative
one, whatever stands behind it, with page ids outside the pool flagged and not followed."""
import pytest
import torch

import vlm_decoder_positional_b200 as pkg
from tests.kv8_model import Cache, i32

pytestmark = pytest.mark.gpu
P, RANGE = 64, pkg.CMR_DEVICE_CACHE_RANGE


def extend(dev, rows, refs, slots, lens):
    """(table, counts, status) after the call, as lists."""
    t, r = i32(rows, dev), i32(refs, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.kv8_extend(t, r, i32(slots, dev), i32(lens, dev), P, device_status=status)
    return t.tolist(), r.tolist(), int(status.item())


def test_extend_counts_up_to_the_first_hole(cuda_device):
    refs = [0, 1, 1, 0, 0, 1, 0, 1]
    # row 0 has one page: two more are given, and 7 is not one of them
    t, r, st = extend(cuda_device, [[5, -1, 7, -1], [1, 2, -1, -1]], refs, [0], [3 * P])
    assert (t, st) == ([[5, 0, 3, -1], [1, 2, -1, -1]], 0) and r == [1, 1, 1, 1, 0, 1, 0, 1]
    # one is given, and the row ends behind it
    t, r, st = extend(cuda_device, [[5, -1, 7, 2], [1, 2, -1, -1]], refs, [1, 0], [2 * P, P + 1])
    assert (t, st) == ([[5, 0, -1, 2], [1, 2, -1, -1]], 0)
    # none is needed, nothing changes
    t, r, st = extend(cuda_device, [[5, -1, 7, 9]], refs, [0], [P])
    assert (t, r, st) == ([[5, -1, 7, 9]], refs, 0)


def test_extend_flags_page_ids_outside_the_pool(cuda_device):
    refs = [0, 1, 1, 0, 0, 1, 0, 1]
    for bad in (8, 2 ** 31 - 1):
        t, r, st = extend(cuda_device, [[5, bad, -1, -1], [1, -1, bad, -1]], refs, [0], [3 * P])
        assert (t, st) == ([[5, bad, 0, -1], [1, -1, bad, -1]], RANGE)
        # behind the end it is not one of the row's
        assert extend(cuda_device, [[5, -1, bad, -1]], refs, [0], [P])[2] == 0
        assert extend(cuda_device, [[5, bad, -1, -1], [1, -1, bad, -1]], refs, [1], [P])[2] == 0


@pytest.mark.parametrize("n", [1, 2, 5, 16, 31, 32, 33, 70])
@pytest.mark.parametrize("cols", [1, 31, 33, 256, 257, 5000])
def test_extend_of_long_rows(cuda_device, n, cols):
    # rows of all lengths: empty, full, ending at the borders of what is read at once
    dev = cuda_device
    ends = [c for c in (0, 1, 31, 32, 255, 256, 257, 511, 512, 2047, 4096, cols - 1, cols)
            if 0 <= c <= cols]
    held = [ends[i % len(ends)] for i in range(n)]
    want = [min(cols, h + i % 3) for i, h in enumerate(held)]
    total = sum(held)
    refs = torch.zeros(total + 2 * n + 3, dtype=torch.int32, device=dev)
    refs[:total] = 1
    t = torch.full((n, cols), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, h in enumerate(held):
        t[i, :h] = torch.arange(at, at + h, dtype=torch.int32, device=dev)
        at += h
        if i % 2 and h + 2 < cols:
            t[i, h + 2:] = 1 << 30                   # nothing to the row
    expected = t.clone()
    for i, (h, w) in enumerate(zip(held, want)):
        expected[i, h:w] = torch.arange(at, at + w - h, dtype=torch.int32, device=dev)
        at += w - h
        if w > h and w < cols:
            expected[i, w] = -1
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.kv8_extend(t, refs, i32(list(range(n)), dev), i32([w * P for w in want], dev), P,
                   device_status=status)
    assert torch.equal(t, expected) and int(status.item()) == 0
    assert (refs[:at] == 1).all() and not refs[at:].any()


def test_a_forked_row_ends_behind_its_pages(cuda_device):
    dev = cuda_device
    c = Cache(dev, [], 1, 1, 64, P, spare=8)
    t, refs = i32([[5, 1, -1, -1], [-1, 7, 6, 2], [-1, 3, 3, 3]], dev), i32([0, 1, 0, 0, 0, 1, 0, 0], dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.kv8_fork(*c.pool(), t, refs, i32([0, 0], dev), i32([1, 2], dev), i32([P, P + 3], dev),
                 device_status=status)
    assert t.tolist() == [[5, 1, -1, -1], [5, -1, 6, 2], [5, 0, -1, 3]]
    assert refs.tolist() == [1, 1, 0, 0, 0, 3, 0, 0] and int(status.item()) == 0


def compact(dev, rows, refs):
    """(table, counts, status) after the call, as lists."""
    c = Cache(dev, [], 2, 1, 64, P, spare=len(refs))
    t, r = i32(rows, dev), i32(refs, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.kv8_compact(*c.pool(), t, r, device_status=status)
    return t.tolist(), r.tolist(), int(status.item())


def test_compact_flags_what_is_no_page_in_use(cuda_device):
    # pages 3 and 5 go to 0 and 2; an id outside the pool, and one of a free page, stay
    refs = [0, 1, 0, 1, 0, 1, 0, 0]
    rows = [[1, 5, -1, -1], [3, -1, -1, -1]]
    assert compact(cuda_device, rows, refs) == ([[1, 2, -1, -1], [0, -1, -1, -1]],
                                                [1, 1, 1, 0, 0, 0, 0, 0], 0)
    for bad in (8, 2 ** 31 - 1, 7):
        t, r, st = compact(cuda_device, [[1, bad, 5, -1], [3, -1, -1, -1]], refs)
        assert (t, st) == ([[1, bad, 2, -1], [0, -1, -1, -1]], RANGE)


def test_compact_looks_at_the_table_where_nothing_moves(cuda_device):
    refs = [1, 1, 1, 0, 0]
    assert compact(cuda_device, [[0, 1, -1], [2, -1, -1]], refs)[2] == 0
    for bad in (5, 4):
        t, r, st = compact(cuda_device, [[0, 1, -1], [2, bad, -1]], refs)
        assert (t, r, st) == ([[0, 1, -1], [2, bad, -1]], refs, RANGE)


def test_compact_leaves_what_stands_behind_a_row(cuda_device):
    refs = [0, 1, 0, 1, 0, 1, 0, 0]
    t, r, st = compact(cuda_device, [[1, -1, 9, 7], [-1, 6, -1, 4], [3, 5, -2, 99]], refs)
    assert (t, st) == ([[1, -1, 9, 7], [-1, 6, -1, 4], [0, 2, -2, 99]], 0)
