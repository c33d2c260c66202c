"""The order of things in the kernels of libcmr_kv8, read from their sources: all are launched
programmatically, so that a CTA may be placed while the kernel ahead of it still runs, and what it
does before its wait has to hold whatever kernel that is."""
import glob
import os
import re

import pytest

from vlm_decoder_positional_b200 import build as libbuild


def kernels():
    """(name, body) of every kernel."""
    for path in sorted(glob.glob(os.path.join(libbuild.KV8_DIR, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
            at = text.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield m.group(1), text[at:end]


KERNELS = dict(kernels())


def test_all_kernels_are_looked_at():
    assert {"attend_rows_kernel", "attend_join_kernel", "attend_join_runs_kernel",
            "attend_tiles_kernel", "attend_tiles_join_kernel", "write_pages_kernel",
            "write_step_kernel", "extend_kernel", "fork_plan_kernel", "fork_copy_kernel",
            "free_kernel", "compact_plan_kernel", "compact_move_kernel"} == set(KERNELS)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_no_tensor_memory_is_held_before_the_wait(name):
    # the kernel ahead may need the columns to end: a CTA that had them and waited for that
    # kernel would wait for good, and so would that kernel's allocation
    before, wait, _ = KERNELS[name].partition("pdl::wait();")
    assert wait and "alloc" not in before


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_no_memory_is_read_before_the_wait(name):
    # no load, none by a function that reads the call's tensors, and no signal to the kernel behind
    before = KERNELS[name].partition("pdl::wait();")[0]
    assert not re.search(r"__ld\w*\(|\bfind_\w+|seq_range|page_id|table_row|planes_of|atomic\w+\(|"
                         r"prefetch\.global|load_\dd|launch_dependents", before)
