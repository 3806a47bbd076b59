"""What can be seen of the paged-cache kernels without a GPU: that each kernel
launched as a programmatic dependent (scheduled while the kernel before it still
runs) waits for that kernel before it touches global memory, and how a pass is
cut into blocks."""

import os
import re

import pytest

from exact_io_aware_bwd_b200 import binding
from exact_io_aware_bwd_b200.build import CSRC, build

KERNELS = [("fa_append.cuh", "fa_append_kernel"), ("fa_paged.cuh", "fa_paged_kernel"),
           ("fa_paged.cuh", "fa_paged_merge_kernel"), ("fa_prefix.cuh", "fa_prefix_own_kernel")]
# the first thing a kernel may do with global memory, as these kernels write it
TOUCHES = re.compile(r"\bp\.(lens|table|new_lens|part_ml|inv_freq|o|lse)\b|paged_seq\(|paged_item_keys\(|tma_load_|"
                     r"copy16_async\(|__ldg\(|\ba\.(q|own_ml|own_o|k_cache|v_cache)\b")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, kernel):
    start = text.index("{", re.search(rf"__global__[^;{{]*\b{kernel}\(", text).end())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(kernel)


@pytest.mark.parametrize("file,kernel", KERNELS, ids=[k for _, k in KERNELS])
def test_waits_before_it_touches_global_memory(file, kernel):
    code = body(source(file), kernel)
    wait = re.search(r"^  grid_dependency_wait\(\);", code, re.M)  # a statement of the body itself: under no condition
    assert wait, "no unconditional wait"
    touch = TOUCHES.search(code)
    assert touch and wait.start() < touch.start(), f"{touch.group()} comes before the wait"


def test_every_dependent_launch_of_the_paged_calls_is_listed():
    text = source("fa_api.cu")
    part = text[text.index("fa_status_t check_paged("):]
    launched = set(re.findall(r"fa::(fa_\w+_kernel)<", part))
    assert {k for _, k in KERNELS} <= launched | {"fa_append_kernel"}
    assert not {k for k in launched if k.startswith(("fa_append", "fa_paged", "fa_prefix"))} - {k for _, k in KERNELS}


@pytest.mark.parametrize("file,kernel", KERNELS, ids=[k for _, k in KERNELS])
def test_tables_and_lengths_are_not_read_as_constants(file, kernel):
    """__ldg (ld.global.nc) asks that nobody writes the data while the kernel
    is resident; a dependent launch is resident before its inputs are written."""
    assert "__ldg" not in body(source(file), kernel)


def test_kernel_ids_differ():
    """The id in the status word says which kernel recorded an error."""
    ids = {}
    for name in sorted(os.listdir(CSRC)):
        for kernel, value in re.findall(r"constexpr uint32_t (kKern[A-Z]\w*) = (\d+);", source(name)):
            ids.setdefault(int(value), []).append(kernel)
    assert len(ids) >= 11 and all(len(k) == 1 for k in ids.values()), ids


# ------------------------------------------------------ how a pass is cut

SMS = 148


def steps(form, n_tiles, owners, key_tiles, S, d):
    """Time of a pass (in us) in whole waves of blocks: a block takes a step
    for each of its row tiles and key tiles and 5 more, in pairs of row tiles
    (an odd one alone, in half the splits) or one by one.  Joining moves
    8 d + 16 bytes of each row and split at 5 TB/s."""
    pairs = n_tiles // 2 if form == "pairs" else 0
    odd = n_tiles - 2 * pairs
    if form == "pairs" and not pairs:
        return float("inf")
    S_odd = (S + 1) // 2 if pairs else S
    blocks = owners * (pairs * S + odd * S_odd)
    of_a_block = max(2 * -(-key_tiles // S) if pairs else 0, -(-key_tiles // S_odd) if odd else 0)
    return -(-blocks // SMS) * (of_a_block + 5) + owners * n_tiles * 128 * S * (8 * d + 16) / 5e6


@pytest.mark.parametrize("n_tiles", [1, 2, 3, 4, 5, 6, 7, 9, 11, 13, 15, 17, 18])
@pytest.mark.parametrize("keys", [8192, 65536])
def test_a_prefix_pass_is_not_cut_into_mostly_empty_waves(n_tiles, keys):
    """The number of splits, read off the workspace, allows a time within a
    tenth of the best one."""
    Hq, Hkv, d, P, seqs = 32, 8, 128, 64, 32
    build()
    nbytes = binding.fa_decode_prefix_workspace_bytes(seqs * n_tiles, Hq, Hkv, 1, d, P, keys // P + 1, keys)
    splits = nbytes // (Hkv * n_tiles * 128 * (4 * d + 8))
    assert splits * Hkv * n_tiles * 128 * (4 * d + 8) == nbytes
    of = lambda form, S: steps(form, n_tiles, Hkv, keys // 128, S, d)
    best = min(of(form, S) for form in ("pairs", "singles") for S in range(1, 65))
    assert min(of("pairs", splits), of("singles", splits)) <= 1.1 * best
