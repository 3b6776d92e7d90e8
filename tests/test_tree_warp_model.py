"""The entry slots of a warp in attn_tree_kernel (csrc/tree.cu, Warp::run), re-enacted on the CPU.

A warp keeps two batches of 32 resolved list entries in shared memory.  Lane l writes entry l of a
batch; a step reads the keys and masks of 16 of them in every lane.  Lanes of a warp may run
apart between the instructions that wait for all of them (barriers, votes, shuffles), so each
slot has to be read for the last time before such an instruction, and written again only
after it.  The model runs the lanes in random order between those points, tags each slot with
its batch, and fails on a read that finds another batch's entry."""

import os
import random
import re

import pytest

from conftest import ROOT

LANES = 32


class SlotError(AssertionError):
    pass


def lane(l, slots, batches, odd, end_barrier):
    """What lane l does; `yield` is an instruction that waits for the whole warp, `yield 0` a
    place where other lanes may run ahead or fall behind."""

    def write(batch):
        slots[(batch & 1) * 32 + l] = batch

    def read(batch, entries):
        for e in entries:
            if slots[(batch & 1) * 32 + e] != batch:
                raise SlotError(f"lane {l} reads entry {e} of batch {batch}, finds batch {slots[(batch & 1) * 32 + e]}")

    def issue(batch, i):  # rows and scales of a step: key[r] of the lane's rows
        read(batch, range(i, i + 16))

    write(0)
    yield 1
    issue(0, 0)
    issue(0, 16)
    for batch in range(batches):
        more = batch + 1 < batches
        yield 0
        if more:
            write(batch + 1)
        for i in (0, 16):
            yield 1  # the step's rows are there
            if more:
                issue(batch + 1, i)
            yield 0
            read(batch, (i + (l >> 2), i + 8 + (l >> 2)))  # the masks of the lane's logits
            yield 1  # the vote on the running maximum
            if odd:  # values key by key
                for kk in range(16):
                    yield 1  # the weights by shuffles
                    yield 0
                    read(batch, (i + kk,))
                if end_barrier:
                    yield 1
            else:  # weights transposed between the lanes, then the products
                yield 1


def run(seed, batches, odd, end_barrier=True):
    rng = random.Random(seed)
    slots = [-1] * 64
    lanes = [lane(l, slots, batches, odd, end_barrier) for l in range(LANES)]
    ready, waiting, done = list(range(LANES)), [], 0
    while ready:
        l = ready.pop(rng.randrange(len(ready)))
        try:
            kind = next(lanes[l])
        except StopIteration:
            done += 1
            kind = None
        if kind == 0:
            ready.append(l)
        elif kind == 1:
            waiting.append(l)
        if not ready and waiting:
            assert done == 0, "lanes that end while others wait"
            ready, waiting = waiting, []
    assert done == LANES


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("batches", [1, 2, 3, 6])
def test_slots_are_read_before_they_are_written_again(batches, odd):
    for seed in range(20):
        run(seed, batches, odd)


def test_key_by_key_needs_a_barrier_at_its_end():
    # without it a lane that is ahead replaces the last entry of a batch that others still read
    with pytest.raises(SlotError):
        for seed in range(20):
            run(seed, 4, True, end_barrier=False)
    run(0, 1, True, end_barrier=False)  # lists of one batch never reuse a slot


def source(name):
    with open(os.path.join(ROOT, "structured_sparse_attention_b200", "csrc", name)) as f:
        return f.read()


def test_the_kernel_has_the_barrier():
    src = source("tree.cu")
    body = src[src.index("void one_by_one("):]
    body = body[:body.index("\n    }\n")]
    assert re.search(r"__syncwarp\(\);[^\n]*$", body.rstrip()), "one_by_one must end in a warp barrier"


def test_tensor_memory_is_read_by_whole_warps():
    # attn_tree_wide_kernel: code that runs in some lanes of a warp (a loop under a lane's own
    # condition, stores of the rows that exist) is followed by a warp barrier before the next
    # access to tensor memory, which is an instruction of the whole warp
    kernel = source("tree_wide.cu")
    loop = kernel.index("in && c < D / 8")
    assert "__syncwarp();" in kernel[loop:kernel.index("tmem_ld8(", loop)]
    last = kernel.index("const bool direct")
    assert "__syncwarp();" in kernel[kernel.index("for (int c", last):kernel.index("tmem_ld32(", last)]
