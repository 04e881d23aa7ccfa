"""Host side of the clipping's tensor lists (no GPU)."""
import numpy as np
import pytest
import torch

import backward_token_expert_amd as bte
from backward_token_expert_amd import lrm


def test_a_list_in_place_may_come_from_an_iterator():
    # as `(p.grad for p in parameters)`: read once, for sources and destinations alike.  Host tensors
    # are turned down for where they are, not for a destination that is missing.
    with pytest.raises(lrm.LrmError, match="on cpu"):
        bte.make_tensor_list(t for t in [torch.zeros(4), torch.zeros(5)])
    with pytest.raises(lrm.LrmError, match="2 sources, 1 destinations"):
        bte.make_tensor_list((torch.zeros(4) for _ in range(2)), iter([torch.zeros(4)]))


def _status(entries, ws_bytes=256):
    """The status of lrm_clip_grads for (src, dst, count, dtype) entries; 3 (the workspace is too small)
    where the list is accepted, so nothing is launched."""
    a = (lrm.Tensor * max(1, len(entries)))(*[lrm.Tensor(*e, 0) for e in entries])
    return bte.load_library().lrm_clip_grads(a, len(entries), 1.0, 0x100000, 0x100000, ws_bytes, None)


def _overlap(entries):
    """The rule itself, pair by pair: no element written by one range is in another."""
    ranges = []
    for src, dst, count, dtype in entries:
        if count:
            size = count * (2 if dtype else 4)
            ranges.append((dst, dst + size, True))
            if src != dst:
                ranges.append((src, src + size, False))
    if not ranges:
        return False
    lo, hi, written = (np.array(c) for c in zip(*ranges))
    meet = (lo[:, None] < hi) & (lo < hi[:, None]) & (written | written[:, None])
    return bool(np.triu(meet, 1).any())


@pytest.mark.parametrize("n", [1, 3, 60, 300, 1100, 1600, 2600])
def test_overlaps_are_found_in_lists_of_any_length_and_order(n):
    import random
    rng = random.Random(n)
    seen = set()
    for trial in range(12 if n < 1000 else 6):
        at, entries = 0x200000, []
        for _ in range(n):
            count, dtype = rng.choice([0, 1, 2, 7, 40, 1000]), rng.randint(0, 1)
            size = count * (2 if dtype else 4) + 15 & ~15
            inplace = rng.random() < 0.5
            entries.append((at, at if inplace else at + size, count, dtype))
            at += size * (1 if inplace else 2)
        rng.shuffle(entries)
        # a few of the lists get one entry moved onto, or beside, another one's place
        for _ in range(trial % 3):
            i, j = rng.randrange(n), rng.randrange(n)
            src, dst, count, dtype = entries[i]
            to = entries[j][rng.randint(0, 1)] + rng.choice([0, 4, 16, -16, 4000])
            entries[i] = (to, dst, count, dtype) if rng.random() < 0.5 else (src, to, count, dtype)
        want = _overlap(entries)
        seen.add(want)
        assert _status(entries) == (1 if want else 3)
    assert n < 60 or seen == {False, True}


def test_a_source_may_be_read_twice():
    shared = [(0x200000, 0x300000 + 0x1000 * i, 16, 0) for i in range(2500)]
    assert _status(shared) == 3
    assert _status(shared + [(0x200000, 0x200000, 16, 0)]) == 1


HEAPLESS = """
import ctypes, resource
import backward_token_expert_amd as bte
from backward_token_expert_amd import lrm
n = 1 << 21
lib = bte.load_library()
a = (lrm.Tensor * n)()
for i in range(n):
    a[i].src = a[i].dst = 0x200000 + 64 * i
    a[i].count = 16
a[1].src = a[1].dst = a[0].src + 32
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (8 << 20),) * 2)
print("status", lib.lrm_clip_grads(a, n, 1.0, 0x100000, 0x100000, 256, None))
"""


def test_a_list_is_checked_without_memory_of_the_librarys_own():
    # with no memory left for a copy of the list, the overlap is still found
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", HEAPLESS], capture_output=True, text=True, cwd=root, timeout=120)
    assert r.stdout.strip() == "status 1", (r.stdout, r.stderr[-500:])
