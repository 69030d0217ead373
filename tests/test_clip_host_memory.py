"""The clipping's checks take no heap memory, however many tensors there are: the
calls find their aliasing (or its absence) in a process that cannot get any (CPU;
fake addresses, never dereferenced)."""
import itertools
import os
import random
import subprocess
import sys

from linear_recurrence_scan_row_amd import rlca as binding
from linear_recurrence_scan_row_amd import sequence as seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ALIAS, HIP = 0, 4, 6
FAR = 1 << 46

CHILD = """
import ctypes, resource
from linear_recurrence_scan_row_amd import rlca as binding, sequence as seq
n = 200_000
tensors = (seq.GradTensor * n)()
for i, t in enumerate(tensors):
    j = i * 7919 % n  # not in the order of their addresses
    t.data = t.out = (1 << 32) + 64 * j
    t.count, t.dtype = 16, 0
tensors[n // 2].data = tensors[n // 2].out = tensors[5].data + 32
lib = binding.lib()
def call():
    return lib.rlca_clip_grad_norm(tensors, n, 1.0, 1e-6, 1 << 46, (1 << 46) + 64,
                                   seq.CLIP_WORKSPACE_BYTES, None)
with open("/proc/self/statm") as f:
    pages = int(f.read().split()[0])
resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + (1 << 20),) * 2)
print("status", call())
"""


def test_checks_without_heap_memory():
    out = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert out.stdout.strip().endswith(f"status {ALIAS}"), out.stdout + out.stderr[-2000:]


def clip(tensors, norm=FAR, workspace=FAR + 64):
    arr = (seq.GradTensor * len(tensors))(*[seq.GradTensor(*t) for t in tensors])
    return binding.lib().rlca_clip_grad_norm(arr, len(tensors), 1.0, 1e-6, norm, workspace,
                                             seq.CLIP_WORKSPACE_BYTES, None)


def overlaps(tensors, extra):
    """Whether a written range overlaps another, by all pairs."""
    ranges = []
    for data, out, count, dtype in tensors:
        nbytes = count * (4 if dtype == binding.RLCA_F32 else 2)
        ranges.append((data, data + nbytes, data == out))
        if data != out:
            ranges.append((out, out + nbytes, True))
    ranges += [(a, a + n, True) for a, n in extra]
    return any((p[2] or q[2]) and p[0] < q[1] and q[0] < p[1]
               for p, q in itertools.combinations(ranges, 2))


def test_against_all_pairs():
    """Random lists on both sides of what one pass over the tensors holds, with
    overlaps anywhere, equal addresses and shared inputs.  Every list has one, so
    that nothing is launched; lists without are told by their last tensor's."""
    r = random.Random(7)
    extra = [(FAR, 8), (FAR + 64, seq.CLIP_WORKSPACE_BYTES)]
    for n in (1, 2, 30, 500, 1500, 3000):
        for _ in range(6):
            tensors, at = [], 1 << 32
            for _ in range(n):
                count = r.randrange(1, 40)
                data = at
                at += 4 * count + 4 * r.randrange(3)
                out = data
                if r.random() < 0.5:
                    out = at
                    at += 4 * count
                tensors.append((data, out, count, r.choice([binding.RLCA_F32, binding.RLCA_BF16])))
            r.shuffle(tensors)
            assert not overlaps(tensors[:40], extra)
            if n > 1:  # inputs may be shared: an out-of-place tensor read twice is no overlap
                a = next((t for t in tensors if t[0] != t[1]), None)
                if a is not None:
                    tensors.append((a[0], at, a[2], a[3]))
            victim = r.choice(tensors)
            place = r.randrange(len(tensors) + 1)
            tensors.insert(place, (victim[1], victim[1], 1, binding.RLCA_F32))
            assert clip(tensors) == ALIAS
            # its neighbour's last byte: the dtype misaligned would be another error
            tensors[place] = (victim[1] + 2 * victim[2] - 2, FAR + (1 << 30), 1, binding.RLCA_BF16)
            assert overlaps(tensors[max(0, place - 1):place + 1] + [victim], extra)
            assert clip(tensors) == ALIAS


def test_lists_without_overlap():
    """They pass the check: without a GPU the launch then fails, with one it is not
    reached (an invalid second list's status comes first)."""
    import torch
    if torch.cuda.is_available():  # the addresses are no memory
        return
    r = random.Random(8)
    for n in (1, 500, 1500, 3000, 5000):
        tensors = [((1 << 32) + 64 * i, (1 << 32) + 64 * i, 16, 0) for i in range(n)]
        r.shuffle(tensors)
        assert clip(tensors) == HIP
        shared = [(1 << 32, (1 << 40) + 64 * i, 16, 0) for i in range(n)]
        r.shuffle(shared)
        assert clip(shared) == HIP
