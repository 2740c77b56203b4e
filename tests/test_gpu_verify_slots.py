"""Slots of a batch that hold no sequence (no row), anywhere among the others:
the drafts of the sequences behind them are still one after the other."""
import pytest

from . import around_ref as ref
from .test_gpu_verify import Case, compare, fh  # noqa: F401 (fh: a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def with_empty(c, empty):
    """The case with empty slots before its sequences empty[i]; (slots of the
    sequences, number of slots)."""
    start, slots = c.row_start.tolist(), []
    new, u = [], []
    for s in range(len(start) - 1):
        for _ in range(empty.count(s)):
            new.append(start[s])
            u.append(0.25)
        slots.append(len(new))
        new.append(start[s])
        u.append(float(c.u_sample[s]))
    for _ in range(empty.count(len(start) - 1)):
        new.append(start[-1])
        u.append(0.75)
    new.append(start[-1])
    c.row_start = torch.tensor(new, dtype=torch.int32, device="cuda")
    c.u_sample = torch.tensor(u, device="cuda")
    return slots, len(u)


def check(fh, counts, empty, v, dtype, mode, draft, room=0):
    c = Case(counts, v, dtype, 31 + len(counts), draft=draft, noise=0.3)
    want = c.want(mode)
    slots, n = with_empty(c, empty)
    if room:                # arrays made for more drafts than there are
        more = torch.full((room,), 3, dtype=torch.int32, device="cuda")
        c.drafts = torch.cat([c.drafts, more])
        c.u_accept = torch.cat([c.u_accept, torch.zeros(room, device="cuda")])
        if c.q is not None:
            c.q = torch.cat([c.q, c.q.new_zeros(room, v)])
            c.q = torch.nn.functional.pad(c.q, (0, -v % 4))[:, :v]
    bufs = c.buffers(fh)
    c.call(fh, bufs, mode)
    torch.cuda.synchronize()
    at = torch.tensor(slots, device="cuda")
    compare([b[at] for b in bufs[:3]], want)
    rest = [s for s in range(n) if s not in slots]
    assert torch.all(bufs[0][rest] == -1) and torch.all(bufs[1][rest] == -1)
    assert torch.all(bufs[2][rest] == 0)


@pytest.mark.parametrize("mode,draft", [("sample", "dense"), ("sample", "point"),
                                        ("greedy", "point")])
@pytest.mark.parametrize("counts,empty", [([2, 2], [1]), ([2, 0, 3, 1], [0]),
                                          ([1, 4, 0, 2], [1, 1, 3, 4, 4]), ([3], [0, 0, 1]),
                                          ([2] * 9, [0, 2, 2, 5, 8, 9])])
def test_empty_slots_anywhere(fh, mode, draft, counts, empty):
    check(fh, counts, empty, 3001, torch.float32, mode, draft)
    check(fh, counts, empty, 3001, torch.bfloat16, mode, draft, room=7)


def test_empty_slots_in_a_large_batch(fh):
    # more slots than the threads of a workgroup, and sequences of many chunks
    n = 700
    check(fh, [s % 3 for s in range(n)], [s for s in range(0, n, 3)] + [5] * 300, 130,
          torch.float32, "sample", "point")
    check(fh, [s % 4 for s in range(40)], [0, 3, 3, 17, 39, 40], 20000, torch.bfloat16, "sample",
          "dense")


def test_one_row_keeps_a_slot(fh):
    # a slot may also be held by one row without a draft: nothing moves
    c = Case([2, 0, 3], 2000, torch.float32, 5)
    bufs = c.check(fh)
    assert bufs[1][1].item() == 0 and bufs[0][1, 0].item() >= 0
