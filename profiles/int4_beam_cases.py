"""Runs the 4-bit head, beam selection and the reordering of states for a
profile: the listed cases of perf/more_operators.py and some more of the same
ranges, through the library, inputs rotated over three sets.

    python3 profiles/int4_beam_cases.py CASES N [--copy]

CASES: names separated by commas, or "all"; N: passes of each.  --copy ends with
a copy-like kernel of known size, by which counters of HBM bytes are scaled.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from perf import more_operators  # noqa: E402

MORE = [
    # forms that the listed cases do not have at these sizes
    dict(name="pack large f32", op="pack", v=128256, d=2048, dtype="f32", group=128, zero=False),
    dict(name="logits prompt 64", op="logits", rows=512, v=128256, d=2048, h="bf16", out="bf16",
         group=64, zero=True),
    dict(name="logits prompt 32", op="logits", rows=512, v=128256, d=2048, h="bf16", out="bf16",
         group=32, zero=False),
    dict(name="logits prompt f32", op="logits", rows=128, v=128256, d=2048, h="f32", out="f32",
         group=128, zero=False),
    dict(name="logits batch", op="logits", rows=32, v=128256, d=2048, h="bf16", out="bf16",
         group=128, zero=False),
    dict(name="logits drafts", op="logits", rows=64, v=128256, d=2048, h="bf16", out="bf16",
         group=128, zero=False),
    dict(name="logits batch f32", op="logits", rows=32, v=128256, d=2048, h="f32", out="f32",
         group=128, zero=False),
    dict(name="beam many", op="beam", B=4, K=16, n=32, v=128256, dtype="bf16", masked=False,
         finished=False),
    dict(name="reorder copy", op="reorder", B=16, K=4, outer=32, inner=8, positions=1000,
         pos_bytes=128, room=1024, place="out", ragged=False),
]


def main():
    want, n = sys.argv[1].split(","), int(sys.argv[2])
    more_operators.own = True
    for case in more_operators.listed() + MORE:
        if want != ["all"] and case["name"] not in want:
            continue
        states = [more_operators.prepare(case, seed) for seed in range(3)]
        torch.cuda.synchronize()
        for i in range(n):
            more_operators.run(states[i % 3])
        torch.cuda.synchronize()
        print("ran", case["name"], flush=True)
        del states
        torch.cuda.empty_cache()
    if "--copy" in sys.argv:
        x = torch.randn(1 << 26, device="cuda")
        for _ in range(3):
            torch.neg(x)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main()
