"""Runs the operators around the head for a profile: the listed cases of
perf/operators.py and some more of the same ranges, through the library, inputs
rotated over three sets.

    python3 profiles/around_head_cases.py CASES N [--copy]

CASES: names separated by commas, or "all"; N: passes of each.  --copy ends with
a copy-like kernel of known size, by which counters of HBM bytes are scaled.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from perf import operators  # noqa: E402

MORE = [
    # forms that the listed cases do not have at these sizes
    dict(name="norm prompts f32", op="norm", rows=8192, d=2048, dtype="f32", residual=True,
         outputs="fp8", offset=0.0),
    dict(name="norm prompts y", op="norm", rows=8192, d=2048, dtype="bf16", residual=True,
         outputs="y", offset=0.0),
    dict(name="logits drafts f32", op="logits", rows=32, v=128256, d=2048, out="f32"),
    dict(name="logits deep", op="logits", rows=300, v=6000, d=4096, out="bf16"),
    dict(name="logits prompts f32", op="logits", rows=2048, v=128256, d=2048, out="f32"),
    dict(name="verify greedy batch", op="verify", B=64, k=7, v=128256, dtype="bf16", mode="greedy",
         draft="point", tau=1.0, masked=False),
]


def main():
    want, n = sys.argv[1].split(","), int(sys.argv[2])
    operators.own = True
    for case in operators.listed() + MORE:
        if want != ["all"] and case["name"] not in want:
            continue
        states = [operators.prepare(case, seed) for seed in range(3)]
        torch.cuda.synchronize()
        for i in range(n):
            operators.run(states[i % 3])
        torch.cuda.synchronize()
        print("ran", case["name"], flush=True)
        del states
    if "--copy" in sys.argv:
        x = torch.randn(1 << 26, device="cuda")
        for _ in range(3):
            torch.neg(x)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main()
