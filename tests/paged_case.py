"""Runs one case of perf/more_operators.py through libclo a few times, for a profiler:

    python tests/paged_case.py chunk_b1_prompt_2000 [passes]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]


def main(name, passes=4):
    import more_operators
    import torch

    more_operators.own = True
    case = next(c for c in more_operators.listed() if c["name"] == name)
    state = more_operators.prepare(case, 1)
    for _ in range(passes):
        more_operators.run(state)
    torch.cuda.synchronize()
    print(f"{name}: {passes} passes")


if __name__ == "__main__":
    main(sys.argv[1], *(int(x) for x in sys.argv[2:]))
