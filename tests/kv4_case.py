"""Runs one case of perf/operators.py through libclo a few times, for a profiler:

    python tests/kv4_case.py attn_b16_64k [passes]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]


def main(name, passes=4):
    import operators
    import torch

    operators.own = True
    case = next(c for c in operators.listed() if c["name"] == name)
    state = operators.prepare(case, 1)
    for _ in range(passes):
        operators.run(state)
    torch.cuda.synchronize()
    flags = int(state["err"].item())
    print(f"{name}: {passes} passes, error flags {flags}")
    return flags


if __name__ == "__main__":
    sys.exit(main(sys.argv[1], *(int(x) for x in sys.argv[2:])))
