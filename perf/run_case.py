"""Calls one case of operators.py four times: a program to profile.

    python perf/run_case.py NAME [SEED]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import operators  # noqa: E402


def main(name, seed=1):
    operators.own = True
    state = operators.prepare(next(c for c in operators.listed() if c["name"] == name), int(seed))
    for _ in range(4):
        operators.run(state)
    torch.cuda.synchronize()
    print("ok", name)


if __name__ == "__main__":
    main(*sys.argv[1:])
