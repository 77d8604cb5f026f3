"""Calls one case of operators.py or more_operators.py four times: a program to
profile.

    python perf/run_case.py NAME [SEED]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import more_operators, operators  # noqa: E402


def main(name, seed=1):
    of, case = next((m, c) for m in (operators, more_operators) for c in m.listed() if c["name"] == name)
    of.own = True
    state = of.prepare(case, int(seed))
    for _ in range(4):
        of.run(state)
    torch.cuda.synchronize()
    print("ok", name)


if __name__ == "__main__":
    main(*sys.argv[1:])
