"""Times the cases of operators.py or more_operators.py on the GPU, or runs one of them under a profiler.

    python perf/time_operators.py [--of more_operators] [--only NAME,NAME] [--seeds 3] [--plain]
    rocprofv3 --pmc ... -- python3 perf/time_operators.py [--of more_operators] --once NAME [--seed 1]

For each case and seed: us per call of a loop of calls through the package (host and device side by side),
and us per call of a replayed HIP graph of calls, the device alone; the least of several rounds. --plain
times the plain forms in a loop instead. --once prepares one case and calls it four times, with nothing
else on the GPU but its inputs' making.
"""
import argparse
import importlib
import os
import sys
import time

import torch

sys.path[:0] = [os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                os.path.dirname(os.path.abspath(__file__))]


def loop_us(ops, state, rounds=7):
    ops.run(state)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    ops.run(state)
    torch.cuda.synchronize()
    calls = max(1, min(300, int(0.03 / (time.perf_counter() - begin))))
    best = float("inf")
    for _ in range(rounds):
        begin = time.perf_counter()
        for _ in range(calls):
            ops.run(state)
        torch.cuda.synchronize()
        best = min(best, (time.perf_counter() - begin) / calls)
    return 1e6 * best


def graph_us(ops, state, calls=30, rounds=10):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.run(state)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            ops.run(state)
    best = float("inf")
    for _ in range(rounds + 3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return 1e3 * best / calls


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--of", default="operators", choices=["operators", "more_operators"], help="the file of the cases")
    p.add_argument("--only", default="", help="names of cases, separated by commas")
    p.add_argument("--seeds", type=int, default=3)
    p.add_argument("--plain", action="store_true")
    p.add_argument("--once", default="", metavar="NAME")
    p.add_argument("--seed", type=int, default=1, help="of --once")
    a = p.parse_args()
    ops = importlib.import_module(a.of)
    ops.own = not a.plain
    cases = {c["name"]: c for c in ops.listed()}
    if a.once:
        state = ops.prepare(cases[a.once], a.seed)
        for _ in range(4):
            ops.run(state)
        torch.cuda.synchronize()
        return
    for name in a.only.split(",") if a.only else cases:
        for seed in range(1, a.seeds + 1):
            state = ops.prepare(cases[name], seed)
            line = f"{name} seed {seed}: {loop_us(ops, state):.1f} us a call"
            if not a.plain:
                line += f", {graph_us(ops, state):.2f} us in a graph"
            print(line, flush=True)
            del state


if __name__ == "__main__":
    main()
