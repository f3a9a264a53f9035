"""Passes of the cases of operators.py through the package's entry points, for a
profiler to watch, and a summary of the trace that it writes.

    rocprofv3 --kernel-trace --stats --output-format csv -d DIR -- python3 perf/passes.py [--passes N] [TEXT ...]
    python3 perf/passes.py --summary DIR/.../..._kernel_trace.csv

Cases whose names hold one of the texts, or all.  The summary gives the median
and the least time of the second half of each kernel's launches: over the first
ones the clock has not settled.
"""
import argparse
import csv
import os
import re
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def passes(texts, n):
    import torch

    from perf import operators
    operators.own = True
    for case in operators.listed():
        if texts and not any(t in case["name"] for t in texts):
            continue
        state = operators.prepare(case, 1)
        for _ in range(n):
            operators.run(state)
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def summary(path):
    with open(path) as f:
        rows = sorted(csv.DictReader(f), key=lambda r: int(r["Start_Timestamp"]))
    times = {}
    for r in rows:
        if "twell::" in r["Kernel_Name"]:
            name = re.sub(r"\(.*", "", r["Kernel_Name"].replace("(anonymous namespace)::", "").replace("void ", ""))
            key = name.replace("twell::", ""), r["Grid_Size_X"], r["Grid_Size_Y"], r["Workgroup_Size_X"]
            times.setdefault(key, []).append((int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3)
    for (name, x, y, wg), t in times.items():
        half = t[len(t) // 2:]
        print(f"median {statistics.median(half):7.2f} us, least {min(half):7.2f}, of {len(half)}: {name}, {x} x {y} threads by {wg}")


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--passes", type=int, default=400)
    ap.add_argument("--summary", metavar="CSV")
    ap.add_argument("texts", nargs="*")
    a = ap.parse_args()
    summary(a.summary) if a.summary else passes(a.texts, a.passes)


if __name__ == "__main__":
    main()
