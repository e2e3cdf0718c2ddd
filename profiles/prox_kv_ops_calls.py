"""Calls of the operators around the paged 8-bit cache for a profiler.

    python3 profiles/prox_kv_ops_calls.py [CASE,CASE]     20 calls of each case of ``perf/more_operators.py``
    python3 profiles/prox_kv_ops_calls.py --summary kernel_trace.csv
                                                          median (least) of the launches of each kernel and grid, us
"""

import csv
import os
import statistics
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

CALLS = 20


def summary(path):
    rows = {}
    with open(path) as f:
        for r in csv.DictReader(f):
            if "prox::" in r["Kernel_Name"]:
                name = r["Kernel_Name"].replace("void ", "").replace("prox::", "").replace("(anonymous namespace)::", "").split("(")[0]
                rows.setdefault((name, int(r["Grid_Size_X"]) // int(r["Workgroup_Size_X"]), r["Workgroup_Size_X"]), []).append(
                    (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3)
    for (name, blocks, threads), us in rows.items():
        print(f"| `{name}` | {blocks} x {threads} | {statistics.median(us):.1f} ({min(us):.1f}) |")


def main():
    if len(sys.argv) > 2 and sys.argv[1] == "--summary":
        return summary(sys.argv[2])
    import torch
    from perf import more_operators as M
    M.own = True
    names = sys.argv[1].split(",") if len(sys.argv) > 1 else None
    for case in M.listed():
        if names and case["name"] not in names:
            continue
        state = M.prepare(case, 1)
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        for _ in range(CALLS):
            M.run(state)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main()
