"""Calls of the paged 8-bit cache's operators for a profiler.

    python3 profiles/prox_kv_calls.py CASE        three calls to warm up, then 12 over three states
    python3 profiles/prox_kv_calls.py --list      names of the cases
    python3 profiles/prox_kv_calls.py --summary kernel_trace.csv
                                                  median (least) of the last 12 launches of each kernel, us
    python3 profiles/prox_kv_calls.py --counter counter_collection.csv
                                                  median of the counter over the last 12 launches of each kernel

CASE is one of those of ``perf/operators.py`` or of FORMS: forms that it does
not list."""

import csv
import os
import statistics
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

CALLS = 12
_ATTEND = dict(op="attend", lengths=1, window=0)
FORMS = [
    dict(_ATTEND, name="prompt_e4m3", kind="fp8", heads=32, kv=8, hd=128, seqs=1, new_lo=4096, new_hi=4096, ctx_lo=4096, ctx_hi=4096),
    dict(_ATTEND, name="long_prompt", kind="int8", heads=32, kv=8, hd=128, seqs=1, new_lo=16384, new_hi=16384, ctx_lo=16384, ctx_hi=16384),
    dict(_ATTEND, name="prompt_heads_of_256", kind="int8", heads=16, kv=4, hd=256, seqs=1, new_lo=4096, new_hi=4096, ctx_lo=4096, ctx_hi=4096),
    dict(_ATTEND, name="tokens_heads_of_192", kind="int8", heads=16, kv=2, hd=192, seqs=16, new_lo=1, new_hi=1, ctx_lo=4000, ctx_hi=16000),
    dict(_ATTEND, name="tokens_heads_of_256", kind="int8", heads=16, kv=2, hd=256, seqs=16, new_lo=1, new_hi=1, ctx_lo=4000, ctx_hi=16000),
    dict(_ATTEND, name="tokens_32_heads_on_1", kind="int8", heads=32, kv=1, hd=128, seqs=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=16384),
    dict(op="read", lengths=1, name="read_prefix_fp32", kind="int8", heads=32, kv=8, hd=128, seqs=1, new_lo=32768, new_hi=32768,
         ctx_lo=32768, ctx_hi=32768, fp32=True),
]


def launches(path, value):
    """Per kernel of the library: `value` of its launches in order."""
    rows = {}
    with open(path) as f:
        for r in csv.DictReader(f):
            if "prox::" in r["Kernel_Name"]:
                name = r["Kernel_Name"].replace("void ", "").replace("prox::(anonymous namespace)::", "").split("(")[0]
                rows.setdefault(name, []).append((int(r["Dispatch_Id"]), value(r)))
    return {k: [x for _, x in sorted(v)] for k, v in rows.items()}


def main(arg, path=None):
    if arg == "--summary":
        for k, v in launches(path, lambda r: (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3).items():
            print(f"`{k}` | {statistics.median(v[-CALLS:]):.1f} ({min(v[-CALLS:]):.1f})")
        return
    if arg == "--counter":
        for k, v in launches(path, lambda r: float(r["Counter_Value"])).items():
            print(f"`{k}` | {statistics.median(v[-CALLS:]):.1f}")
        return
    import torch
    from perf import operators as ops
    ops.own = True
    cases = {c["name"]: c for c in ops.listed() + FORMS}
    if arg == "--list":
        print("\n".join(cases))
        return
    case = cases[arg]

    def call(st):
        if not case.get("fp32"):
            return ops.run(st)
        P, cache, batch = ops._handles(st)
        return P.kv_read(cache, batch, dtype=torch.float32)

    states = [ops.prepare(case, s) for s in (1, 2, 3)]
    for i in range(3 + CALLS):
        call(states[i % 3])
    torch.cuda.synchronize()
    print(arg, "work", ops.work(case), flush=True)


if __name__ == "__main__":
    main(*sys.argv[1:])
