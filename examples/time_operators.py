"""Times one call of an operator around the layer at a size of your own.

    python examples/time_operators.py lora  M K N R L [mixed|requests] [bf16|fp16]
    python examples/time_operators.py gate  M E top_k [forward|backward] [fp32|bf16|fp16]
    python examples/time_operators.py sort  M H E top_k [forward|backward] [bf16|fp16|fp32]
    python examples/time_operators.py unsort  (as sort)

Inputs are those of perf/operators.py (lora: a token's adapter drawn evenly from L, or runs of
one).  Whole calls through the Python binding, one after another on three rotating inputs:
microseconds a call, the median of seven runs of 60 (which is how the sizes in the sources'
comments and the design notes were timed), and the operator's floor, its bytes and operations
at the rates given by --hbm (GB/s) and --flops (TFLOP/s).  Needs a GB300 and the built library.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from perf import operators as cases  # noqa: E402


def case(op, args):
    sizes = [int(a) for a in args if a.lstrip("-").isdigit()]
    words = [a for a in args if not a.lstrip("-").isdigit()]
    dtype = [w for w in words if w in ("bf16", "fp16", "fp32")]
    how = {"dtype": dtype[0]} if dtype else {}
    for w in words:
        if w in ("forward", "backward"):
            how["direction"] = w
        elif w in ("mixed", "requests"):
            how["tokens"] = w
        elif w not in dtype:
            raise SystemExit(f"what is {w!r}?")
    return {"lora": cases._lora, "gate": cases._gate, "sort": cases._sort,
            "unsort": cases._unsort}[op]("", *sizes, **how)


def time_call(c, runs=7, calls=60):
    """Seconds a call."""
    cases.own = True
    inputs = [cases.prepare(c, seed) for seed in range(3)]
    for i in range(12):
        cases.run(inputs[i % 3])
    took = []
    for _ in range(runs):
        torch.cuda.synchronize()
        start = time.perf_counter()
        for i in range(calls):
            cases.run(inputs[i % 3])
        torch.cuda.synchronize()
        took.append((time.perf_counter() - start) / calls)
    return sorted(took)[runs // 2]


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__,
                                formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("op", choices=["lora", "gate", "sort", "unsort"])
    p.add_argument("sizes", nargs="+")
    p.add_argument("--hbm", type=float, default=6673.5)
    p.add_argument("--flops", type=float, default=1880.1)
    a = p.parse_args(argv)
    c = case(a.op, a.sizes)
    work = cases.work(c)
    floor = max(work["bytes"] / (a.hbm * 1e9), work["flops"] / (a.flops * 1e12))
    print("%s %s: %.2f us a call, floor %.2f us" % (a.op, " ".join(a.sizes), time_call(c) * 1e6,
                                                    floor * 1e6))


if __name__ == "__main__":
    main()
