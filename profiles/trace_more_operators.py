"""What rocprofv3 traces: each listed case of perf/more_operators.py, and forms beside them, prepared
three times over and called 13 times in turn.

    rocprofv3 --kernel-trace --stats -d prof -o p --output-format csv -- python3 profiles/trace_more_operators.py [NAME,NAME]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_grouped_amd as bs  # noqa: E402
from perf import more_operators as mo  # noqa: E402

mo.own = True
BOTH = bs.ROWWISE | bs.COLWISE
ROUTE = {"tokens": 131072, "experts": 128, "top_k": 8, "type": "fp32", "masked": 0.0, "renormalize": True}
MOVE = {"op": "dispatch", "tokens": 16384, "experts": 32, "top_k": 4, "cols": 4096, "dropped": 0.0, "weighted": False}
GLU = {"act": "swiglu", "rows": 65536, "pad": 0, "experts": 32, "ffn": 2048}
SRELU = GLU | {"act": "srelu", "ffn": 4096}

#: beside the listed ones: (name, case, recipe)
MORE = [("route_sigmoid", ROUTE | {"op": "route", "scoring": "sigmoid", "bias": True, "sum": False}, None),
        ("route_grad_chosen", ROUTE | {"op": "route_grad", "scoring": "softmax", "bias": False, "sum": False}, None),
        ("dispatch_bf16", MOVE | {"out": "bf16"}, None), ("dispatch_rowwise", MOVE | {"out": "mxfp8_row"}, None),
        ("dispatch_weighted", MOVE | {"out": "mxfp8", "weighted": True}, None),
        ("dispatch_mxfp4", MOVE | {"out": "mxfp8"}, bs.RECIPE_MX4),
        ("act_layer", GLU | {"op": "act"}, None), ("act_layer_mxfp4", GLU | {"op": "act"}, bs.RECIPE_MX4),
        ("act_srelu", SRELU | {"op": "act"}, None),
        ("act_grad_mxfp4", GLU | {"op": "act_grad"}, bs.RECIPE_MX4), ("act_grad_srelu", SRELU | {"op": "act_grad"}, None)]


def call(s, recipe):
    """A case's call, or the same with MXFP4 outputs (the MXFP8 buffers hold them)."""
    if recipe is None:
        return mo.run(s)
    if s["op"] == "dispatch":
        return bs.dispatch_quantize(s["x"], s["plan"], recipe, BOTH, s["q"], weights=s["weights"])
    act = bs.ACT_SRELU if s["act"] == "srelu" else bs.ACT_SWIGLU
    if s["op"] == "act":
        return bs.grouped_act_checkpoint(act, s["h"], s["splits"], recipe, BOTH, s["q"], s["kept"], probs=s["probs"])
    return bs.grouped_act_checkpoint_grad(act, s["kept"], s["dy"], s["splits"], recipe, BOTH, s["q"], probs=s["probs"],
                                          y=s["y"], dprobs=s["dprobs"])


def main():
    names = sys.argv[1].split(",") if len(sys.argv) > 1 else None
    for name, case, recipe in [(c["name"], c, None) for c in mo.listed()] + MORE:
        if names and name not in names:
            continue
        print(name, flush=True)
        states = [mo.prepare(case, seed) for seed in range(3)]
        for i in range(13):
            call(states[i % 3], recipe)
        torch.cuda.synchronize()
        del states
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
