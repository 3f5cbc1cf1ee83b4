"""Tensors on another device than the current one are refused before the library is called, each argument by itself (no GPU
needed: the tensors say that they lie on one, their pointers are never dereferenced)."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

BOTH = bs.ROWWISE | bs.COLWISE


class Placed(torch.Tensor):
    """A tensor that says that it lies on device `at`."""
    is_cuda = True

    def get_device(self):
        return self.at

    def data_ptr(self):
        return 1 << 20


def on(t, at=0):
    p = torch.Tensor._make_subclass(Placed, t)
    p.at = at
    return p


def layouts(rows, cols, experts, which):
    return {n: on(t) for n, t in bs.alloc_quantized(rows, cols, experts, bs.RECIPE_MX, which, "cpu").items()}


def zeros(*shape, dtype=torch.float32):
    return on(torch.zeros(shape, dtype=dtype))


BF16, I32 = torch.bfloat16, torch.int32


def calls():
    """Each call and its tensors by name; (dict, key) where they lie."""
    plan = dict(rows=zeros(4, 2, dtype=I32), choices=zeros(8, dtype=I32), splits=zeros(3, dtype=I32))
    q, kept, wide, y = layouts(8, 64, 3, BOTH), layouts(8, 128, 3, bs.ROWWISE), layouts(8, 128, 3, BOTH), layouts(8, 64, 3, bs.COLWISE)
    t = dict(x=zeros(4, 64, dtype=BF16), w=zeros(4, 2), status=zeros(1, dtype=I32), h=zeros(8, 128, dtype=BF16),
             dy=zeros(8, 64, dtype=BF16), p=zeros(8), dp=zeros(8), ws=zeros(1 << 16, dtype=torch.uint8))
    every = {
        "quantize": (lambda: bs.dispatch_quantize(t["x"], plan, bs.RECIPE_MX, BOTH, q, weights=t["w"], status=t["status"],
                                                  stream=0),
                     [(t, "x"), (t, "w"), (t, "status"), (plan, "rows"), (plan, "choices"), (plan, "splits")] +
                     [(q, n) for n in q]),
        "keep": (lambda: bs.grouped_act_checkpoint(bs.ACT_SWIGLU, t["h"], plan["splits"], bs.RECIPE_MX, BOTH, q, kept,
                                                   probs=t["p"], status=t["status"], stream=0),
                 [(t, "h"), (t, "p"), (t, "status"), (plan, "splits")] + [(d, n) for d in (q, kept) for n in d]),
        "grad": (lambda: bs.grouped_act_checkpoint_grad(bs.ACT_SWIGLU, kept, t["dy"], plan["splits"], bs.RECIPE_MX, BOTH,
                                                        wide, probs=t["p"], y=y, dprobs=t["dp"], workspace=t["ws"],
                                                        status=t["status"], stream=0),
                 [(t, n) for n in ("dy", "p", "dp", "ws", "status")] + [(plan, "splits")] +
                 [(d, n) for d in (kept, wide, y) for n in d])}
    return every


@pytest.mark.parametrize("call,i", [(name, i) for name, (_, at) in calls().items() for i in range(len(at))])
def test_each_tensor_is_on_the_current_device(monkeypatch, call, i):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    run, places = calls()[call]
    where, name = places[i]
    where[name].at = 1
    with pytest.raises(ValueError, match="the current device is cuda:0"):
        run()
