"""What the AdamW step with stochastic rounding refuses, before any HIP call (no GPU needed): the fake pointers are
never dereferenced."""
import warnings

import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

P = 1 << 20
OK, NULL, SHAPE, ALIGN, ARG = 0, -1, -4, -5, -7


def step(plan=P, n=1, chunks=1, pd=0, gd=0, st=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, lr_dev=None,
         step_dev=None, gs=None, noop=None, seed=1):
    return bs.lib().bsfp8_adamw_step_stochastic(plan, n, chunks, pd, gd, st, lr, b1, b2, eps, wd, t, lr_dev, step_dev, gs,
                                                noop, seed, None)


@pytest.mark.parametrize("change,code", [
    (dict(pd=2), ARG), (dict(gd=-1), ARG), (dict(st=2), ARG), (dict(lr=-1.0), ARG), (dict(b1=1.0), ARG),
    (dict(b2=float("nan")), ARG), (dict(eps=-1e-9), ARG), (dict(wd=float("inf")), ARG), (dict(t=0), ARG), (dict(n=0), SHAPE),
    (dict(chunks=-1), SHAPE), (dict(chunks=1 << 31), SHAPE), (dict(plan=None), NULL), (dict(plan=P + 8), ALIGN),
    (dict(gs=P + 2), ALIGN), (dict(step_dev=P + 1), ALIGN), (dict(chunks=0, plan=None), OK),
    (dict(chunks=0, plan=None, seed=(1 << 64) - 1), OK),
])
def test_refuses(change, code):
    assert step(**change) == code


def test_binding_warns_of_nearest_rounding():
    for state, seed, warned in ((bs.STATE_8BIT, None, 1), (bs.STATE_8BIT, 3, 0), (bs.STATE_F32, None, 0)):
        plan = bs.AdamWPlan(torch.zeros(1), 1, 0, bs.F32, bs.F32, state, ())  # only empty tensors: nothing is launched
        with warnings.catch_warnings(record=True) as got:
            warnings.simplefilter("always")
            bs.adamw_step(plan, 1e-3, stream=0, seed=seed)
        assert len(got) == warned and all("seed" in str(w.message) for w in got)
    with pytest.raises(bs.BSFP8Error, match="invalid"):
        bs.adamw_step(plan, -1.0, stream=0, seed=-1)
