"""Tokens' rows quantized along their rows alone, few (which are taken as they lie) and many (in their groups' turns): the
sizes decide what is written either way, as with both layouts.  Bytes, no tolerance."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, MX4 = bs.RECIPE_MX, bs.RECIPE_MX4
ROW, BOTH = bs.ROWWISE, bs.ROWWISE | bs.COLWISE


def poisoned(rows, cols, experts, recipe, which):
    q = bs.alloc_quantized(rows, cols, experts, recipe, which, DEV)
    for t in q.values():
        t.fill_(0xEE)
    return q


def routed(tokens, experts, k, cols, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    e = torch.randint(0, experts, (tokens, k), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn((tokens, cols), generator=g, device=DEV).bfloat16()
    w = torch.rand((tokens, k), generator=g, device=DEV)
    return bs.dispatch_plan(e, experts), x, w


@pytest.mark.parametrize("tokens", [1, 40, 2047, 2048, 16383, 16384])
@pytest.mark.parametrize("experts", [1, 7, 65, 257, 1024])
@pytest.mark.parametrize("recipe,which", [(MX, ROW), (MX4, ROW), (MX, BOTH)])
def test_bad_sizes_set_the_status_and_write_nothing(tokens, experts, recipe, which):
    plan, x, w = routed(tokens, experts, 2, 64)
    rows, good = 2 * tokens, plan["splits"]
    for at in {0, experts // 2, experts - 1}:
        for bad, bits in (([-1], bs.STATUS_NEGATIVE_SPLIT), ([rows + 1], bs.STATUS_EXCEEDS_CAPACITY),
                          ([int(good[at]) + 1], bs.STATUS_EXCEEDS_CAPACITY), ([2 ** 31 - 1], bs.STATUS_EXCEEDS_CAPACITY),
                          ([-2 ** 31], bs.STATUS_NEGATIVE_SPLIT),
                          ([-5, rows + 9], bs.STATUS_NEGATIVE_SPLIT | bs.STATUS_EXCEEDS_CAPACITY)):
            if len(bad) > experts:
                continue
            plan["splits"] = good.clone()
            for i, b in enumerate(bad):
                plan["splits"][(at + i) % experts] = b
            for weights in (None, w):
                q, status = poisoned(rows, 64, experts, recipe, which), torch.zeros(1, dtype=torch.int32, device=DEV)
                bs.dispatch_quantize(x, plan, recipe, which, q, weights=weights, status=status)
                assert int(status) == bits and all((t == 0xEE).all() for t in q.values()), (at, bad)


@pytest.mark.parametrize("tokens,experts,k", [(3, 2, 1), (40, 7, 3), (1000, 65, 4), (1365, 9, 3), (4096, 33, 1), (2500, 300, 2), (20000, 40, 2)])
@pytest.mark.parametrize("recipe,which", [(MX, ROW), (MX4, ROW), (MX, BOTH)])
@pytest.mark.parametrize("cols", [32, 160])
def test_rows_past_the_sizes_are_left(tokens, experts, k, recipe, which, cols):
    """Sizes that end before the choices do."""
    plan, x, _ = routed(tokens, experts, k, cols, 1)
    plan["splits"] = plan["splits"] * 2 // 3
    live, n = int(plan["splits"].sum()), tokens * k
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = bs.dispatch_quantize(x, plan, recipe, which, poisoned(n, cols, experts, recipe, which), status=status)
    rows = x[plan["choices"].long() // k]
    want = bs.grouped_quantize(rows, plan["splits"], recipe, which, poisoned(n, cols, experts, recipe, which))
    assert int(status) == 0 and (got["row_q"][live:] == 0xEE).all() and (got["row_s"][:, live:] == 0xEE).all()
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("rows", [1, 31, 32, 127, 129, 4095, 4097, 32767, 32768, 40001])
@pytest.mark.parametrize("experts", [1, 64, 65, 256, 257])
@pytest.mark.parametrize("recipe", [MX, MX4])
def test_few_rows_and_many(rows, experts, recipe):
    plan, x, _ = routed(rows, experts, 1, 160, 2)
    got = bs.dispatch_quantize(x, plan, recipe, ROW, poisoned(rows, 160, experts, recipe, ROW))
    want = bs.grouped_quantize(x[plan["choices"].long()], plan["splits"], recipe, ROW, poisoned(rows, 160, experts, recipe, ROW))
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("tokens,experts,k", [(3, 1, 2), (50, 7, 3), (1365, 9, 3), (2047, 300, 2), (4096, 33, 1), (3000, 128, 4), (10000, 128, 4)])
@pytest.mark.parametrize("recipe,which", [(MX, ROW), (MX4, ROW), (MX, BOTH), (MX4, BOTH)])
@pytest.mark.parametrize("weighted", [False, True])
def test_a_row_without_a_choice_is_zeros(tokens, experts, k, recipe, which, weighted):
    """Choices outside [0, tokens * top_k) before the last row: that row alone is zeros, codes and scales of the rows behind
    it are theirs.  (Weights that are powers of two make the products exact in bf16.)"""
    plan, x, _ = routed(tokens, experts, k, 96, 3)
    n = tokens * k
    g = torch.Generator(device=DEV).manual_seed(4)
    gone = torch.rand(n, generator=g, device=DEV) < 0.3
    gone[n // 3] = True
    plan["choices"][gone] = torch.tensor([-1, n, -9, 1 << 30, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)[
        torch.randint(0, 6, (int(gone.sum()),), generator=g, device=DEV)]
    w = torch.exp2(torch.randint(-3, 4, (tokens, k), generator=g, device=DEV).float()) if weighted else None
    c = torch.where(gone, 0, plan["choices"]).long()
    rows = x[c // k] * (w.view(-1)[c].bfloat16()[:, None] if weighted else 1)
    rows[gone] = 0
    got = bs.dispatch_quantize(x, plan, recipe, which, poisoned(n, 96, experts, recipe, which), weights=w)
    want = bs.grouped_quantize(rows, plan["splits"], recipe, which, poisoned(n, 96, experts, recipe, which))
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("recipe,which", [(MX, BOTH), (MX4, BOTH), (MX, ROW), (MX4, bs.COLWISE)])
@pytest.mark.parametrize("weighted", [False, True])
def test_several_column_tiles_a_workgroup(recipe, which, weighted):
    """A launch of more row tiles than it has segments for, random values in all rows, a width that ends inside a tile."""
    tokens, experts, k, cols = 16400, 37, 2, 4128
    plan, x, _ = routed(tokens, experts, k, cols, 5)
    w = torch.exp2(torch.randint(-3, 4, (tokens, k), device=DEV).float()) if weighted else None
    want = bs.grouped_quantize(bs.dispatch(x, plan, w), plan["splits"], recipe, which,
                               poisoned(tokens * k, cols, experts, recipe, which))
    for _ in range(3):
        got = bs.dispatch_quantize(x, plan, recipe, which, poisoned(tokens * k, cols, experts, recipe, which), weights=w)
        for name in want:
            assert torch.equal(got[name], want[name]), name
