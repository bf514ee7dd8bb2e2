"""mamba_batch_plan on the GPU against one request after another; whole numbers, so all of them equal."""
import numpy as np
import pytest

import la_ref as ref
from recurrent_state_update_gb300 import binding as bd
from recurrent_state_update_gb300 import build as bld
from recurrent_state_update_gb300 import workloads as wl

from gpu_util import guarded, to_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    bld.build()
    bd.lib()
    torch.cuda.set_device(0)


def check(new, past, table, block, num_slots, max_tokens, max_ckpt=3, skip=(), spread=0):
    import torch
    rows = len(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = {n: guarded(torch.full(shape, 77, **i32)) for n, shape in dict(
        cu_seqlens=(rows + 1,), slot_ids=(rows,), copy_src=(rows,), copy_dst=(rows,), ckpt_slots=(rows, max_ckpt),
        positions=(max_tokens,), token_rows=(max_tokens,)).items() if n not in skip}
    if "has_initial_state" not in skip:
        outs["has_initial_state"] = guarded(torch.full((rows,), 77, dtype=torch.uint8, device="cuda"))
    err = torch.zeros(1, **i32)
    table = np.asarray(table, np.int32).reshape(rows, -1)
    pages = to_i32(np.pad(table, ((0, 0), (0, spread)), constant_values=-9))[:, :table.shape[1]]
    bd.mamba_batch_plan(to_i32(new), to_i32(past), pages, block, num_slots, err_word=err, **{n: o.t for n, o in outs.items()})
    want, bits = ref.batch_plan([int(x) for x in new], [int(x) for x in past], table.tolist(), block, num_slots, max_tokens, max_ckpt)
    for n, o in outs.items():
        o.check(n)
        assert o.t.cpu().tolist() == want[n], n
    assert int(err.item()) == bits
    return bits


def batch(seed, rows, block, longest, columns):
    g = wl.rng(seed, 0)
    new = g.integers(0, longest + 1, rows)
    new[g.random(rows) < 0.2] = 0
    past = g.integers(0, 4 * (block or 50), rows)
    if block:
        past = np.where(g.random(rows) < 0.5, past // block * block, past)
    return new, past, g.permutation(rows * columns).reshape(rows, columns)


@pytest.mark.parametrize("rows,block,longest", [(1, 64, 1), (1, 64, 900), (7, 0, 5), (33, 16, 50), (256, 128, 1), (300, 128, 400),
                                                (4096, 64, 3), (4097, 64, 3), (20000, 8, 20)])
def test_plan(rows, block, longest):
    columns = 1 + (4 * block + longest) // block if block else 1
    new, past, table = batch(40, rows, block, longest, columns)
    assert check(new, past, table, block, table.size, int(new.sum()) + 13, spread=rows % 3) == 0


def test_plan_of_exactly_the_most_tokens_and_one_more():
    new, past, table = [3, 0, 5], [0, 4, 64], np.arange(9).reshape(3, 3)
    assert check(new, past, table, 32, 9, 8) == 0
    assert check(new, past, table, 32, 9, 7) == bd.MAMBA_ERR_SEQLENS


@pytest.mark.parametrize("new,past", [([-1, 2], [0, 0]), ([1, 2], [0, -5]), ([2 ** 31 - 1, 2 ** 31 - 1], [0, 0]),
                                      ([1, 1], [0, 2 ** 31 - 1])])
@pytest.mark.parametrize("more", [0, 5000])
def test_plan_refuses_bad_lengths(new, past, more):
    table = np.arange(2 * (2 + more)).reshape(-1, 2)
    assert check(new + [1] * more, past + [0] * more, table, 0, table.size, 9000) == bd.MAMBA_ERR_SEQLENS


def test_plan_flags_pages_that_are_missing_or_outside_the_pool():
    table = [[0, 1, 2], [3, -1, 4], [5, 99, 6], [-1, 7, 8], [9, 10, 11], [12, -3, 13], [14, -1, 15]]
    # the last state's column past the table; -1; outside the pool; the first state's page; fine; a bad checkpoint; one skipped
    new, past = [40, 8, 8, 8, 8, 24, 24], [8, 8, 8, 8, 8, 0, 0]
    assert check(new, past, table, 8, 16, 200) == bd.MAMBA_ERR_SLOT_RANGE


def test_plan_checkpoints_need_a_start_on_a_border():
    table = np.arange(12).reshape(2, 6)
    assert check([33, 33], [8, 9], table, 8, 12, 66, max_ckpt=5) == 0


@pytest.mark.parametrize("skip", ["has_initial_state", "positions", "token_rows", "ckpt_slots", ("copy_src", "copy_dst"),
                                  ("positions", "token_rows")])
def test_plan_without_some_outputs(skip):
    new, past, table = batch(41, 50, 16, 40, 8)
    assert check(new, past, table, 16, table.size, 3000, skip=(skip,) if isinstance(skip, str) else skip) == 0


def test_plan_of_no_rows():
    import torch
    cu = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    bd.mamba_batch_plan(none, none, none.view(0, 1), 8, 4, cu_seqlens=cu, slot_ids=none, positions=pos)
    assert cu.tolist() == [0] and pos.tolist() == [-1] * 4
