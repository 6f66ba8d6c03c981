"""build_block_tables against Python integers: equal in every output."""
import random

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref

pytestmark = pytest.mark.gpu


def _run(context, new, width, block, spare, taken=0, pad=0, extra_cols=0, seed=0):
    rng = random.Random(seed)
    R = len(context)
    pool = list(range(R * max(width, 1) + spare + 8))
    rng.shuffle(pool)
    held = [min(-(-max(0, c) // block), width) for c in context]
    table = [[pool.pop() if c < h else -7 for c in range(width)] for h in held]
    need = sum(max(0, min(-(-(max(0, c) + max(0, n)) // block), width) - h) for c, n, h in zip(context, new, held))
    free = pool[: max(0, need + spare)]
    max_tokens = sum(max(0, n) for n in new) + pad
    store = torch.full((R, width + extra_cols), -9, dtype=torch.int32)
    if width:
        store[:, :width] = torch.tensor(table, dtype=torch.int32).reshape(R, width)
    dev = store.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = i8.build_block_tables(i32(context), i32(new), dev[:, :width], i32(free), block, max(0, max_tokens),
                                 taken=i32([taken]) if taken else None)
    i8.sync_check()
    want = ref.tables_reference(context, new, table, free, taken, block, max(0, max_tokens))
    after = dev.cpu()
    if width:
        assert after[:, :width].tolist() == want[0]
    assert (after[:, width:] == -9).all()
    assert plan.cu_new.tolist() == want[1]
    assert plan.seq_lens.tolist() == want[2]
    assert plan.slots.tolist() == want[3]
    assert plan.positions.tolist() == want[4]
    assert plan.counts.tolist() == want[5]


@pytest.mark.parametrize("block", [16, 48, 64])
@pytest.mark.parametrize("R", [1, 2, 31, 64, 511, 512, 513, 2048])
def test_random_steps(R, block):
    rng = random.Random(R * 7 + block)
    context = [rng.choice([0, 0, 1, block - 1, block, block + 1, rng.randrange(400)]) for _ in range(R)]
    new = [rng.choice([0, 1, 1, 1, block, rng.randrange(90)]) for _ in range(R)]
    width = max(-(-(c + n) // block) for c, n in zip(context, new)) + 1
    _run(context, new, width, block, 5, taken=3, pad=rng.randrange(9), extra_cols=2, seed=R)


def test_edges():
    _run([0], [0], 1, 16, 0)                       # nothing to do
    _run([0, 0, 0], [0, 0, 0], 2, 16, 0, pad=5)    # empty requests, padded buffers
    _run([0, 5, 0, 7], [0, 1, 0, 0], 3, 16, 0)     # one token between empty requests
    _run([15, 16, 17], [1, 1, 1], 2, 16, 0)        # a block's last, first and second offset
    _run([-3, 4], [2, -1], 2, 16, 0)               # negative lengths count as 0
    _run([0], [100000], 6250, 16, 0)               # one long request
    _run([70000, 1], [1, 1], 1100, 64, 0)


def test_free_list_or_width_runs_out():
    _run([0, 0, 10], [40, 40, 30], 4, 16, -2)      # two blocks short
    _run([0, 0], [40, 40], 4, 16, -6)              # an empty free list
    _run([0, 30], [40, 40], 2, 16, 0)              # tables too narrow
    _run([0], [40], 0, 16, 0)                      # no columns at all
    _run([0, 0], [64, 64], 8, 16, 0, taken=5)      # the list's tail is short by what is taken
    _run([0], [20], 2, 16, 0, taken=50)            # taken past the list's end


def test_capacity_smaller_than_the_step():
    _run([3, 4], [50, 60], 8, 16, 0, pad=-37)
    _run([3, 4], [50, 60], 8, 16, 0, pad=-110)


def test_most_requests_and_graph():
    R = 16384
    rng = random.Random(1)
    context, new = [rng.randrange(100) for _ in range(R)], [rng.randrange(3) for _ in range(R)]
    _run(context, new, 8, 16, 1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    c, n, free = i32([10, 0, 33]), i32([1, 1, 1]), i32(list(range(50, 60)))
    table = i32([[1, -1, -1], [-1, -1, -1], [2, 3, 4]])
    out = i8.BlockPlan.empty(3, 8)
    i8.build_block_tables(c, n, table.clone(), free, 16, 8, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i8.build_block_tables(c, n, table, free, 16, 8, out=out)
    n.copy_(i32([7, 2, 0]))
    graph.replay()
    i8.sync_check()
    want = ref.tables_reference([10, 0, 33], [7, 2, 0], [[1, -1, -1], [-1, -1, -1], [2, 3, 4]], list(range(50, 60)), 0, 16, 8)
    assert [table.tolist(), out.cu_new.tolist(), out.seq_lens.tolist(), out.slots.tolist(), out.positions.tolist(),
            out.counts.tolist()] == list(want)


def test_operands_between_the_table_s_rows():
    """Vectors in the gaps of a row-strided table share no memory with it."""
    R, width, ld = 3, 2, 16
    buf = torch.full((R, ld), -9, dtype=torch.int32, device="cuda")
    table, context, new, free = buf[:, :width], buf[0, 2:5], buf[1, 2:5], buf[2, 2:8]
    context.copy_(torch.tensor([0, 5, 17]))
    new.copy_(torch.tensor([1, 1, 3]))
    free.copy_(torch.tensor([11, 12, 13, 14, 15, 16]))
    table.copy_(torch.tensor([[-7, -7], [3, -7], [4, 5]]))
    plan = i8.build_block_tables(context, new, table, free, 16, 5)
    i8.sync_check()
    want = ref.tables_reference([0, 5, 17], [1, 1, 3], [[-7, -7], [3, -7], [4, 5]], [11, 12, 13, 14, 15, 16], 0, 16, 5)
    assert table.tolist() == want[0] and plan.slots.tolist() == want[3] and plan.counts.tolist() == want[5]


def test_kept_in_place_is_refused():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = i8.BlockPlan.empty(2, 4)
    table, free = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda")
    plan.seq_lens.copy_(i32([1, 2]))
    plan.counts.copy_(i32([0, 0, 0]))
    for args, kw in (((plan.seq_lens, i32([1, 1])), {}), ((i32([1, 2]), i32([1, 1])), {"taken": plan.counts[1:2]})):
        with pytest.raises(i8.I8Error) as e:
            i8.build_block_tables(*args, table, free, 16, 4, out=plan, **kw)
        assert e.value.status == 1
