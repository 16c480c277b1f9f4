"""Lists of free pages that run out where the host does not know it: behind the pages that are free a list holds -1, no page of an
earlier list, and the calls that take from it report it."""
import numpy as np
import pytest

import decode_reference as ref
import page_reference as pages
from test_decode_gpu import dev, kvx, slot_inputs, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def ints(*shape, fill=-7, dtype=torch.int32):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


@pytest.mark.parametrize("n,ctx_hi,new_hi", [(1, 0, 40), (16, 900, 1), (300, 500, 90), (1025, 40, 3), (3000, 200, 200)])
@pytest.mark.parametrize("bs", [1, 16, 24])
def test_slot_map_of_a_list_that_ends_in_negative_ids(n, ctx_hi, new_hi, bs):
    ctx, new, free, table = slot_inputs(n, bs, ctx_hi, new_hi, n + bs)
    new[0] += bs + 1                                                       # some block is taken
    width, total = table.shape[1] + 3, int(new.sum())
    table = np.concatenate([table, np.full((n, width - table.shape[1]), -1, np.int32)], 1)
    ids = np.concatenate([free, 10 ** 6 + np.arange(2 * n + 9, dtype=np.int32)])
    taken = ref.slot_map(ctx, new, bs, ids, table, width, total)[6]
    assert 0 < taken <= len(ids)
    for held in (taken, taken - 1, taken // 2, 0):
        short = np.where(np.arange(len(ids)) < held, ids, -1).astype(np.int32)
        want = ref.slot_map(ctx, new, bs, short, table, width, total)
        d_table, result = dev(table), ints(3, dtype=torch.int64)
        tok_off, slots, seq = ints(n + 1, dtype=torch.int64), ints(total, dtype=torch.int64), ints(n)
        kvx.kvx_slot_map(dev(ctx), dev(new), n, bs, dev(short), len(short), d_table, width, width, total, tok_off, slots, None, seq, result)
        assert result.tolist() == [want[5], taken, kvx.KVX_OK if held == taken else kvx.KVX_ERANGE]
        assert np.array_equal(slots.cpu().numpy(), want[1]) and np.array_equal(d_table.cpu().numpy(), want[4])
        assert (held == taken) == bool((want[1] >= 0).all())


def test_captured_steps_until_a_pool_runs_out():
    """Free list, slots and tokens of a decode step, captured once. While pages are left no two rows hold one; when they run out the step
    says so and gives none away."""
    bs, width, n, n_blocks = 4, 12, 6, 40
    table, ctx, seq = ints(n, width, fill=-1), ints(n, fill=0), ints(n, fill=0)
    one = ints(n, fill=1)
    refs, free = ints(n_blocks), ints(n_blocks)
    found, result = ints(3, dtype=torch.int64), ints(3, dtype=torch.int64)
    tok_off, slots, positions = ints(n + 1, dtype=torch.int64), ints(n, dtype=torch.int64), ints(n)
    side = torch.cuda.Stream()

    def step():
        ctx.copy_(seq)
        free.fill_(-1)
        kvx.kvx_pages_free(table, width, width, ctx, n, bs, n_blocks, refs, free, found, side)
        kvx.kvx_slot_map(ctx, one, n, bs, free, n, table, width, width, n, tok_off, slots, positions, seq, result, side)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    ran_out = 0
    for t in range(width * bs):
        before, lens = table.cpu().numpy(), seq.cpu().numpy()
        _, ids, _ = pages.free(before, lens, bs, n_blocks)
        graph.replay()
        torch.cuda.synchronize()
        need = n if t % bs == 0 else 0                                     # every request begins a page at the same step
        now = table.cpu().numpy()
        if len(ids) >= need:
            assert result[2].item() == kvx.KVX_OK and (slots >= 0).all()
            held = np.concatenate([now[r, :-(-(t + 1) // bs)] for r in range(n)])
            assert len(np.unique(held)) == len(held) and (held >= 0).all()
        else:
            ran_out += 1
            assert result.tolist() == [n, need, kvx.KVX_ERANGE]
            got = now[:, t // bs]
            assert got.tolist() == ids.tolist() + [-1] * (n - len(ids)) and (slots[len(ids):] == -1).all()
            break
    assert ran_out == 1 and t == n_blocks // n * bs                        # 36 pages of 6 rows, then 4 for 6


def test_captured_fork_of_a_pool_that_runs_out():
    """Six rows of one request with a page in part filled take five pages of their own; of fewer that are free none is given twice."""
    bs, width, n, n_blocks = 16, 5, 6, 12
    table, lens = ints(n, width, fill=-1), ints(n, fill=0)
    parent = ints(n, fill=0)
    refs, free, found = ints(n_blocks), ints(n_blocks), ints(3, dtype=torch.int64)
    new, new_len, src, dst, scratch, result = ints(n, width), ints(n), ints(n), ints(n), ints(n), ints(3, dtype=torch.int64)
    side = torch.cuda.Stream()

    def step():
        free.fill_(-1)
        kvx.kvx_pages_free(table, width, width, lens, n, bs, n_blocks, refs, free, found, side)
        kvx.kvx_pages_fork(table, width, width, lens, n, parent, n, bs, free, n, new, width, new_len, src, dst, scratch, result, side)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for others in (0, 1, 3, 4):                                            # pages that a second request holds: 8, 7, 5, 4 are left
        t = np.full((n, width), -1, np.int32)
        t[0, :4] = (3, 1, 7, 5)
        t[1, :others] = (0, 2, 4, 6)[:others]
        length = np.array([60, others * bs, 0, 0, 0, 0], np.int32)
        table.copy_(dev(t))
        lens.copy_(dev(length))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        left = np.setdiff1d(np.arange(n_blocks), t)
        got = new[:, 3].cpu().numpy()
        assert got[0] == 5 and got[1:].tolist() == (left.tolist() + [-1] * n)[:n - 1]
        assert result[2].item() == (kvx.KVX_OK if len(left) >= n - 1 else kvx.KVX_ERANGE)
