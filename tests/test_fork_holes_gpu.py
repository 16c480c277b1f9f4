"""kvx_pages_fork of rows that lack a page they should hold: reported wherever it stands, and only where a row goes on from it."""
import numpy as np
import pytest

from test_pages_gpu import dev, ints, kvx, torch

pytestmark = pytest.mark.gpu
BS = 4


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def fork(table, lens, parent):
    n, width = table.shape
    n_out = len(parent)
    new, new_len, src, dst, result = ints(n_out, width), ints(n_out), ints(n_out), ints(n_out), ints(3, dtype=torch.int64)
    kvx.kvx_pages_fork(dev(table), width, width, dev(lens), n, dev(np.asarray(parent, np.int32)), n_out, BS, dev(np.arange(9000, 9000 + n_out, dtype=np.int32)),
                       n_out, new, width, new_len, src, dst, ints(n), result)
    return new.cpu().numpy(), result[2].item()


# (row, column): a full page in the middle, the first one, one far into a row, the last page in part filled (of the row that keeps it
# and of those that would copy it), the last page filled to its end
@pytest.mark.parametrize("row,col", [(1, 1), (1, 0), (2, 150), (2, 299), (3, 2), (4, 1)])
@pytest.mark.parametrize("what", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("copies", [1, 3])
def test_a_hole_is_reported(row, col, what, copies):
    lens = np.array([5, 11, 1200, 9, 8, 0], np.int32)
    width = 301
    table = np.full((6, width), -1, np.int32)
    for r, k in enumerate(-(-lens // BS)):
        table[r, :k] = 1000 * r + np.arange(k)
    parent = [p for p in range(6) for _ in range(copies)] + [-1]
    assert fork(table, lens, parent)[1] == kvx.KVX_OK
    table[row, col] = what
    new, status = fork(table, lens, parent)
    assert status == kvx.KVX_ERANGE
    assert (new[row * copies, :-(-lens[row] // BS)] == table[row, :-(-lens[row] // BS)]).all()
    others = [p for p in parent if p != row]
    assert fork(table, lens, others)[1] == kvx.KVX_OK                      # no row goes on from it
    table[row] = np.where(np.arange(width) < col, table[row], -1)
    lens[row] = col * BS                                                   # behind the row's end it is no hole
    assert fork(table, lens, parent)[1] == kvx.KVX_OK


def test_a_hole_in_a_late_row_of_many():
    """More rows than a pass of the kernel takes."""
    n = 20000
    lens = np.full(n, 8, np.int32)
    table = np.arange(2 * n, dtype=np.int32).reshape(n, 2)
    assert fork(table, lens, np.arange(n))[1] == kvx.KVX_OK
    table[n - 3, 0] = -1
    assert fork(table, lens, np.arange(n))[1] == kvx.KVX_ERANGE
