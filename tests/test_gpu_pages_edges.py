"""Page calls at the edges of their contract, against plain implementations."""
import numpy as np
import pytest
import torch

from paged_block_sparse_kv_b200 import vx
from test_gpu_pages import DEV, Pool, dev, err_word, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 50, 2 ** 31 - 1])
@pytest.mark.parametrize("parent", [[0, 1], [1, 1], [1], [-1, 0]])
def test_update_reports_a_page_outside_the_pool_in_any_old_row(bad, parent):
    """However many children its row has (one: no reference changes), a bad id sets the bit, is passed on and not counted."""
    pool = Pool("int8", 50, Hkv=1, D=64, P=16, seed=9, batch=2)
    table = vx.PageTable(dev([0, 4]), dev([7, bad, 9, 0, 11, 12]), dev([48, 32]), 4)
    refs = np.zeros(50, int)
    refs[[7, 9, 11, 12]] = 1
    new = vx.PageTable(dev(8 * np.arange(len(parent))), torch.full((16,), -5, dtype=torch.int32, device=DEV),
                       torch.zeros(len(parent), dtype=torch.int32, device=DEV), 4)
    new_ref, err = torch.full((50,), -5, dtype=torch.int32, device=DEV), err_word()
    vx.vx_update_table(pool.geo, pool.vx, table, dev(refs), dev(parent), dev(np.zeros(len(parent))), new, new_ref,
                       workspace(pool.geo, 2), err=err)
    assert int(err.item()) == vx.VX_DATA_BAD_PAGE_ID
    old, want, idx = [[7, bad, 9], [11, 12]], refs.copy(), np.full(16, -5)
    for row in old:
        for p in row:
            if p != bad:
                want[p] -= 1
    for i, p in enumerate(parent):
        row = old[p] if p >= 0 else []
        idx[8 * i:8 * i + len(row)] = row
        for page in row:
            if page != bad:
                want[page] += 1
    assert np.array_equal(new.page_indices.cpu().numpy(), idx)
    assert np.array_equal(new_ref.cpu().numpy(), want)
    assert new.seq_lens.tolist() == [[48, 32][p] if p >= 0 else 0 for p in parent]
    pool.check()
