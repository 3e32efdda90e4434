"""The 8-bit paged cache's calls at the ends of what their descriptions allow."""
import numpy as np
import pytest

from tests import kv8_ref as R
from tests.test_gpu_kv8 import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


@pytest.mark.parametrize("pages,before,huge,after", [(64, [20, 0, 33], 17, [3, 40, 0, 5]), (5, [100], 33, [7]), (2100, [], 16, [1, 1])])
def test_growth_past_32_bits_of_pages(torch, pages, before, huge, after):
    """Rows that ask for 2^27 pages each, 2^31 and more together, which the pool
    does not have: they stay as they were, like every later row that needs a
    page; the rows before them, and those that need none, grow."""
    from scratch_decoder_only_b200.kv8 import KV8Pool
    P, wide = 16, 2 ** 27 - 16
    rows = len(before) + huge + len(after) + 1
    table = torch.empty(rows, wide, dtype=torch.int32, device="cuda")     # (only its first columns are looked at)
    table[:, :200] = -1
    lens, ref = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    pool = KV8Pool(table, lens, ref, P)
    # the last row has room for its token
    lens[-1], table[-1, 0], ref[2] = 15, 2, 1
    add = np.array(before + [wide * P] * huge + after + [1], np.int64)
    pool.extend(i32(torch, add))
    want = R.Pool(rows, 200, pages, P)
    want.lens[-1], want.t[-1, 0], want.ref[2] = 15, 2, 1
    n = len(before)
    want.extend(np.where(np.arange(rows) < n, add, 0))     # (a row before them may find too few pages too)
    want.lens[-1] = 16
    assert pool.status() == 32
    assert np.array_equal(lens.cpu().numpy(), want.lens) and np.array_equal(ref.cpu().numpy(), want.ref)
    assert np.array_equal(table[:, :200].cpu().numpy(), want.t)
    # and a row that asks for one page more than there are, by itself
    add = np.zeros(rows, np.int64)
    add[n], add[n + 1] = (pages + 1) * P, 1
    pool.extend(i32(torch, add))
    assert pool.status() == 32 and np.array_equal(lens.cpu().numpy(), want.lens) and np.array_equal(ref.cpu().numpy(), want.ref)
    # all that are left: served
    free = int((want.ref == 0).sum())
    add[n], add[n + 1] = free * P, 0
    pool.extend(i32(torch, add))
    assert pool.status() == 0 and int(lens[n]) == free * P and bool((ref == 1).all())
    assert np.array_equal(table[n, :free].cpu().numpy(), np.nonzero(want.ref == 0)[0])


def test_a_count_without_its_table_is_refused(torch):
    """ref alone, or with one of the two that belong to it, is a ValueError like the other bad descriptions."""
    from scratch_decoder_only_b200.kv8 import KV8Cache
    c = KV8Cache.empty(1, 8, 2, 64, n_rows=3, max_pages=4)
    four = (c.k, c.v, c.k_scale, c.v_scale)
    for more in (dict(ref=c.ref), dict(table=c.table, ref=c.ref), dict(lens=c.lens, ref=c.ref),
                 dict(table=c.table, lens=c.lens, ref=c.ref.long())):
        with pytest.raises(ValueError):
            KV8Cache(*four, **more)
    assert KV8Cache(*four, c.table, c.lens, c.ref).pool.n_pages == 8
