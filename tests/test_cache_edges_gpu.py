"""Page bookkeeping at its edges, against the list model of the histories' test."""
import pytest
import torch

from tests.test_cache_pages_gpu import Model, Pool, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def test_a_table_without_rows(da):
    """Every index is past its end (-2); padding is nothing to do (0)."""
    p = Pool(0, 4, 6)
    for seqs, want in (([0], -2), ([-1, 3], -2), ([-1, -5], 0), ([], 0)):
        assert da.cache_free(p.table, p.L, p.refs, _ints(seqs)).tolist() == [want]
    for a, c, want in (([0], [1], -2), ([-1, 0], [0, 0], -2), ([-1, 0], [0, -1], 0), ([], [], 0)):
        copies, res = da.cache_fork(p.table, p.L, p.refs, _ints(a), _ints(c), 8)
        assert res.tolist() == [want] and copies.shape == (len(a), 2) and copies.eq(-1).all()
    assert da.cache_extend(p.table, p.L, p.refs, _ints([]), 8).tolist() == [0]
    assert da.cache_trim(p.table, p.L, p.refs, 8, 4, 1).tolist() == [0]
    p.refs[4] = 1  # a page that no row of this table names
    table, refs, moves, live = da.cache_compact(p.table, p.refs)
    assert table.shape == (0, 4) and live.tolist() == [1] and refs.tolist() == [1, 0, 0, 0, 0, 0]
    assert moves.tolist() == [[4, 0], [-1, -1], [-1, -1]]
    assert da.device_error() == 0
