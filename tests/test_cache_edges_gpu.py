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


@pytest.mark.parametrize("page", [8, 64, 4096])
def test_free_and_trim_of_shared_pages(da, page):
    """Pages that branches share come back when the last of them lets go."""
    m, p = Model(6, 5, 40, page), Pool(6, 5, 40)
    ext = [3 * page, 2 * page + 5, 0, 0, 0, 0]
    assert da.cache_extend(p.table, p.L, p.refs, _ints(ext), page).tolist() == [m.extend(ext)]
    for a, c in (([0, 0, 1], [2, 3, 4]), ([4, -1], [5, 5])):  # two of sequence 0, a chain from 1 to 4 to 5
        copies, got = da.cache_fork(p.table, p.L, p.refs, _ints(a), _ints(c), page)
        ref, res = m.fork(a, c)
        assert got.tolist() == [res] and [tuple(x) for x in copies.tolist()] == ref
        p.same(m)
    for op in ("free 0 0 -1", "trim", "free 4", "free 2 3", "free 1 5 5"):
        if op == "trim":
            got, want = da.cache_trim(p.table, p.L, p.refs, page, page, 1), m.trim(page, 1)
        else:
            seqs = [int(x) for x in op.split()[1:]]
            got, want = da.cache_free(p.table, p.L, p.refs, _ints(seqs)), m.free(seqs)
        assert got.tolist() == [want], op
        p.same(m)
    assert p.refs.eq(0).all() and p.table.eq(-1).all()


def test_pairs_read_the_state_before_the_call(da):
    """A child that is also a parent was empty when the call began, so its own child stays empty."""
    for a, c in (([0, 1], [1, 2]), ([1, 0], [2, 1])):
        m, p = Model(3, 4, 9, 8), Pool(3, 4, 9)
        da.cache_extend(p.table, p.L, p.refs, _ints([12, 0, 0]), 8)
        m.extend([12, 0, 0])
        copies, got = da.cache_fork(p.table, p.L, p.refs, _ints(a), _ints(c), 8)
        assert got.tolist() == [1] and p.L.tolist() == [12, 12, 0]
        assert p.table[2].eq(-1).all() and p.table[1].tolist() == [0, 2, -1, -1] and p.refs[:3].tolist() == [2, 1, 1]
        assert copies.tolist() == ([[1, 2], [-1, -1]] if a[0] == 0 else [[-1, -1], [1, 2]])


def test_a_serving_loop_in_a_graph(da):
    """Extend, trim, free and fork captured once and replayed on the state as it moves on."""
    m, p = Model(4, 12, 60, 8), Pool(4, 12, 60)
    grow, drop = _ints([5, 3, 0, 0]), _ints([2, -1])
    parents, children = _ints([0, -1]), _ints([2, 3])

    def step():
        r = [da.cache_extend(p.table, p.L, p.refs, grow, 8), da.cache_free(p.table, p.L, p.refs, drop)]
        copies, took = da.cache_fork(p.table, p.L, p.refs, parents, children, 8)
        return [*r, copies, took, da.cache_trim(p.table, p.L, p.refs, 8, 20, 3)]

    def model():
        r = [[m.extend([5, 3, 0, 0])], [m.free([2, -1])]]
        copies, took = m.fork([0, -1], [2, 3])
        return [*r, [list(c) for c in copies], [took], [m.trim(20, 3)]]

    assert [t.tolist() for t in step()] == model()
    torch.cuda.synchronize()
    state = [t.clone() for t in (p.table, p.L, p.refs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, s in zip((p.table, p.L, p.refs), state):
        t.copy_(s)
    for _ in range(12):
        graph.replay()
        torch.cuda.synchronize()
        assert [t.tolist() for t in out] == model()
        p.same(m)
