"""Rotary positions at their edges: calls that the first tests do not make."""
import pytest
import torch

from tests.test_rope_gpu import _close, _inputs, _turn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def test_an_output_without_its_input_is_refused(da):
    q, k, pos, inv = (t.cuda() for t in _inputs(4, 2, 1, 64, (16, 16), torch.bfloat16, seed=1))
    out = torch.full_like(k, 3.0)
    with pytest.raises(ValueError):
        da.rope(q, None, pos, inv, (16, 16), k_out=out)
    torch.cuda.synchronize()
    assert out.eq(3.0).all()
    assert da.rope(q, None, pos, inv, (16, 16))[1] is None


def _append_case(Hq, Hkv, D, sections, new, page, dtype, seed):
    B, T = len(new), sum(new)
    g = torch.Generator().manual_seed(seed)
    q, k, pos, inv = _inputs(T, Hq, Hkv, D, sections, dtype, seed=seed)
    v = torch.randn(T, Hkv, D, generator=g).to(dtype)
    old = torch.randint(0, 60, (B,), generator=g)
    per = (60 + max(new)) // page + 1
    N = B * per + 2
    table = torch.randperm(N, generator=g)[: B * per].view(B, per).int()
    kc, vc = (torch.randn(N, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist()).int()
    rows = []  # (page, row) of every token
    for b, n in enumerate(new):
        at = [int(old[b]) + i for i in range(n)]
        rows += [(int(table[b, a // page]), a % page) for a in at]
    return q, k, v, pos, inv, kc, vc, table, (old + torch.tensor(new)).int(), cu, rows


def _check_append(da, case, sections, interleaved, wrap=lambda t: t.cuda()):
    """`wrap` puts q, k and v into the memory that the call reads them from."""
    q, k, v, pos, inv, kc, vc, table, seqlens, cu, rows = case
    kd, vd = kc.cuda(), vc.cuda()
    qo = da.rope_append_paged(wrap(q), wrap(k), wrap(v), pos.cuda(), inv.cuda(), sections, kd, vd, table.cuda(),
                              seqlens.cuda(), cu_seqlens=cu.cuda(), interleaved=interleaved)
    _close(qo, _turn(q, pos, inv, sections, interleaved=interleaved), q)
    turned = _turn(k, pos, inv, sections, interleaved=interleaved)
    pg, r = (torch.tensor(x) for x in zip(*rows))
    _close(kd[pg.cuda(), r.cuda()], turned, k)
    assert torch.equal(vd.cpu()[pg, r], v)
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    seen[pg, r] = True
    assert torch.equal(kd.cpu()[~seen], kc[~seen]) and torch.equal(vd.cpu()[~seen], vc[~seen])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D,sections", [
    (4, 2, 128, (16, 24, 24)), (64, 8, 128, (64,)), (6, 3, 64, (8, 0, 16)), (4, 1, 96, (5, 7, 3)), (2, 2, 80, (2, 4, 6, 8)),
    (2, 1, 2, (1,)), (16, 4, 512, (100, 100, 56)), (3, 5, 128, (16, 16)),
])
def test_append_of_every_shape(da, Hq, Hkv, D, sections, dtype, interleaved):
    """Vectors of every width, both pairings, both types; heads that pass through in part; more KV heads than
    query heads."""
    new, page = ([1, 1, 1], 16) if D == 128 and Hq == 64 else ([7, 0, 40, 1], 8)
    _check_append(da, _append_case(Hq, Hkv, D, sections, new, page, dtype, seed=D + Hq), sections, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 4, 1])
def test_append_of_columns_at_any_alignment(da, pad, interleaved):
    sections = (16, 24, 24)
    case = _append_case(4, 2, 128, sections, [33, 2], 64, torch.bfloat16, seed=pad)

    def columns(t):
        wide = torch.zeros(t.shape[0], pad + t[0].numel() + 3 * pad, dtype=t.dtype, device="cuda")
        view = wide[:, pad: pad + t[0].numel()].view(t.shape)
        view.copy_(t)
        return view

    _check_append(da, case, sections, interleaved, wrap=columns)


def test_append_to_many_sequences(da):
    """More sequences than a warp has lanes, empty ones among them."""
    g = torch.Generator().manual_seed(4)
    new = torch.randint(0, 4, (150,), generator=g).tolist()
    _check_append(da, _append_case(4, 2, 128, (64,), new, 8, torch.bfloat16, seed=9), (64,), False)


def test_rope_and_append_in_a_graph(da):
    """Captured once and replayed on other lengths and pages, as a decode step is."""
    sections, B, page = (16, 24, 24), 5, 8
    q, k, pos, inv = (t.cuda() for t in _inputs(B, 4, 2, 128, sections, torch.bfloat16, seed=6))
    v = torch.randn(B, 2, 128, device="cuda").bfloat16()
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    lens = torch.tensor([1, 5, 9, 30, 32], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(B * 4, page, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def step():
        da.rope(q, k, pos, inv, sections, q_out=qo, k_out=ko)
        return da.rope_append_paged(q, k, v, pos, inv, sections, kc, vc, table, lens)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qa = step()
    for shift in range(3):
        kc.zero_()
        table.copy_(table.roll(1, 1))
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        ref_q, ref_k = da.rope(q, k, pos, inv, sections)
        assert torch.equal(qo, ref_q) and torch.equal(qa, ref_q) and torch.equal(ko, ref_k)
        at = (lens - 1).long()
        page_of = table[torch.arange(B, device="cuda"), at // page].long()
        assert torch.equal(kc[page_of, at % page], ref_k)
        kc[page_of, at % page] = 0
        assert torch.count_nonzero(kc).item() == 0
