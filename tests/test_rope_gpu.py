"""Rotary positions with several axes on the GPU, alone and fused with the write to a paged cache,
against complex rotations in 64 bits.

Tolerances. The angle reaches sincospif as a fraction of a turn in fp32, |2t| <= 1, rounded by at most
half a step: pi * 2^-25 * 2 radians at most, 1.9e-7; sincospif adds 2 ulp (2^-23 of 1). Two products
and a sum of fp32 add three roundings of 2^-24 each: |error| <= (|a| + |b|) * (1.9e-7 + 2.4e-7 + 1.8e-7)
< 1e-6 * (|a| + |b|). bf16 outputs add half a step of the result, 2^-8 of it at most (2^-9 relative to the
binade's top; the bound used is torch.finfo(bfloat16).eps / 2 = 2^-8).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def _turn(x, positions, inv_freq, sections, inverse=False, interleaved=False):
    """[T, H, D] fp64: every pair times exp(+-i angle)."""
    P = sum(sections)
    ang = torch.cat([positions[a].double()[:, None] * f.double() for a, f in
                     enumerate(torch.split(inv_freq.cpu(), list(sections)))], 1)
    z = torch.exp(1j * (-ang if inverse else ang))[:, None]
    y = x.double().cpu().clone()
    a, b = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    w = torch.complex(y[..., a].clone(), y[..., b].clone()) * z
    y[..., a], y[..., b] = w.real, w.imag
    return y


def _close(got, ref, x):
    assert got.shape == ref.shape
    reach = 2 * x.double().abs().amax(-1, keepdim=True).cpu()
    tol = 1e-6 * reach + (torch.finfo(torch.bfloat16).eps / 2 * ref.abs() if got.dtype == torch.bfloat16 else 0)
    assert bool(((got.double().cpu() - ref).abs() <= tol).all())


def _inputs(T, Hq, Hkv, D, sections, dtype, seed, far=200000):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hq, D, generator=g).to(dtype)
    k = torch.randn(T, max(Hkv, 1), D, generator=g).to(dtype)
    pos = torch.randint(-5, far, (len(sections), T), generator=g).int()
    P = sum(sections)
    inv = (10000.0 ** (-torch.arange(P).double() / P)).float()
    return q, k, pos, inv


CASES = [
    # T, Hq, Hkv, D, sections
    (1, 2, 1, 128, (64,)),
    (5, 64, 8, 128, (16, 24, 24)),
    (130, 4, 2, 128, (8, 0, 16)),        # an empty section, dimensions that pass through
    (33, 6, 3, 64, (8, 12, 12)),
    (17, 4, 1, 96, (5, 7, 3)),           # odd sections: one pair at a time
    (9, 2, 2, 80, (2, 4, 6, 8)),         # four axes, two pairs at a time
    (3, 2, 1, 2, (1,)),                  # the smallest head
    (2, 2, 1, 512, (100, 100, 56)),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,sections", CASES)
def test_rope_matches_complex_rotations(da, T, Hq, Hkv, D, sections, dtype, interleaved):
    q, k, pos, inv = _inputs(T, Hq, Hkv, D, sections, dtype, seed=T + D)
    for inverse in (False, True):
        qo, ko = da.rope(q.cuda(), k.cuda(), pos.cuda(), inv.cuda(), sections, inverse=inverse, interleaved=interleaved)
        for got, x in ((qo, q), (ko, k)):
            _close(got, _turn(x, pos, inv, sections, inverse, interleaved), x)


def test_far_positions(da):
    q, k, pos, inv = _inputs(40, 2, 1, 128, (64,), torch.float32, seed=3)
    pos[0, :] = 2**31 - 1 - torch.arange(40).int()
    pos[0, 20:] = -(2**31) + torch.arange(20).int()
    qo, _ = da.rope(q.cuda(), None, pos.cuda(), inv.cuda(), (64,))
    # positions of 2^31: the product of position and frequency rounds by 2^-53 of up to 2^31, 2.4e-7
    ref = _turn(q, pos, inv, (64,))
    assert float((qo.double().cpu() - ref).abs().max()) <= 2e-6 * 2 * float(q.abs().max())


def test_strided_inputs_in_place_and_odd_alignment(da):
    T, Hq, Hkv, D, sections = 21, 6, 2, 128, (16, 24, 24)
    q, k, pos, inv = _inputs(T, Hq, Hkv, D, sections, torch.bfloat16, seed=8)
    ref_q, ref_k = _turn(q, pos, inv, sections), _turn(k, pos, inv, sections)
    for pad in (0, 8, 2, 1):  # the columns start at 16-, 4- and 2-byte boundaries
        wide = torch.zeros(T, pad + (Hq + Hkv) * D, dtype=torch.bfloat16, device="cuda")
        qv, kv = wide[:, pad: pad + Hq * D].view(T, Hq, D), wide[:, pad + Hq * D:].view(T, Hkv, D)
        qv.copy_(q)
        kv.copy_(k)
        a, b = da.rope(qv, kv, pos.cuda(), inv.cuda(), sections)
        _close(a, ref_q, q)
        _close(b, ref_k, k)
        a, b = da.rope(qv, kv, pos.cuda(), inv.cuda(), sections, q_out=qv, k_out=kv)
        assert a.data_ptr() == qv.data_ptr()
        _close(qv, ref_q, q)
        _close(kv, ref_k, k)
        assert torch.count_nonzero(wide[:, :pad]).item() == 0


def test_inverse_is_the_gradient(da):
    """<rope(x + h e) - rope(x - h e), g> / 2h = <e, rope(g, inverse)>, exactly linear."""
    T, H, D, sections = 7, 3, 32, (6, 10)
    q, _, pos, inv = _inputs(T, H, 1, D, sections, torch.float32, seed=4)
    g, e = torch.randn(T, H, D), torch.randn(T, H, D)
    run = lambda x, **kw: da.rope(x.cuda(), None, pos.cuda(), inv.cuda(), sections, **kw)[0].double().cpu()  # noqa: E731
    diff = ((run(q + e) - run(q - e)) / 2 * g.double()).sum()
    grad = (run(g, inverse=True) * e.double()).sum()
    # each side sums T*H*D terms of size about 1 with errors below 1e-6 * 2 * max
    assert abs(float(diff - grad)) <= T * H * D * 1e-6 * 2 * 4 * 4


def test_empty_and_refused(da):
    q, k, pos, inv = (t.cuda() for t in _inputs(4, 2, 1, 64, (16, 16), torch.bfloat16, seed=1))
    a, b = da.rope(q[:0], k[:0], pos[:, :0].contiguous(), inv, (16, 16))
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)
    with pytest.raises(ValueError):
        da.rope(q, k, pos, inv, (32,))            # one axis, two rows of positions
    with pytest.raises(ValueError):
        da.rope(q, k, pos, inv[:20], (16, 16))    # frequencies and sections disagree
    with pytest.raises(da.DiffAttnError):
        da.rope(q, k, pos, torch.ones(40, device="cuda"), (20, 20))  # more pairs than D / 2
    with pytest.raises(da.DiffAttnError):
        da.rope(q, k, torch.zeros(5, 4, dtype=torch.int32, device="cuda"), inv[:5].contiguous(), (1,) * 5)
    with pytest.raises(TypeError):
        da.rope(q.half(), k, pos, inv, (16, 16))
    with pytest.raises(ValueError):
        da.rope(q.transpose(0, 1), None, pos, inv, (16, 16))
    assert da.device_error() == 0


# ----------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,page", [([1, 1, 1], 16), ([7, 0, 30, 1], 8), ([100, 3], 64), ([1], 8)])
def test_append_writes_the_right_rows_and_no_others(da, new, page, dtype):
    B, Hq, Hkv, D, sections = len(new), 4, 2, 128, (16, 24, 24)
    T = sum(new)
    q, k, pos, inv = _inputs(T + 2, Hq, Hkv, D, sections, dtype, seed=T + page)
    v = torch.randn(T + 2, Hkv, D, generator=torch.Generator().manual_seed(5)).to(dtype)
    g = torch.Generator().manual_seed(6)
    old = torch.randint(0, 50, (B,), generator=g)
    per = (50 + max(new)) // page + 1
    table = torch.randperm(B * per + 3, generator=g)[: B * per].view(B, per).int()
    kc = torch.randn(B * per + 3, page, Hkv, D, generator=g).to(dtype)
    vc = torch.randn(B * per + 3, page, Hkv, D, generator=g).to(dtype)
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist()).int()
    seqlens = (old + torch.tensor(new)).int()
    kd, vd, qo = kc.cuda(), vc.cuda(), torch.full((T + 2, Hq, D), 9.0, dtype=dtype, device="cuda")
    # two rows behind the last sequence
    da.rope_append_paged(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), inv.cuda(), sections, kd, vd, table.cuda(),
                         seqlens.cuda(), cu_seqlens=cu.cuda(), q_out=qo)
    assert bool((qo[T:] == 9.0).all())
    _close(qo[:T], _turn(q, pos, inv, sections)[:T], q[:T])
    turned = _turn(k, pos, inv, sections)
    seen = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b in range(B):
        for i in range(new[b]):
            at, t = int(old[b]) + i, int(cu[b]) + i
            pg, r = int(table[b, at // page]), at % page
            seen[pg, r] = True
            _close(kd[pg, r], turned[t], k[t])
            assert torch.equal(vd[pg, r].cpu(), v[t])
    assert torch.equal(kd.cpu()[~seen], kc[~seen]) and torch.equal(vd.cpu()[~seen], vc[~seen])
    assert da.device_error() == 0


def test_append_one_token_each_and_without_a_page(da):
    B, Hq, Hkv, D, page, sections = 4, 4, 2, 128, 8, (64,)
    q, k, pos, inv = (t.cuda() for t in _inputs(B, Hq, Hkv, D, sections, torch.bfloat16, seed=2))
    v = torch.randn(B, Hkv, D, device="cuda").bfloat16()
    kc = torch.zeros(6, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[0, 1], [2, -1], [3, 99], [4, 5]], dtype=torch.int32, device="cuda")
    seqlens = torch.tensor([9, 9, 16, 0], dtype=torch.int32, device="cuda")  # page 1 row 0; none; none; before the start
    qo = da.rope_append_paged(q, k, v, pos, inv, sections, kc, vc, table, seqlens)
    ref_q, ref_k = da.rope(q, k, pos, inv, sections)
    assert torch.equal(qo, ref_q)
    assert torch.equal(kc[1, 0], ref_k[0]) and torch.equal(vc[1, 0], v[0])
    kc[1, 0] = 0
    vc[1, 0] = 0
    assert torch.count_nonzero(kc).item() == 0 and torch.count_nonzero(vc).item() == 0
    long = torch.tensor([17, 9, 16, 0], dtype=torch.int32, device="cuda")  # past the table's row
    da.rope_append_paged(q, k, v, pos, inv, sections, kc, vc, table, long)
    assert torch.count_nonzero(kc).item() == 0
    with pytest.raises(da.DiffAttnError):
        da.rope_append_paged(q, k, v, pos, inv, sections, kc[:, :7].contiguous(), vc[:, :7].contiguous(), table, seqlens)
    with pytest.raises(ValueError):
        da.rope_append_paged(q, k, v, pos, inv, sections, kc, vc, table[:3], seqlens)
    assert da.device_error() == 0
