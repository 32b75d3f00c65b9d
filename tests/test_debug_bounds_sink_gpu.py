"""The bounds-checking build on small cases of the window attention with sinks, the rotary positions and
the page operations: a zero error word and the usual agreement with the oracle. (No case here is meant to
violate a bound.)"""
import numpy as np
import pytest
import torch

import workloads
from oracle import diffattn_f64 as ora
from tests.parity import bf16_close, grad_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg():
    """The binding's wrappers, calling into the bounds-checking library for this module."""
    import differential_attention_v2_b200 as da
    from differential_attention_v2_b200 import _lib
    from differential_attention_v2_b200.build import DEBUG_LIB_PATH, build

    assert torch.cuda.is_available()
    build(debug_bounds=True)  # a no-op when the library is up to date
    saved = _lib.LIB
    _lib.LIB = _lib.load(DEBUG_LIB_PATH)
    try:
        yield da
    finally:
        _lib.LIB = saved


def _clean(da):
    torch.cuda.synchronize()
    assert da.device_error() == 0


@pytest.mark.parametrize("S,Hq,Hkv,window,sink", [(1, 2, 1, 1, 1), (300, 8, 2, 64, 4), (700, 16, 1, 130, 200)])
def test_training_pass_in_bounds(dbg, S, Hq, Hkv, window, sink):
    case = workloads.PrefillCase(B=2, S=S, Hq=Hq, Hkv=Hkv, D=128, seed=S)
    inp = workloads.make_prefill(case)
    inp["dout"] = workloads.make_prefill_grad(case)
    d = {k: v.cuda() for k, v in inp.items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    out, ob, lse = dbg.prefill_train(*x, window=window, sink=sink)
    _clean(dbg)
    grads = dbg.backward(*x, ob, lse, d["dout"], window=window, sink=sink)
    _clean(dbg)
    host = (inp["q"], inp["k"], inp["v"], inp["lam"])
    bf16_close(out, ora.prefill(*host, window=window, sink=sink), "debug sink prefill")
    for g, r, n in zip(grads, ora.prefill_backward(*host, inp["dout"], window=window, sink=sink), "qkvl"):
        grad_close(g, r, f"debug sink d{n}")


def test_packed_training_pass_in_bounds(dbg):
    lens = [300, 1, 0, 129, 64]
    case = workloads.PrefillCase(B=1, S=sum(lens), Hq=8, Hkv=2, D=128, seed=5)
    inp = {k: v[0] for k, v in {**workloads.make_prefill(case), "dout": workloads.make_prefill_grad(case)}.items()}
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    d = {k: v.cuda() for k, v in inp.items()}
    x, tail = (d["q"], d["k"], d["v"], d["lam"]), (cu.cuda(), max(lens))
    out, ob, lse = dbg.prefill_varlen_train(*x, *tail, window=50, sink=4)
    _clean(dbg)
    grads = dbg.backward_varlen(*x, ob, lse, d["dout"], *tail, window=50, sink=4)
    _clean(dbg)
    host = (inp["q"], inp["k"], inp["v"], inp["lam"])
    bf16_close(out, ora.prefill_varlen(*host, cu, window=50, sink=4), "debug packed sink prefill")
    for g, r, n in zip(grads, ora.prefill_backward_varlen(*host, inp["dout"], cu, window=50, sink=4), "qkvl"):
        grad_close(g, r, f"debug packed sink d{n}")


@pytest.mark.parametrize("page", [8, 16, 64])
@pytest.mark.parametrize("Hq,Hkv,window,sink,lens", [(16, 2, 64, 4, [300, 1, 0, 69]), (32, 2, 100, 70, [900, 171])])
def test_decode_in_bounds(dbg, Hq, Hkv, window, sink, lens, page):
    smax = -(-max(lens) // page) * page
    inp = workloads.make_decode(workloads.DecodeCase(B=len(lens), Smax=smax, Hq=Hq, Hkv=Hkv, D=128, len_lo=1, len_hi=smax,
                                                     seed=page))
    n = torch.tensor(lens, dtype=torch.int32)
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], n, inp["lam"], window=window, sink=sink)
    out = dbg.decode(d["q"], d["kcache"], d["vcache"], n.cuda(), d["lam"], window=window, sink=sink)
    _clean(dbg)
    bf16_close(out, ref, "debug sink decode")
    B, per = len(lens), smax // page
    shape = (B * per, page, Hkv, 128)
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    out = dbg.decode_paged(d["q"], d["kcache"].view(shape), d["vcache"].view(shape), table, n.cuda(), d["lam"],
                           window=window, sink=sink)
    _clean(dbg)
    bf16_close(out, ref, "debug paged sink decode")


def test_rotary_append_and_pages_in_bounds(dbg):
    B, page, N = 4, 8, 40
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    new = torch.tensor([20, 9, 0, 0], dtype=torch.int32, device="cuda")
    assert dbg.cache_extend(table, seqlens, refs, new, page).item() == 5
    q, k, v = (torch.randn(29, h, 128, device="cuda").bfloat16() for h in (4, 2, 2))
    kc, vc = (torch.zeros(N, page, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(29, dtype=torch.int32, device="cuda")[None]
    inv = torch.rand(64, device="cuda")
    cu = torch.tensor([0, 20, 29, 29, 29], dtype=torch.int32, device="cuda")
    dbg.rope_append_paged(q, k, v, pos, inv, (64,), kc, vc, table, seqlens, cu_seqlens=cu)
    kr = dbg.rope(k, None, pos, inv, (64,))[0]
    rows = kc[table[0, :3].long()].flatten(0, 1)[:20]
    assert torch.equal(rows, kr[:20])
    copies, took = dbg.cache_fork(table, seqlens, refs, new[:1] * 0, new[:1] * 0 + 2, page)
    assert took.item() == 1
    dbg.cache_copy_pages(kc, vc, copies)
    assert torch.equal(kc[table[2, :3].long()].flatten(0, 1)[:20], kr[:20])
    dbg.cache_trim(table, seqlens, refs, page, 4, 1)
    dbg.cache_free(table, seqlens, refs, new[:1] * 0)
    table, refs, moves, live = dbg.cache_compact(table, refs)
    dbg.cache_copy_pages(kc, vc, moves)
    last = table[2, 2].item()
    assert torch.equal(kc[last, :4], kr[16:20])
    _clean(dbg)
