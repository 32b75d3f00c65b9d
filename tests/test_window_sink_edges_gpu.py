"""Window attention with sinks at its edges: no sinks at all, padded packed batches, large and uneven decode
batches, caches past 32 bits."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import diffattn_f64 as ora
from tests.parity import bf16_close, grad_close
from tests.test_window_sink_gpu import _case, _decode_inputs, _grads_close, _hide, _packed, _pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def _ok(da):
    torch.cuda.synchronize()
    assert da.device_error() == 0


@pytest.mark.parametrize("S,Hq,Hkv,window", [(1, 2, 1, 1), (300, 8, 2, 64), (513, 16, 1, 1), (700, 4, 2, 130), (260, 4, 1, 260)])
def test_training_pass_without_sinks(da, S, Hq, Hkv, window):
    """sink = 0 is the window alone, with fp32 O_b."""
    inp = _case(1, S, Hq, Hkv, seed=S + 7)
    d = {k: v.cuda() for k, v in inp.items()}
    x, host = (d["q"], d["k"], d["v"], d["lam"]), (inp["q"], inp["k"], inp["v"], inp["lam"])
    out, ob, lse = da.prefill_train(*x, window=window, sink=0)
    grads = da.backward(*x, ob, lse, d["dout"], window=window, sink=0)
    _ok(da)
    assert ob.dtype == torch.float32
    bf16_close(out, ora.prefill(*host, window=window), "train out")
    _grads_close(grads, ora.prefill_backward(*host, inp["dout"], window=window), f"S={S} W={window}")


def test_packed_training_pass_without_sinks(da):
    lens = [300, 1, 0, 129, 64]
    inp, cu = _packed(lens, 8, 2, seed=3)
    d = {k: v.cuda() for k, v in inp.items()}
    x, host, tail = (d["q"], d["k"], d["v"], d["lam"]), (inp["q"], inp["k"], inp["v"], inp["lam"]), (cu.cuda(), max(lens))
    out, ob, lse = da.prefill_varlen_train(*x, *tail, window=50, sink=0)
    grads = da.backward_varlen(*x, ob, lse, d["dout"], *tail, window=50, sink=0)
    _ok(da)
    bf16_close(out, ora.prefill_varlen(*host, cu, window=50), "train out")
    _grads_close(grads, ora.prefill_backward_varlen(*host, inp["dout"], cu, window=50), "packed")


@pytest.mark.parametrize("page", [0, 8, 16, 64])
@pytest.mark.parametrize("Hq,Hkv,window,sink,lens", [
    (16, 2, 64, 0, [300, 1, 0, 64, 65]),
    (8, 4, 1, 0, [700, 129, 2, 1]),              # the newest key alone
    (16, 1, 40, 3, [20000, 1, 0, 45, 700]),      # one long sequence among short ones
    (4, 1, 9, 24, [int(n) for n in np.random.default_rng(1).integers(0, 90, 200)]),  # many sequences
    (16, 8, 33, 7, [100] * 70),                  # more clusters than SMs
])
def test_decode(da, Hq, Hkv, window, sink, lens, page):
    inp = _decode_inputs(Hq, Hkv, lens, seed=Hq + window + page)
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], inp["seqlens"], inp["lam"], window=window, sink=sink)
    _hide(inp, window, sink)
    if page:
        kp, vp, table = _pages(inp, page, window, sink, seed=page)
        out = da.decode_paged(inp["q"].cuda(), kp.cuda(), vp.cuda(), table.cuda(), inp["seqlens"].cuda(),
                              inp["lam"].cuda(), window=window, sink=sink)
    else:
        d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
        out = da.decode(d["q"], d["kcache"], d["vcache"], d["seqlens"], d["lam"], window=window, sink=sink)
    _ok(da)
    bf16_close(out, ref, "decode")


def test_decode_over_a_contiguous_cache_past_32_bits(da):
    """The last of three sequences lies behind 2^31 elements."""
    B, Smax, Hq, Hkv, n = 3, 1 << 20, 16, 8, 200
    kc = torch.zeros(B, Smax, Hkv, 128, dtype=torch.bfloat16, device="cuda")  # 6.4 GB
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(n, Hkv, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, 128, generator=g, device="cuda").bfloat16()
    lam = torch.rand(B, Hq // 2, generator=g, device="cuda")
    # sequence 2: sinks at its start, the window at the cache's end
    kc[2, :10], vc[2, :10], kc[2, -(n - 10):], vc[2, -(n - 10):] = k[:10], v[:10], k[10:], v[10:]
    lens = torch.tensor([1, 1, Smax], dtype=torch.int32, device="cuda")
    out = da.decode(q, kc, vc, lens, lam, window=n - 10, sink=10)
    _ok(da)
    ref = ora.decode(q[2:].cpu(), k[None].cpu(), v[None].cpu(), [n], lam[2:].cpu(), window=n, sink=0)
    bf16_close(out[2:], ref, "behind 2^31")


@pytest.mark.parametrize("pad", [1, 70, 200])
@pytest.mark.parametrize("sink", [0, 4, 150])
def test_rows_behind_the_last_sequence_are_left_as_they_were(da, sink, pad):
    """A padded packed batch: cu_seqlens ends before the tensors do."""
    lens, Hq, Hkv, window = [150, 0, 61], 8, 2, 40
    inp, cu = _packed([*lens, pad], Hq, Hkv, seed=pad)
    cu, T = cu[:-1].contiguous(), sum(lens)
    d = {k: v.cuda() for k, v in inp.items()}
    x, host = (d["q"], d["k"], d["v"], d["lam"]), [inp[n][:T] for n in ("q", "k", "v", "lam")]
    total, c = T + pad, cu.cuda()
    new = lambda *s, dtype=torch.bfloat16: torch.full((total, *s), 9.0, dtype=dtype, device="cuda")  # noqa: E731
    ref = ora.prefill_varlen(*host, cu, window=window, sink=sink)
    out = new(Hq // 2, 128)
    da.prefill_varlen_window(*x, c, max(lens), window, sink=sink, out=out)
    bf16_close(out[:T], ref, "prefill")
    f32 = dict(dtype=torch.float32)
    train = new(Hq // 2, 128), new(Hq, 128, **f32), new(Hq, **f32)
    da.prefill_varlen_train(*x, c, max(lens), *train, window=window, sink=sink)
    bf16_close(train[0][:T], ref, "train")
    grads = new(Hq, 128), new(Hkv, 128), new(Hkv, 128), new(Hq // 2, **f32)
    args = (len(lens), max(lens), total, Hq, Hkv)
    ws = torch.empty(da.LIB.diffattn_v2_backward_varlen_window_sink_workspace_size(*args, window, sink),
                     dtype=torch.uint8, device="cuda")
    ptr = lambda *ts: [ctypes.c_void_p(t.data_ptr()) for t in ts]  # noqa: E731
    assert da.LIB.diffattn_v2_backward_varlen_window_sink(
        *ptr(*x, train[1], train[2], d["dout"], *grads, c), *args, 128, window, sink, *ptr(ws), ws.numel(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    _ok(da)
    for g, r, n in zip(grads, ora.prefill_backward_varlen(*host, inp["dout"][:T], cu, window=window, sink=sink), "qkvl"):
        grad_close(g[:T], r, f"d{n}")
    for t in (out, *train, *grads):
        assert t[T:].eq(9.0).all()


@pytest.mark.parametrize("lens,window,sink", [([1500, 40, 900], 100, 513), ([1300], 60, 900), ([700, 650], 50, 640)])
def test_packed_training_with_many_sinks(da, lens, window, sink):
    """Sinks past the first 512, sequences shorter than the sinks among them."""
    inp, cu = _packed(lens, 4, 1, seed=sink)
    d = {k: v.cuda() for k, v in inp.items()}
    x, host, tail = (d["q"], d["k"], d["v"], d["lam"]), (inp["q"], inp["k"], inp["v"], inp["lam"]), (cu.cuda(), max(lens))
    out, ob, lse = da.prefill_varlen_train(*x, *tail, window=window, sink=sink)
    grads = da.backward_varlen(*x, ob, lse, d["dout"], *tail, window=window, sink=sink)
    _ok(da)
    bf16_close(out, ora.prefill_varlen(*host, cu, window=window, sink=sink), "train out")
    _grads_close(grads, ora.prefill_backward_varlen(*host, inp["dout"], cu, window=window, sink=sink), f"packed {lens}")


def test_largest_masks_are_the_causal_one(da):
    """Windows and sinks up to the largest int."""
    top = 2**31 - 1
    inp = _case(1, 300, 4, 1, seed=8)
    d = {k: v.cuda() for k, v in inp.items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    ref = da.prefill(*x)
    step = (d["q"][:, -1].clone(), d["k"], d["v"], torch.tensor([300], dtype=torch.int32, device="cuda"),
            d["lam"][:, -1].clone())
    for w, s in ((top, 0), (top, top), (1, top), (300, 5), (5, 300)):
        assert torch.equal(da.prefill_window(*x, w, sink=s), ref)
        out, ob, lse = da.prefill_train(*x, window=w, sink=s)
        bf16_close(out, ora.prefill(inp["q"], inp["k"], inp["v"], inp["lam"]), "train")
        got = da.backward(*x, ob, lse, d["dout"], window=w, sink=s)
        _grads_close(got, ora.prefill_backward(inp["q"], inp["k"], inp["v"], inp["lam"], inp["dout"]), f"{w} {s}")
        bf16_close(da.decode(*step, window=w, sink=s), ora.prefill(inp["q"], inp["k"], inp["v"], inp["lam"])[:, -1], "decode")
    _ok(da)


@pytest.mark.parametrize("Hq,Hkv,B", [(8, 1, 1), (16, 1, 7), (8, 4, 2), (32, 8, 1)])
@pytest.mark.parametrize("window,sink", [(500, 4), (513, 0), (600, 100), (2100, 17)])
def test_decode_of_few_units_by_large_clusters(da, Hq, Hkv, B, window, sink):
    """One to nine (KV head, sequence) units: clusters of 16 CTAs or 8, with lists from two chunks a CTA on,
    one CTA of a shorter sequence left without any."""
    lens = [2500, 700, 1, 520, 0, 2499, 33][:B]
    inp = _decode_inputs(Hq, Hkv, lens, seed=window + B)
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], inp["seqlens"], inp["lam"], window=window, sink=sink)
    _hide(inp, window, sink)
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    out = da.decode(d["q"], d["kcache"], d["vcache"], d["seqlens"], d["lam"], window=window, sink=sink)
    _ok(da)
    bf16_close(out, ref, "few units")


@pytest.mark.parametrize("page", [1024, 4096])
def test_large_pages(da, page):
    """Appended to and decoded from; a page holds the sinks, the window and rows that nobody wrote."""
    Hq, Hkv, n, window, sink = 16, 2, 5000, 700, 9
    g = torch.Generator(device="cuda").manual_seed(page)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, lam = r(n, Hq, 128), r(n, Hkv, 128), r(n, Hkv, 128), torch.rand(1, Hq // 2, generator=g, device="cuda")
    N = -(-n // page) + 2
    kc = torch.full((N, page, Hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    ints = dict(dtype=torch.int32, device="cuda")
    table, lens, refs = torch.full((1, N - 1), -1, **ints), torch.zeros(1, **ints), torch.zeros(N, **ints)
    refs[0] = 1  # taken by another table
    assert da.cache_extend(table, lens, refs, torch.full((1,), n, **ints), page).item() == N - 2
    pos = torch.arange(n, **ints)[None]
    inv = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    qr = da.rope_append_paged(q, k, v, pos, inv, (64,), kc, vc, table, lens, cu_seqlens=torch.tensor([0, n], **ints))
    kr = da.rope(k, None, pos, inv, (64,))[0]
    out = da.decode_paged(qr[-1:].clone(), kc, vc, table, lens, lam, window=window, sink=sink)
    _ok(da)
    ref = ora.decode(qr[-1:].cpu(), kr[None].cpu(), v[None].cpu(), [n], lam.cpu(), window=window, sink=sink)
    bf16_close(out, ref, "large pages")
