"""Sliding-window attention with sinks on the GPU against the float64 oracle: prefill ([B,S] and
packed), training pass, single-token decode over contiguous and paged caches."""
import numpy as np
import pytest
import torch

import workloads
from oracle import diffattn_f64 as ora
from tests.parity import bf16_close, grad_close, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def _case(B, S, Hq, Hkv, seed):
    case = workloads.PrefillCase(B=B, S=S, Hq=Hq, Hkv=Hkv, D=128, seed=seed)
    inp = workloads.make_prefill(case)
    inp["dout"] = workloads.make_prefill_grad(case)
    return inp


def _ok(da):
    torch.cuda.synchronize()
    assert da.device_error() == 0


PREFILL = [
    # B, S, Hq, Hkv, window, sink
    (1, 1, 2, 1, 1, 1),          # one token
    (1, 300, 4, 2, 1, 1),        # each query sees itself and key 0
    (2, 300, 8, 2, 64, 4),       # ragged tail; sinks before the window in the second and third tile
    (1, 513, 16, 1, 100, 64),    # group of 16, window starting inside tiles
    (1, 700, 8, 4, 130, 200),    # sinks over two tiles, the second half covered
    (1, 600, 4, 1, 128, 128),    # a wholly covered sink tile
    (1, 500, 4, 1, 40, 300),     # sinks wider than the window, across tiles
    (1, 400, 4, 1, 400, 3),      # a window of every key: plain causal
    (1, 400, 4, 1, 7, 400),      # sinks of every key: plain causal
    (3, 257, 32, 4, 90, 17),
]


@pytest.mark.parametrize("B,S,Hq,Hkv,window,sink", PREFILL)
def test_prefill_matches_oracle(da, B, S, Hq, Hkv, window, sink):
    inp = _case(B, S, Hq, Hkv, seed=S + window)
    d = {k: v.cuda() for k, v in inp.items()}
    out = da.prefill_window(d["q"], d["k"], d["v"], d["lam"], window, sink=sink)
    _ok(da)
    bf16_close(out, ora.prefill(inp["q"], inp["k"], inp["v"], inp["lam"], window=window, sink=sink), "prefill")


def test_no_sinks_is_the_window(da):
    d = {k: v.cuda() for k, v in _case(2, 500, 8, 2, seed=5).items()}
    a = da.prefill_window(d["q"], d["k"], d["v"], d["lam"], 70, sink=0)
    assert torch.equal(a, da.prefill_window(d["q"], d["k"], d["v"], d["lam"], 70))
    _ok(da)


PACKED = [
    # lengths, Hq, Hkv, window, sink
    ([300, 1, 0, 129, 64], 8, 2, 50, 4),
    ([5], 2, 1, 2, 1),
    ([0, 700, 0, 33], 16, 4, 128, 130),
    ([128, 128, 128], 4, 1, 1, 2),
    ([1] * 5, 4, 2, 3, 3),
]


def _packed(lens, Hq, Hkv, seed):
    inp = {k: v[0] for k, v in _case(1, sum(lens), Hq, Hkv, seed).items()}
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    return inp, cu


@pytest.mark.parametrize("lens,Hq,Hkv,window,sink", PACKED)
def test_packed_prefill_matches_oracle(da, lens, Hq, Hkv, window, sink):
    inp, cu = _packed(lens, Hq, Hkv, seed=sum(lens))
    d = {k: v.cuda() for k, v in inp.items()}
    out = da.prefill_varlen_window(d["q"], d["k"], d["v"], d["lam"], cu.cuda(), max(lens), window, sink=sink)
    _ok(da)
    bf16_close(out, ora.prefill_varlen(inp["q"], inp["k"], inp["v"], inp["lam"], cu, window=window, sink=sink), "packed")


def test_many_sequences_equal_the_batch(da):
    """300 sequences (one CTA per item) give the bits of the batched call."""
    d = {k: v.cuda() for k, v in _case(300, 150, 4, 1, seed=9).items()}
    ref = da.prefill_window(d["q"], d["k"], d["v"], d["lam"], 20, sink=3)
    cu = (torch.arange(301, device="cuda") * 150).int()
    flat = [d[n].flatten(0, 1) for n in ("q", "k", "v", "lam")]
    out = da.prefill_varlen_window(*flat, cu, 150, 20, sink=3)
    _ok(da)
    assert torch.equal(out, ref.flatten(0, 1))


def _grads_close(got, ref, what):
    for g, r, n in zip(got, ref, ("dq", "dk", "dv", "dlam")):
        grad_close(g, r, f"{what} {n}")


TRAIN = [
    (1, 1, 2, 1, 1, 1),
    (1, 200, 4, 1, 2, 1),
    (2, 300, 8, 2, 64, 4),
    (1, 513, 16, 1, 100, 64),
    (1, 700, 8, 4, 130, 200),
    (1, 400, 4, 2, 400, 3),
    (1, 1000, 4, 1, 60, 5),     # many query blocks behind the sinks' window
    (1, 640, 32, 4, 200, 128),
    (1, 1500, 8, 2, 33, 300),   # sinks over three key tiles
]


@pytest.mark.parametrize("B,S,Hq,Hkv,window,sink", TRAIN)
def test_training_pass_matches_oracle(da, B, S, Hq, Hkv, window, sink):
    inp = _case(B, S, Hq, Hkv, seed=2 * S + window)
    d = {k: v.cuda() for k, v in inp.items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    out, ob, lse = da.prefill_train(*x, window=window, sink=sink)
    grads = da.backward(*x, ob, lse, d["dout"], window=window, sink=sink)
    _ok(da)
    assert ob.dtype == torch.float32
    bf16_close(out, ora.prefill(inp["q"], inp["k"], inp["v"], inp["lam"], window=window, sink=sink), "train out")
    ref = ora.prefill_backward(inp["q"], inp["k"], inp["v"], inp["lam"], inp["dout"], window=window, sink=sink)
    _grads_close(grads, ref, f"S={S} W={window} s={sink}")
    assert torch.count_nonzero(grads[0][:, 0]).item() == 0  # query 0 sees one key


@pytest.mark.parametrize("lens,Hq,Hkv,window,sink", PACKED)
def test_packed_training_pass_matches_oracle(da, lens, Hq, Hkv, window, sink):
    inp, cu = _packed(lens, Hq, Hkv, seed=3 + sum(lens))
    d = {k: v.cuda() for k, v in inp.items()}
    x, tail = (d["q"], d["k"], d["v"], d["lam"]), (cu.cuda(), max(lens))
    out, ob, lse = da.prefill_varlen_train(*x, *tail, window=window, sink=sink)
    grads = da.backward_varlen(*x, ob, lse, d["dout"], *tail, window=window, sink=sink)
    _ok(da)
    bf16_close(out, ora.prefill_varlen(inp["q"], inp["k"], inp["v"], inp["lam"], cu, window=window, sink=sink), "train out")
    ref = ora.prefill_backward_varlen(inp["q"], inp["k"], inp["v"], inp["lam"], inp["dout"], cu, window=window, sink=sink)
    _grads_close(grads, ref, f"packed {lens}")


def test_dq_where_many_alike_sinks_share_the_weight(da):
    """Sinks that resemble one another: the roundings of their dS add up in dQ along the common direction
    unless they are kept apart. Relative to dQ its own rounding is at most half a bf16 step, 2^-8; a
    common-mode error of dS products rounded at 2^-8 each would be of that size again."""
    S, sink, window = 500, 64, 60
    g = torch.Generator().manual_seed(6)
    u = torch.randn(128, generator=g)
    u /= u.norm()
    inp = _case(1, S, 4, 1, seed=78)
    inp["q"] = (inp["q"].float() + 2 * u).bfloat16()
    inp["k"][:, :sink] = (inp["k"][:, :sink].float() + 18 * u).bfloat16()
    d = {k: v.cuda() for k, v in inp.items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    for w, s in ((window, sink), (S, sink), (window, S)):  # and where the mask is the plain causal one
        out, ob, lse = da.prefill_train(*x, window=w, sink=s)
        grads = da.backward(*x, ob, lse, d["dout"], window=w, sink=s)
        _ok(da)
        ref = ora.prefill_backward(inp["q"], inp["k"], inp["v"], inp["lam"], inp["dout"], window=w, sink=s)
        _grads_close(grads, ref, f"alike sinks W={w} s={s}")
        off = np.linalg.norm(to64(grads[0]) - ref[0]) / np.linalg.norm(ref[0])
        assert off <= 2.0 ** -8, off


def test_gradients_where_one_sink_takes_nearly_all_weight(da):
    """dS is a small difference of large terms there: A (dP - E) with A near 1 on the sink."""
    inp = _case(1, 260, 4, 1, seed=77)
    inp["q"] = (inp["q"].float() * 0.5).bfloat16()
    u = torch.zeros(128)
    u[::2] = 1.0
    inp["q"] = (inp["q"].float() + u).bfloat16()
    inp["k"][:, 0] = (u * 1.0).bfloat16()  # logit about 64 / sqrt(128) = 5.7 above the others
    d = {k: v.cuda() for k, v in inp.items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    _, ob, lse = da.prefill_train(*x, window=3, sink=1)
    grads = da.backward(*x, ob, lse, d["dout"], window=3, sink=1)
    _ok(da)
    ref = ora.prefill_backward(inp["q"], inp["k"], inp["v"], inp["lam"], inp["dout"], window=3, sink=1)
    _grads_close(grads, ref, "dominant sink")


def test_backward_is_deterministic_and_ignores_its_workspace(da):
    d = {k: v.cuda() for k, v in _case(1, 900, 16, 2, seed=21).items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    _, ob, lse = da.prefill_train(*x, window=50, sink=9)
    need = da.LIB.diffattn_v2_backward_window_sink_workspace_size(1, 900, 16, 2, 50, 9)
    a = da.backward(*x, ob, lse, d["dout"], window=50, sink=9)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    b = da.backward(*x, ob, lse, d["dout"], window=50, sink=9, workspace=ws)
    _ok(da)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ws[need:].eq(255).all()


# ----------------------------------------------------------------------------------- decode
DECODE = [
    # Hq, Hkv, window, sink, lengths
    (16, 2, 64, 4, [300, 1, 0, 64, 68, 69]),
    (8, 4, 1, 1, [700, 129, 2, 1]),            # the newest key and key 0
    (32, 2, 100, 70, [900, 333, 170, 171]),    # group of 16, sinks past a stage
    (64, 8, 500, 64, [1000, 564, 565, 63]),
    (4, 2, 2000, 3, [1500, 7]),                # a window wider than every sequence
    (8, 1, 3000, 130, [5000, 4999, 3131]),     # several stages per CTA
    (16, 4, 7, 900, [1000, 905, 910]),         # sinks wider than the window
]


def _decode_inputs(Hq, Hkv, lens, seed, smax=None):
    smax = smax or max(max(lens), 1)
    inp = workloads.make_decode(workloads.DecodeCase(B=len(lens), Smax=smax, Hq=Hq, Hkv=Hkv, D=128, len_lo=1,
                                                     len_hi=smax, seed=seed))
    inp["seqlens"] = torch.tensor(lens, dtype=torch.int32)
    return inp


def _hide(inp, window, sink):
    """NaN and infinities wherever no key is visible."""
    for b, n in enumerate(inp["seqlens"].tolist()):
        for j in range(inp["kcache"].shape[1]):
            if not (j < n and (j < sink or j >= n - window)):
                inp["kcache"][b, j] = float("nan")
                inp["vcache"][b, j] = float("inf") if j % 2 else float("nan")


@pytest.mark.parametrize("Hq,Hkv,window,sink,lens", DECODE)
def test_decode_matches_oracle(da, Hq, Hkv, window, sink, lens):
    inp = _decode_inputs(Hq, Hkv, lens, seed=Hq + window)
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], inp["seqlens"], inp["lam"], window=window, sink=sink)
    _hide(inp, window, sink)
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    out = da.decode(d["q"], d["kcache"], d["vcache"], d["seqlens"], d["lam"], window=window, sink=sink)
    _ok(da)
    bf16_close(out, ref, "decode")
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.count_nonzero(out[b]).item() == 0


def _pages(inp, page, window, sink, seed):
    """The caches of `inp` on scattered pages; pages without a visible key have entry -1 or one that
    names a page of NaN."""
    B, smax = inp["kcache"].shape[:2]
    per = -(-smax // page)
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(B * per + 1, generator=g)
    kp = torch.full((B * per + 1, page, *inp["kcache"].shape[2:]), float("nan"), dtype=torch.bfloat16)
    vp = kp.clone()
    table = torch.full((B, per), -1, dtype=torch.int32)
    for b, n in enumerate(inp["seqlens"].tolist()):
        for i in range(per):
            rows = range(i * page, min((i + 1) * page, smax))
            if any(j < n and (j < sink or j >= n - window) for j in rows):
                pg = int(perm[b * per + i])
                kp[pg, : len(rows)] = inp["kcache"][b, rows[0]: rows[-1] + 1]
                vp[pg, : len(rows)] = inp["vcache"][b, rows[0]: rows[-1] + 1]
                table[b, i] = pg
            elif i % 2:
                table[b, i] = int(perm[-1])
    return kp, vp, table


@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("Hq,Hkv,window,sink,lens", DECODE)
def test_paged_decode_matches_oracle(da, Hq, Hkv, window, sink, lens, page):
    inp = _decode_inputs(Hq, Hkv, lens, seed=Hq + window + page)
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], inp["seqlens"], inp["lam"], window=window, sink=sink)
    _hide(inp, window, sink)
    kp, vp, table = _pages(inp, page, window, sink, seed=page)
    out = da.decode_paged(inp["q"].cuda(), kp.cuda(), vp.cuda(), table.cuda(), inp["seqlens"].cuda(), inp["lam"].cuda(),
                          window=window, sink=sink)
    _ok(da)
    bf16_close(out, ref, f"paged decode page={page}")


def test_decode_equals_the_prefills_last_rows(da):
    d = {k: v.cuda() for k, v in _case(2, 700, 16, 2, seed=13).items()}
    ref = da.prefill_window(d["q"], d["k"], d["v"], d["lam"], 200, sink=5)[:, -1]
    n = torch.full((2,), 700, dtype=torch.int32, device="cuda")
    out = da.decode(d["q"][:, -1].contiguous(), d["k"], d["v"], n, d["lam"][:, -1].contiguous(), window=200, sink=5)
    _ok(da)
    bf16_close(out, to64(ref), "decode against the prefill's last row")


def test_decode_clamps_lengths_to_the_cache(da):
    inp = _decode_inputs(16, 2, [300, 10], seed=4)
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    ref = da.decode(d["q"], d["kcache"], d["vcache"], torch.tensor([300, 0], dtype=torch.int32, device="cuda"), d["lam"],
                    window=50, sink=4)
    out = da.decode(d["q"], d["kcache"], d["vcache"], torch.tensor([5000, -3], dtype=torch.int32, device="cuda"),
                    d["lam"], window=50, sink=4)
    _ok(da)
    assert torch.equal(out, ref)


def test_decode_of_a_long_window_by_sixteen_ctas(da):
    """One sequence and one KV head over more than 16,384 keys: the largest cluster."""
    inp = _decode_inputs(8, 1, [20011], seed=16)
    ref = ora.decode(inp["q"], inp["kcache"], inp["vcache"], inp["seqlens"], inp["lam"], window=18000, sink=40)
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor)}
    out = da.decode(d["q"], d["kcache"], d["vcache"], d["seqlens"], d["lam"], window=18000, sink=40)
    _ok(da)
    bf16_close(out, ref, "long window")


def test_a_cache_past_32_bits(da):
    """Pages whose elements lie behind 2^31: append, copy and decode there."""
    page, Hkv, Hq, N = 64, 8, 16, 40000
    kc = torch.empty(N, page, Hkv, 128, dtype=torch.bfloat16, device="cuda")  # 5.2 GB
    vc = torch.empty_like(kc)
    n = 100
    table = torch.tensor([[N - 1, N - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(n, Hq, 128), r(n, Hkv, 128), r(n, Hkv, 128)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    inv = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    qr = da.rope_append_paged(q, k, v, pos, inv, (64,), kc, vc, table, lens, cu_seqlens=cu)
    kr = da.rope(k, None, pos, inv, (64,))[0]
    lam = torch.rand(1, Hq // 2, generator=g, device="cuda")
    ref = ora.decode(qr[-1:].cpu(), kr[None].cpu(), v[None].cpu(), [n], lam.cpu(), window=50, sink=4)
    last = qr[-1:].contiguous()
    bf16_close(da.decode_paged(last, kc, vc, table, lens, lam, window=50, sink=4), ref, "behind 2^31")
    copies = torch.tensor([[N - 1, N - 2], [N - 3, 5]], dtype=torch.int32, device="cuda")
    da.cache_copy_pages(kc, vc, copies)
    moved = torch.tensor([[N - 2, 5]], dtype=torch.int32, device="cuda")
    bf16_close(da.decode_paged(last, kc, vc, moved, lens, lam, window=50, sink=4), ref, "copied")
    _ok(da)


def test_calls_from_two_threads(da):
    """The binding gives up the interpreter lock during a call; each thread has its own stream."""
    import threading

    inp = _decode_inputs(16, 2, [900, 450, 1, 777], seed=3)
    d = [inp[n].cuda() for n in ("q", "kcache", "vcache", "seqlens", "lam")]
    ref = da.decode(*d, window=300, sink=6)
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                if not torch.equal(da.decode(*d, window=300, sink=6), ref):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok(da)
    assert not bad


def test_decode_in_graphs_and_on_two_streams(da):
    """Two captured decodes and an eager one share nothing: replayed together they give their bits."""
    cases = []
    for seed, (Hq, Hkv) in enumerate([(16, 2), (32, 2), (64, 8)]):
        inp = _decode_inputs(Hq, Hkv, [900, 450, 1, 777], seed=seed)
        d = [inp[n].cuda() for n in ("q", "kcache", "vcache", "seqlens", "lam")]
        cases.append((d, da.decode(*d, window=300, sink=6)))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d, ref in cases[:2]:
        out, g = torch.zeros_like(ref), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            da.decode(*d, out=out, window=300, sink=6)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        extra = da.decode(*cases[2][0], window=300, sink=6, stream=streams[2])
    _ok(da)
    for out, (_, ref) in zip([*outs, extra], cases):
        assert torch.equal(out, ref)


def test_training_pass_in_a_graph(da):
    d = {k: v.cuda() for k, v in _case(1, 400, 8, 2, seed=31).items()}
    x = (d["q"], d["k"], d["v"], d["lam"])

    def step():
        out, ob, lse = da.prefill_train(*x, window=70, sink=4)
        return (out, *da.backward(*x, ob, lse, d["dout"], window=70, sink=4))

    ref = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in got:
        t.zero_()
    g.replay()
    _ok(da)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals(da):
    d = {k: v.cuda() for k, v in _case(1, 64, 8, 2, seed=1).items()}
    x = (d["q"], d["k"], d["v"], d["lam"])
    with pytest.raises(da.DiffAttnError):
        da.prefill_window(*x, 0, sink=1)
    with pytest.raises(da.DiffAttnError):
        da.prefill_window(*x, 8, sink=-1)
    with pytest.raises(ValueError):
        da.prefill_window(d["q"], d["k"], d["v"][:, :32], d["lam"], 8, sink=1)
    with pytest.raises(ValueError):
        da.prefill_train(*x, sink=1)  # no window
    with pytest.raises(TypeError):
        out, ob, lse = da.prefill_train(*x, window=8, sink=1)
        da.backward(*x, ob.bfloat16(), lse, d["dout"], window=8, sink=1)
    with pytest.raises(da.DiffAttnError):
        da.backward(*x, ob, lse, d["dout"], window=8, sink=1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        da.prefill_window(*x, 2**40, sink=1)
    with pytest.raises(TypeError):
        da.prefill_window(*x, 8.5, sink=1)
    with pytest.raises(TypeError):
        da.prefill_window(None, *x[1:], 8, sink=1)
    with pytest.raises(ValueError):
        da.prefill_window(*x, 8, sink=1, out=torch.empty(1, 64, 128, 4, dtype=torch.bfloat16, device="cuda").mT)
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        da.decode(d["q"][:, 0].contiguous(), d["k"], d["v"], n, d["lam"][:, 0].contiguous(), sink=1)
    with pytest.raises(ValueError):
        da.decode(d["q"][:, 0], d["k"].cpu(), d["v"], n, d["lam"][:, 0].contiguous(), window=4, sink=1)
    _ok(da)
