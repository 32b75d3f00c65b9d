"""Calls with an explicit stream. What a call allocates has to come from the memory pool of the stream that
it runs on: the allocator hands out a block of the current stream's pool while work queued there may still
use it, and the given stream does not wait for that work. The outputs, which the caller reads on its own
stream, must not go back to the pool while work queued there still reads them."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


@pytest.fixture(scope="module")
def x():
    """Small inputs of every call below."""
    case = workloads.PrefillCase(B=1, S=200, Hq=8, Hkv=2, D=128, seed=1)
    d = {k: v.cuda() for k, v in workloads.make_prefill(case).items()}
    d["dout"] = workloads.make_prefill_grad(case).cuda()
    d["qkvl"] = tuple(d[n] for n in ("q", "k", "v", "lam"))
    d["packed"] = tuple(t[0].contiguous() for t in d["qkvl"])
    d["cu"] = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    d["step"] = (d["q"][:, -1].contiguous(), d["k"], d["v"], torch.tensor([200], dtype=torch.int32, device="cuda"),
                 d["lam"][:, -1].contiguous())
    d["pages"] = (d["step"][0], d["k"].view(25, 8, 2, 128), d["v"].view(25, 8, 2, 128),
                  torch.arange(25, dtype=torch.int32, device="cuda").view(1, 25), *d["step"][3:])
    d["pos"] = torch.arange(200, dtype=torch.int32, device="cuda")[None]
    d["inv"] = torch.rand(64, device="cuda")
    d["pool"] = (d["pages"][3].clone(), torch.tensor([200], dtype=torch.int32, device="cuda"),
                 torch.ones(25, dtype=torch.int32, device="cuda"))
    return d


def _backward(da, x, s, **kw):
    _, ob, lse = da.prefill_train(*x["qkvl"], **kw)
    torch.cuda.synchronize()
    return lambda: da.backward(*x["qkvl"], ob, lse, x["dout"], stream=s, **kw)


def _backward_varlen(da, x, s, **kw):
    _, ob, lse = da.prefill_varlen_train(*x["packed"], x["cu"], 150, **kw)
    torch.cuda.synchronize()
    return lambda: da.backward_varlen(*x["packed"], ob, lse, x["dout"][0], x["cu"], 150, stream=s, **kw)


W = dict(window=50, sink=3)


def _append(da, x, s):
    k, v, cu = x["pages"][1].clone(), x["pages"][2].clone(), x["cu"][::2].contiguous()
    torch.cuda.synchronize()
    return lambda: da.rope_append_paged(x["q"][0], x["k"][0], x["v"][0], x["pos"], x["inv"], (64,), k, v,
                                        *x["pages"][3:5], cu_seqlens=cu, stream=s)


def _pages(call):
    """A bookkeeping call that changes nothing: no new tokens, padding, a window of every key."""
    def make(da, x, s):
        none, zero = torch.full((1,), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        return lambda: call(da, x["pool"], none, zero, s)
    return make


SINK_ROPE_CACHE = {
    "prefill_window": lambda da, x, s: lambda: da.prefill_window(*x["qkvl"], 50, sink=3, stream=s),
    "prefill_varlen_window": lambda da, x, s: lambda: da.prefill_varlen_window(*x["packed"], x["cu"], 150, 50, sink=3,
                                                                               stream=s),
    "prefill_train": lambda da, x, s: lambda: da.prefill_train(*x["qkvl"], stream=s, **W),
    "prefill_varlen_train": lambda da, x, s: lambda: da.prefill_varlen_train(*x["packed"], x["cu"], 150, stream=s, **W),
    "backward": lambda da, x, s: _backward(da, x, s, **W),
    "backward_varlen": lambda da, x, s: _backward_varlen(da, x, s, **W),
    "decode": lambda da, x, s: lambda: da.decode(*x["step"], stream=s, **W),
    "decode_paged": lambda da, x, s: lambda: da.decode_paged(*x["pages"], stream=s, **W),
    "rope": lambda da, x, s: lambda: da.rope(x["q"][0], x["k"][0], x["pos"], x["inv"], (64,), stream=s),
    "rope_append_paged": _append,
    "cache_extend": _pages(lambda da, pool, none, zero, s: da.cache_extend(*pool, zero, 8, stream=s)),
    "cache_fork": _pages(lambda da, pool, none, zero, s: da.cache_fork(*pool, zero, none, 8, stream=s)),
    "cache_trim": _pages(lambda da, pool, none, zero, s: da.cache_trim(*pool, 8, 500, 3, stream=s)),
    "cache_free": _pages(lambda da, pool, none, zero, s: da.cache_free(*pool, none, stream=s)),
    "cache_compact": _pages(lambda da, pool, none, zero, s: da.cache_compact(pool[0], pool[2], stream=s)),
}


def _lambda_v2(da, x, s, fused):
    g = torch.Generator(device="cuda").manual_seed(2)
    t, w = (torch.randn(*n, generator=g, device="cuda").bfloat16() for n in ((200, 256), (256, 32)))
    wt = w[:, :4].t().contiguous()
    torch.cuda.synchronize()
    if fused:
        return lambda: da.prefill_fused_lambda(*x["qkvl"][:3], t[None], wt, stream=s)
    return lambda: da.lambda_v2(t, w, stream=s)


def _multi(da, x, s):
    q, lam = x["q"][:, -2:].contiguous(), x["lam"][:, -2:].contiguous()
    torch.cuda.synchronize()
    return lambda: da.decode_multi(q, *x["step"][1:4], lam, stream=s)


def _f32(da, x, s, decode):
    y = [t.float() if t.is_floating_point() else t for t in (x["step"] if decode else x["qkvl"])]
    torch.cuda.synchronize()
    return (lambda: da.decode_f32(*y, stream=s)) if decode else (lambda: da.prefill_f32(*y, stream=s))


def _lambda_v1(da, x, s):
    y = [torch.rand(4, 64, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    return lambda: da.lambda_v1(*y, stream=s)


PLAIN = {
    "prefill": lambda da, x, s: lambda: da.prefill(*x["qkvl"], stream=s),
    "prefill_window": lambda da, x, s: lambda: da.prefill_window(*x["qkvl"], 50, stream=s),
    "prefill_varlen": lambda da, x, s: lambda: da.prefill_varlen(*x["packed"], x["cu"], 150, stream=s),
    "prefill_varlen_window": lambda da, x, s: lambda: da.prefill_varlen_window(*x["packed"], x["cu"], 150, 50, stream=s),
    "prefill_train": lambda da, x, s: lambda: da.prefill_train(*x["qkvl"], stream=s),
    "prefill_varlen_train": lambda da, x, s: lambda: da.prefill_varlen_train(*x["packed"], x["cu"], 150, stream=s),
    "backward": _backward,
    "backward_varlen": _backward_varlen,
    "decode": lambda da, x, s: lambda: da.decode(*x["step"], stream=s),
    "decode_window": lambda da, x, s: lambda: da.decode(*x["step"], stream=s, window=50),
    "decode_paged": lambda da, x, s: lambda: da.decode_paged(*x["pages"], stream=s),
    "decode_multi": _multi,
    "decode_noalloc": lambda da, x, s: lambda: da.decode_noalloc(*x["step"], stream=s),
    "prefill_f32": lambda da, x, s: _f32(da, x, s, False),
    "decode_f32": lambda da, x, s: _f32(da, x, s, True),
    "lambda_v1": _lambda_v1,
    "lambda_v2": lambda da, x, s: _lambda_v2(da, x, s, False),
    "prefill_fused_lambda": lambda da, x, s: _lambda_v2(da, x, s, True),
}


def _tensors(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else (out,)) if t is not None]


def _pool_of(t):
    """Handle of the stream whose pool holds t, and the state of its block."""
    for seg in torch.cuda.memory_snapshot():
        at = seg["address"]
        for block in seg["blocks"]:
            if at <= t < at + block["size"]:
                return seg["stream"], block["state"]
            at += block["size"]
    raise AssertionError("not an allocated block")


def _check_pool(call, s):
    handle = s if isinstance(s, int) else s.cuda_stream
    ref = _tensors(call())
    torch.cuda.synchronize()
    where = [_pool_of(t.data_ptr())[0] for t in ref if t.numel()]
    assert where and all(w == handle for w in where), (where, handle)
    # an output dropped while the caller's stream is busy stays out of the pool until that work is done
    ptr = ref[0].data_ptr()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    del ref
    assert _pool_of(ptr)[1] == "active_pending_free"
    torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", SINK_ROPE_CACHE)
def test_allocations_belong_to_the_given_stream(da, x, name, raw):
    s = torch.cuda.Stream()
    _check_pool(SINK_ROPE_CACHE[name](da, x, s.cuda_stream if raw else s), s)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", PLAIN)
def test_allocations_of_the_other_calls_belong_to_it_too(da, x, name, raw):
    s = torch.cuda.Stream()
    _check_pool(PLAIN[name](da, x, s.cuda_stream if raw else s), s)


@pytest.mark.parametrize("name,calls", [("backward", SINK_ROPE_CACHE), ("backward_varlen", SINK_ROPE_CACHE),
                                        ("backward", PLAIN), ("backward_varlen", PLAIN), ("decode", PLAIN),
                                        ("decode_window", PLAIN), ("decode_paged", PLAIN), ("decode_multi", PLAIN)],
                         ids=lambda v: v if isinstance(v, str) else "plain" if v is PLAIN else "sink")
def test_workspaces_belong_to_the_given_stream(da, x, name, calls):
    """Every allocation that the call makes, the workspace that it drops included."""
    s = torch.cuda.Stream()
    call = calls[name](da, x, s)
    torch.cuda.memory._record_memory_history(enabled="all", context=None, max_entries=10000, clear_history=True)
    try:
        out = call()
        torch.cuda.synchronize()
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    made = [e["stream"] for e in trace if e["action"] == "alloc"]
    assert len(made) > len(_tensors(out)) and all(h == s.cuda_stream for h in made), made


def test_results_on_a_given_stream(da, x):
    """The same bits as on the current stream, for torch streams, raw handles and the default stream."""
    ref = _tensors(_backward(da, x, None, **W)())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = _tensors(_backward(da, x, s, **W)())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert da.device_error() == 0


NOTHING = {  # calls on nothing, which launch no kernel: (call, B)
    "extend": (lambda da, pool, n, **kw: da.cache_extend(*pool, n, 8, **kw), 0),
    "fork": (lambda da, pool, n, **kw: da.cache_fork(*pool, n, n, 8, **kw)[1], 3),
    "trim": (lambda da, pool, n, **kw: da.cache_trim(*pool, 8, 4, 1, **kw), 0),
    "free": (lambda da, pool, n, **kw: da.cache_free(*pool, n, **kw), 3),
}


@pytest.mark.parametrize("which", ["none", "torch", "raw", "default"])
@pytest.mark.parametrize("name", NOTHING)
def test_the_result_of_nothing_is_written_in_the_streams_order(da, name, which):
    call, B = NOTHING[name]
    ints = dict(dtype=torch.int32, device="cuda")
    pool = (torch.full((B, 4), -1, **ints), torch.zeros(B, **ints), torch.zeros(5, **ints))
    result, n = torch.zeros(1, **ints), torch.zeros(0, **ints)
    torch.cuda.synchronize()
    side = torch.cuda.default_stream() if which == "default" else torch.cuda.Stream()
    given = {"none": None, "torch": side, "raw": side.cuda_stream, "default": 0}[which]
    with torch.cuda.stream(side):  # a value that the call has to come after
        torch.cuda._sleep(100_000_000)
        result.fill_(7)
    with torch.cuda.stream(side if which == "none" else torch.cuda.Stream()):
        got = call(da, pool, n, result=result, stream=given)
        fresh = call(da, pool, n, stream=given)
    torch.cuda.synchronize()
    assert got is result and got.tolist() == [0] and fresh.tolist() == [0]


@pytest.mark.parametrize("name", NOTHING)
def test_a_refused_result_keeps_its_value(da, name):
    call, B = NOTHING[name]
    ints = dict(dtype=torch.int32, device="cuda")
    pool = (torch.full((B, 4), -1, **ints), torch.zeros(B, **ints), torch.zeros(5, **ints))
    for bad, error in ((torch.full((1,), 7, device="cuda"), TypeError), (torch.full((2,), 7, **ints), ValueError)):
        with pytest.raises(error):
            call(da, pool, torch.zeros(0, **ints), result=bad)
        assert bad.eq(7).all()
    if name != "trim":  # (takes no list)
        with pytest.raises(TypeError):
            call(da, pool, [])


ALL = {**{f"sink {n}": c for n, c in SINK_ROPE_CACHE.items()}, **{f"plain {n}": c for n, c in PLAIN.items()}}


@pytest.mark.parametrize("name", ALL)
def test_the_first_call_of_a_host_thread(da, x, name):
    """A thread that has made no CUDA call yet, as a server's worker. (All that the call allocates is cached by
    then, so that not even the allocator calls the runtime before it.)"""
    import threading

    call = ALL[name](da, x, None)
    ref = _tensors(call())
    torch.cuda.synchronize()
    ref = [t.clone() for t in ref]
    got = []

    def work():
        try:
            got.append(_tensors(call()))
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not isinstance(got[0], Exception), got[0]
    assert all(torch.equal(a, b) for a, b in zip(got[0], ref))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("calls", [SINK_ROPE_CACHE, PLAIN], ids=["sink", "plain"])
def test_a_captured_call_on_a_forked_stream(da, x, calls, raw):
    """stream= names a stream that joined the capture: outputs and workspaces come from the graph's pool, and
    a replay after other work has used the memory gives the same bits."""
    s = torch.cuda.Stream()
    given = s.cuda_stream if raw else s
    names = ["prefill_train", "backward", "backward_varlen", "decode", "decode_paged"]
    made = [calls[n](da, x, given) for n in names]
    refs = []
    for call in made:
        out = _tensors(call())
        torch.cuda.synchronize()
        refs.append([t.clone() for t in out])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        outs = [_tensors(call()) for call in made]
        torch.cuda.current_stream().wait_stream(s)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for o in outs:
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    del junk
    for o, r, n in zip(outs, refs, names):
        assert all(torch.equal(a, b) for a, b in zip(o, r)), n
    assert da.device_error() == 0
