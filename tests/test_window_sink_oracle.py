"""CPU: the oracle's window with sinks against a definition written out key by key and against finite
differences; the host-side refusals of the window-with-sinks, rotary and cache entry points."""
import ctypes
import math

import numpy as np
import pytest

from oracle import diffattn_f64 as ora


def _naive(q, k, v, lam, window, sink):
    S, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((S, Hq // 2, D))
    for i in range(S):
        keys = [j for j in range(i + 1) if i - j < window or j < sink]
        for p in range(Hq // 2):
            o = []
            for h in (2 * p, 2 * p + 1):
                w = [math.exp(sum(q[i, h] * k[j, h // G]) / math.sqrt(D)) for j in keys]
                o.append(sum(x * v[j, h // G] for x, j in zip(w, keys)) / sum(w))
            out[i, p] = o[0] - lam[i, p] * o[1]
    return out


def _random(S, Hq, Hkv, D, seed):
    r = np.random.default_rng(seed)
    return (r.normal(size=(S, Hq, D)), r.normal(size=(S, Hkv, D)), r.normal(size=(S, Hkv, D)), r.uniform(size=(S, Hq // 2)))


@pytest.mark.parametrize("window,sink", [(1, 1), (3, 2), (2, 7), (20, 1), (4, 30)])
def test_prefill_with_sinks(window, sink):
    q, k, v, lam = _random(11, 4, 2, 3, seed=window)
    got = ora.prefill(q[None], k[None], v[None], lam[None], window=window, sink=sink)[0]
    np.testing.assert_allclose(got, _naive(q, k, v, lam, window, sink), rtol=1e-12, atol=1e-12)
    cu = [0, 4, 4, 11]
    got = ora.prefill_varlen(q, k, v, lam, cu, window=window, sink=sink)
    for a, b in zip(cu, cu[1:]):
        np.testing.assert_allclose(got[a:b], _naive(q[a:b], k[a:b], v[a:b], lam[a:b], window, sink), atol=1e-12)
    n = [11]
    last = ora.decode(q[None, -1], k[None], v[None], n, lam[None, -1], window=window, sink=sink)
    np.testing.assert_allclose(last[0], _naive(q, k, v, lam, window, sink)[-1], atol=1e-12)


def test_gradients_with_sinks_by_differences():
    x = list(_random(9, 4, 2, 3, seed=4))
    r = np.random.default_rng(5)
    g = r.normal(size=(9, 2, 3))
    grads = ora.prefill_backward(*(t[None] for t in x), g[None], window=3, sink=2)
    h = 1e-6
    for n in range(4):
        e = r.normal(size=x[n].shape)
        f = []
        for s in (h, -h):
            y = [t + s * e if i == n else t for i, t in enumerate(x)]
            f.append(float((ora.prefill(*(t[None] for t in y), window=3, sink=2)[0] * g).sum()))
        # central differences: h^2 times third derivatives of order 10, and 1e-16 / h of rounding
        assert abs((f[0] - f[1]) / (2 * h) - float((grads[n][0] * e).sum())) < 1e-7


def test_no_sinks_is_the_window_mask():
    np.testing.assert_array_equal(ora.window_mask(9, 9, 3), ora.window_mask(9, 9, 3, sink=0))
    m = ora.window_mask(6, 6, 2, sink=1)
    assert [int((row == 0).sum()) for row in m] == [1, 2, 3, 3, 3, 3]


# ------------------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from differential_attention_v2_b200.build import build

    build()
    import differential_attention_v2_b200 as da

    return da.LIB


P = 1 << 20  # aligned placeholders: every call below is refused, or a no-op, before any CUDA call
A = [P + 4096 * i for i in range(16)]
INV, UNS, OK = -1, -2, 0


def test_window_sink_refusals(lib):
    f = lib.diffattn_v2_prefill_window_sink
    x = A[:5]
    for tail, want in [((1, 64, 8, 2, 128, 0, 1), INV), ((1, 64, 8, 2, 128, 4, -1), INV), ((1, 64, 6, 2, 128, 4, 1), INV),
                       ((1, 64, 8, 2, 64, 4, 1), UNS), ((0, 64, 8, 2, 128, 4, 1), OK), ((1, 0, 8, 2, 128, 4, 1), OK),
                       ((-1, 64, 8, 2, 128, 4, 1), INV), ((1, 128 * 65536, 8, 2, 128, 4, 1), UNS),
                       ((1 << 20, 1 << 20, 64, 8, 128, 4, 1), UNS)]:
        assert f(*x, *tail, None) == want, tail
    assert f(*x[:4], A[4] + 8, 1, 64, 8, 2, 128, 4, 1, None) == INV
    assert f(None, *x[1:], 1, 64, 8, 2, 128, 4, 1, None) == INV
    g = lib.diffattn_v2_prefill_varlen_window_sink
    assert g(*x, None, 1, 64, 64, 8, 2, 128, 4, 1, None) == INV
    assert g(*x, A[5], 1, 64, -1, 8, 2, 128, 4, 1, None) == INV
    assert g(*x, A[5], 0, 64, 64, 8, 2, 128, 4, 1, None) == OK
    t = lib.diffattn_v2_prefill_window_sink_train
    assert t(*x, None, A[6], 1, 64, 8, 2, 128, 4, 1, None) == INV
    assert t(*x, A[5], A[6] + 4, 1, 64, 8, 2, 128, 4, 1, None) == INV
    assert t(*x, A[5], A[6], 1, 64, 8, 2, 64, 4, 1, None) == UNS


def test_backward_window_sink_refusals(lib):
    size = lib.diffattn_v2_backward_window_sink_workspace_size
    need = size(2, 300, 8, 2, 64, 4)
    assert need >= lib.diffattn_v2_backward_workspace_size(2, 300, 8) and size(2, 300, 8, 2, 0, 4) == 0
    assert size(2, 300, 6, 2, 64, 4) == 0 and size(0, 300, 8, 2, 64, 4) == 0
    f = lib.diffattn_v2_backward_window_sink
    x, tail = A[:11], (2, 300, 8, 2, 128)
    assert f(*x, *tail, 64, 4, A[12], need - 4, None) == INV
    assert f(*x, *tail, 0, 4, A[12], need, None) == INV
    assert f(*x, *tail, 64, -4, A[12], need, None) == INV
    assert f(*x, *tail, 64, 4, None, need, None) == INV
    assert f(*x, 2, 300, 8, 2, 64, 64, 4, A[12], 1 << 40, None) == UNS
    assert f(*x, 0, 300, 8, 2, 128, 64, 4, A[12], need, None) == OK
    g, size = lib.diffattn_v2_backward_varlen_window_sink, lib.diffattn_v2_backward_varlen_window_sink_workspace_size
    need = size(3, 200, 500, 8, 2, 64, 4)
    assert need >= lib.diffattn_v2_backward_varlen_workspace_size(3, 500, 8)
    assert g(*x, A[11], 3, 200, 500, 8, 2, 128, 64, 4, A[12], need - 4, None) == INV
    assert g(*x, None, 3, 200, 500, 8, 2, 128, 64, 4, A[12], need, None) == INV
    assert g(*x, A[11], 3, 200, 500, 8, 2, 64, 64, 4, A[12], 1 << 40, None) == UNS


def test_decode_window_sink_refusals(lib):
    f = lib.diffattn_v2_decode_window_sink
    x = A[:6]
    for tail, want in [((2, 100, 8, 2, 128, 0, 1), INV), ((2, 100, 8, 2, 128, 4, -1), INV), ((2, 0, 8, 2, 128, 4, 1), INV),
                       ((2, 100, 8, 2, 64, 4, 1), UNS), ((2, 100, 12, 2, 128, 4, 1), UNS), ((0, 100, 8, 2, 128, 4, 1), OK),
                       ((70000, 100, 8, 2, 128, 4, 1), UNS)]:
        assert f(*x, *tail, None) == want, tail
    g = lib.diffattn_v2_decode_paged_window_sink
    x = A[:7]
    for tail, want in [((2, 8, 12, 9, 8, 2, 128, 4, 1), INV), ((2, 8, 4, 9, 8, 2, 128, 4, 1), INV),
                       ((2, 0, 16, 9, 8, 2, 128, 4, 1), INV), ((2, 8, 16, 0, 8, 2, 128, 4, 1), INV),
                       ((2, 1 << 20, 4096, 9, 8, 2, 128, 4, 1), INV), ((2, 8, 16, 9, 8, 2, 64, 4, 1), UNS)]:
        assert g(*x, *tail, None) == want, tail
    assert g(*x[:3], None, *x[4:], 2, 8, 16, 9, 8, 2, 128, 4, 1, None) == INV


def test_rope_refusals(lib):
    sec = (ctypes.c_int * 5)(16, 24, 24, 0, 0)
    neg = (ctypes.c_int * 2)(70, -10)

    def f(q=A[0], k=A[1], qo=A[2], ko=A[3], pos=A[4], inv=A[5], sections=sec, n=3, T=5, Hq=4, Hkv=2, D=128, qs=512, ks=256,
          qos=512, kos=256, dtype=0, inter=0, inverse=0):
        return lib.diffattn_v2_rope(q, k, qo, ko, pos, inv, sections, n, T, Hq, Hkv, D, qs, ks, qos, kos, dtype, inter,
                                    inverse, None)

    assert f(T=0) == OK
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(pos=None), dict(inv=A[5] + 2), dict(T=-1), dict(Hq=0),
                dict(Hkv=-1), dict(D=127), dict(n=0), dict(qs=511), dict(kos=255), dict(dtype=2), dict(inter=2),
                dict(inverse=-1), dict(sections=neg, n=2), dict(D=64), dict(q=A[0] + 1),
                dict(sections=(ctypes.c_int * 1)(0), n=1)):
        assert f(**bad) == INV, bad
    assert f(n=5) == UNS
    assert f(D=8192, qs=1 << 20, ks=1 << 20, qos=1 << 20, kos=1 << 20) == UNS


def test_append_refusals(lib):
    sec = (ctypes.c_int * 1)(64)

    def f(T=5, B=5, cu=None, page=16, table=A[7], v=A[2], Hkv=2, vs=256, max_pages=8, num_pages=9, kp=A[5]):
        return lib.diffattn_v2_rope_append_paged(A[0], A[1], v, A[3], A[4], A[12], sec, 1, kp, A[6], table, A[8], cu, T, B,
                                                 max_pages, page, num_pages, 4, Hkv, 128, 512, 256, vs, 512, 0, 0, None)

    assert f(T=0) == OK
    for bad in (dict(T=4), dict(page=12), dict(table=None), dict(v=None), dict(Hkv=0), dict(vs=200), dict(max_pages=0),
                dict(num_pages=0), dict(kp=A[5] + 1), dict(cu=A[9] + 2)):
        assert f(**bad) == INV, bad


def test_cache_refusals(lib):
    e, fk, tr, fr = (getattr(lib, "diffattn_v2_cache_" + n) for n in ("extend", "fork", "trim", "free"))
    assert e(*A[:5], 4, 8, 12, 9, None) == INV and e(*A[:5], 4, 0, 16, 9, None) == INV
    assert e(*A[:4], None, 4, 8, 16, 9, None) == INV and e(*A[:4], A[4] + 2, 4, 8, 16, 9, None) == INV
    assert e(*A[:5], 2049, 8, 16, 9, None) == UNS and e(*A[:5], 0, 8, 16, 9, None) == OK
    assert fk(*A[:7], -1, 4, 8, 16, 9, None) == INV and fk(*A[:5], A[5] + 4, A[6], 2, 4, 8, 16, 9, None) == INV
    assert fk(*A[:7], 2049, 4, 8, 16, 9, None) == UNS and fk(*A[:7], 0, 4, 8, 16, 9, None) == OK
    assert tr(*A[:4], 4, 8, 16, 9, 0, 1, None) == INV and tr(*A[:4], 4, 8, 16, 9, 4, -1, None) == INV
    assert fr(*A[:5], -1, 4, 8, 9, None) == INV and fr(*A[:3], None, A[4], 1, 4, 8, 9, None) == INV
    c = lib.diffattn_v2_cache_compact
    assert c(*A[:4], None, A[5], 4, 8, 9, None) == INV and c(*A[:6], 4, 8, 0, None) == INV
    y = lib.diffattn_v2_cache_copy_pages
    assert y(A[0], A[0], A[1], 3, 9, 64, None) == INV and y(A[0], A[1], None, 3, 9, 64, None) == INV
    assert y(A[0], A[1], A[2], 3, 9, 24, None) == UNS and y(A[0], A[1] + 8, A[2], 3, 9, 64, None) == INV
    assert y(A[0], A[1], A[2], 0, 9, 64, None) == OK


def test_cache_size_limits(lib):
    """Index arithmetic in 32 bits: pools of more than 2^30 pages, and tables whose entries cannot be
    counted in an int, are refused."""
    e, fk, tr, fr, c = (getattr(lib, "diffattn_v2_cache_" + n) for n in ("extend", "fork", "trim", "free", "compact"))
    big = (1 << 30) + 1
    assert e(*A[:5], 4, 8, 16, big, None) == INV
    assert fk(*A[:7], 2, 4, 8, 16, big, None) == INV
    assert tr(*A[:4], 4, 8, 16, big, 64, 4, None) == INV
    assert fr(*A[:5], 1, 4, 8, big, None) == INV
    assert c(*A[:6], 4, 8, big, None) == INV
    assert e(*A[:5], 2048, 1 << 20, 8, 9, None) == UNS  # 2^31 entries
    assert e(*A[:5], 0, 1 << 20, 8, 9, None) == OK


def test_backward_launch_limits(lib):
    """Many packed sequences beside a very long one: a grid whose CTAs cannot be counted in an int is
    refused (its count used to wrap)."""
    g = lib.diffattn_v2_backward_varlen_window_sink
    x = A[:11]
    # 16384 sequences of at most 2^20 tokens, 32 pairs: 2^32 query tiles
    assert g(*x, A[11], 16384, 1 << 20, 1 << 21, 64, 8, 128, 1024, 4, A[12], 1 << 60, None) == UNS
    assert g(*x, A[11], 16384, 1 << 20, 1 << 21, 64, 8, 128, 1 << 20, 4, A[12], 1 << 60, None) == UNS
