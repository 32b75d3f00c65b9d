"""The page bookkeeping of a paged cache on the GPU against a list model, and one serving run that uses
it together with the rotary append and the window decode with sinks."""
import random

import pytest
import torch

from oracle import diffattn_f64 as ora
from tests.parity import bf16_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


class Model:
    """The definition, entry by entry."""

    def __init__(self, B, max_pages, num_pages, page):
        self.table = [[-1] * max_pages for _ in range(B)]
        self.L, self.refs, self.page = [0] * B, [0] * num_pages, page

    def need(self, n):
        return -(-n // self.page)

    def take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def drop(self, p):
        self.refs[p] -= 1
        return self.refs[p] == 0

    def extend(self, n_new):
        new = [a + max(b, 0) for a, b in zip(self.L, n_new)]
        want = sum(self.need(b) - self.need(a) for a, b in zip(self.L, new))
        if want > self.refs.count(0) or max(map(self.need, new)) > len(self.table[0]):
            return -1
        for b, n in enumerate(new):
            for i in range(self.need(self.L[b]), self.need(n)):
                self.table[b][i] = self.take()
        self.L = new
        return want

    def fork(self, parents, children):
        none, B = [(-1, -1)] * len(parents), len(self.L)
        real = [(a, c) for a, c in zip(parents, children) if a >= 0 and c >= 0]
        if any(a >= B or c >= B or a == c or self.L[c] for a, c in real) or len({c for _, c in real}) < len(real):
            return none, -2
        part = [a >= 0 and c >= 0 and self.L[a] % self.page != 0 for a, c in zip(parents, children)]
        if sum(part) > self.refs.count(0):
            return none, -1
        fresh = [self.take() if x else -1 for x in part]
        lens = list(self.L)
        for a, c, x, p in zip(parents, children, part, fresh):
            if a < 0 or c < 0:
                continue
            last, n = lens[a] // self.page, lens[a]
            self.L[c] = n
            for i in range(self.need(n)):
                e = p if x and i == last else self.table[a][i]
                self.table[c][i] = e
                if e >= 0 and not (x and i == last):
                    self.refs[e] += 1
        return [(self.table[a][lens[a] // self.page], p) if x else (-1, -1)
                for a, x, p in zip(parents, part, fresh)], sum(part)

    def trim(self, window, sink):
        freed = 0
        for b, row in enumerate(self.table):
            for i, e in enumerate(row):
                if e >= 0 and i * self.page >= sink and (i + 1) * self.page <= self.L[b] - window:
                    freed += self.drop(e)
                    row[i] = -1
        return freed

    def free(self, seqs):
        if any(s >= len(self.L) for s in seqs):
            return -2
        freed = 0
        for s in {s for s in seqs if s >= 0}:
            freed += sum(self.drop(e) for e in self.table[s] if e >= 0)
            self.table[s], self.L[s] = [-1] * len(self.table[s]), 0
        return freed

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p, r in enumerate(self.refs) if r > 0 and p >= n],
                         [p for p in range(n) if self.refs[p] == 0]))
        to = dict(moves)
        self.table = [[to.get(e, e) for e in row] for row in self.table]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves, n


class Pool:
    def __init__(self, B, max_pages, num_pages):
        dev = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((B, max_pages), -1, **dev)
        self.L, self.refs = torch.zeros(B, **dev), torch.zeros(num_pages, **dev)

    def same(self, m):
        assert self.L.tolist() == m.L
        assert self.table.tolist() == m.table
        assert self.refs.tolist() == m.refs
        flat = [e for row in m.table for e in row if e >= 0]
        assert all(m.refs[p] == flat.count(p) for p in set(flat))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,max_pages,num_pages,page", [
    (1, 1, 1, 8), (5, 9, 40, 8), (70, 33, 1500, 16), (8, 300, 1037, 8), (12, 140, 5000, 64),
])
def test_random_histories_match_the_model(da, B, max_pages, num_pages, page):
    r = random.Random(B * num_pages)
    m, p = Model(B, max_pages, num_pages, page), Pool(B, max_pages, num_pages)
    for step in range(25):
        op = r.choice(["extend", "extend", "fork", "trim", "free", "compact"])
        if op == "extend":
            top = r.choice([2, page, 3 * page, max_pages * page // 2])
            n = [r.randint(-1, top) if r.random() < 0.6 else 0 for _ in range(B)]
            got = da.cache_extend(p.table, p.L, p.refs, _ints(n), page).tolist()
            assert got == [m.extend(n)], (step, op)
        elif op == "fork":
            empty = [b for b in range(B) if m.L[b] == 0]
            k = r.randint(0, len(empty))
            children = [c if r.random() < 0.9 else -1 for c in r.sample(empty, k)]
            full = [b for b in range(B) if m.L[b]] or [-1]
            parents = [r.choice(full) for _ in children]
            copies, got = da.cache_fork(p.table, p.L, p.refs, _ints(parents), _ints(children), page)
            ref, res = m.fork(parents, children)
            assert got.tolist() == [res] and [tuple(c) for c in copies.tolist()] == ref, (step, op)
        elif op == "trim":
            w, s = r.randint(1, 4 * page), r.choice([0, 1, page, page + 1])
            assert da.cache_trim(p.table, p.L, p.refs, page, w, s).tolist() == [m.trim(w, s)], (step, op)
        elif op == "free":
            seqs = [r.randrange(-1, B) for _ in range(r.randint(0, B))]  # with repeats and padding
            assert da.cache_free(p.table, p.L, p.refs, _ints(seqs)).tolist() == [m.free(seqs)], (step, op)
        else:
            own = step % 2 == 0  # into the state's own tensors, or into new ones
            out = (p.table, p.refs) if own else (None, None)
            p.table, p.refs, moves, live = da.cache_compact(p.table, p.refs, *out)
            ref, n = m.compact()
            got = [tuple(c) for c in moves.tolist()]
            assert live.tolist() == [n] and got[: len(ref)] == ref and set(got[len(ref):]) <= {(-1, -1)}, (step, op)
        p.same(m)
    assert da.device_error() == 0


def test_calls_refuse_as_a_whole(da):
    m, p = Model(4, 3, 5, 8), Pool(4, 3, 5)
    assert da.cache_extend(p.table, p.L, p.refs, _ints([20, 9, 0, 0]), 8).tolist() == [5] == [m.extend([20, 9, 0, 0])]
    p.same(m)
    for n in ([0, 8, 0, 0], [10, 0, 0, 0], [0, 0, 25, 0], [2**31 - 1, 0, 0, 0]):  # no page; row full; row too short
        assert da.cache_extend(p.table, p.L, p.refs, _ints(n), 8).tolist() == [-1]
        p.same(m)
    for a, c, want in (([0], [2], -1), ([0], [0], -2), ([0], [1], -2), ([0, 1], [2, 2], -2), ([0], [4], -2),
                       ([4], [2], -2), ([0, -1], [2, 3], -1)):
        copies, res = da.cache_fork(p.table, p.L, p.refs, _ints(a), _ints(c), 8)
        assert res.tolist() == [want] and copies.eq(-1).all()
        p.same(m)
    assert da.cache_free(p.table, p.L, p.refs, _ints([0, 4])).tolist() == [-2]
    p.same(m)
    with pytest.raises(da.DiffAttnError):
        da.cache_extend(p.table, p.L, p.refs, _ints([0] * 4), 12)
    with pytest.raises(da.DiffAttnError):
        da.cache_trim(p.table, p.L, p.refs, 8, 0, 4)
    with pytest.raises(TypeError):
        da.cache_free(p.table, p.L, p.refs, torch.tensor([0], device="cuda"))
    with pytest.raises(ValueError):
        da.cache_extend(p.table, p.L[:3], p.refs, _ints([0] * 4), 8)
    with pytest.raises(da.DiffAttnError):
        big = Pool(2049, 1, 4)
        da.cache_extend(big.table, big.L, big.refs, torch.zeros_like(big.L), 8)
    assert da.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,Hkv,D", [(8, 1, 8), (16, 8, 128), (64, 3, 64)])
def test_copy_pages(da, page, Hkv, D, dtype):
    N = 50
    k = torch.randn(N, page, Hkv, D, device="cuda").to(dtype)
    v = torch.randn(N, page, Hkv, D, device="cuda").to(dtype)
    pairs = [(0, 49), (0, 48), (-1, -1), (7, 20), (3, -1), (50, 1), (2, 50), (5, 21)]
    rk, rv = k.clone(), v.clone()
    for a, b in pairs:
        if 0 <= a < N and 0 <= b < N:
            rk[b], rv[b] = k[a], v[a]
    da.cache_copy_pages(k, v, _ints(pairs))
    assert torch.equal(k, rk) and torch.equal(v, rv)
    da.cache_copy_pages(k, v, _ints(pairs)[:0])
    with pytest.raises(da.DiffAttnError):
        da.cache_copy_pages(k, k, _ints(pairs))
    with pytest.raises(ValueError):
        da.cache_copy_pages(k, v[:10], _ints(pairs))


def test_large_pool(da):
    """A pool of a million pages, of which the last few thousand are free or used."""
    N = 1 << 20
    p = Pool(3, 4000, N)
    p.refs[: N - 3000] = 1
    assert da.cache_extend(p.table, p.L, p.refs, _ints([16000, 8, 0]), 8).tolist() == [2001]
    assert p.table[0, :2000].tolist() == list(range(N - 3000, N - 1000))
    assert p.table[1, 0].item() == N - 1000
    p.refs[:500000] = 0
    live = int((p.refs > 0).sum())
    table, refs, moves, got = da.cache_compact(p.table, p.refs)
    assert got.tolist() == [live] and bool((refs[:live] > 0).all()) and int(refs[live:].abs().sum()) == 0
    k = int((p.refs[live:] > 0).sum())
    assert bool((moves[k:] == -1).all())
    src = torch.nonzero(p.refs[live:] > 0).flatten().int() + live
    dst = torch.nonzero(p.refs[:live] == 0).flatten().int()
    assert torch.equal(moves[:k, 0], src) and torch.equal(moves[:k, 1], dst)
    to = torch.arange(N, device="cuda", dtype=torch.int32)
    to[src.long()] = dst
    assert torch.equal(table[p.table >= 0], to[p.table[p.table >= 0].long()])


def test_a_serving_run(da):
    """Prompts, a fork, decode steps, trimming, dropping, compaction: at every step the attention over
    the pages equals the oracle on each sequence's own keys."""
    B, Hq, Hkv, D, page, window, sink, N = 5, 8, 2, 128, 8, 24, 5, 40
    sections = (16, 24, 24)
    P = sum(sections)
    inv = (10000.0 ** (-torch.arange(P, device="cuda").double() / P)).float()
    pool = Pool(B, 16, N)
    kc = torch.full((N, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    keys = [([], []) for _ in range(B)]  # every sequence's turned keys and values, kept apart
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731

    def grow(n_new):
        assert da.cache_extend(pool.table, pool.L, pool.refs, _ints(n_new), page).item() >= 0
        T = sum(n_new)
        q, k, v = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D)
        cu = _ints([0] + torch.tensor(n_new).cumsum(0).tolist())
        at = torch.cat([torch.arange(n - a, n) for a, n in zip(n_new, pool.L.tolist())])
        pos = torch.stack((at, at // 4, at % 4)).int().cuda()
        qr = da.rope_append_paged(q, k, v, pos, inv, sections, kc, vc, pool.table, pool.L, cu_seqlens=cu)
        kr = da.rope(k, None, pos, inv, sections)[0]
        for b in range(B):
            for t in range(int(cu[b]), int(cu[b + 1])):
                keys[b][0].append(kr[t].cpu())
                keys[b][1].append(v[t].cpu())
        return qr, cu

    def attend(qr, cu):
        live = [b for b in range(B) if int(cu[b + 1]) > int(cu[b])]
        q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        for b in live:
            q[b] = qr[int(cu[b + 1]) - 1]
        lam = torch.sigmoid(torch.randn(B, Hq // 2, generator=g, device="cuda"))
        out = da.decode_paged(q, kc, vc, pool.table, pool.L, lam, window=window, sink=sink)
        for b in live:
            kk, vv = (torch.stack(x)[None] for x in keys[b])
            ref = ora.decode(q[b:b + 1].cpu(), kk, vv, [len(keys[b][0])], lam[b:b + 1].cpu(), window=window, sink=sink)
            bf16_close(out[b:b + 1], ref, f"sequence {b} of {len(keys[b][0])} keys")

    attend(*grow([30, 3, 57, 0, 0]))
    copies, took = da.cache_fork(pool.table, pool.L, pool.refs, _ints([2, 1]), _ints([3, 4]), page)
    assert took.tolist() == [2]
    da.cache_copy_pages(kc, vc, copies)
    keys[3], keys[4] = ([list(x) for x in keys[i]] for i in (2, 1))
    for step in range(14):
        attend(*grow([1, 1, 1, 1, 1]))
        da.cache_trim(pool.table, pool.L, pool.refs, page, window, sink)
        if step == 6:
            assert da.cache_free(pool.table, pool.L, pool.refs, _ints([2])).item() > 0
            keys[2] = ([], [])
            pool.table, pool.refs, moves, live = da.cache_compact(pool.table, pool.refs)
            da.cache_copy_pages(kc, vc, moves)
            kc[live.item():] = float("nan")
            vc[live.item():] = float("nan")
    attend(*grow([4, 0, 9, 1, 2]))
    assert da.device_error() == 0


def test_chained_calls_without_synchronisation(da):
    """Steps queued one behind the other give the bits of steps with a wait after every call."""
    B, Hq, Hkv, page, N, steps, window, sink = 6, 8, 2, 16, 90, 60, 70, 3
    inv = 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    g = torch.Generator(device="cuda").manual_seed(11)
    toks = torch.randn(steps, B, Hq + 2 * Hkv, 128, generator=g, device="cuda").bfloat16()
    lam = torch.rand(steps, B, Hq // 2, generator=g, device="cuda")
    one = torch.ones(B, dtype=torch.int32, device="cuda")

    def run(wait):
        def done(x=None):
            if wait:
                torch.cuda.synchronize()
            return x

        pool = Pool(B, 16, N)
        kc = torch.zeros(N, page, Hkv, 128, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        outs = []
        for i in range(steps):
            done(da.cache_extend(pool.table, pool.L, pool.refs, one, page))
            q, k, v = toks[i].split([Hq, Hkv, Hkv], 1)
            pos = done((pool.L[None] - 1).contiguous())
            qr = done(da.rope_append_paged(q, k, v, pos, inv, (64,), kc, vc, pool.table, pool.L))
            outs.append(done(da.decode_paged(qr * 1.0, kc, vc, pool.table, pool.L, lam[i], window=window, sink=sink)))
            done(da.cache_trim(pool.table, pool.L, pool.refs, page, window, sink))
            if i == 30:
                done(da.cache_free(pool.table, pool.L, pool.refs, _ints([1, 4])))
                c, _ = done(da.cache_fork(pool.table, pool.L, pool.refs, _ints([0, 5]), _ints([1, 4]), page))
                done(da.cache_copy_pages(kc, vc, c))
                pool.table, pool.refs, m, _ = done(da.cache_compact(pool.table, pool.refs))
                done(da.cache_copy_pages(kc, vc, m))
        torch.cuda.synchronize()
        return torch.stack(outs), pool.table, pool.refs, pool.L, kc, vc

    ref = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), ref))
    assert da.device_error() == 0
