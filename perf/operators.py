"""Measured cases of the sliding-window layer with attention sinks, its rotary positions and its paged cache.

The operators: DiffAttn attention whose queries see the first `sink` keys of their sequence besides the
last `window` ones (prefill, training step and single-token decode over a paged cache), rotary positions
with several axes (on q and k, and fused with the write of k and v into the paged cache), and the page
bookkeeping of such a cache (drop, fork, copy, extend, trim, compact).

`run` computes a case either in elementary torch operations (`own` false) or through this package's entry
points (`own` true); `exact` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

D = 128  # head dimension of the bf16 attention kernels
DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # long-document prefill of a hybrid model's window layer: the repository's 64/8-head layout
        {"name": "prefill", "op": "prefill", "B": 2, "S": 4096, "Hq": 64, "Hkv": 8, "window": 1024, "sink": 4},
        # a serving batch of prompts packed without padding, one token to long, a smaller model
        {"name": "prefill_packed", "op": "prefill", "lens": "1500,1,130,777,64,0,391,1025", "Hq": 16, "Hkv": 4,
         "window": 256, "sink": 16},
        # training step (forward and gradients) of such a layer on one long sequence
        {"name": "train", "op": "train", "B": 1, "S": 4096, "Hq": 32, "Hkv": 8, "window": 1024, "sink": 4},
        # training step on packed documents of odd lengths, sinks wider than a chat preamble
        {"name": "train_packed", "op": "train", "lens": "997,63,1,800,255,414", "Hq": 16, "Hkv": 4, "window": 512,
         "sink": 64},
        # one user's chat, one token: latency
        {"name": "decode_one", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "len_lo": 5003, "len_hi": 5003,
         "window": 1024, "sink": 4, "page": 16, "lens_seed": 1},
        # a full serving batch, one token per sequence: bandwidth
        {"name": "decode_batch", "op": "decode", "B": 64, "Hq": 64, "Hkv": 8, "len_lo": 1024, "len_hi": 8192,
         "window": 4096, "sink": 4, "page": 64, "lens_seed": 2},
        # q and k of a packed batch with image patches, sections for time, height and width
        {"name": "rope", "op": "rope", "T": 16384, "Hq": 64, "Hkv": 8, "D": 128, "sections": "16,24,24",
         "dtype": "bf16", "inverse": False, "interleaved": False},
        # gradients through the rotation, fp32 heads of 64, adjacent pairs, an odd number of tokens
        {"name": "rope_grad_f32", "op": "rope", "T": 2049, "Hq": 16, "Hkv": 4, "D": 64, "sections": "8,12,12",
         "dtype": "f32", "inverse": True, "interleaved": True},
        # decode step: rotate q and k of one token per sequence and write k, v to their pages
        {"name": "append_decode", "op": "append", "B": 64, "chunk": 1, "Hq": 64, "Hkv": 8, "page": 64,
         "ctx": 4096, "sections": "16,24,24"},
        # chunked prefill: the same for 2048 new tokens of each of 4 sequences
        {"name": "append_chunk", "op": "append", "B": 4, "chunk": 2048, "Hq": 64, "Hkv": 8, "page": 64,
         "ctx": 5000, "sections": "16,24,24"},
        # parallel sampling: drop 24 losing branches, fork 24 from the winners, extend, trim behind the window
        {"name": "branch", "op": "branch", "B": 64, "n": 24, "Hkv": 8, "page": 16, "pages": 4096, "max_pages": 512,
         "len_lo": 400, "len_hi": 4000, "grow": 40, "window": 1024, "sink": 4, "lens_seed": 3},
        # giving memory back: the live pages of a fragmented pool move to its front
        {"name": "compact", "op": "compact", "B": 32, "Hkv": 8, "page": 64, "pages": 4001, "max_pages": 128,
         "lens_seed": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([2, 4, 8, 16])
    while hkv * group > 64:
        group //= 2
    return hkv * group, hkv


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "decode", "decode", "rope", "append", "branch", "compact"])
    if op in ("prefill", "train"):
        Hq, Hkv = _heads(rng)
        c = {"op": op, "Hq": Hq, "Hkv": Hkv, "window": _log(rng, 1 if op == "prefill" else 8, 4096),
             "sink": _log(rng, 1, 512)}
        # the plain form's scores bound the size: heads x rows x rows
        budget = 2 * 64 * 4096 ** 2 if op == "prefill" else 32 * 4096 ** 2
        top = int(min(8192, math.sqrt(budget / Hq)))
        if rng.random() < 0.5:
            c["S"] = _log(rng, 1 if op == "prefill" else 16, top)
            c["B"] = max(1, min(4, budget // (Hq * c["S"] ** 2)))
        else:
            n, left, lens = rng.randint(1, 12), min(top, 4096), []
            for _ in range(n):
                lens.append(min(left, rng.choice([0, 1, rng.randint(1, 700), _log(rng, 1, 2500)])))
                left -= lens[-1]
            lens[0] = max(lens[0], 1 if op == "prefill" else 16)
            c["lens"] = ",".join(map(str, lens))
        return c
    if op == "decode":
        Hq, Hkv = _heads(rng)
        ctx = _log(rng, 1, 131072)
        window, sink = _log(rng, 1, 32768), _log(rng, 1, 512)
        most = 64 * 4100 * 8  # keys x KV heads of the largest listed case
        B = max(1, min(_log(rng, 1, 128), most // (min(ctx, window + sink) * Hkv + 1)))
        return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "len_lo": max(1, ctx // rng.choice([1, 2, 8])), "len_hi": ctx,
                "window": window, "sink": sink, "page": rng.choice([8, 16, 32, 64, 128, 256]),
                "lens_seed": rng.randrange(1 << 20)}
    if op == "rope":
        Dh = rng.choice([64, 128])
        a = [4 * rng.randint(0, Dh // 24) for _ in range(3)]
        a[rng.randrange(3)] += 4
        Hq, Hkv = _heads(rng)
        return {"op": op, "T": _log(rng, 1, 16384), "Hq": Hq, "Hkv": Hkv, "D": Dh, "sections": ",".join(map(str, a)),
                "dtype": rng.choice(["bf16", "bf16", "f32"]) if Dh == 64 else "bf16",
                "inverse": rng.random() < 0.5, "interleaved": rng.random() < 0.5}
    if op == "append":
        Hq, Hkv = _heads(rng)
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "chunk": rng.choice([1, 1, _log(rng, 1, max(1, 8192 // B))]), "Hq": Hq, "Hkv": Hkv,
                "page": rng.choice([8, 16, 64, 128]), "ctx": _log(rng, 1, 4096),
                "sections": rng.choice(["16,24,24", "64", "24,40", "8,8,16"])}
    if op == "branch":
        n = rng.randint(1, 24)
        hi = _log(rng, 40, 4000)
        return {"op": op, "B": 2 * n + rng.randint(0, 16), "n": n, "Hkv": rng.choice([2, 4, 8]),
                "page": rng.choice([16, 32]), "pages": rng.randint(6000, 8000), "max_pages": 512,
                "len_lo": 1 + hi // 10, "len_hi": hi, "grow": rng.randint(0, 100), "window": _log(rng, 16, 1024),
                "sink": _log(rng, 1, 128), "lens_seed": rng.randrange(1 << 20)}
    return {"op": "compact", "B": rng.randint(1, 48), "Hkv": rng.choice([2, 4, 8]), "page": rng.choice([8, 16, 32, 64]),
            "pages": _log(rng, 200, 4000), "max_pages": 96, "lens_seed": rng.randrange(1 << 20)}


# ------------------------------------------------------------------------------------------- inputs
def _lens(case):
    """Host-side lengths of a packed batch, or None."""
    return [int(x) for x in case["lens"].split(",")] if "lens" in case else None


def _seqlens(case, n=None):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n or case["B"])]


def _attention_inputs(case, gen, lead, sink_rows):
    """q, k, v bf16 and lambda fp32; the sink keys share a direction with every query, as trained sinks do."""
    Hq, Hkv = case["Hq"], case["Hkv"]
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    u = r(D)
    u = u / u.norm()
    q = r(*lead, Hq, D) + 2 * u
    k = r(*lead, Hkv, D)
    k.view(-1, Hkv, D)[sink_rows] += 18 * u
    lam = torch.sigmoid(r(*lead, Hq // 2))
    return q.bfloat16(), k.bfloat16(), r(*lead, Hkv, D).bfloat16(), lam


def _live_pages(length, case):
    """Logical pages that a window layer still holds for a sequence: its sinks' and its window's."""
    ps = case["page"]
    pages = -(-length // ps)
    keep = min(pages, -(-case["sink"] // ps))
    return [*range(keep), *range(max(keep, max(0, length - case["window"]) // ps), pages)]


def _table(rows, max_pages, num_pages, gen):
    """Block table with the listed logical pages of each sequence on distinct random pages; -1 elsewhere."""
    b = [i for i, row in enumerate(rows) for _ in row]
    p = [x for row in rows for x in row]
    ids = torch.randperm(num_pages, generator=gen, device=DEV)[: len(p)].int()
    table = torch.full((len(rows), max_pages), -1, dtype=torch.int32, device=DEV)
    if p:
        table[torch.tensor(b, device=DEV), torch.tensor(p, device=DEV)] = ids
    return table


def _rope_inputs(case, gen, T, Dh):
    sections = tuple(int(x) for x in case["sections"].split(","))
    P = sum(sections)
    # text runs on the first axis, patches add rows and columns: positions into the hundred thousands
    base = int(torch.randint(0, 120000, (1,), generator=gen, device=DEV))
    pos = torch.stack([base + torch.arange(T, device=DEV)]
                      + [torch.randint(0, 2048, (T,), generator=gen, device=DEV) for _ in sections[1:]]).int()
    inv = (10000.0 ** (-torch.arange(P, dtype=torch.float64, device=DEV) / P)).float()
    return {"positions": pos.contiguous(), "inv_freq": inv, "sections": sections}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("prefill", "train"):
        lens = _lens(case)
        if lens is None:
            B, S = case["B"], case["S"]
            lead = (B, S)
            at = torch.arange(B * S, device=DEV) % S
        else:
            lead = (sum(lens),)
            at = torch.cat([torch.arange(n, device=DEV) for n in lens])
            cu = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
            st.update(cu=cu, max_seqlen=max(lens))
        st["q"], st["k"], st["v"], st["lam"] = _attention_inputs(case, gen, lead, at < case["sink"])
        if op == "train":
            st["dout"] = torch.randn(*lead, case["Hq"] // 2, D, generator=gen, device=DEV).bfloat16()
    elif op == "decode":
        lens = _seqlens(case)
        rows = [_live_pages(n, case) for n in lens]
        held = sum(map(len, rows))
        num_pages = held + held // 8 + 1
        table = _table(rows, -(-case["len_hi"] // case["page"]), num_pages, gen)
        sinks = torch.zeros(num_pages, case["page"], dtype=torch.bool, device=DEV)
        for p in range(min(-(-case["sink"] // case["page"]), table.shape[1])):
            ids = table[:, p]
            sinks[ids[ids >= 0].long(), : case["sink"] - p * case["page"]] = True
        q, _, _, lam = _attention_inputs({**case, "Hkv": 1}, gen, (case["B"],), slice(0, 0))
        _, k, v, _ = _attention_inputs({**case, "Hq": 2}, gen, (num_pages, case["page"]), sinks.view(-1))
        st.update(q=q, k=k, v=v, lam=lam, table=table, seqlens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    elif op == "rope":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        st.update(_rope_inputs(case, gen, case["T"], case["D"]))
        st["q"] = torch.randn(case["T"], case["Hq"], case["D"], generator=gen, device=DEV).to(dt)
        st["k"] = torch.randn(case["T"], case["Hkv"], case["D"], generator=gen, device=DEV).to(dt)
    elif op == "append":
        B, n, ps, Hq, Hkv = case["B"], case["chunk"], case["page"], case["Hq"], case["Hkv"]
        T = B * n
        st.update(_rope_inputs(case, gen, T, D))
        # q, k and v as the columns of one projection's output
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=DEV).bfloat16()
        st["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        old = torch.randint(0, case["ctx"] + 1, (B,), generator=gen, device=DEV)
        per = -(-(case["ctx"] + n) // ps)
        table = _table([list(range(per))] * B, per, B * per + 5, gen)
        st.update(table=table, seqlens=(old + n).int(), cu=(torch.arange(B + 1, device=DEV) * n).int())
        st["kc"] = torch.randn(B * per + 5, ps, Hkv, D, generator=gen, device=DEV).bfloat16()
        st["vc"] = torch.randn(B * per + 5, ps, Hkv, D, generator=gen, device=DEV).bfloat16()
    elif op == "branch":
        B, n, N = case["B"], case["n"], case["pages"]
        parents_n = B - n
        lens = _seqlens(case, parents_n) + [0] * n
        rows = [_live_pages(x, case) if x else [] for x in lens]
        table = _table(rows, case["max_pages"], N, gen)
        refs = torch.zeros(N, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        st.update(table=table, refs=refs, seqlens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        st["children"] = (parents_n + torch.randperm(n, generator=gen, device=DEV)).int()
        st["parents"] = torch.randint(0, parents_n, (n,), generator=gen, device=DEV).int()
        st["n_new"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        st["n_new"][parents_n:] = torch.randint(0, case["grow"] + 1, (n,), generator=gen, device=DEV).int()
        for c in ("kc", "vc"):
            st[c] = torch.randn(N, case["page"], case["Hkv"], D, generator=gen, device=DEV).bfloat16()
    else:
        N, B, width = case["pages"], case["B"], case["max_pages"]
        r = random.Random(case["lens_seed"])
        # sequences hold about 60 % of the pool, on scattered pages
        count = [r.randint(1, width) for _ in range(B)]
        scale = min(1.0, 0.6 * N / sum(count))
        table = _table([list(range(int(c * scale))) for c in count], width, N, gen)
        refs = torch.zeros(N, dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        # the last sequence is a fork of the first
        table[-1] = table[0] if B > 1 else table[-1]
        refs.zero_()
        flat = table.view(-1)
        refs.index_add_(0, flat.clamp(min=0).long(), (flat >= 0).int())
        st.update(table=table, refs=refs)
        for c in ("kc", "vc"):
            st[c] = torch.randn(N, case["page"], case["Hkv"], D, generator=gen, device=DEV).bfloat16()
    return st


# ------------------------------------------------------------------------------------------- run
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_prefill(st):
    import differential_attention_v2_b200 as da

    c = st["case"]
    if "cu" in st:
        return da.prefill_varlen_window(st["q"], st["k"], st["v"], st["lam"], st["cu"], st["max_seqlen"], c["window"],
                                        sink=c["sink"])
    return da.prefill_window(st["q"], st["k"], st["v"], st["lam"], c["window"], sink=c["sink"])


def _own_train(st):
    import differential_attention_v2_b200 as da

    c, x = st["case"], (st["q"], st["k"], st["v"], st["lam"])
    if "cu" in st:
        tail = (st["cu"], st["max_seqlen"])
        out, ob, lse = da.prefill_varlen_train(*x, *tail, window=c["window"], sink=c["sink"])
        dq, dk, dv, dlam = da.backward_varlen(*x, ob, lse, st["dout"], *tail, window=c["window"], sink=c["sink"])
    else:
        out, ob, lse = da.prefill_train(*x, window=c["window"], sink=c["sink"])
        dq, dk, dv, dlam = da.backward(*x, ob, lse, st["dout"], window=c["window"], sink=c["sink"])
    # lambda's gradient goes on into the bf16 projection that lambda came from
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dlam": dlam.bfloat16()}


def _own_decode(st):
    import differential_attention_v2_b200 as da

    c = st["case"]
    return da.decode_paged(st["q"], st["k"], st["v"], st["table"], st["seqlens"], st["lam"], window=c["window"],
                           sink=c["sink"])


def _own_rope(st):
    import differential_attention_v2_b200 as da

    c = st["case"]
    return da.rope(st["q"], st["k"], st["positions"], st["inv_freq"], st["sections"], inverse=c["inverse"],
                   interleaved=c["interleaved"])


def _own_append(st):
    import differential_attention_v2_b200 as da

    q = da.rope_append_paged(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["sections"], st["kc"],
                             st["vc"], st["table"], st["seqlens"], cu_seqlens=st["cu"])
    return {"q": q, "kc": st["kc"], "vc": st["vc"]}


def _own_branch(st):
    import differential_attention_v2_b200 as da

    c, pool = st["case"], (st["table"], st["seqlens"], st["refs"])
    freed = da.cache_free(*pool, st["children"])
    copies, forked = da.cache_fork(*pool, st["parents"], st["children"], c["page"])
    da.cache_copy_pages(st["kc"], st["vc"], copies)
    grown = da.cache_extend(*pool, st["n_new"], c["page"])
    trimmed = da.cache_trim(*pool, c["page"], c["window"], c["sink"])
    return {"table": st["table"], "seqlens": st["seqlens"], "refs": st["refs"], "copies": copies, "forked": forked,
            "grown": grown, "trimmed": trimmed, "kc": st["kc"], "vc": st["vc"]}


def _own_compact(st):
    import differential_attention_v2_b200 as da

    table, refs, moves, live = da.cache_compact(st["table"], st["refs"])
    da.cache_copy_pages(st["kc"], st["vc"], moves)
    return {"table": table, "refs": refs, "moves": moves, "live": live, "kc": st["kc"], "vc": st["vc"]}


_own = {"prefill": _own_prefill, "train": _own_train, "decode": _own_decode, "rope": _own_rope, "append": _own_append,
        "branch": _own_branch, "compact": _own_compact}


# --------------------------------------------------------------------------------- plain forms
def _visible(st):
    """[S, S] (one mask for every batch row): key j is seen from query i of its sequence iff j <= i and
    (i - j < window or j < sink)."""
    c = st["case"]
    if "cu" in st:
        T = st["q"].shape[0]
        t = torch.arange(T, device=DEV, dtype=torch.int32)
        seq = torch.searchsorted(st["cu"][1:].contiguous(), t, right=True)
        at = t - st["cu"][seq]
    else:
        at = torch.arange(st["q"].shape[1], device=DEV)
        seq = torch.zeros_like(at)
    d = at[:, None] - at[None, :]
    return (seq[:, None] == seq[None, :]) & (d >= 0) & ((d < c["window"]) | (at < c["sink"])[None, :])


def _split_heads(x, Hkv):
    """[B,S,H,D] -> fp32 [B,Hkv,(H/Hkv)*S,D]: the heads of one KV head as rows."""
    B, S, H, d = x.shape
    return x.float().reshape(B, S, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)


def _join_heads(x, S):
    B, Hkv, R, d = x.shape
    return x.reshape(B, Hkv, R // S, S, d).permute(0, 3, 1, 2, 4).reshape(B, S, -1, d)


def _weights(q, k, visible):
    """fp32 softmax weights [B,Hkv,G*S,S]."""
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    S = k.shape[-2]
    s = s.view(*s.shape[:2], -1, S, S).masked_fill_(~visible, -math.inf).view(s.shape)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    return s / s.sum(-1, keepdim=True)


def _batched(st, *names):
    return [st[n][None] if "cu" in st else st[n] for n in names]


def _plain_prefill(st):
    c = st["case"]
    q, k, v, lam = _batched(st, "q", "k", "v", "lam")
    S = q.shape[1]
    a = _weights(_split_heads(q, c["Hkv"]), _split_heads(k, c["Hkv"]), _visible(st))
    o = _join_heads(torch.matmul(a, _split_heads(v, c["Hkv"])), S)
    out = (o[:, :, 0::2] - lam[..., None] * o[:, :, 1::2]).bfloat16()
    return out[0] if "cu" in st else out


def _plain_train(st):
    c = st["case"]
    q, k, v, lam, dout = _batched(st, "q", "k", "v", "lam", "dout")
    S = q.shape[1]
    qs, ks, vs = (_split_heads(x, c["Hkv"]) for x in (q, k, v))
    a = _weights(qs, ks, _visible(st))
    o = _join_heads(torch.matmul(a, vs), S)
    o1, o2 = o[:, :, 0::2], o[:, :, 1::2]
    g = dout.float()
    out = o1 - lam[..., None] * o2
    dlam = -(g * o2).sum(-1)
    do = _split_heads(torch.stack((g, -lam[..., None] * g), 3).flatten(2, 3), c["Hkv"])  # per query head
    dv = torch.matmul(a.transpose(-1, -2), do)
    dp = torch.matmul(do, vs.transpose(-1, -2))
    ds = a * (dp - (a * dp).sum(-1, keepdim=True)) / math.sqrt(D)
    dq = _join_heads(torch.matmul(ds, ks), S)
    dk = torch.matmul(ds.transpose(-1, -2), qs)
    r = {"out": out, "dq": dq, "dk": dk.transpose(1, 2), "dv": dv.transpose(1, 2), "dlam": dlam}
    return {n: (x[0] if "cu" in st else x).bfloat16() for n, x in r.items()}


def _plain_decode(st):
    c = st["case"]
    B, ps = c["B"], c["page"]
    L = st["seqlens"].long()[:, None]
    lo = (L - c["window"]).clamp(min=0)
    # the visible positions of each sequence: its sinks below the window, then the window
    n_sink, n_win = min(c["sink"], c["len_hi"]), min(c["window"], c["len_hi"])
    j = torch.cat((torch.arange(n_sink, device=DEV).expand(B, -1), lo + torch.arange(n_win, device=DEV)), 1)
    ok = torch.cat((j[:, :n_sink] < torch.minimum(lo, L), j[:, n_sink:] < L), 1)
    j = torch.where(ok, j, torch.zeros_like(j))
    row = st["table"].long().gather(1, j // ps).clamp(min=0) * ps + j % ps
    k = st["k"].view(-1, c["Hkv"], D)[row].float().transpose(1, 2)
    v = st["v"].view(-1, c["Hkv"], D)[row].float().transpose(1, 2)
    q = st["q"].float().view(B, c["Hkv"], -1, D)
    s = (torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)).masked_fill(~ok[:, None, None], -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(s / s.sum(-1, keepdim=True), v).reshape(B, c["Hq"], D)
    return (o[:, 0::2] - st["lam"][..., None] * o[:, 1::2]).bfloat16()


def _angles(st, sign):
    """cos and sin [T, P] of each token's rotation angles; angles of far positions need 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device=DEV),
                                   torch.tensor(st["sections"], device=DEV), output_size=sum(st["sections"]))
    a = st["positions"].double()[axis].T * st["inv_freq"].double()
    return torch.cos(a).float(), sign * torch.sin(a).float()


def _rotate(x, cos, sin, interleaved):
    P = cos.shape[1]
    x = x.float()
    rot, rest = x[..., : 2 * P], x[..., 2 * P:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :P], rot[..., P:])
    cos, sin = cos[:, None], sin[:, None]
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, rest), -1)


def _plain_rope(st):
    c = st["case"]
    cos, sin = _angles(st, -1.0 if c["inverse"] else 1.0)
    return tuple(_rotate(st[n], cos, sin, c["interleaved"]).to(st[n].dtype) for n in ("q", "k"))


def _plain_append(st):
    c = st["case"]
    cos, sin = _angles(st, 1.0)
    t = torch.arange(st["q"].shape[0], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:].contiguous(), t, right=True)
    at = (st["seqlens"][b] - st["cu"][b + 1] + t).long()
    row = st["table"][b, at // c["page"]].long() * c["page"] + at % c["page"]
    st["kc"].view(-1, c["Hkv"], D)[row] = _rotate(st["k"], cos, sin, False).bfloat16()
    st["vc"].view(-1, c["Hkv"], D)[row] = st["v"]
    return {"q": _rotate(st["q"], cos, sin, False).bfloat16(), "kc": st["kc"], "vc": st["vc"]}


def _count(refs, pages, by):
    """refs[p] += by for every entry p >= 0; returns how many pages came to rest at 0."""
    pages = pages.reshape(-1)
    before = refs > 0
    refs.index_add_(0, pages.clamp(min=0).long(), by * (pages >= 0).int())
    return (before & (refs == 0)).sum().int().view(1)


def _take(refs, want):
    """The free pages, lowest first, for the true entries of `want` in their order; -1 for the others."""
    order = torch.argsort((refs != 0).int(), stable=True).int()
    rank = torch.cumsum(want.reshape(-1).int(), 0) - 1
    ids = torch.where(want.reshape(-1), order[rank.clamp(min=0)], -1).view(want.shape)
    _count(refs, ids, 1)
    return ids, want.sum().int().view(1)


def _copy_pages(st, copies):
    c = copies[copies[:, 0] >= 0].long()
    for x in (st["kc"], st["vc"]):
        x[c[:, 1]] = x[c[:, 0]]


def _plain_branch(st):
    c = st["case"]
    table, seqlens, refs, ps = st["table"], st["seqlens"], st["refs"], c["page"]
    child, parent = st["children"].long(), st["parents"].long()
    _count(refs, table[child], -1)
    table[child], seqlens[child] = -1, 0
    # fork: whole pages are shared, a partly filled last page is copied to a page of its own
    L = seqlens[parent]
    rows, last = table[parent], (L // ps).long()
    part = L % ps != 0
    src = torch.where(part, rows.gather(1, last.clamp(max=rows.shape[1] - 1)[:, None])[:, 0], -1)
    dst, forked = _take(refs, part)
    logical = torch.arange(rows.shape[1], device=DEV)
    own_page = (logical == last[:, None]) & part[:, None]
    _count(refs, torch.where(own_page, -1, rows), 1)
    table[child], seqlens[child] = torch.where(own_page, dst[:, None], rows), L
    copies = torch.stack((src, dst), 1)
    _copy_pages(st, copies)
    # extend
    new = seqlens + st["n_new"]
    want = (logical >= ((seqlens + ps - 1) // ps)[:, None]) & (logical < ((new + ps - 1) // ps)[:, None])
    ids, grown = _take(refs, want)
    table.copy_(torch.where(want, ids, table))
    seqlens.copy_(new)
    # trim: pages that hold neither a sink nor a key of the window
    gone = (logical >= -(-c["sink"] // ps)) & (logical < ((seqlens - c["window"]).clamp(min=0) // ps)[:, None])
    trimmed = _count(refs, torch.where(gone, table, -1), -1)
    table.masked_fill_(gone, -1)
    return {"table": table, "seqlens": seqlens, "refs": refs, "copies": copies, "forked": forked, "grown": grown,
            "trimmed": trimmed, "kc": st["kc"], "vc": st["vc"]}


def _plain_compact(st):
    refs, N = st["refs"], st["refs"].numel()
    i = torch.arange(N, device=DEV, dtype=torch.int32)
    live = refs > 0
    n = live.sum().int()
    src, dst = i[live & (i >= n)], i[~live & (i < n)]
    moves = torch.full((N // 2, 2), -1, dtype=torch.int32, device=DEV)
    moves[: src.numel()] = torch.stack((src, dst), 1)
    to = i.clone()
    to[src.long()] = dst
    new_refs = torch.zeros_like(refs)
    new_refs[to[live].long()] = refs[live]
    table = torch.where(st["table"] >= 0, to[st["table"].clamp(min=0).long()], -1)
    _copy_pages(st, moves)
    return {"table": table, "refs": new_refs, "moves": moves, "live": n.view(1), "kc": st["kc"], "vc": st["vc"]}


_plain = {"prefill": _plain_prefill, "train": _plain_train, "decode": _plain_decode, "rope": _plain_rope,
          "append": _plain_append, "branch": _plain_branch, "compact": _plain_compact}


# ------------------------------------------------------------------------------------------- work
def _pairs(n, window, sink):
    """Visible (query, key) pairs of a causal sequence of n tokens."""
    full = sum(min(i + 1, window) for i in range(n))
    return full + sum(min(sink, max(0, i + 1 - window)) for i in range(n))


def work(case):
    op = case["op"]
    if op in ("prefill", "train"):
        lens = _lens(case) or [case["S"]] * case["B"]
        T, Hq, Hkv = sum(lens), case["Hq"], case["Hkv"]
        pairs = sum(_pairs(n, case["window"], case["sink"]) for n in lens)
        io = 2 * D * T * (Hq + 2 * Hkv) + 4 * T * Hq // 2  # q, k, v, lambda
        out = 2 * D * T * Hq // 2
        if op == "prefill":
            return {"bytes": io + out, "flops": 4 * D * Hq * pairs}
        # forward (scores, values) and, per pair of heads, one dP, dV, and per head scores, dQ, dK
        return {"bytes": io + 2 * out + 2 * D * T * (Hq + 2 * Hkv) + 2 * T * Hq // 2,
                "flops": 4 * D * Hq * pairs + (2 * 2 + 2 * 3 * 2) * D * (Hq // 2) * pairs}
    if op == "decode":
        keys = sum(min(n, case["window"]) + min(case["sink"], max(0, n - case["window"])) for n in _seqlens(case))
        rows = case["B"] * case["Hq"]
        return {"bytes": 4 * D * case["Hkv"] * keys + 3 * D * rows + 2 * rows, "flops": 4 * D * keys * case["Hq"]}
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        size = 4 if case["dtype"] == "f32" else 2
        sections = case["sections"].split(",")
        return {"bytes": 2 * size * n + 4 * case["T"] * len(sections), "flops": 3 * n}
    if op == "append":
        T = case["B"] * case["chunk"]
        n = T * (case["Hq"] + 2 * case["Hkv"]) * D
        return {"bytes": 4 * n + 4 * T * len(case["sections"].split(",")), "flops": 3 * n}
    page = 2 * 2 * case["page"] * case["Hkv"] * D  # k and v
    if op == "branch":
        return {"bytes": 2 * page * case["n"] + 8 * case["B"] * case["max_pages"] + 8 * case["pages"],
                "flops": case["B"] * case["max_pages"]}
    # about 40 % of the live pages lie behind the front, and move
    moved = 0.24 * min(case["pages"], sum(random.Random(case["lens_seed"]).randint(1, case["max_pages"])
                                          for _ in range(case["B"])) / 0.6)
    return {"bytes": 2 * page * moved + 8 * case["B"] * case["max_pages"] + 12 * case["pages"], "flops": case["pages"]}


# ------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    return {"prefill": _exact_attention, "train": _exact_attention, "decode": _exact_decode, "rope": _exact_rope,
            "append": _exact_append, "branch": _exact_branch, "compact": _exact_compact}[case["op"]](prepare(case, seed))


def _exact_head(q, k, v, window, sink):
    """One head of one sequence in 64 bits: sum over keys of exp(s - logsumexp(s)) v."""
    n = q.shape[0]
    i = torch.arange(n, device=DEV)
    hidden = (i[None, :] > i[:, None]) | ((i[None, :] <= i[:, None] - window) & (i[None, :] >= sink))
    s = (q @ k.T) * D ** -0.5
    s = s.masked_fill(hidden, -math.inf)
    return torch.exp(s - torch.logsumexp(s, 1, keepdim=True)) @ v


def _exact_attention(st):
    c = st["case"]
    names = ("q", "k", "v", "lam")
    if "cu" in st:
        ends = torch.tensor(_lens(c)).cumsum(0).tolist()
        spans = [slice(e - n, e) for n, e in zip(_lens(c), ends)]
    else:
        spans = range(c["B"])
    grads = c["op"] == "train"
    r = {n: torch.zeros(st[n].shape, dtype=torch.float64, device=DEV) for n in names}
    out = torch.zeros(*st["lam"].shape, D, dtype=torch.float64, device=DEV)
    group = c["Hq"] // c["Hkv"]
    for at in spans:
        for p in range(c["Hq"] // 2):
            g = 2 * p // group
            leaves = [st["q"][at][:, 2 * p].double(), st["q"][at][:, 2 * p + 1].double(), st["k"][at][:, g].double(),
                      st["v"][at][:, g].double(), st["lam"][at][:, p].double()]
            if leaves[0].shape[0] == 0:
                continue
            for x in leaves:
                x.requires_grad_(grads)
            q1, q2, k, v, lam = leaves
            o = (_exact_head(q1, k, v, c["window"], c["sink"])
                 - lam[:, None] * _exact_head(q2, k, v, c["window"], c["sink"]))
            out[at][:, p] = o.detach()
            if grads:
                d = torch.autograd.grad(o, leaves, st["dout"][at][:, p].double())
                r["q"][at][:, 2 * p], r["q"][at][:, 2 * p + 1], r["lam"][at][:, p] = d[0], d[1], d[4]
                r["k"][at][:, g] += d[2]
                r["v"][at][:, g] += d[3]
    return out if not grads else {"out": out, "dq": r["q"], "dk": r["k"], "dv": r["v"], "dlam": r["lam"]}


def _exact_decode(st):
    c, out = st["case"], []
    table = st["table"].cpu()
    for b, n in enumerate(st["seqlens"].tolist()):
        keys = torch.tensor([j for j in range(n) if j < c["sink"] or j >= n - c["window"]])
        page, row = table[b][keys // c["page"]].long().to(DEV), (keys % c["page"]).to(DEV)
        k, v = st["k"][page, row].double(), st["v"][page, row].double()
        q = st["q"][b].double().view(c["Hkv"], -1, D)
        s = torch.einsum("ghd,ngd->ghn", q, k) * D ** -0.5
        a = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
        o = torch.einsum("ghn,ngd->ghd", a, v).reshape(c["Hq"] // 2, 2, D)
        out.append(o[:, 0] - st["lam"][b].double()[:, None] * o[:, 1])
    return torch.stack(out)


def _exact_turn(x, st, inverse=False, interleaved=False):
    """Each pair as a complex number times exp(i angle)."""
    f, turn = 0, []
    for a, s in enumerate(st["sections"]):
        turn.append(st["positions"][a].double()[:, None] * st["inv_freq"][f: f + s].double())
        f += s
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.cat(turn, 1))[:, None]
    z = z.conj() if inverse else z
    y = x.double().clone()
    if interleaved:
        y[..., : 2 * f] = torch.view_as_real(torch.view_as_complex(y[..., : 2 * f].unflatten(-1, (f, 2)).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(y[..., :f].contiguous(), y[..., f: 2 * f].contiguous()) * z
        y[..., :f], y[..., f: 2 * f] = w.real, w.imag
    return y


def _exact_rope(st):
    c = st["case"]
    return tuple(_exact_turn(st[n], st, c["inverse"], c["interleaved"]) for n in ("q", "k"))


def _exact_append(st):
    c = st["case"]
    k, kc, vc = _exact_turn(st["k"], st), st["kc"].double(), st["vc"].double()
    table, L = st["table"].tolist(), st["seqlens"].tolist()
    page, row = [], []
    for b in range(c["B"]):
        for i in range(c["chunk"]):
            at = L[b] - c["chunk"] + i
            page.append(table[b][at // c["page"]])
            row.append(at % c["page"])
    page, row = torch.tensor(page, device=DEV), torch.tensor(row, device=DEV)
    kc[page, row], vc[page, row] = k, st["v"].double()
    return {"q": _exact_turn(st["q"], st), "kc": kc, "vc": vc}


def _exact_pool(st, copies):
    """The caches after the copies, in their order; no page is written before it is read."""
    for a, b in copies:
        for x in (st["kc"], st["vc"]):
            x[b] = x[a]
    return {"kc": st["kc"].double(), "vc": st["vc"].double()}


def _exact_branch(st):
    # entry by entry on lists, from the definition
    c, ps = st["case"], st["case"]["page"]
    table, L, refs = st["table"].tolist(), st["seqlens"].tolist(), st["refs"].tolist()
    children, n_new = st["children"].tolist(), st["n_new"].tolist()

    def take():
        p = refs.index(0)
        refs[p] = 1
        return p

    copies = []
    parents = st["parents"].tolist()
    part = [L[a] % ps != 0 for a in parents]
    fresh = [take() if x else -1 for x in part]
    for a, b, x, p in zip(parents, children, part, fresh):
        last = L[a] // ps
        table[b], L[b] = list(table[a]), L[a]
        copies.append((table[a][last], p) if x else (-1, -1))
        if x:
            table[b][last] = p
        for i, e in enumerate(table[b]):
            if e >= 0 and not (x and i == last):
                refs[e] += 1
    grown = 0
    for b in range(c["B"]):
        new = L[b] + n_new[b]
        for i in range(-(-L[b] // ps), -(-new // ps)):
            table[b][i] = take()
            grown += 1
        L[b] = new
    trimmed = 0
    for b in range(c["B"]):
        for i, e in enumerate(table[b]):
            if e >= 0 and i * ps >= c["sink"] and (i + 1) * ps <= L[b] - c["window"]:
                refs[e] -= 1
                trimmed += refs[e] == 0
                table[b][i] = -1
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"table": whole(table), "seqlens": whole(L), "refs": whole(refs), "copies": whole(copies),
            "forked": whole([sum(part)]), "grown": whole([grown]), "trimmed": whole([trimmed]),
            **_exact_pool(st, [x for x in copies if x[0] >= 0])}


def _exact_compact(st):
    refs, table = st["refs"].tolist(), st["table"].tolist()
    n = sum(r > 0 for r in refs)
    moves = list(zip([p for p in range(n, len(refs)) if refs[p] > 0], [p for p in range(n) if refs[p] == 0]))
    to = dict(moves)
    table = [[to.get(e, e) for e in row] for row in table]
    new = [0] * len(refs)
    for p, r in enumerate(refs):
        if r > 0:
            new[to.get(p, p)] = r
    pad = moves + [(-1, -1)] * (len(refs) // 2 - len(moves))
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"table": whole(table), "refs": whole(new), "moves": whole(pad), "live": whole([n]), **_exact_pool(st, moves)}
