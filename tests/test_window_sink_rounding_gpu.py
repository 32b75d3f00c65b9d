"""The two-bf16-term products of the training pass with sinks: O_b and dQ against 64 bits where the sinks
resemble one another, at bounds that a product with one term exceeds.

Where the bounds come from. What the kernels round is rounded here in 64-bit arithmetic: the weights P of the
forward and dS of the backward to bf16, with a second bf16 term for keys below a limit, and dQ to bf16; all else
(scores, exponentials, sums) is fp32 in the kernels and exact here, 2^-24 against roundings of 2^-9 to 2^-8. The
model's error with the second term for all sinks is `right`; without it, or with it for the first sinks only,
forward or backward, it is larger by the gap that the test is about. The kernels have to be below the middle of
`right` and the smallest of the wrong ones, and the case counts only where that gap is at least 10 %: some 20
times what the order of the fp32 sums changes of it."""
import functools

import numpy as np
import pytest
import torch

import workloads
from oracle import diffattn_f64 as ora
from tests.parity import grad_close, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def _bf16(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


def _terms(x, two):
    """x rounded to bf16, in the columns (keys) where `two` is true to the sum of two bf16 terms."""
    hi = _bf16(x)
    return np.where(two[None, :], hi + _bf16(x - hi), hi)


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@functools.lru_cache(maxsize=None)
def _exact(S, Hq, lo, sink, window, seed):
    """Inputs whose keys lo .. sink-1 share a direction with every query, and in 64 bits per head: exp(s - max),
    dP, O_b and dQ."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(128, generator=g)
    u /= u.norm()
    case = workloads.PrefillCase(B=1, S=S, Hq=Hq, Hkv=1, D=128, seed=seed + 1)
    inp = workloads.make_prefill(case)
    inp["dout"] = workloads.make_prefill_grad(case)
    inp["q"] = (inp["q"].float() + 2 * u).bfloat16()
    inp["k"][:, lo:sink] = (inp["k"][:, lo:sink].float() + 18 * u).bfloat16()
    q, k, v, _, dout = (inp[n][0].double().numpy() for n in ("q", "k", "v", "lam", "dout"))
    mask = ora.window_mask(S, S, window, sink=sink)
    e, ob = [], []
    for h in range(Hq):
        s = q[:, h] @ k[:, 0].T / np.sqrt(128) + mask
        e.append(np.exp(s - s.max(1, keepdims=True)))
        ob.append(e[h] @ v[:, 0] / e[h].sum(1, keepdims=True))
    dp = [dout[:, p] @ v[:, 0].T for p in range(Hq // 2)]
    host = [inp[n] for n in ("q", "k", "v", "lam", "dout")]
    return inp, e, dp, np.stack(ob, 1), ora.prefill_backward(*host, window=window, sink=sink)


def _model(args, forward, backward):
    """Relative errors of O_b and dQ with the second term for keys below `forward` in P and `backward` in dS."""
    inp, e, dp, ob, ref = _exact(*args)
    k, v, lam, dout = (inp[n][0].double().numpy() for n in ("k", "v", "lam", "dout"))
    keys = np.arange(k.shape[0])
    o_all, dq = np.empty_like(ob), np.empty_like(ob)
    for h in range(ob.shape[1]):
        total = e[h].sum(1, keepdims=True)
        o = _terms(e[h], keys < forward) @ v[:, 0] / total
        ds = e[h] / total * (dp[h // 2] - (dout[:, h // 2] * o).sum(1, keepdims=True))
        ds = -lam[:, h // 2, None] * ds if h % 2 else ds
        ds[0] = 0.0  # one visible key
        o_all[:, h], dq[:, h] = o, _bf16(_terms(ds, keys < backward) @ k[:, 0] / np.sqrt(128))
    return _rel(o_all, ob), _rel(dq, ref[0][0])


CASES = [
    # S, heads, first alike sink, sinks, window
    (500, 4, 0, 64, 60),
    (500, 4, 0, 64, 500),        # the causal mask: a window of every key
    (700, 4, 100, 200, 130),     # a sink tile whose first keys are like any other
    (1300, 4, 512, 640, 60),     # alike sinks past the first 512
    (1300, 4, 512, 1000, 200),
    (1100, 4, 600, 1100, 90),    # the causal mask: sinks of every key
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("S,Hq,lo,sink,window", CASES)
def test_both_terms_of_alike_sinks(da, S, Hq, lo, sink, window, packed):
    args = (S, Hq, lo, sink, window, S + sink)
    inp, _, _, ob_ref, ref = _exact(*args)
    right = _model(args, sink, sink)
    # one term; the second for the first 512 sinks or for the tile before the alike ones only
    some = {0, max(0, lo // 128 * 128)} | ({512} if sink > 512 else set())
    no_forward = [_model(args, f, sink) for f in some]
    no_backward = [_model(args, sink, b) for b in some]
    bound_ob = (right[0] + min(x[0] for x in no_forward)) / 2
    bound_dq = (right[1] + min(x[1] for x in no_forward + no_backward)) / 2
    assert min(bound_ob / right[0], bound_dq / right[1]) >= 1.05, "no case for this test"
    d = {n: t.cuda() for n, t in inp.items()}
    x = [d[n] for n in ("q", "k", "v", "lam")]
    if packed:
        cu = torch.tensor([0, S], dtype=torch.int32, device="cuda")
        x = [t[0] for t in x]
        _, ob, lse = da.prefill_varlen_train(*x, cu, S, window=window, sink=sink)
        grads = da.backward_varlen(*x, ob, lse, d["dout"][0], cu, S, window=window, sink=sink)
        ob, grads = ob[None], [t[None] for t in grads]
    else:
        _, ob, lse = da.prefill_train(*x, window=window, sink=sink)
        grads = da.backward(*x, ob, lse, d["dout"], window=window, sink=sink)
    torch.cuda.synchronize()
    assert da.device_error() == 0
    off_ob, off_dq = _rel(to64(ob[0]), ob_ref), _rel(to64(grads[0][0]), ref[0][0])
    print(f"O_b {off_ob:.2e} (model {right[0]:.2e}, bound {bound_ob:.2e})  dQ {off_dq:.2e} (model {right[1]:.2e}, "
          f"bound {bound_dq:.2e})")
    assert off_ob <= bound_ob, (off_ob, right, no_forward)
    assert off_dq <= bound_dq, (off_dq, right, no_forward, no_backward)
    for g, r, n in zip(grads, ref, ("dq", "dk", "dv", "dlam")):
        grad_close(g, r, f"alike sinks {n}")
