"""Verification of chains drafted and verified under sampling settings, on the
GPU, against the 64-bit rule in sample_ref.py: lengths and tokens have to be
equal (the sums' 2^-40 meets no decision of the seeded inputs)."""
import numpy as np
import pytest
import torch

import sample_ref
from speculative_decoding_draft_depth_gb300 import ddt
from test_gpu_sample import make_ctx, rows, settings, to_filter

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"bf16": ddt.BF16, "f32": ddt.F32}


def inputs(R, L, V, seed, draft="bf16", target="bf16", spread=3.0, noise=0.5, sd=None):
    """Draft rows, target rows near them, guesses from the draft rows' distributions."""
    base = rows(R * (L + 1), V, seed, spread, torch.float32).view(R, L + 1, V)
    t = (base + noise * rows(R * (L + 1), V, seed + 1, 1.0, torch.float32).view(R, L + 1, V)).to(TYPES[target])
    d = base[:, :L].to(TYPES[draft]).contiguous()
    rng = np.random.default_rng(seed)
    sd = sd or settings(R)
    tok = np.array([[sample_ref.pick(sample_ref.distribution(z, *(x[i] for x in sd)), rng.random())
                     for z in d[i].double().cpu().numpy()] for i in range(R)], dtype=np.int32).reshape(R, L)
    return d, t.contiguous(), tok, rng.random((R, L), dtype=np.float32), rng.random(R, dtype=np.float32)


def run(ctx, d, t, tok, u, r, sd=None, st=None, n=None):
    R, L = tok.shape
    al = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    at = torch.full((R, L + 1), -7, dtype=torch.int32, device="cuda")
    ctx.ddt_accept_sampled(d, t, torch.from_numpy(tok).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda(), R,
                           al, at, draft_filter=None if sd is None else to_filter(sd),
                           target_filter=None if st is None else to_filter(st),
                           n_guess=None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    return al.tolist(), at.tolist(), ctx.ddt_device_status()


def check(d, t, tok, u, r, sd=None, st=None, n=None, ctx=None, status=0):
    R, L = tok.shape
    V = d.shape[2]
    code = lambda x: ddt.F32 if x.dtype == torch.float32 else ddt.BF16  # noqa: E731
    ctx = ctx or make_ctx(V, R, L, code(d), code(t))
    al, at, got = run(ctx, d, t, tok, u, r, sd, st, n)
    f32 = lambda s, i: tuple(x[i] if j == 1 else float(np.float32(x[i])) for j, x in enumerate(s or settings(R)))  # noqa: E731
    for i in range(R):
        m = L if n is None else min(max(n[i], 0), L)
        wl, wt = sample_ref.chain(d[i].double().cpu().numpy(), t[i].double().cpu().numpy(), tok[i], u[i], float(r[i]), m,
                                  f32(sd, i), f32(st, i))
        assert (al[i], at[i]) == (wl, wt), i
    assert got == status
    return al, at


CASES = {
    "none": (dict(), dict()),
    "temperature": (dict(T=0.7), dict(T=1.2)),
    "top_k": (dict(T=0.9, k=20), dict(T=0.9, k=20)),
    "top_p": (dict(p=0.9), dict(p=0.8)),
    "min_p": (dict(m=0.02), dict(T=1.3, m=0.1)),
    "all": (dict(T=0.8, k=64, p=0.95, m=0.01), dict(T=0.9, k=50, p=0.9, m=0.02)),
    "greedy_target": (dict(T=0.5), dict(T=0.0)),
    "greedy_both": (dict(T=0.0), dict(T=0.0)),
    "greedy_draft": (dict(T=0.0), dict(T=1.0, p=0.9)),
}


@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-bf16", "f32-f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_settings(name, types):
    draft, target = types.split("-")
    R, L, V = 7, 4, 5003
    sd, st = (settings(R, **x) for x in CASES[name])
    d, t, tok, u, r = inputs(R, L, V, 31, draft, target, sd=sd)
    check(d, t, tok, u, r, sd, st)


@pytest.mark.parametrize("V", [1, 2, 9, 100, 1025, 32000])
@pytest.mark.parametrize("L", [1, 6, 18])
def test_sizes(V, L):
    R = 3
    sd, st = settings(R, T=[0.6, 1.0, 1.4], p=[0.9, 1.0, 0.7]), settings(R, T=1.1, k=[0, 12, 300])
    for draft, target in (("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")):
        check(*inputs(R, L, V, 7 + V, draft, target, sd=sd), sd, st)


def test_full_vocabulary():
    R, L, V = 4, 5, 151936
    sd, st = settings(R, T=[1.0, 0.8, 0.0, 1.2], k=[0, 50, 0, 0], p=[1.0, 0.9, 1.0, 0.95]), settings(R, T=0.9, p=[1.0, 0.9, 0.95, 0.99])
    check(*inputs(R, L, V, 3, spread=2.5, noise=0.3, sd=sd), sd, st)


def test_prefixes_and_counts_out_of_range():
    R, L, V = 6, 5, 3001
    d, t, tok, u, r = inputs(R, L, V, 5, noise=0.1)
    st = settings(R, k=40)
    check(d, t, tok, u, r, None, st, n=[0, 1, 3, 5, 2, 4])
    check(d, t, tok, u, r, None, st, n=[0, -2, 3, 9, 2, 4], status=ddt.DEV_BAD_TREE)


def test_rows_behind_a_prefix_are_not_read():
    R, L, V = 3, 4, 3001
    d, t, tok, u, r = inputs(R, L, V, 6, noise=0.05)
    n = [0, 2, 4]
    for i in range(R):
        d[i, n[i]:] = torch.nan
        t[i, n[i] + 1:] = torch.nan
    check(d, t, tok, u, r, settings(R, p=0.9), settings(R, p=0.9), n=n)


def test_guesses_out_of_range():
    R, L, V = 3, 3, 2000
    d, t, tok, u, r = inputs(R, L, V, 8, noise=0.01)
    tok[0, 0], tok[1, 1], tok[2, 2] = -1, V, 2 ** 31 - 1
    check(d, t, tok, u * 0.01, r, status=ddt.DEV_BAD_TREE)


def test_guess_outside_the_drafter_s_kept_set():
    """q(x) = 0 counts as ratio 1, even where p(x) = 0 as well."""
    R, L, V = 2, 2, 500
    d, t, tok, u, r = inputs(R, L, V, 9, noise=0.01)
    tok[:, 0] = d[:, 0].float().argmin(1).cpu().numpy()
    check(d, t, tok, u, r, settings(R, k=5), settings(R, k=5))


def test_same_rows_are_always_kept():
    R, L, V = 5, 6, 4001
    d, t, tok, u, r = inputs(R, L, V, 10, noise=0.0)
    st = settings(R, T=0.8, k=30, p=0.9)
    sd = [list(x) for x in st]
    tok = inputs(R, L, V, 10, noise=0.0, sd=sd)[2]
    al, _ = check(d, t, tok, u, r, sd, st)
    assert al == [L + 1] * R


def test_empty_rows_and_special_values():
    R, L, V = 5, 2, 1000
    d, t, tok, u, r = inputs(R, L, V, 11, noise=0.2)
    d[0, 0] = -torch.inf          # no draft weights: ratio 1
    t[1, 0] = -torch.inf          # no target weights: the guess is dropped, nothing to draw
    t[2, :, ::2] = -torch.inf
    d[3, 0, 17] = torch.inf
    t[3, 0, 17] = t[3, 0, 400] = torch.inf
    tok[3, 0] = 17
    t[4] = torch.finfo(torch.bfloat16).min
    al, at = check(d, t, tok, u, r, settings(R, p=0.9), settings(R, T=1.2))
    assert al[1] == 1 and at[1][0] == -1


def test_nan_logits_are_reported():
    R, L, V = 2, 2, 1000
    d, t, tok, u, r = inputs(R, L, V, 12, noise=0.2)
    d[0, 0, 3] = torch.nan
    t[1, 1, 5] = torch.nan
    check(d, t, tok, u, r, settings(R, p=0.9), settings(R), status=ddt.DEV_NAN_LOGITS)


def test_bad_settings():
    R, L, V = 3, 2, 1000
    d, t, tok, u, r = inputs(R, L, V, 13, noise=0.0)
    ctx = make_ctx(V, R, L)
    good = run(ctx, d, t, tok, u, r)
    al, at, st = run(ctx, d, t, tok, u, r, settings(R, T=[1.0, -1.0, 1.0]), settings(R, p=[1.0, 1.0, 2.0]))
    assert st == ddt.DEV_BAD_SETTING
    assert al[1:] == [1, 1] and at[1:] == [[-1] * (L + 1)] * 2
    assert (al[0], at[0]) == (good[0][0], good[1][0])


def test_without_settings_it_is_the_rule_at_temperature_1():
    R, L, V = 16, 5, 20011
    d, t, tok, u, r = inputs(R, L, V, 14)
    ctx = make_ctx(V, R, L)
    al, at, _ = run(ctx, d, t, tok, u, r)
    b = [torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, L + 1, dtype=torch.int32, device="cuda")]
    ctx.ddt_accept_stochastic(d, t, torch.from_numpy(tok).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda(), R, *b)
    assert al == b[0].tolist() and at == b[1].tolist()


def test_captured():
    R, L, V = 5, 3, 9001
    sd = settings(R, T=0.8, p=0.9)
    d, t, tok, u, r = inputs(R, L, V, 15, sd=sd)
    ctx, f = make_ctx(V, R, L), to_filter(sd)
    g = [torch.from_numpy(x).cuda() for x in (tok, u, r)]
    al, at = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, L + 1, dtype=torch.int32, device="cuda")
    call = lambda: ctx.ddt_accept_sampled(d, t, *g, R, al, at, draft_filter=f, target_filter=f)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    d2, t2, *rest = inputs(R, L, V, 16, sd=sd)
    d.copy_(d2)
    t.copy_(t2)
    for a, b in zip(g, rest):
        a.copy_(torch.from_numpy(b))
    graph.replay()
    torch.cuda.synchronize()
    want = run(ctx, d2, t2, *rest, sd, sd)
    assert (al.tolist(), at.tolist()) == want[:2]
    check(d2, t2, *rest, sd, sd)


def test_keeps_the_target_s_distribution():
    """One guess drawn from q, verified against p: over evenly spaced uniforms of the guess,
    the decision and the draw, the committed token has p's probabilities. With n points an
    axis, an axis moves a token's count by at most its own share of the jumps: 3 V^2 / n
    bounds the sum over tokens."""
    V, n = 6, 24
    d, t = rows(1, V, 3, 1.0, torch.float32), rows(1, V, 4, 1.0, torch.float32)
    fd, ft = (0.9, 5, 1.0, 0.0), (1.2, 0, 0.9, 0.0)
    q = sample_ref.distribution(d[0].double().cpu().numpy(), *fd)
    p = sample_ref.distribution(t[0].double().cpu().numpy(), 1.2, 0, float(np.float32(0.9)), 0.0)
    axis = ((np.arange(n) + 0.5) / n).astype(np.float32)
    guess = np.array([sample_ref.pick(q, x) for x in axis], dtype=np.int32)
    tok, u, r = (x.reshape(-1).copy() for x in np.meshgrid(guess, axis, axis, indexing="ij"))
    count = np.zeros(V)
    for a in range(0, len(tok), 1728):
        m = min(1728, len(tok) - a)
        ctx = make_ctx(V, m, 1, ddt.F32, ddt.F32)
        at = run(ctx, d.expand(m, V).reshape(m, 1, V).contiguous(), t.expand(2 * m, V).reshape(m, 2, V).contiguous(),
                 tok[a:a + m, None].astype(np.int32), u[a:a + m, None], r[a:a + m], settings(m, *fd), settings(m, *ft))[1]
        count += np.bincount([x[0] for x in at], minlength=V)
    assert np.abs(count / len(tok) - p).sum() <= 3.0 * V * V / n / n * 4
