"""Sampling under temperature, top-k, top-p and min-p on the GPU against the
64-bit definition in sample_ref.py.

Tokens have to be equal. The kernel's weights and sums are good to about 2^-40
and the reference's to 2^-50, so a drawn border falls between them with a chance
of 1e-9 a row at the sizes here; the inputs are seeded and none does. A
log-probability is a difference of two fp32 numbers, each rounded a few times:
(z - z_max) / T with two roundings, log1p with an error of 2 ulp and an argument
of two roundings, and the difference's own: together below 8 * 2^-24 of the
larger of the two. Beside that the sum itself, which is 1 or more, is off by 2^-40 of
itself and by 2^-44 for each 16 bytes of a row (a rounding to units of 2^-44), and so its
logarithm by as much: of a sum next to 1, whose logarithm is next to 0, this is what counts.
Where no top-k and no top-p apply, the sum may be one of the hardware's 2^x, off by 2^-20 of
itself: 2^-22 for a weight, 2^-24 each for three roundings of it and 4 * 2^-24 for a sum of
eight, in all 13 * 2^-24 (the draw is made anew with exact sums where that could decide it)."""
import numpy as np
import pytest
import torch

import sample_ref
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu


def make_ctx(V, R_max=1, L=1, draft=ddt.BF16, target=ddt.BF16):
    K = min(8, V)
    return ddt.Context(ddt.make_config(R_max=R_max, L=L, V=V, B=K, K=K, Hq=4, Hkv=1, d=64, page_size=16,
                                       max_pages_per_req=1, num_pages=1, draft_dtype=draft, target_dtype=target))


def settings(n, T=1.0, k=0, p=1.0, m=0.0):
    """Four lists of n from numbers or lists."""
    return [list(x) if isinstance(x, (list, tuple, np.ndarray)) else [x] * n for x in (T, k, p, m)]


def to_filter(s):
    f32 = dict(dtype=torch.float32, device="cuda")
    return ddt.Filter(torch.tensor(s[0], **f32), torch.tensor(s[1], dtype=torch.int32, device="cuda"),
                      torch.tensor(s[2], **f32), torch.tensor(s[3], **f32))


def run(logits, u, s=None, ctx=None, stream=None):
    N, V = logits.shape
    ctx = ctx or make_ctx(V)
    tokens = torch.full((N + 2,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((N + 2,), 7.0, device="cuda")
    ctx.ddt_sample(logits, torch.as_tensor(u, dtype=torch.float32).cuda(), tokens[:N],
                   filter=None if s is None else to_filter(s), logprobs=lp[:N], stream=stream)
    torch.cuda.synchronize()
    assert tokens[N:].tolist() == [-7, -7] and lp[N:].tolist() == [7.0, 7.0]
    return tokens[:N].tolist(), lp[:N].double().cpu().numpy(), ctx.ddt_device_status()


def want(logits, u, s=None):
    N = logits.shape[0]
    z = logits.double().cpu().numpy()
    s = s or settings(N)
    f = [np.asarray(x, dtype=np.int64 if i == 1 else np.float32).astype(np.int64 if i == 1 else np.float64)
         for i, x in enumerate(s)]
    u = np.asarray(u, dtype=np.float32).astype(np.float64)
    d = [sample_ref.distribution(z[i], *(x[i] for x in f)) for i in range(N)]
    tok = [sample_ref.pick(d[i], u[i]) for i in range(N)]
    with np.errstate(divide="ignore"):
        lp = np.array([np.log(d[i][t]) if t >= 0 else -np.inf for i, t in enumerate(tok)])
    return tok, lp, d


def check(logits, u, s=None, status=0, **kw):
    tok, lp, st = run(logits, u, s, **kw)
    wtok, wlp, _ = want(logits, u, s)
    assert tok == wtok
    assert st == status
    z = logits.double().cpu().numpy()
    N = len(tok)
    T = [x if x > 0 else 1.0 for x in (s or settings(N))[0]]
    for i, t in enumerate(tok):
        if t < 0 or not np.isfinite(z[i][t]):
            assert lp[i] == wlp[i] or abs(lp[i] - wlp[i]) <= 8 * 2.0 ** -24 * abs(wlp[i]) + 2.0 ** -40
            continue
        big = abs((np.nanmax(z[i]) - z[i][t]) / T[i])
        quick = s is None or (not 0 < s[1][i] < len(z[i]) and s[2][i] >= 1)
        of_sum = 2.0 ** -40 + len(z[i]) / 4 * 2.0 ** -44 + quick * 2.0 ** -20
        assert abs(lp[i] - wlp[i]) <= 8 * 2.0 ** -24 * max(big, abs(wlp[i]) + big) + of_sum
    return tok


def rows(N, V, seed, spread=3.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(N, V, generator=g, device="cuda") * spread).to(dtype)


def uniforms(N, seed):
    return np.random.default_rng(seed).random(N, dtype=np.float32)


SETTINGS = {
    "none": dict(),
    "hot": dict(T=1.7),
    "cold": dict(T=0.05),
    "greedy": dict(T=0.0, k=40, p=0.5, m=0.2),
    "k1": dict(k=1),
    "k50": dict(T=0.8, k=50),
    "k256": dict(k=256),
    "k257": dict(T=1.3, k=257),
    "k5000": dict(T=2.0, k=5000),
    "p0": dict(p=0.0),
    "p5": dict(p=0.5),
    "p95": dict(T=1.2, p=0.95),
    "p9999": dict(T=1.5, p=0.9999),
    "m1": dict(m=1.0),
    "m05": dict(T=1.5, m=0.05),
    "all": dict(T=0.9, k=64, p=0.9, m=0.01),
    "wide": dict(T=3.0, k=3000, p=0.97, m=1e-4),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 255, 257, 1000, 4099, 32003])
def test_sizes(V, dtype):
    """Every setting, rows that begin off 16 bytes, a few and many values a row."""
    ctx = make_ctx(V)
    for i, (name, s) in enumerate(SETTINGS.items()):
        N = 5
        z = rows(N, V, 100 + i, spread=(0.5, 3.0, 8.0)[i % 3], dtype=dtype)
        check(z, uniforms(N, i), settings(N, **s), ctx=ctx)
    check(rows(3, V, 7, dtype=dtype), uniforms(3, 1), ctx=ctx)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(SETTINGS))
def test_full_vocabulary(name, dtype):
    z = torch.cat((rows(3, 151936, 1, 1.0, dtype), rows(3, 151936, 2, 4.0, dtype)))
    check(z, uniforms(6, 3), settings(6, **SETTINGS[name]))


def test_mixed_rows():
    """Settings of their own for each of many rows."""
    rng = np.random.default_rng(5)
    N, V = 67, 50021
    s = [np.where(rng.random(N) < 0.1, 0.0, rng.uniform(0.3, 2.0, N)).astype(np.float32),
         np.where(rng.random(N) < 0.5, 0, rng.integers(1, 3000, N)),
         np.where(rng.random(N) < 0.5, 1.0, rng.uniform(0, 1, N)).astype(np.float32),
         np.where(rng.random(N) < 0.5, 0.0, 10.0 ** rng.uniform(-5, 0, N)).astype(np.float32)]
    check(rows(N, V, 11, 2.5), uniforms(N, 12), [list(x) for x in s])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_large_vocabulary(dtype):
    z = rows(1, 524288, 3, 2.0, dtype)
    for s in (dict(), dict(k=100, p=0.9), dict(p=0.9, T=1.5)):
        check(z, [0.61], settings(1, **s))


def test_very_large_vocabulary():
    """A row of 2 MB: the largest that a configuration takes."""
    z = rows(2, 1048576, 3, 2.0)
    for s in (dict(), dict(k=1000, p=0.9), dict(p=0.97, T=1.5)):
        check(z, [0.61, 0.07], settings(2, **s))


@pytest.mark.parametrize("kind", ["equal", "two", "few", "steps"])
def test_ties(kind):
    """Rows of few distinct values: borders cut runs of equal logits, lowest index first."""
    N, V = 4, 40009
    g = torch.Generator().manual_seed(9)
    if kind == "equal":
        z = torch.full((N, V), 1.5)
    elif kind == "two":
        z = torch.randint(0, 2, (N, V), generator=g).float()
    elif kind == "few":
        z = torch.randint(-3, 4, (N, V), generator=g).float()
    else:
        z = torch.round(torch.randn(N, V, generator=g) * 8) / 4
    for dtype in (torch.bfloat16, torch.float32):
        for s in (dict(), dict(k=1), dict(k=17), dict(k=700), dict(k=20011), dict(p=0.3), dict(p=0.77, T=0.6),
                  dict(k=30000, p=0.5), dict(m=0.3), dict(k=900, p=0.2, m=0.1)):
            check(z.to(dtype).cuda(), [0.0, 0.3, 0.8, 0.9999999], settings(N, **s))


def test_masks():
    """Logits of -infinity, the types' lowest value, NaN and +infinity."""
    V = 3001
    for dtype in (torch.bfloat16, torch.float32):
        low = torch.finfo(dtype).min
        z = rows(8, V, 4, 2.0, dtype)
        z[0] = -torch.inf                      # nothing left
        z[1] = -torch.inf
        z[1, 1234] = -5.0                      # one left
        z[2, 10:] = low
        z[3] = low                             # all masked, with one value
        z[4, ::3] = -torch.inf
        z[5, 7] = torch.inf
        z[5, 2000] = torch.inf
        z[6, :V - 2] = low
        z[7, 5:100] = -1e9
        for s in (dict(), dict(k=5), dict(k=1000), dict(p=0.9), dict(m=0.01), dict(T=0.0), dict(T=100.0, k=700, p=0.99)):
            check(z, uniforms(8, 21), settings(8, **s))
        n = z.clone()
        n[4, 17] = torch.nan
        n[6] = torch.nan
        for s in (dict(), dict(p=0.9), dict(k=3)):
            check(n, uniforms(8, 22), settings(8, **s), status=ddt.DEV_NAN_LOGITS)


def test_ranges():
    """Very large, very small and log-probability-like logits; far temperatures."""
    for dtype in (torch.bfloat16, torch.float32):
        for z in (rows(2, 2003, 1, 1e4, dtype), rows(2, 2003, 2, 1e-4, dtype), rows(2, 2003, 3, 1e-30, dtype),
                  rows(2, 2003, 4, 1e30, dtype),
                  torch.log_softmax(rows(2, 2003, 5, 3.0, torch.float32), 1).to(dtype)):
            for s in (dict(), dict(T=1e-3), dict(T=1e6), dict(T=1e30), dict(T=1e-30), dict(p=0.9), dict(k=300),
                      dict(T=50.0, p=0.5, m=0.5)):
                check(z, uniforms(2, 9), settings(2, **s))


def test_uniforms_at_the_ends():
    V = 5003
    z = rows(6, V, 8)
    u = [0.0, 1.0 - 2.0 ** -24, 1.0, float("nan"), -1.0, 2.0 ** -149]
    for s in (dict(), dict(k=20), dict(p=0.8)):
        check(z, u, settings(6, **s))


def test_bad_settings():
    V, bad = 1000, float("nan")
    s = [[-1.0, float("inf"), bad, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0], [0, 0, 0, 0, 0, 0, 0, 0, -3],
         [1.0, 1.0, 1.0, -0.1, 1.5, bad, 1.0, 1.0, 1.0], [0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 1.01, bad, 0.0]]
    z, u = rows(9, V, 6), uniforms(9, 6)
    tok, lp, st = run(z, u, s)
    assert tok[:8] == [-1] * 8 and np.isneginf(lp[:8]).all() and st == ddt.DEV_BAD_SETTING
    assert tok[8] == want(z[8:], u[8:])[0][0]  # (a negative top-k is off)


def test_greedy_is_argmax():
    z = torch.round(rows(33, 7001, 5) * 2) / 2
    tok = check(z, uniforms(33, 5), settings(33, T=0.0))
    first = (z == z.max(1, keepdim=True).values).int().argmax(1)
    assert tok == first.tolist()


def test_settings_one_by_one():
    """A filter with some arrays missing."""
    V, N = 3000, 4
    z, u = rows(N, V, 3), uniforms(N, 3)
    ctx = make_ctx(V)
    for s in (dict(T=0.7), dict(k=9), dict(p=0.6), dict(m=0.2)):
        full = settings(N, **s)
        f = to_filter(full)
        part = ddt.Filter(**{n: getattr(f, n) for n, key in (("temperature", "T"), ("top_k", "k"), ("top_p", "p"),
                                                             ("min_p", "m")) if key in s})
        tokens = torch.empty(N, dtype=torch.int32, device="cuda")
        ctx.ddt_sample(z, torch.from_numpy(u).cuda(), tokens, filter=part)
        assert tokens.tolist() == want(z, u, full)[0]


def test_no_rows():
    ctx = make_ctx(100)
    e = torch.empty(0, device="cuda")
    ctx.ddt_sample(torch.empty(0, 100, device="cuda"), e, torch.empty(0, dtype=torch.int32, device="cuda"), logprobs=e)


def test_far_rows():
    """Element offsets beyond 32 bits."""
    V, N = 151936, 14400
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    z[:8] = rows(8, V, 1)
    z[8:] = z[:1]
    z[-3:] = rows(3, V, 2)
    u, s = uniforms(N, 4), settings(N, k=30, p=0.9)
    tok, _, _ = run(z, u, s)
    for i in (0, 5, N // 2, N - 3, N - 1):
        assert tok[i] == want(z[i:i + 1], u[i:i + 1], [x[i:i + 1] for x in s])[0][0], i


def test_captured_and_on_two_streams():
    """A captured call replays on new inputs; calls of one context on two streams at once."""
    V, N = 30011, 6
    ctx = make_ctx(V)
    z, u = rows(N, V, 1), torch.from_numpy(uniforms(N, 1)).cuda()
    s = settings(N, T=[0.0, 0.5, 1.0, 1.5, 1.0, 1.0], k=[0, 10, 400, 0, 0, 3], p=[1.0, 0.9, 0.9, 0.99, 1.0, 0.5])
    f, tokens = to_filter(s), torch.empty(N, dtype=torch.int32, device="cuda")
    ctx.ddt_sample(z, u, tokens, filter=f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ctx.ddt_sample(z, u, tokens, filter=f)
    for seed in (2, 3):
        z.copy_(rows(N, V, seed))
        un = uniforms(N, seed)
        u.copy_(torch.from_numpy(un))
        graph.replay()
        torch.cuda.synchronize()
        assert tokens.tolist() == want(z, un, s)[0]
    z2, t2 = rows(N, V, 9), torch.empty(N, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        ctx.ddt_sample(z, u, tokens, filter=f)
        ctx.ddt_sample(z2, u, t2, filter=f, stream=side)
    torch.cuda.synchronize()
    assert tokens.tolist() == want(z, un, s)[0] and t2.tolist() == want(z2, un, s)[0]


def test_repeats_bit_for_bit():
    z = rows(9, 151936, 1, 1.2)
    s = settings(9, T=1.3, k=[0, 0, 0, 9000, 9000, 9000, 20, 20, 20], p=[1.0, 0.9, 0.5] * 3)
    first = run(z, uniforms(9, 2), s)
    for _ in range(5):
        again = run(z, uniforms(9, 2), s)
        assert again[0] == first[0] and np.array_equal(again[1], first[1])


def test_draws_follow_the_distribution():
    """4096 evenly spaced uniforms of one row: each token's count is its share, to one."""
    N, V = 4096, 997
    z = rows(1, V, 1, 1.5, torch.float32).expand(N, V).contiguous()
    u = ((np.arange(N) + 0.5) / N).astype(np.float32)
    s = settings(N, T=0.8, k=50, p=0.95)
    tok, _, _ = run(z, u, s)
    p = want(z[:1], u[:1], [x[:1] for x in s])[2][0]
    count = np.bincount(tok, minlength=V)
    assert count[p == 0].sum() == 0
    assert (np.abs(count - N * p) <= 1.0 + 1e-6).all()  # (evenly spaced uniforms: the running sums, rounded)
