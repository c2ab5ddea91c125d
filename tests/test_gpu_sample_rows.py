"""Sampling of many rows, where each has a CTA of its own that reads it from global memory:
tokens and log probabilities against the plain 64-bit form, as for few rows (the tolerance's
terms are those of test_gpu_sample), and drafted chains of many requests."""
import ctypes

import numpy as np
import pytest
import torch

import sample_ref
import test_gpu_accept_sampled as accept
from speculative_decoding_draft_depth_gb300 import ddt
from test_gpu_sample import check, make_ctx, settings

pytestmark = pytest.mark.gpu
N = 640  # (rows enough to have a CTA each)


def logits(n, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, V, generator=g) * spread * (0.2 + torch.rand(n, 1, generator=g))
    z.scatter_add_(1, torch.randint(0, V, (n, 5), generator=g), 6.0 * torch.rand(n, 5, generator=g))
    return z.to(dtype).cuda()


def uniforms(n, seed):
    return np.random.default_rng(seed).random(n, dtype=np.float32)


@pytest.mark.parametrize("V", [1, 7, 1000, 8191, 24575, 25001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mixed_settings(V, dtype):
    rng = np.random.default_rng(V)
    s = settings(N, T=rng.choice([0.0, 0.3, 1.0, 2.5], N), k=rng.choice([0, 0, 1, 5, 300, 5000], N),
                 p=rng.choice([1.0, 1.0, 0.0, 0.3, 0.9, 0.99], N), m=rng.choice([0.0, 0.0, 0.05, 0.9], N))
    check(logits(N, V, dtype, V), uniforms(N, V), s)


@pytest.mark.parametrize("p", [0.1, 0.8, 0.95, 0.999])
@pytest.mark.parametrize("spread", [0.3, 2.0])
def test_top_p_of_wide_rows(p, spread):
    """Deep borders: nearly flat rows, of which most is kept."""
    check(logits(N, 25003, torch.bfloat16, 5, spread), uniforms(N, 6), settings(N, p=p, T=1.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [25001, 515])
@pytest.mark.parametrize("N", [N, 48])
def test_odd_rows(dtype, V, N):
    """Equal logits, masked ones, infinities, NaN, tiny and large values, hot and cold rows."""
    z = logits(N, V, dtype, 3)
    inf = float("inf")
    z[0] = 1.5
    z[1] = -inf
    z[2] = -inf
    z[2, V - 1] = -3.0
    z[3, 5] = inf
    z[3, V // 2] = inf
    z[4, 7] = float("nan")
    z[5] = float("nan")
    z[6] = 1e-30
    z[6, 3] = -1e-35
    z[7] = 300.0
    z[7, V // 3:] = 299.0
    z[8] = -500.0
    z[9, ::2] = -inf
    z[10] = torch.finfo(dtype).min
    z[10, 2] = torch.finfo(dtype).max
    z[11] = (torch.arange(V) % 3).to(dtype)
    z[12, 1:] = 2.0 ** -31
    z[12, 0] = 0.0
    z[13] = 0.0
    z[14, : V // 2] = -0.0
    z[15, 0] = inf
    z[15, 1] = float("nan")
    rng = np.random.default_rng(1)
    reps = np.arange(N) // 16
    z = z[torch.arange(N) % 16].clone()
    s = settings(N, T=np.array([1.0, 0.0, 0.7, 20.0, 1.0])[reps % 5], k=np.array([0, 3, 0, 400])[reps % 4],
                 p=np.array([1.0, 0.5, 0.97])[reps % 3], m=np.array([0.0, 0.0, 0.2])[(reps // 3) % 3])
    check(z, rng.random(N, dtype=np.float32), s, status=ddt.DEV_NAN_LOGITS)


def test_ends_of_u():
    z = logits(N, 25001, torch.bfloat16, 9)
    u = np.array([0.0, np.nextafter(np.float32(1), np.float32(0)), 0.5, 1e-30], dtype=np.float32)[np.arange(N) % 4]
    check(z, u, settings(N, p=np.where(np.arange(N) % 8 < 4, 1.0, 0.9)))


def chain_settings(R, seed):
    rng = np.random.default_rng(seed)
    return settings(R, T=rng.choice([0.0, 0.7, 1.2], R), k=rng.choice([0, 0, 8, 400], R), p=rng.choice([1.0, 1.0, 0.9], R),
                    m=rng.choice([0.0, 0.0, 0.1], R))


@pytest.mark.parametrize("V", [33, 25001])
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-bf16", "f32-f32"])
def test_chains(types, V):
    """Chains of 160 requests (rows enough to have a CTA each) under every setting, some of them short."""
    R, L = 160, 4
    sd, st = chain_settings(R, 1), chain_settings(R, 2)
    d, t, tok, u, r = accept.inputs(R, L, V, 41, *types.split("-"), sd=sd)
    accept.check(d, t, tok, u, r, sd, st)
    accept.check(d, t, tok, u, r, sd, st, n=[i % (L + 1) for i in range(R)])


@pytest.mark.parametrize("types", ["bf16-bf16", "f32-bf16"])
def test_draws_next_to_the_ratio(types):
    """u two steps of fp32 beside p(x) / q(x), nearer than quick sums tell."""
    R, L, V = 130, 5, 2501
    s = settings(R, T=0.9, m=np.where(np.arange(R) % 3 == 0, 0.01, 0.0))
    d, t, tok, u, r = accept.inputs(R, L, V, 51, *types.split("-"), noise=0.2, sd=s)
    f = [tuple(x[i] if j == 1 else float(np.float32(x[i])) for j, x in enumerate(s)) for i in range(R)]
    for i in range(R):
        for j in range(L):
            q = sample_ref.distribution(d[i, j].double().cpu().numpy(), *f[i])[tok[i, j]]
            ratio = np.float32(sample_ref.distribution(t[i, j].double().cpu().numpy(), *f[i])[tok[i, j]] / q)
            if 0 < ratio < 1:
                end = np.float32(0 if j < i % (L + 1) else 2)
                u[i, j] = np.nextafter(np.nextafter(ratio, end), end)
    accept.check(d, t, tok, u, r, s, s)


def test_rows_larger_than_a_cluster_holds():
    """4 MB a row."""
    z = logits(2, 1048576, torch.float32, 61)
    for s in (dict(), dict(k=40, p=0.9), dict(p=0.9, T=0.8)):
        check(z, [0.3, 0.97], settings(2, **s), ctx=make_ctx(1048576))


def test_refusals():
    """Null and misaligned pointers, unknown types, outputs that overlap: an error, and nothing is written."""
    n, V = 4, 64
    ctx = make_ctx(V, n, 2)
    lib, h = ddt.load(), ctx._h
    buf = torch.zeros(4096, dtype=torch.int32, device="cuda")
    z = torch.zeros(n * 3 * V + 8, dtype=torch.bfloat16, device="cuda")
    p, zp = buf.data_ptr(), z.data_ptr()
    null = ctypes.POINTER(ddt.FilterArgs)()

    def sample(logits=zp, dtype=ddt.BF16, rows=n, filter=null, u=p, tokens=p + 64, logprobs=p + 128):
        return lib.ddt_sample(h, logits, dtype, rows, filter, u, tokens, logprobs, None)

    def odd(**kw):
        return ctypes.byref(ddt.FilterArgs(**kw))

    assert sample() == ddt.OK and sample(logprobs=None) == ddt.OK and sample(rows=0, logits=None) == ddt.OK
    torch.cuda.synchronize()
    buf.fill_(-9)
    for bad in (dict(logits=None), dict(logits=zp + 2), dict(dtype=2), dict(rows=-1), dict(u=None), dict(u=p + 1),
                dict(tokens=None), dict(tokens=p + 66), dict(logprobs=p + 130), dict(tokens=p), dict(logprobs=p + 76),
                dict(tokens=zp), dict(filter=odd(temperature=p + 258)), dict(filter=odd(top_k=p + 64)),
                dict(filter=odd(min_p=p + 124))):
        assert sample(**bad) == ddt.EINVAL, bad
    a = dict(d=zp, t=zp, tok=p, u=p + 512, r=p + 1024, R=n, fd=null, ft=null, al=p + 2048, at=p + 3200, ng=None)

    def accept_(**kw):
        x = {**a, **kw}
        return lib.ddt_accept_sampled(h, x["d"], x["t"], x["tok"], x["u"], x["r"], x["R"], x["fd"], x["ft"], x["al"], x["at"],
                                      x["ng"], None)

    for bad in (dict(d=None), dict(t=zp + 2), dict(tok=None), dict(u=p + 513), dict(r=None), dict(R=n + 1), dict(R=-1),
                dict(al=None), dict(at=p + 3201), dict(al=p + 512), dict(at=p + 1000), dict(al=p + 3200), dict(ng=p + 2049),
                dict(ng=p + 2052), dict(fd=odd(top_p=p + 2)), dict(ft=odd(min_p=p + 2048))):
        assert accept_(**bad) == ddt.EINVAL, bad
    torch.cuda.synchronize()
    assert buf.unique().tolist() == [-9]
    assert accept_(R=0, d=None) == ddt.OK
    big = make_ctx(1048576, 1, 1)
    assert lib.ddt_accept_sampled(big._h, zp, zp, p, p, p, 0, null, null, p, p, None, None) == ddt.EUNSUPPORTED


def test_strided_tensors_are_refused():
    ctx = make_ctx(64, 4, 2)
    z, f, i = torch.zeros(4, 65, device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    good = dict(logits=z[:, :64].contiguous(), u=f[:4], tokens=i[:4])
    ctx.ddt_sample(**good)
    for bad in (dict(logits=z[:, :64]), dict(u=f[::2]), dict(tokens=i[::2]), dict(filter=ddt.Filter(top_p=f[:1].expand(4))),
                dict(filter=ddt.Filter(top_k=i[::2])), dict(u=f[:4].cpu())):
        with pytest.raises(ValueError):
            ctx.ddt_sample(**{**good, **bad})
