"""ddt_prefix_attention / ddt_prefix_attention_kvq against causal attention in fp64
(tolerances: see packed_ref.Packed.attention64; a row's sums over a prefix and over
its own keys are joined in fp32, within the 2^-20 that the tolerance has for sums),
what they leave alone, skip or refuse, and a run of continuations of one prompt."""
import numpy as np
import pytest
import torch

import sample_ref
from packed_ref import SENTINEL, Packed, check_close
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu

SHAPES = [  # Hq, Hkv, d, page
    (32, 8, 128, 16), (4, 1, 64, 16), (8, 8, 64, 64), (16, 1, 128, 32), (10, 5, 128, 256), (16, 2, 64, 16),
]


class Shared(Packed):
    """Groups [(prefix, [(new tokens, own cached tokens), ...]), ...] and, ahead of
    and behind them, requests of no group. A prefix's whole pages are held once; the
    page that its end lies in is a copy of each member's."""

    def __init__(self, groups, ahead=(), behind=(), prefix_tokens=None, **kw):
        lens = [n for n, _ in ahead] + [n for _, m in groups for n, _ in m] + [n for n, _ in behind]
        ctx = [c for _, c in ahead] + [p + c for p, m in groups for _, c in m] + [c for _, c in behind]
        super().__init__(lens, ctx, **kw)
        c = self.h.cfg
        T = self.T if prefix_tokens is None else prefix_tokens
        self.h = ddt.Context(ddt.make_config(R_max=c.R_max, L=4, V=32, B=8, Hq=c.Hq, Hkv=c.Hkv, d=c.d,
                                             page_size=c.page_size, max_pages_per_req=c.max_pages_per_req,
                                             num_pages=c.num_pages, prefix_tokens=T))
        self.prefixes = [p for p, _ in groups]
        self.first = [len(ahead)]
        for _, m in groups:
            self.first.append(self.first[-1] + len(m))
        self.group_start = torch.tensor(self.first, dtype=torch.int32, device="cuda")
        self.prefix_lens = torch.tensor(self.prefixes, dtype=torch.int32, device="cuda")

    def share(self, tables=True):
        """Members' first slots as the group's first request has them."""
        pools = (self.k_cache, self.v_cache) if self.bits == 16 else tuple(
            getattr(self.kv4, n) for n in ("k_codes", "v_codes", "k_scales", "v_scales"))
        for g, p in enumerate(self.prefixes):
            lead = self.first[g]
            for r in range(lead + 1, self.first[g + 1]):
                full = p // self.page if tables else 0
                self.table[r, :full] = self.table[lead, :full]
                (pa, ra), (pb, rb) = (self.slots(x, full * self.page, p) for x in (lead, r))
                for t in pools:
                    if self.bits == 16:
                        t[pb, rb] = t[pa, ra]
                    else:
                        t[pb, :, rb] = t[pa, :, ra]

    def fill(self, tables=True):
        self.fill_context()
        self.share(tables)
        self.fill_new()

    def attend(self, q=None, out=None, stream=None):
        q = self.q if q is None else q
        out = torch.full((self.T, self.Hq, self.d), SENTINEL, device="cuda").bfloat16() if out is None else out
        a = (q, self.q_start, self.ctx_lens, self.table, self.R, self.group_start, self.prefix_lens)
        if self.bits == 16:
            self.h.ddt_prefix_attention(*a, self.k_cache, self.v_cache, out, stream=stream)
        else:
            self.h.ddt_prefix_attention_kvq(*a, self.kv4, out, stream=stream)
        return out


def check(p, **kw):
    got = p.attend(**kw)
    want, tol = p.attention64(kw.get("q"))
    check_close(got, want, tol)
    assert p.h.ddt_device_status() == 0
    return got


def run(p, **kw):
    p.fill()
    return check(p, **kw)


def same(got, first):
    assert torch.equal(got.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("groups", [
    [(128, [(1, 0), (1, 1)])],
    [(1000, [(1, 0), (1, 5), (1, 200)])],
    [(700, [(1, 40)] * 9), (127, [(1, 3), (1, 0)]), (129, [(2, 0), (1, 300)])],
    [(300, [(16, 10), (16, 0), (5, 77)]), (2000, [(1, 1)])],
    [(0, [(3, 5), (1, 0)]), (640, [(0, 0), (1, 9), (0, 3), (7, 128)])],
    [(512, [(130, 0), (90, 31), (1, 600)])],
    [(257, [(1, i) for i in range(70)])],
])
def test_groups(bits, shape, groups):
    Hq, Hkv, d, page = shape
    run(Shared(groups, ahead=[(2, 50)], behind=[(1, 300), (40, 0)], Hq=Hq, Hkv=Hkv, d=d, page=page, bits=bits, seed=3,
               lead=1, tail=3))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("seed", range(6))
def test_ragged_groups(bits, seed):
    rng = np.random.default_rng(200 + seed)
    Hq, Hkv, d, page = SHAPES[seed % len(SHAPES)]

    def log(lo, hi):
        return int(np.exp(rng.uniform(np.log(lo), np.log(hi))))

    groups = [(log(1, 6000), [(int(rng.random() > 0.1) * log(1, 20), log(1, 500) - 1) for _ in range(log(1, 40))])
              for _ in range(int(rng.integers(1, 6)))]
    run(Shared(groups, ahead=[(1, 900)] * int(rng.integers(0, 3)), behind=[(log(1, 300), log(1, 900))] * int(rng.integers(0, 2)),
               Hq=Hq, Hkv=Hkv, d=d, page=page, bits=bits, seed=seed))


@pytest.mark.parametrize("bits", [16, 4])
def test_no_groups(bits):
    run(Shared([], ahead=[(1, 700), (30, 0), (1, 0)], Hq=8, Hkv=2, d=64, bits=bits, seed=5))


@pytest.mark.parametrize("bits", [16, 4])
def test_many_requests(bits):
    rng = np.random.default_rng(7)
    groups = [(int(rng.integers(0, 700)), [(int(rng.integers(0, 3)), int(rng.integers(0, 60))) for _ in range(n)])
              for n in (300, 1, 250, 2, 3)]
    run(Shared(groups, behind=[(1, 5)] * 200, Hq=4, Hkv=1, d=64, bits=bits, seed=8))


@pytest.mark.parametrize("gain", [0.05, 8.0])
def test_scores_far_apart(gain):
    """Prefixes whose scores lie far below the own keys', and far above."""
    p = Shared([(900, [(1, 100), (4, 30), (1, 0)])], Hq=8, Hkv=2, d=128, seed=9)
    p.fill()
    pg, row = p.slots(0, 0, 900)
    p.k_cache[pg, row] *= gain
    p.share()
    check(p)


@pytest.mark.parametrize("bits", [16, 4])
def test_a_prefix_held_in_copies(bits):
    """Members whose tables name pages of their own with equal contents."""
    p = Shared([(520, [(1, 10), (3, 0), (1, 77)])], Hq=16, Hkv=4, d=64, bits=bits, seed=10)
    p.fill(tables=False)
    check(p)


@pytest.mark.parametrize("bits", [16, 4])
def test_strided_queries(bits):
    p = Shared([(300, [(1, 10), (9, 0)])], Hq=8, Hkv=2, d=64, bits=bits, seed=11)
    wide = torch.randn(p.T, 8 * 64 + 40, device="cuda").bfloat16()
    run(p, q=wide[:, 8:8 + 512].view(p.T, 8, 64))


@pytest.mark.parametrize("bits", [16, 4])
def test_stale_slots_are_not_seen(bits):
    """The pools hold NaN wherever no request has a token."""
    run(Shared([(391, [(1, 0), (2, 3), (1, 130)]), (130, [(1, 0), (1, 0)])], Hq=8, Hkv=2, d=128, page=64, bits=bits,
               seed=12, stale=float("nan")))


def _bad(bits):
    p = Shared([(300, [(1, 10), (2, 0), (1, 5)]), (256, [(1, 1), (3, 40)])], behind=[(2, 9)], Hq=8, Hkv=2, d=64,
               bits=bits, seed=13)
    p.fill()
    return p


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("change,skipped", [
    (("prefix_lens", 0, -1), {0, 1, 2}),
    (("prefix_lens", 0, 10 ** 6), {0, 1, 2}),
    (("prefix_lens", 1, 2 ** 31 - 1), {3, 4}),
    (("prefix_lens", 0, 304), {1}),   # one member has no more than 300 cached tokens
    (("group_start", 2, 9), {3, 4, 5}),  # beyond the requests
    (("ctx_lens", 1, -4), {1}),
    (("group_start", 0, -3), {0, 1, 2}),
])
def test_bad_groups_and_members(bits, change, skipped):
    p = _bad(bits)
    want, tol = p.attention64()
    name, at, value = change
    getattr(p, name)[at] = value
    got = p.attend()
    for r in range(p.R):
        s = slice(int(p.starts[r]), int(p.starts[r + 1]))
        if r in skipped:
            assert bool((got[s] == SENTINEL).all()), r
        else:
            check_close(got[s], want[s], tol[s])
    assert p.h.ddt_device_status() == ddt.DEV_BAD_LENGTH


@pytest.mark.parametrize("bits", [16, 4])
def test_bad_pages(bits):
    """A page out of range reads as zeros, in a prefix through its first request's table."""
    p = Shared([(384, [(1, 5), (1, 20)])], Hq=4, Hkv=1, d=64, bits=bits, seed=14)
    p.fill()
    pg = int(p.table[0, 3])
    for t in (p.k_cache, p.v_cache) if bits == 16 else (p.kv4.k_codes, p.kv4.v_codes, p.kv4.k_scales, p.kv4.v_scales):
        t[pg] = 0
    want, tol = p.attention64()
    p.table[0, 3] = p.num_pages
    check_close(p.attend(), want, tol)
    assert p.h.ddt_device_status() == ddt.DEV_BAD_PAGE


def test_refusals():
    p = Shared([(300, [(1, 10), (2, 0)])], Hq=4, Hkv=2, d=64, seed=15)
    p.fill()
    lib = ddt.load()
    out = torch.empty_like(p.q)
    base = dict(q=p.q.data_ptr(), qs=0, s=p.q_start.data_ptr(), c=p.ctx_lens.data_ptr(), R=2, T=p.T, k=p.k_cache.data_ptr(),
                v=p.v_cache.data_ptr(), b=p.table.data_ptr(), g=p.group_start.data_ptr(), l=p.prefix_lens.data_ptr(), G=1,
                o=out.data_ptr())

    def call(**kw):
        a = dict(base, **kw)
        return lib.ddt_prefix_attention(p.h._h, a["q"], a["qs"], a["s"], a["c"], a["R"], a["T"], a["k"], a["v"], a["b"],
                                        a["g"], a["l"], a["G"], a["o"], None)

    assert call() == ddt.OK and call(R=0) == ddt.OK and call(T=0, q=None, o=None) == ddt.OK
    assert call(G=0, g=None, l=None) == ddt.OK
    for bad in (dict(R=3), dict(G=-1), dict(G=3), dict(g=None), dict(l=None), dict(g=base["g"] + 1), dict(l=base["l"] + 2),
                dict(q=None), dict(k=None), dict(v=None), dict(b=None), dict(o=None), dict(o=base["q"]), dict(o=base["k"]),
                dict(qs=8), dict(q=base["q"] + 8), dict(o=base["o"] + 8), dict(g=base["o"]), dict(l=base["o"] + 16)):
        assert call(**bad) == ddt.EINVAL, bad
    for tokens in (p.T - 1, 0):
        x = Shared([(300, [(1, 10), (2, 0)])], Hq=4, Hkv=2, d=64, seed=15, prefix_tokens=tokens)
        with pytest.raises(ddt.DdtError) as e:
            x.attend()
        assert e.value.status == ddt.EUNSUPPORTED
    with pytest.raises(ValueError):
        p.h.ddt_prefix_attention(p.q, p.q_start, p.ctx_lens, p.table, 2, p.group_start[:1], p.prefix_lens, p.k_cache,
                                 p.v_cache, out)
    torch.cuda.synchronize()
    assert p.h.ddt_device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_repeats_agree_on_other_streams_and_behind_other_calls(bits):
    p = Shared([(1500, [(1, 20)] * 12), (300, [(4, 0), (1, 50)])], behind=[(1, 3000)], Hq=16, Hkv=4, d=128, bits=bits, seed=16)
    first = run(p)
    s = torch.cuda.Stream()
    for _ in range(3):
        Packed.attend(p)  # (prompt attention between them uses the workspace)
        out = torch.full_like(first, SENTINEL)
        s.wait_stream(torch.cuda.current_stream())
        p.attend(out=out, stream=s)
        s.synchronize()
        same(out, first)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("groups", [[(128, [(1, 0), (1, 1)])], [(3000, [(1, 20)] * 20)], [(1, [(1, 0), (1, 3)])]])
def test_what_comes_next_sees_the_whole_output(bits, groups):
    p = Shared(groups, Hq=32, Hkv=8, d=128, bits=bits, seed=17)
    first = run(p)
    out, copies = torch.empty_like(first), []
    for _ in range(50):
        out.fill_(SENTINEL)
        p.attend(out=out)
        copies.append(out.clone())
    for c in copies:
        same(c, first)


@pytest.mark.parametrize("bits", [16, 4])
def test_captured_steps_follow_the_lengths(bits):
    p = Shared([(260, [(1, 30), (2, 5), (1, 0)]), (140, [(1, 9), (1, 60)])], Hq=8, Hkv=2, d=64, bits=bits, seed=18)
    p.fill()
    out = torch.empty_like(p.q)
    p.attend(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.attend(out=out)
    for step in range(3):
        p.q.normal_()
        p.prefix_lens.copy_(torch.tensor([260 - 70 * step, 140 - 20 * step], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, tol = p.attention64()
        check_close(out, want, tol)
    assert p.h.ddt_device_status() == 0


def test_two_contexts_at_once():
    a = Shared([(900, [(1, 20)] * 6)], Hq=16, Hkv=2, d=128, seed=19)
    b = Shared([(400, [(3, 9), (1, 0)])], Hq=8, Hkv=8, d=64, bits=4, seed=20)
    want = [run(a), run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    for i in range(20):
        for p, s, o in zip((a, b), streams, outs):
            p.attend(out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for x in o:
            same(x, w)


def test_a_wait_that_runs_out():
    """As prompt attention's: reported, and the next call is whole."""
    p = Shared([(600, [(1, 20)] * 3)], Hq=8, Hkv=2, d=64, seed=21)
    first = run(p)
    p.h.ddt_debug_arm_prompt_timeout(100000)
    p.attend()
    torch.cuda.synchronize()
    assert p.h.ddt_device_status() & ddt.DEV_TIMEOUT
    same(p.attend(), first)
    assert p.h.ddt_device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_continuations_of_one_prompt(bits):
    """Eight continuations of a prompt, as a server runs them: steps that append a token to
    each, attend with the prompt shared, project to logits and sample. Attentions against
    fp64, and prompt attention's; tokens against the 64-bit draw of the same logits."""
    n, P, Hq, Hkv, d, V, steps = 8, 200, 8, 2, 64, 499, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    p = Shared([(P, [(1, steps)] * n)], Hq=Hq, Hkv=Hkv, d=d, bits=bits, seed=22)
    p.fill()
    emb = torch.randn(V, (Hq + 2 * Hkv) * d, generator=g, device="cuda").bfloat16()
    head = torch.randn(Hq * d, V, generator=g, device="cuda") * 0.2
    rot = ddt.Rotary(ddt.rotary_table(P + steps + 2, d), d)
    smp = ddt.Context(ddt.make_config(R_max=n, L=1, V=V, B=8, Hq=Hq, Hkv=Hkv, d=d, page_size=16, max_pages_per_req=1,
                                      num_pages=1))
    f = ddt.Filter(torch.full((n,), 0.8, device="cuda"), torch.full((n,), 40, dtype=torch.int32, device="cuda"),
                   torch.full((n,), 0.95, device="cuda"))
    settings = (float(np.float32(0.8)), 40, float(np.float32(0.95)))
    tokens = torch.arange(n, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), P, dtype=torch.int32, device="cuda")
    for step in range(steps):
        rows = emb[tokens.long()].view(n, Hq + 2 * Hkv, d)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        qo, new = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(lens)
        out, alone = torch.empty_like(qo), torch.empty_like(qo)
        a = (p.q_start, lens, p.table, n)
        shared = a + (p.group_start, p.prefix_lens)
        if bits == 16:
            p.h.ddt_append_kv(q, k, v, *a, p.k_cache, p.v_cache, q_out=qo, rotary=rot, new_lens=new)
            p.h.ddt_prefix_attention(qo, *shared, p.k_cache, p.v_cache, out)
            p.h.ddt_prompt_attention(qo, *a, p.k_cache, p.v_cache, alone)
        else:
            p.h.ddt_append_kvq(q, k, v, *a, p.kv4, q_out=qo, rotary=rot, new_lens=new)
            p.h.ddt_prefix_attention_kvq(qo, *shared, p.kv4, out)
            p.h.ddt_prompt_attention_kvq(qo, *a, p.kv4, alone)
        p.lens, p.ctx = [1] * n, [P + step] * n
        want, tol = p.attention64(qo)
        check_close(out, want, tol)
        check_close(alone, want, tol)
        logits = out.float().flatten(1) @ head
        u = torch.rand(n, generator=g, device="cuda")
        smp.ddt_sample(logits, u, tokens, filter=f)
        z, un = logits.double().cpu().numpy(), u.double().cpu().numpy()
        assert tokens.tolist() == [sample_ref.pick(sample_ref.distribution(z[i], *settings), un[i]) for i in range(n)]
        lens.copy_(new)
    assert p.h.ddt_device_status() == 0 and smp.ddt_device_status() == 0
