"""ddt_prompt_attention / ddt_prompt_attention_kvq against causal attention in
fp64 (tolerances: see packed_ref.Packed.attention64), what they leave alone,
skip or refuse, and runs of append and attention as a server makes them."""
import ctypes

import numpy as np
import pytest
import torch

from packed_ref import SENTINEL, Packed, check_close
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu


def run(p, **kw):
    p.fill_context()
    p.fill_new()
    got = p.attend(**kw)
    want, tol = p.attention64(kw.get("q"))
    check_close(got, want, tol)
    assert p.h.ddt_device_status() == 0
    return got


SHAPES = [  # Hq, Hkv, d, page
    (32, 8, 128, 16), (4, 1, 64, 16), (8, 8, 64, 64), (16, 1, 128, 32), (10, 5, 128, 256), (16, 2, 64, 16),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens,ctx", [
    ([1], [0]),
    ([1], [1000]),
    ([1, 1, 1, 1, 1], [0, 126, 127, 128, 255]),
    ([16, 16, 16], [500, 0, 111]),
    ([0, 5, 0, 130, 1], [40, 3, 0, 0, 129]),
    ([63, 64, 65], [0, 64, 63]),
    ([127, 129], [1, 127]),
    ([300], [0]),
    ([257, 2], [513, 700]),
])
def test_attention(bits, shape, lens, ctx):
    Hq, Hkv, d, page = shape
    run(Packed(lens, ctx, Hq, Hkv, d, page, bits, seed=21, lead=1, tail=4))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("seed", range(6))
def test_ragged_batches(bits, seed):
    rng = np.random.default_rng(100 + seed)
    Hq, Hkv, d, page = SHAPES[seed % len(SHAPES)]
    R = int(rng.integers(3, 40))
    lens = np.exp(rng.uniform(0, np.log(400), R)).astype(int) * (rng.random(R) > 0.1)
    ctx = np.exp(rng.uniform(0, np.log(3500), R)).astype(int) - 1
    run(Packed(lens.tolist(), ctx.tolist(), Hq, Hkv, d, page, bits, seed=seed, tail=int(rng.integers(0, 3))))


@pytest.mark.parametrize("bits", [16, 4])
def test_one_token_far_along(bits):
    run(Packed([1], [70001], 8, 2, 128, 16, bits, seed=22))


@pytest.mark.parametrize("bits", [16, 4])
def test_more_requests_than_threads(bits):
    rng = np.random.default_rng(7)
    run(Packed(rng.integers(0, 3, 900).tolist(), rng.integers(0, 80, 900).tolist(), 4, 1, 64, 16, bits, seed=23))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("shape", SHAPES)
def test_few_tokens_unevenly_spread(bits, shape):
    """Few tokens on average, all of them with two requests (for the 4-bit cache:
    the few-rows kernel with items of several query tiles), and two each."""
    Hq, Hkv, d, page = shape
    run(Packed([37, 0, 0, 0, 0, 0, 0, 0, 0, 0, 43] + [0] * 69, [300, 5] * 40, Hq, Hkv, d, page, bits, seed=45, tail=1))
    run(Packed([2, 1, 2, 2, 0, 2], [90, 0, 1000, 127, 3, 14], Hq, Hkv, d, page, bits, seed=46))


def test_long_prompt():
    run(Packed([2500], [0], 8, 2, 128, 16, 16, seed=24))


def test_large_scores():
    """Scores of several hundred: one key carries each row, the maximum moves often."""
    p = Packed([200, 1], [300, 600], 8, 2, 128, 16, 16, seed=25)
    p.q *= 8
    p.k *= 4
    run(p)


def test_growing_scores():
    """Keys that grow along the sequence: every tile raises the running maximum."""
    p = Packed([1, 70], [1500, 900], 8, 2, 64, 16, 16, seed=26)
    p.fill_context()
    for r, c in enumerate(p.ctx):
        pg, row = p.slots(r, 0, c)
        p.k_cache[pg, row] *= (torch.arange(c, device="cuda") / 40.0)[:, None, None].bfloat16()
    p.fill_new()
    got = p.attend()
    want, tol = p.attention64()
    check_close(got, want, tol)


@pytest.mark.parametrize("kind", ["creep", "leap", "fall", "flat"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [16, 4])
def test_scores_that_change_along_the_keys(bits, d, kind):
    """Keys whose first channel, which every query weighs by 4, moves the scores in
    64-key steps that no mask touches: up by some three bits a step, by far at two
    keys, down from the first on, or not at all (every key equal)."""
    p = Packed([1, 300, 40], [1500, 900, 1300], 8, 2, d, 16, bits, seed=36)
    p.q[..., 0] = 4
    p.fill_context()
    p.fill_new()
    for r, (n, c) in enumerate(zip(p.lens, p.ctx)):
        k, v = p._normal(n + c, 2, d).bfloat16(), p._normal(n + c, 2, d).bfloat16()
        at = torch.arange(n + c, device="cuda")
        if kind == "flat":
            k.zero_()
        else:
            h = {"creep": at / 64 * (d ** 0.5 / 2), "leap": ((at == 700) | (at == 1203)) * 60.0,
                 "fall": (n + c - at) / 20.0}[kind]
            k[..., 0] = h[:, None].bfloat16()
        p.put(r, 0, n + c, k, v)
    got = p.attend()
    want, tol = p.attention64()
    check_close(got, want, tol)
    assert p.h.ddt_device_status() == 0


def test_global_scales():
    run(Packed([3, 40, 1], [90, 200, 400], 8, 2, 128, 16, 4, seed=27, k_scale=0.37, v_scale=1.0 / 1024, v_gain=1e-3))


def test_strided_queries():
    p = Packed([5, 60], [9, 100], 8, 2, 128, 16, 16, seed=28)
    rows = torch.cat((p.q.flatten(1), p.k.flatten(1), p.v.flatten(1)), 1)
    q = rows.split((8 * 128, 256, 256), 1)[0].unflatten(1, (8, 128))
    assert not q.is_contiguous()
    run(p, q=q)


def test_infinite_and_nan_rows_stay_with_their_request():
    """A request whose values hold NaN and infinities gives what it gives; its
    neighbours' rows are not touched by them."""
    p = Packed([4, 50, 3], [30, 60, 128], 8, 2, 64, 16, 16, seed=29)
    p.fill_context()
    p.fill_new()
    pg, row = p.slots(1, 0, 110)
    p.v_cache[pg, row] = float("nan")
    p.k_cache[pg[:50], row[:50]] = float("inf")
    got = p.attend()
    want, tol = p.attention64()
    a, b = int(p.starts[1]), int(p.starts[2])
    assert bool(got[a:b].isnan().all())
    for sl in (slice(0, a), slice(b, p.T)):
        check_close(got[sl], want[sl], tol[sl])


@pytest.mark.parametrize("bits", [16, 4])
def test_bad_pages_read_as_zeros(bits):
    p = Packed([2, 3], [60, 40], 8, 2, 64, 16, bits, seed=30, stale=0.0)
    p.fill_context()
    p.fill_new()
    pg = int(p.table[0, 1])
    for t in ((p.k_cache, p.v_cache) if bits == 16 else (p.kv4.k_codes, p.kv4.v_codes)):
        t[pg] = 0
    want, tol = p.attention64()
    p.table[0, 1] = p.num_pages + 7
    got = p.attend()
    assert p.h.ddt_device_status() == ddt.DEV_BAD_PAGE
    check_close(got, want, tol)
    p.table[0, 1] = -1
    check_close(p.attend(), want, tol)
    assert p.h.ddt_device_status() == ddt.DEV_BAD_PAGE


@pytest.mark.parametrize("kind", ["negative", "past_the_table", "past_T"])
def test_bad_lengths_skip_their_request(kind):
    p = Packed([4, 6, 5], [3, 8, 2], 4, 2, 64, 16, 16, seed=31)
    p.fill_context()
    p.fill_new()
    want, tol = p.attention64()
    r = 2 if kind == "past_T" else 1
    if kind == "negative":
        p.ctx_lens[1] = -1
    elif kind == "past_the_table":
        p.ctx_lens[1] = p.max_pages * p.page - 5
    else:
        p.q_start[3] = 99
    a, b = int(p.starts[r]), int(p.starts[r + 1])
    want[a:b], tol[a:b] = SENTINEL, 0.0
    check_close(p.attend(), want, tol)
    assert p.h.ddt_device_status() == ddt.DEV_BAD_LENGTH


@pytest.mark.parametrize("bits", [16, 4])
def test_the_last_slot_of_the_table(bits):
    """A request whose tokens end with the block table's last page."""
    p = Packed([5, 130], [40, 300], 8, 2, 64, 16, bits, seed=37)
    free = sorted(set(range(p.num_pages)) - set(p.table.flatten().tolist()))
    assert int(p.table[1, -1]) < 0 and bool((p.table[1, :-1] >= 0).all())
    p.table[1, -1] = free[0]
    p.ctx[1] = p.max_pages * 16 - 130
    p.ctx_lens.copy_(torch.tensor(p.ctx, dtype=torch.int32))
    run(p)


@pytest.mark.parametrize("bits", [16, 4])
def test_requests_that_share_pages(bits):
    """A prefix held once: both tables begin with the same pages."""
    p = Packed([3, 70], [200, 260], 8, 2, 128, 16, bits, seed=38)
    p.table[1, :12] = p.table[0, :12]
    run(p)


@pytest.mark.parametrize("bits", [16, 4])
def test_rows_of_no_request(bits):
    """Rows, but not a token of any request: nothing is written."""
    p = Packed([0, 0, 0], [5, 0, 90], 8, 2, 64, 16, bits, seed=39, lead=2, tail=40)
    p.fill_context()
    assert bool((p.attend() == SENTINEL).all())
    assert p.h.ddt_device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_rows_that_two_requests_name(bits):
    """q_start that falls: the request with the fall is skipped, and rows that the
    two around it both name hold the result of either."""
    p = Packed([6, 3, 7], [30, 4, 50], 8, 2, 64, 16, bits, seed=40)
    p.fill_context()
    p.fill_new()
    want, tol = p.attention64()
    p.q_start.copy_(torch.tensor([0, 6, 2, 9], dtype=torch.int32))
    got = p.attend()
    assert p.h.ddt_device_status() == ddt.DEV_BAD_LENGTH
    check_close(got[:2], want[:2], tol[:2])
    assert bool((got[9:] == SENTINEL).all())
    assert bool(got[:9].isfinite().all()) and not bool((got[:9] == SENTINEL).all(-1).any())


def test_refusals():
    p = Packed([4, 4], [0, 3], 4, 2, 64, 16, 16, seed=32)
    lib = ddt.load()
    out = torch.empty_like(p.q)
    base = dict(q=p.q.data_ptr(), qs=0, s=p.q_start.data_ptr(), c=p.ctx_lens.data_ptr(), R=2, T=p.T,
                k=p.k_cache.data_ptr(), v=p.v_cache.data_ptr(), b=p.table.data_ptr(), o=out.data_ptr())

    def call(**kw):
        a = dict(base, **kw)
        return lib.ddt_prompt_attention(p.h._h, a["q"], a["qs"], a["s"], a["c"], a["R"], a["T"], a["k"], a["v"],
                                        a["b"], a["o"], None)

    p.fill_context()
    p.fill_new()
    assert call() == ddt.OK and call(R=0) == ddt.OK and call(T=0, q=None, o=None) == ddt.OK
    for bad in (dict(R=3), dict(R=-1), dict(T=-1), dict(T=2 ** 31 - 1), dict(q=None), dict(s=None), dict(c=None),
                dict(k=None), dict(v=None), dict(b=None), dict(o=None), dict(qs=8), dict(qs=258), dict(qs=-256),
                dict(q=base["q"] + 8), dict(o=base["o"] + 8), dict(k=base["k"] + 2), dict(v=base["v"] + 2),
                dict(s=base["s"] + 1), dict(o=base["q"]), dict(o=base["q"] + 16)):
        assert call(**bad) == ddt.EINVAL, bad
    with pytest.raises(ValueError):
        p.attend(q=p.q.cpu())
    with pytest.raises(ValueError):
        p.attend(out=torch.empty((p.T, 4, 64), device="cuda"))
    torch.cuda.synchronize()
    assert p.h.ddt_device_status() == 0


def test_another_stream_and_repeats_agree():
    """The same call again, on another stream, and after another call used the
    workspace: equal bits (no result depends on the order of arrival)."""
    p = Packed([1, 90, 33], [5000, 700, 0], 16, 2, 128, 16, 16, seed=33)
    first = run(p)
    o = Packed([300], [100], 16, 2, 128, 16, 16, seed=34, R_max=4)
    run(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = torch.full_like(first, SENTINEL)
        s.wait_stream(torch.cuda.current_stream())
        p.attend(out=out, stream=s)
        s.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens,ctx", [([1], [10]), ([1, 1, 1], [10, 700, 0]), ([20], [3000])])
def test_what_comes_next_sees_the_whole_output(bits, lens, ctx):
    """Work right behind the call on its stream, with and without items that share
    boundaries cut (whose merge is staged while the attention still runs)."""
    p = Packed(lens, ctx, 32, 8, 128, 16, bits, seed=47)
    first = run(p)
    out, copies = torch.empty_like(first), []
    for _ in range(50):
        out.fill_(SENTINEL)
        p.attend(out=out)
        copies.append(out.clone())
    for c in copies:
        assert torch.equal(c.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("bits", [16, 4])
def test_two_contexts_at_once(bits):
    """Two contexts on two streams share nothing."""
    a = Packed([1, 40], [2000, 300], 16, 2, 128, 16, bits, seed=48)
    b = Packed([3, 1], [900, 4000], 8, 8, 64, 16, bits, seed=49)
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
            assert torch.equal(x.view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("bits", [16, 4])
def test_captured_steps_follow_the_lengths(bits):
    """An append and its attention captured once; the replays read the lengths,
    pages and tokens of their own time."""
    p = Packed([2, 9], [30, 100], 8, 2, 64, 16, bits, seed=35)
    p.fill_context()
    qo, out = torch.empty_like(p.q), torch.empty_like(p.q)
    p.append(q_out=qo)
    p.attend(q=qo, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.append(q_out=qo)
        p.attend(q=qo, out=out)
    for step in range(3):
        p.q.normal_(), p.k.normal_(), p.v.normal_()
        if step:  # other lengths, on the pages that the requests have
            p.ctx = [30 - 9 * step, 100 - 7 * step]
            p.ctx_lens.copy_(torch.tensor(p.ctx, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, tol = p.attention64()
        check_close(out, want, tol)
    assert p.h.ddt_device_status() == 0


def test_pool_past_32_bits():
    p = Packed([1, 3], [40, 20], 8, 8, 128, 16, 16, seed=36, stale=0.0, extra_pages=2 ** 31 // (16 * 8 * 128) + 4)
    n = p.num_pages
    p.table[0, :3] = torch.tensor([n - 1, n - 3, n - 2], dtype=torch.int32)
    p.table[1, :2] = torch.tensor([n - 5, n - 4], dtype=torch.int32)
    run(p)


@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_then_steps(bits):
    """A prompt in two chunks, then drafted chains of 5 tokens of which 2 are
    kept, then single tokens: lengths move by new_lens or by what was kept, and
    every attention equals the one of the whole sequence at once."""
    R, Hq, Hkv, d = 3, 8, 2, 64
    total = [150, 33, 260]
    g = torch.Generator(device="cuda")
    g.manual_seed(40)
    rot = ddt.Rotary(ddt.rotary_table(400, d), d)
    full = Packed(total, [0] * R, Hq, Hkv, d, 16, bits, seed=41)
    qo = full.append(rot)
    want, tol = full.attention64(qo)
    step = Packed(total, [0] * R, Hq, Hkv, d, 16, bits, seed=42)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    done = [0] * R

    def feed(counts, keep):
        """counts[r] next tokens of each request, of which keep[r] stay."""
        rows = torch.cat([torch.arange(done[r], done[r] + counts[r]) + int(full.starts[r]) for r in range(R)]).cuda()
        starts = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
        q, k, v = full.q[rows], full.k[rows], full.v[rows]
        out, new = torch.empty_like(q), torch.empty_like(lens)
        kw = dict(q_out=q, rotary=rot, new_lens=new)
        if bits == 16:
            step.h.ddt_append_kv(q, k, v, starts, lens, step.table, R, step.k_cache, step.v_cache, **kw)
            step.h.ddt_prompt_attention(q, starts, lens, step.table, R, step.k_cache, step.v_cache, out)
        else:
            step.h.ddt_append_kvq(q, k, v, starts, lens, step.table, R, step.kv4, **kw)
            step.h.ddt_prompt_attention_kvq(q, starts, lens, step.table, R, step.kv4, out)
        check_close(out, want[rows], tol[rows])
        for r in range(R):
            done[r] += keep[r]
        if keep == counts:
            lens.copy_(new)
        else:
            lens.copy_(torch.tensor(done, dtype=torch.int32))

    feed([100, 1, 128], [100, 1, 128])
    feed([30, 20, 0], [30, 20, 0])
    for _ in range(3):
        feed([5, 4, 5], [2, 2, 2])
    for _ in range(2):
        feed([1, 1, 1], [1, 1, 1])
    assert step.h.ddt_device_status() == 0


def test_beside_the_tree():
    """A chain as a tree (each position's parent the one before it): tree
    attention of its unappended keys equals prompt attention of the appended
    ones, and the round's compaction leaves the rows that the append writes."""
    R, B, Hq, Hkv, d, page = 3, 8, 8, 2, 128, 16
    P = B + 1
    p = Packed([P] * R, [50, 0, 131], Hq, Hkv, d, page, 16, seed=43, stale=0.0)
    p.fill_context()
    mask = torch.zeros((R, P, 1), dtype=torch.int32, device="cuda")
    for i in range(P):
        mask[:, i, 0] = (1 << (i + 1)) - 1
    tree = torch.empty((R, P, Hq, d), dtype=torch.float32, device="cuda")
    p.h.ddt_tree_attention(p.q, p.k, p.v, p.k_cache, p.v_cache, p.table, p.ctx_lens, mask, R, tree)
    # accept three nodes of each chain: slots ctx .. ctx + 3
    nodes = torch.tensor([[1, 2, 3, -1]] * R, dtype=torch.int32, device="cuda")
    acc = torch.full((R,), 4, dtype=torch.int32, device="cuda")
    kc, vc, cl = p.k_cache.clone(), p.v_cache.clone(), p.ctx_lens.clone()
    p.h.ddt_compact(kc, vc, p.table, cl, p.k, p.v, nodes, acc, R)
    p.append()
    got = p.attend()
    want, tol = p.attention64()
    check_close(got, want, tol)
    # (the tree's result is fp32: no rounding of the result, the same bound otherwise)
    check_close(tree.view(-1, Hq, d), want, tol)
    for r, c in enumerate(p.ctx):
        pg, row = p.slots(r, c, c + 4)
        assert torch.equal(kc[pg, row], p.k_cache[pg, row]) and torch.equal(vc[pg, row], p.v_cache[pg, row])
    assert cl.tolist() == [c + 4 for c in p.ctx]
