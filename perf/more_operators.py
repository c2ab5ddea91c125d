"""Sampled decoding of many continuations, as cases to be measured.

Three operators: a token of each logit row drawn under its temperature, top-k,
top-p and min-p from given random numbers; drafted chains verified by the
probability rule when both the drafter's and the target's tokens are drawn
under such settings; and attention of a batch whose requests share long
prefixes in the paged KV cache (in bf16, or held in 4 bits), each prefix read
once for all its requests. `run` computes them in elementary torch operations,
or, with `own` set, through this repository's calls.

A case's lengths follow from the case alone (its "shape" number), the values
from the seed.
"""
import math
import random

import torch

own = False

MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1 magnitudes by code
#: nearest e2m1: the midpoints, and whether a value on one goes up (ties to the even code)
MIDS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


def _sample(name, rows, V, dtype, settings, spread_lo, spread_hi):
    c = {"kind": "sample", "rows": rows, "V": V, "dtype": dtype, "settings": settings, "spread_lo": spread_lo,
         "spread_hi": spread_hi}
    return c if name is None else {"name": name, **c}


def _accept(name, R, L, V, draft, target, settings, cut, spread_lo, spread_hi, shape=1):
    c = {"kind": "accept", "R": R, "L": L, "V": V, "dtype": target, "draft": draft, "settings": settings, "cut": cut,
         "spread_lo": spread_lo, "spread_hi": spread_hi, "shape": shape}
    return c if name is None else {"name": name, **c}


def _prefix(name, groups, mem_lo, mem_hi, pre_lo, pre_hi, own_lo, own_hi, tok_lo, tok_hi, bits=16, Hq=32, Hkv=8, d=128,
            page=16, shape=1):
    c = {"kind": "prefix", "groups": groups, "mem_lo": mem_lo, "mem_hi": mem_hi, "pre_lo": pre_lo, "pre_hi": pre_hi,
         "own_lo": own_lo, "own_hi": own_hi, "tok_lo": tok_lo, "tok_hi": tok_hi, "bits": bits, "Hq": Hq, "Hkv": Hkv,
         "d": d, "page": page, "shape": shape}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # the next token of a single request under every setting: latency
        _sample("sample_one", 1, 151936, "bf16", "all", 2.0, 4.0),
        # a decoding step of 64 requests, each with settings of its own (some greedy, some without any)
        _sample("sample_step", 64, 151936, "bf16", "mixed", 1.0, 4.0),
        # a large step at temperatures alone, fp32 logits, an odd vocabulary
        _sample("sample_wide", 256, 100003, "f32", "temperature", 1.0, 4.0),
        # hot, nearly flat rows under top-p: the kept set is most of the vocabulary
        _sample("sample_flat", 96, 151936, "bf16", "nucleus", 1.0, 1.4),
        # one drafted chain of 15 guesses: latency
        _accept("accept_one", 1, 15, 151936, "bf16", "bf16", "mixed", False, 2.0, 4.0),
        # the drafted chains of 64 requests
        _accept("accept_chains", 64, 15, 151936, "bf16", "bf16", "mixed", False, 2.0, 4.0),
        # prefixes of short chains that a scheduler kept, an fp32 drafter, an odd vocabulary
        _accept("accept_kept", 48, 5, 32003, "f32", "bf16", "mixed", True, 1.0, 4.0),
        # a few continuations of one short prompt: latency
        _prefix("prefix_few", 1, 8, 8, 1000, 1000, 1, 60, 1, 1),
        # 64 continuations of one prompt, a token each
        _prefix("prefix_step", 1, 64, 64, 8192, 8192, 1, 1024, 1, 1),
        # several system prompts, chains of drafted tokens under verification, groups of one among them
        _prefix("prefix_chains", 8, 1, 24, 500, 12000, 1, 700, 1, 16),
        # many continuations of long documents, narrow heads, larger pages
        _prefix("prefix_wide", 2, 96, 128, 9000, 16384, 1, 600, 1, 2, Hq=16, Hkv=4, d=64, page=64),
        # the step over a cache held in 4 bits
        _prefix("prefix4_step", 1, 64, 64, 8192, 8192, 1, 1024, 1, 1, bits=4),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    while True:
        kind = rng.choice(("sample", "accept", "prefix"))
        lo = rng.uniform(1.0, 3.0)
        hi = rng.uniform(lo, 4.0)
        if kind == "sample":
            c = _sample(None, log_int(1, 512), log_int(500, 262144), rng.choice(("bf16", "f32")),
                        rng.choice(("all", "mixed", "temperature", "nucleus")), lo, hi)
            if c["rows"] * c["V"] > 25_600_000:
                continue
            return c
        if kind == "accept":
            c = _accept(None, log_int(1, 96), rng.randint(1, 18), log_int(500, 152000), rng.choice(("bf16", "f32")),
                        rng.choice(("bf16", "f32")), rng.choice(("all", "mixed", "temperature", "nucleus")),
                        rng.random() < 0.4, lo, hi, rng.randrange(1 << 20))
            if c["R"] * (2 * c["L"] + 1) * c["V"] > 100_000_000:
                continue
            return c
        d = rng.choice((64, 128, 128))
        hkv = rng.choice((1, 2, 4, 5, 8, 8))
        g = rng.choice((1, 2, 4, 4, 8, 16))
        mem_hi, pre_hi, own_hi, tok_hi = log_int(1, 128), log_int(1, 16384), log_int(1, 1500), log_int(1, 16)
        c = _prefix(None, log_int(1, 8), log_int(1, mem_hi), mem_hi, log_int(1, pre_hi), pre_hi, log_int(1, own_hi),
                    own_hi, log_int(1, tok_hi), tok_hi, rng.choice((16, 16, 4)), hkv * g, hkv, d,
                    rng.choice((16, 16, 32, 64, 256)), rng.randrange(1 << 20))
        if hkv * g > 64:
            continue
        groups, lens, ctx = _lengths(c)
        R, S, n = len(lens), max(x + y for x, y in zip(lens, ctx)), max(lens)
        # (the plain form spreads every request's keys out, and its scores)
        if R * S * hkv * d > 1.2e9 or R * S * hkv * g * n > 2.5e9 or work(c)["flops"] > 4e11:
            continue
        return c


def _lengths(case):
    """Members and prefix of each group; tokens and context (the prefix in it) of each request."""
    rng = random.Random(case["shape"] * 7919 + case["groups"])
    groups = [(rng.randint(case["mem_lo"], case["mem_hi"]), rng.randint(case["pre_lo"], case["pre_hi"]))
              for _ in range(case["groups"])]
    lens, ctx = [], []
    for m, p in groups:
        for _ in range(m):
            lens.append(rng.randint(case["tok_lo"], case["tok_hi"]))
            ctx.append(p + rng.randint(case["own_lo"], case["own_hi"]) - 1)
    return groups, lens, ctx


def _guesses(case):
    rng = random.Random(case["shape"] * 104729 + case["R"])
    return [rng.randint(0, case["L"]) if case["cut"] else case["L"] for _ in range(case["R"])]


def work(case):
    if case["kind"] == "sample":
        n = case["rows"] * case["V"]
        return {"bytes": n * _size(case["dtype"]) + case["rows"] * 28, "flops": 4 * n}
    if case["kind"] == "accept":
        rows = sum(_guesses(case))
        byts = rows * case["V"] * _size(case["draft"]) + (rows + case["R"]) * case["V"] * _size(case["dtype"])
        return {"bytes": byts + case["R"] * (16 * case["L"] + 48), "flops": 4 * (2 * rows + case["R"]) * case["V"]}
    groups, lens, ctx = _lengths(case)
    T, Hq, d = sum(lens), case["Hq"], case["d"]
    n = case["Hkv"] * d
    keys, r = 0, 0  # a prefix once, and what each request has behind it
    for m, p in groups:
        keys += p + sum(lens[i] + ctx[i] - p for i in range(r, r + m))
        r += m
    pairs = sum(x * c + x * (x + 1) // 2 for x, c in zip(lens, ctx))
    row = 2 * n if case["bits"] == 16 else n // 2 + n // 16
    return {"bytes": 2 * T * Hq * d * 2 + 2 * keys * row, "flops": 4 * pairs * Hq * d}


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if case["kind"] == "sample":
        st = _prepare_sample(case, gen, dev)
    elif case["kind"] == "accept":
        st = _prepare_accept(case, gen, dev)
    else:
        st = _prepare_prefix(case, gen, dev)
    st["case"] = case
    if own:
        _prepare_own(st, case)
    return st


def _uniform(gen, dev, *shape):
    return torch.rand(*shape, generator=gen, device=dev)


def _logits(gen, dev, rows, V, lo, hi):
    """Rows as a model gives them: a spread of their own, and a few likely tokens at the front."""
    spread = lo + (hi - lo) * _uniform(gen, dev, rows, 1)
    z = torch.randn(rows, V, generator=gen, device=dev) * spread
    boost = 8.0 * torch.arange(1, 21, device=dev).float() ** -1.1
    at = torch.randint(0, V, (rows, 20), generator=gen, device=dev)
    return z.scatter_add_(1, at, boost.expand(rows, 20).contiguous())


def _settings(gen, dev, n, which):
    """temperature, top_k, top_p, min_p of n rows or requests (temperature 0: greedy; top_k 0, top_p 1, min_p 0: off)."""
    t = 0.5 + 0.8 * _uniform(gen, dev, n)
    k = torch.zeros(n, dtype=torch.int32, device=dev)
    p, m = torch.ones(n, device=dev), torch.zeros(n, device=dev)
    if which == "nucleus":
        p = 0.8 + 0.19 * _uniform(gen, dev, n)
    if which in ("all", "mixed"):
        k = torch.randint(5, 101, (n,), generator=gen, device=dev, dtype=torch.int32)
        p = 0.7 + 0.29 * _uniform(gen, dev, n)
        m = 0.1 * _uniform(gen, dev, n)
    if which == "mixed":  # each of them on for about half of the requests; one request in sixteen is greedy
        on = _uniform(gen, dev, 4, n)
        t = torch.where(on[3] < 0.0625, torch.zeros_like(t), t)
        k = torch.where(on[0] < 0.5, k, torch.zeros_like(k))
        p = torch.where(on[1] < 0.5, p, torch.ones_like(p))
        m = torch.where(on[2] < 0.5, m, torch.zeros_like(m))
    return t, k, p, m


def _of_type(z, dtype):
    return z.bfloat16() if dtype == "bf16" else z


def _prepare_sample(case, gen, dev):
    rows, V = case["rows"], case["V"]
    return {"logits": _of_type(_logits(gen, dev, rows, V, case["spread_lo"], case["spread_hi"]), case["dtype"]),
            "settings": _settings(gen, dev, rows, case["settings"]), "u": _uniform(gen, dev, rows),
            "tokens": torch.empty(rows, dtype=torch.int32, device=dev),
            "logprobs": torch.empty(rows, dtype=torch.float32, device=dev)}


def _prepare_accept(case, gen, dev):
    R, L, V = case["R"], case["L"], case["V"]
    draft = torch.empty(R, L, V, dtype=_of_type(torch.empty(0), case["draft"]).dtype, device=dev)
    target = torch.empty(R, L + 1, V, dtype=_of_type(torch.empty(0), case["dtype"]).dtype, device=dev)
    tokens = torch.empty(R, L, dtype=torch.int32, device=dev)
    settings = _settings(gen, dev, R, case["settings"])
    for i in range(R):
        z = _logits(gen, dev, L + 1, V, case["spread_lo"], case["spread_hi"])
        target[i] = (z + torch.randn(L + 1, V, generator=gen, device=dev) * (0.1 + 0.5 * _uniform(gen, dev, 1)))
        draft[i] = z[:L]
        # the drafter draws its guesses from the rows it gives, among the most likely tokens
        top = draft[i].float().topk(min(V, 40), dim=1)
        g = -torch.log(-torch.log(_uniform(gen, dev, *top.values.shape).clamp(1e-9, 1 - 1e-7)))
        pick = (top.values / settings[0][i].clamp(min=0.05) + g * (settings[0][i] > 0)).argmax(1, keepdim=True)
        tokens[i] = top.indices.gather(1, pick).squeeze(1).int()
    return {"draft": draft, "target": target, "tokens": tokens, "settings": settings, "u": _uniform(gen, dev, R, L),
            "r": _uniform(gen, dev, R),
            "n_guess": torch.tensor(_guesses(case), dtype=torch.int32, device=dev) if case["cut"] else None,
            "acc_len": torch.empty(R, dtype=torch.int32, device=dev),
            "acc_tokens": torch.empty(R, L + 1, dtype=torch.int32, device=dev)}


def _prepare_prefix(case, gen, dev):
    groups, lens, ctx = _lengths(case)
    R, Hq, Hkv, d, page = len(lens), case["Hq"], case["Hkv"], case["d"], case["page"]
    T = sum(lens)
    # a prefix's whole pages are held once; the page that its end lies in, and what follows, by each request
    rows, num_pages, r = [], 0, 0
    for m, p in groups:
        full = p // page
        shared = list(range(num_pages, num_pages + full))
        num_pages += full
        for i in range(r, r + m):
            n = (lens[i] + ctx[i] + page - 1) // page - full
            rows.append(shared + list(range(num_pages, num_pages + n)))
            num_pages += n
        r += m
    max_pages = max(len(x) for x in rows) + 1
    order = torch.randperm(num_pages + 3, generator=gen, device=dev).int()
    at = torch.tensor([x + [0] * (max_pages - len(x)) for x in rows], device=dev)
    used = torch.tensor([[1] * len(x) + [0] * (max_pages - len(x)) for x in rows], device=dev)
    table = (order[at] * used).int()
    num_pages += 3

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    starts, firsts = [0], [0]
    for n in lens:
        starts.append(starts[-1] + n)
    for m, _ in groups:
        firsts.append(firsts[-1] + m)
    i32 = dict(dtype=torch.int32, device=dev)
    # rows of queries and keys as projections give them: a few channels carry more
    gain = 1.0 + 2.0 * (torch.rand(d, generator=gen, device=dev) > 0.95).float()
    st = {"R": R, "T": T, "lens": lens, "ctx": ctx, "max_pages": max_pages, "num_pages": num_pages, "table": table,
          "q_start": torch.tensor(starts, **i32), "ctx_lens": torch.tensor(ctx, **i32),
          "group_start": torch.tensor(firsts, **i32), "prefix_lens": torch.tensor([p for _, p in groups], **i32),
          "q": (normal(T, Hq, d) * gain).bfloat16()}
    st["out"] = torch.empty_like(st["q"])
    kv = {}
    for n in ("k", "v"):
        if case["bits"] == 16:
            st[n + "_cache"] = kv[n] = normal(num_pages, page, Hkv, d).bfloat16()
        else:
            codes = torch.empty((num_pages, Hkv, page, d // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((num_pages, Hkv, page, d // 16), dtype=torch.uint8, device=dev)
            for i in range(0, num_pages, 4096):  # in pieces: the spread-out codes are wide
                j = min(num_pages, i + 4096)
                codes[i:j], scales[i:j] = _pack4(normal(j - i, Hkv, page, d))
            st[n + "_codes"], st[n + "_scales"] = codes, scales
    # the members of a group hold equal rows of the page that the prefix ends in
    end = st["prefix_lens"].long() % page
    lead = torch.repeat_interleave(st["group_start"][:-1].long(), torch.tensor([m for m, _ in groups], device=dev))
    of = torch.repeat_interleave(torch.arange(len(groups), device=dev), torch.tensor([m for m, _ in groups], device=dev))
    last = st["prefix_lens"].long()[of] // page
    src, dst = table[lead, last].long(), table[torch.arange(R, device=dev), last].long()
    here = torch.arange(page, device=dev)[None, :] < end[of][:, None]
    for n in [x for x in st if x.endswith(("_cache", "_codes", "_scales"))]:
        a, b = st[n][src], st[n][dst]
        mask = here[:, :, None, None] if n.endswith("_cache") else here[:, None, :, None]
        # (where the prefix fills its pages, a request without own tokens there writes back what it holds)
        st[n][dst] = torch.where(mask, a, b)
    return st


def _prepare_own(st, case):
    from speculative_decoding_draft_depth_gb300 import ddt
    kinds = {"bf16": ddt.BF16, "f32": ddt.F32}
    if case["kind"] == "prefix":
        st["handle"] = ddt.Context(ddt.make_config(
            R_max=st["R"], L=4, V=32, B=8, Hq=case["Hq"], Hkv=case["Hkv"], d=case["d"], page_size=case["page"],
            max_pages_per_req=st["max_pages"], num_pages=st["num_pages"], prefix_tokens=st["T"]))
        if case["bits"] == 4:
            st["kv4"] = ddt.Kv4Cache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"])
        return
    accept = case["kind"] == "accept"
    st["handle"] = ddt.Context(ddt.make_config(
        R_max=case["R"] if accept else 1, L=case["L"] if accept else 1, V=case["V"], B=8, Hq=8, Hkv=8, d=64, page_size=16,
        max_pages_per_req=1, num_pages=1, draft_dtype=kinds[case["draft"] if accept else case["dtype"]],
        target_dtype=kinds[case["dtype"]]))
    st["filter"] = ddt.Filter(*st["settings"])


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["kind"] == "sample":
        return _plain_sample(st)
    return _plain_accept(st, case) if case["kind"] == "accept" else _plain_prefix(st, case)


def _run_own(st, case):
    h = st["handle"]
    if case["kind"] == "sample":
        h.ddt_sample(st["logits"], st["u"], st["tokens"], filter=st["filter"], logprobs=st["logprobs"])
        return st["tokens"], st["logprobs"]
    if case["kind"] == "accept":
        h.ddt_accept_sampled(st["draft"], st["target"], st["tokens"], st["u"], st["r"], case["R"], st["acc_len"],
                             st["acc_tokens"], draft_filter=st["filter"], target_filter=st["filter"],
                             n_guess=st["n_guess"])
        return st["acc_len"], st["acc_tokens"]
    if case["bits"] == 16:
        h.ddt_prefix_attention(st["q"], st["q_start"], st["ctx_lens"], st["table"], st["R"], st["group_start"],
                               st["prefix_lens"], st["k_cache"], st["v_cache"], st["out"])
    else:
        h.ddt_prefix_attention_kvq(st["q"], st["q_start"], st["ctx_lens"], st["table"], st["R"], st["group_start"],
                                   st["prefix_lens"], st["kv4"], st["out"])
    return st["out"]


# ---------------------------------------------------------------- plain forms
def _kept(logits, settings):
    """Weights of the kept tokens, [n, V] fp64 (0: not kept; not divided by their sum). settings: four [n] tensors."""
    t, k, p, m = (x[:, None] for x in settings)
    greedy = t == 0
    t, k = torch.where(greedy, torch.ones_like(t), t), torch.where(greedy, torch.ones_like(k), k)
    z, order = logits.float().sort(dim=1, descending=True, stable=True)  # equal values: lower index first
    # in 64 bits: a sum next to the border decides which token is kept or drawn
    w = ((z.double() - z[:, :1].double()) / t.double()).exp()
    w = w.masked_fill_(w < m.double(), 0.0)
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    w = w.masked_fill_((rank >= k) & (k > 0), 0.0)
    before = w.cumsum(1)
    enough = p.double() * before[:, -1:]
    before = torch.cat((torch.zeros_like(enough), before[:, :-1]), 1)
    w = w.masked_fill_((before >= enough) & (rank > 0) & (p < 1), 0.0)
    return torch.empty_like(w).scatter_(1, order, w)


def _first_above(w, u):
    """First index whose running sum of the weights w [n, V] exceeds u [n] times their sum; -1 without weights."""
    s = w.cumsum(1)
    at = (s <= u.double()[:, None] * s[:, -1:]).sum(1)
    last = w.shape[1] - 1 - (w.flip(1) > 0).to(torch.int32).argmax(1)
    return torch.where(s[:, -1] > 0, torch.minimum(at, last), torch.full_like(at, -1)), s[:, -1]


def _plain_sample(st):
    w = _kept(st["logits"], st["settings"])
    at, total = _first_above(w, st["u"])
    st["tokens"].copy_(at)
    st["logprobs"].copy_((w.gather(1, at.clamp(min=0)[:, None]).squeeze(1) / total).log())
    return st["tokens"], st["logprobs"]


def _plain_accept(st, case):
    R, L, V = case["R"], case["L"], case["V"]
    dev = st["u"].device
    n = st["n_guess"].long() if case["cut"] else torch.full((R,), L, device=dev)
    wq = _kept(st["draft"].flatten(0, 1), tuple(x.repeat_interleave(L) for x in st["settings"])).view(R, L, V)
    wp = _kept(st["target"].flatten(0, 1), tuple(x.repeat_interleave(L + 1) for x in st["settings"])).view(R, L + 1, V)
    q, p = wq / wq.sum(2, keepdim=True), wp / wp.sum(2, keepdim=True)
    x = st["tokens"].long()
    qx, px = q.gather(2, x[:, :, None]).squeeze(2), p[:, :L].gather(2, x[:, :, None]).squeeze(2)
    ratio = torch.where(qx > 0, px / qx, torch.ones_like(qx)).clamp(max=1.0)
    step = torch.arange(L, device=dev)[None, :]
    keep = (st["u"].double() < ratio) & (step < n[:, None])
    first = keep.long().cumprod(1).sum(1)  # guesses kept
    row = torch.arange(R, device=dev)
    w = p[row, first]
    w = torch.where((first < n)[:, None], w - q[row, first.clamp(max=L - 1)], w).clamp(min=0.0)
    at, _ = _first_above(w, st["r"])
    step = torch.arange(L + 1, device=dev)[None, :]
    guess = torch.cat((x, torch.full((R, 1), -1, device=dev)), 1)
    none = torch.full_like(guess, -1)
    st["acc_tokens"].copy_(torch.where(step < first[:, None], guess, torch.where(step == first[:, None], at[:, None], none)))
    st["acc_len"].copy_(first + 1)
    return st["acc_len"], st["acc_tokens"]


def _plain_prefix(st, case):
    R, Hq, Hkv, d, page = st["R"], case["Hq"], case["Hkv"], case["d"], case["page"]
    G, n, S = Hq // Hkv, max(st["lens"]), max(x + c for x, c in zip(st["lens"], st["ctx"]))
    start, ctx = st["q_start"].long(), st["ctx_lens"].long()
    pg = st["table"][:, :(S + page - 1) // page].long()
    if case["bits"] == 16:
        k, v = (st[x][pg].flatten(1, 2)[:, :S].permute(0, 2, 1, 3).float() for x in ("k_cache", "v_cache"))
    else:
        k, v = (_unpack4(st[x + "_codes"][pg], st[x + "_scales"][pg]).permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :S]
                for x in ("k", "v"))
    i = torch.arange(n, device=start.device)
    q = st["q"][(start[:-1, None] + i).clamp(max=st["T"] - 1)].float()  # [R, n, Hq, d], rows behind a request's last unused
    q = q.view(R, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, d)
    s = (q @ k.transpose(2, 3) / math.sqrt(d)).view(R, Hkv, n, G, S)
    ahead = torch.arange(S, device=s.device)[None, None, :] > (ctx[:, None] + i)[:, :, None]
    s.masked_fill_(ahead[:, None, :, None, :], -math.inf)
    w = (s - s.amax(-1, keepdim=True)).exp_()
    w = (w / w.sum(-1, keepdim=True)).view(R, Hkv, n * G, S)
    # (slots behind a request's last hold other requests' values or zeros: weight 0)
    o = (w @ v).view(R, Hkv, n, G, d).permute(0, 2, 1, 3, 4).reshape(R, n, Hq, d)
    t = torch.arange(st["T"], device=start.device)
    r = torch.searchsorted(start, t, right=True) - 1
    st["out"].copy_(o[r, t - start[r]])
    return st["out"]


def _pack4(x):
    """[..., d] fp32 -> codes [..., d/2] u8 and block scales [..., d/16] u8 (e4m3 bits); global scale 1."""
    d = x.shape[-1]
    b = x.reshape(*x.shape[:-1], d // 16, 16)
    sig = torch.clamp(b.abs().amax(-1) / 6.0, max=448.0).to(torch.float8_e4m3fn)
    s = sig.float().unsqueeze(-1)
    mag = torch.zeros_like(b, dtype=torch.int64)
    for mid, up in MIDS:
        mag += (b.abs() >= s * mid) if up else (b.abs() > s * mid)
    mag = torch.where(s > 0, mag, torch.zeros_like(mag))
    code = mag + 8 * torch.signbit(b).long()
    # eight codes in four bytes: even elements in the low half's nibbles, odd ones in the high half's
    e = code.reshape(*x.shape[:-1], d // 8, 4, 2)
    byts = (e[..., 0::2, :] + 16 * e[..., 1::2, :]).transpose(-1, -2).reshape(*x.shape[:-1], d // 2)
    return byts.to(torch.uint8), sig.view(torch.uint8)


def _unpack4(codes, scales, dtype=torch.float32):
    d = codes.shape[-1] * 2
    c = codes.reshape(*codes.shape[:-1], d // 8, 2, 2)  # [.., even/odd, byte]
    nib = torch.stack((c & 15, c >> 4), dim=-1)  # [.., even/odd, byte, nibble]
    e = nib.reshape(*codes.shape[:-1], d // 8, 2, 4).transpose(-1, -2).reshape(*codes.shape[:-1], d)
    value = torch.tensor(MAG + tuple(-x for x in MAG), dtype=dtype, device=codes.device)[e.int()]
    s = scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)
    return (value.reshape(*codes.shape[:-1], d // 16, 16) * s).reshape(*codes.shape[:-1], d)


# ---------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "sample":
        return _exact_sample(st, case)
    return _exact_accept(st, case) if case["kind"] == "accept" else _exact_prefix(st, case)


def _distribution(z, t, k, p, m):
    """The kept tokens' probabilities of one row z [V], from its distinct values and how often each occurs."""
    z = z.double()
    value, where, count = torch.unique(z, sorted=True, return_inverse=True, return_counts=True)
    value, count, where = value.flip(0), count.flip(0), len(value) - 1 - where
    if t == 0.0:
        t, k = 1.0, 1
    w = torch.exp((value - value[0]) / t)
    n = count.double() * (w >= m)
    before = n.cumsum(0) - n
    if k > 0:
        n = torch.minimum(n, (k - before).clamp(min=0))
    if p < 1.0:
        mass = (n * w).cumsum(0)
        need = p * mass[-1]
        short = need - (mass - n * w)  # what is still to be reached before each value
        n = torch.where(short > 0, torch.minimum(n, torch.ceil(short / w.clamp(min=1e-300))), torch.zeros_like(n))
        n[0] = n[0].clamp(min=1)
    out = (w * (n == count))[where]
    for v in torch.nonzero((n > 0) & (n < count)).flatten().tolist():  # the value that the border cuts: lowest indices first
        out[torch.nonzero(where == v).flatten()[:int(n[v])]] = w[v]
    return out / out.sum()


def _pick(w, u):
    """First index whose running sum exceeds u times the sum."""
    s = torch.cumsum(w, 0)
    if not s[-1] > 0:
        return -1
    at = int(torch.searchsorted(s, u * s[-1], right=True))
    return min(at, int(torch.nonzero(w).max()))


def _exact_sample(st, case):
    rows = list(zip(*(x.tolist() for x in st["settings"])))
    u, tokens, lp = st["u"].tolist(), [], []
    for i, row in enumerate(rows):
        d = _distribution(st["logits"][i], *row)
        tokens.append(_pick(d, u[i]))
        lp.append(float(torch.log(d[tokens[-1]])))
    dev = st["u"].device
    return torch.tensor(tokens, dtype=torch.int32, device=dev), torch.tensor(lp, dtype=torch.float64, device=dev)


def _exact_accept(st, case):
    R, L = case["R"], case["L"]
    n, u, r, x = _guesses(case), st["u"].tolist(), st["r"].tolist(), st["tokens"].tolist()
    rows = list(zip(*(s.tolist() for s in st["settings"])))
    lens, toks = [], []
    for i in range(R):
        done = []
        for k in range(n[i] + 1):
            p = _distribution(st["target"][i, k], *rows[i])
            if k == n[i]:
                done.append(_pick(p, r[i]))
                break
            q = _distribution(st["draft"][i, k], *rows[i])
            a, b = float(p[x[i][k]]), float(q[x[i][k]])
            if not u[i][k] < (min(1.0, a / b) if b > 0 else 1.0):
                done.append(_pick((p - q).clamp(min=0), r[i]))
                break
            done.append(x[i][k])
        lens.append(len(done))
        toks.append(done + [-1] * (L + 1 - len(done)))
    i32 = dict(dtype=torch.int32, device=st["u"].device)
    return torch.tensor(lens, **i32), torch.tensor(toks, **i32)


def _exact_prefix(st, case):
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    if st["R"] * Hkv > 1500:
        return None
    G, out, t0 = Hq // Hkv, torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device), 0
    for r in range(st["R"]):
        n, c = st["lens"][r], st["ctx"][r]
        at = torch.arange(c + n, device=out.device)
        pg, row = st["table"][r, at // page].long(), at % page
        hidden = at[None, None, :] > at[c:][:, None, None]
        for h in range(Hkv):
            if case["bits"] == 16:
                k, v = st["k_cache"][pg, row, h].double(), st["v_cache"][pg, row, h].double()
            else:
                k, v = (_unpack4(st[x + "_codes"][pg, h, row], st[x + "_scales"][pg, h, row], torch.float64)
                        for x in ("k", "v"))
            q = st["q"][t0:t0 + n, h * G:(h + 1) * G].double()
            s = torch.einsum("mgd,nd->mgn", q, k) * d ** -0.5
            out[t0:t0 + n, h * G:(h + 1) * G] = torch.einsum("mgn,nd->mgd", torch.softmax(s.masked_fill(hidden, -math.inf), -1), v)
        t0 += n
    return out
