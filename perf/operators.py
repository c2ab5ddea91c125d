"""The serving operators around the paged KV cache, as cases to be measured.

Three operators: keys and values of new tokens appended to the paged cache
with the position rotation applied on the way (into a bf16 cache or one held
in 4 bits), causal attention of packed sequences over that cache (a prompt, a
chunk of one, a drafted chain, a single token), and the same attention over
the cache held in 4 bits. `run` computes them in elementary torch operations,
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


def _case(name, kind, bits, R, len_lo, len_hi, ctx_lo, ctx_hi, Hq=32, Hkv=8, d=128, page=16, rot=None,
          inter=False, shape=1):
    c = {"kind": kind, "bits": bits, "R": R, "len_lo": len_lo, "len_hi": len_hi, "ctx_lo": ctx_lo,
         "ctx_hi": ctx_hi, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "rot": d if rot is None else rot,
         "inter": inter, "shape": shape}
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decoded token of a single request: the launch is what it costs
        _case("append_one", "append", 16, 1, 1, 1, 4096, 4096),
        # a verification step: 64 requests' drafted chains and their roots (15 + 1 tokens)
        _case("append_chains", "append", 16, 64, 16, 16, 512, 2048),
        # a batch of ragged prompts behind earlier turns
        _case("append_prompts", "append", 16, 24, 1, 2047, 0, 1500),
        # the drafted chains into a cache held in 4 bits
        _case("append4_chains", "append", 4, 64, 16, 16, 512, 2048),
        # ragged prompts into it: narrow heads, half of each rotated in neighbouring pairs, larger pages
        _case("append4_prompts", "append", 4, 24, 1, 2047, 0, 1500, Hq=16, Hkv=16, d=64, page=64, rot=32,
              inter=True),
        # one token of a single request: latency
        _case("attend_one", "attend", 16, 1, 1, 1, 4096, 4096),
        # a decoding step of 64 requests with mixed contexts: reads the cache once
        _case("attend_decode", "attend", 16, 64, 1, 1, 512, 16384),
        # the same requests' drafted chains, 16 tokens each
        _case("attend_chains", "attend", 16, 64, 16, 16, 512, 16384),
        # one long prompt from the start: matrix products
        _case("attend_prompt", "attend", 16, 1, 16384, 16384, 0, 0),
        # packed short and middling prompts, one KV head for each query head, narrow heads
        _case("attend_packed", "attend", 16, 32, 1, 2047, 0, 300, Hq=8, Hkv=8, d=64, page=64),
        # the decoding step over a cache held in 4 bits
        _case("attend4_decode", "attend", 4, 64, 1, 1, 512, 16384),
        # chunks of prompts behind long contexts over it
        _case("attend4_chunks", "attend", 4, 4, 1500, 2048, 4000, 16000),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    while True:
        kind = rng.choice(("append", "attend", "attend"))
        d = rng.choice((64, 128, 128))
        hkv = rng.choice((1, 2, 4, 5, 8, 8))
        g = rng.choice((1, 2, 4, 4, 8, 16))
        if hkv * g > 64:
            continue
        R = log_int(1, 96)
        len_hi = log_int(1, 12000)
        len_lo = log_int(1, len_hi)
        ctx_hi = log_int(1, 30000) if kind == "attend" else log_int(1, 2000)
        ctx_lo = rng.randint(0, ctx_hi)
        c = _case(None, kind, rng.choice((16, 16, 4)), R, len_lo, len_hi, ctx_lo, ctx_hi, hkv * g, hkv, d,
                  rng.choice((16, 16, 32, 64, 256)), rng.choice((d, d, d // 2)), rng.random() < 0.4,
                  rng.randrange(1 << 20))
        lens, ctx = _lengths(c)
        w = work(c)
        if w["flops"] > 1.5e12 or w["bytes"] > 1.5e9 or sum(x + y for x, y in zip(lens, ctx)) * hkv * d > 4e8 or \
                sum(lens) * hkv * g * d > 2e8:
            continue
        return c


def _lengths(case):
    rng = random.Random(case["shape"] * 7919 + case["R"])
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["R"])]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["R"])]
    return lens, ctx


def _row_bytes(case):
    """Bytes of one token's key (or value) row of the cache."""
    n = case["Hkv"] * case["d"]
    return 2 * n if case["bits"] == 16 else n // 2 + n // 16


def work(case):
    lens, ctx = _lengths(case)
    T, Hq, Hkv, d = sum(lens), case["Hq"], case["Hkv"], case["d"]
    if case["kind"] == "append":
        held = 2 * T * Hkv * d * 2 if case["bits"] == 4 else 0  # the values that the new codes stand for
        rows = 2 * T * Hq * d * 2 + 2 * T * Hkv * d * 2 + 2 * T * _row_bytes(case) + held
        tab = len({p for n, c in zip(lens, ctx) for p in range(c, c + n)}) * case["rot"] * 4
        return {"bytes": rows + tab, "flops": T * (Hq + Hkv) * case["rot"] * 3}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(lens, ctx))
    byts = 2 * T * Hq * d * 2 + 2 * sum(n + c for n, c in zip(lens, ctx)) * _row_bytes(case)
    return {"bytes": byts, "flops": 4 * pairs * Hq * d}


def _pack4(x):
    """[..., d] fp32 -> codes [..., d/2] u8 and block scales [..., d/16] u8 (e4m3 bits); global scale 1."""
    d = x.shape[-1]
    b = x.reshape(*x.shape[:-1], d // 16, 16)
    amax = b.abs().amax(-1)
    sig = torch.clamp(amax / 6.0, max=448.0).to(torch.float8_e4m3fn)
    s = sig.float().unsqueeze(-1)
    mag = torch.zeros_like(b, dtype=torch.int64)
    for mid, up in MIDS:
        mag += (b.abs() >= s * mid) if up else (b.abs() > s * mid)
    mag = torch.where(s > 0, mag, torch.zeros_like(mag))
    code = mag + 8 * torch.signbit(b).long()
    # eight codes in four bytes: even elements in the low half's nibbles, odd ones in the high half's
    e = code.reshape(*x.shape[:-1], d // 8, 4, 2)
    lo = e[..., 0::2, :] + 16 * e[..., 1::2, :]  # [.., 2 bytes, even/odd]
    byts = lo.transpose(-1, -2).reshape(*x.shape[:-1], d // 2)
    return byts.to(torch.uint8), sig.view(torch.uint8)


def _unpack4(codes, scales, dtype=torch.float32):
    d = codes.shape[-1] * 2
    c = codes.reshape(*codes.shape[:-1], d // 8, 2, 2).long()  # [.., even/odd, byte]
    nib = torch.stack((c & 15, c >> 4), dim=-1)  # [.., even/odd, byte, nibble]
    e = nib.reshape(*codes.shape[:-1], d // 8, 2, 4).transpose(-1, -2).reshape(*codes.shape[:-1], d)
    mag = torch.tensor(MAG, dtype=dtype, device=codes.device)[e & 7]
    val = torch.where(e >= 8, -mag, mag).reshape(*codes.shape[:-1], d // 16, 16)
    return (val * scales.view(torch.float8_e4m3fn).to(dtype).unsqueeze(-1)).reshape(*codes.shape[:-1], d)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens, ctx = _lengths(case)
    R, Hq, Hkv, d, page = case["R"], case["Hq"], case["Hkv"], case["d"], case["page"]
    T = sum(lens)
    need = [(n + c + page - 1) // page for n, c in zip(lens, ctx)]
    max_pages, num_pages = max(need) + 1, sum(need) + 3
    perm = torch.randperm(num_pages, generator=gen, device=dev)[:sum(need)].int()
    table = torch.full((R, max_pages), 0, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    st = {"case": case, "T": T, "lens": lens, "ctx": ctx, "table": table,
          "q_start": torch.tensor(starts, dtype=torch.int32, device=dev),
          "ctx_lens": torch.tensor(ctx, dtype=torch.int32, device=dev),
          "max_pages": max_pages, "num_pages": num_pages}
    # rows of queries and keys as projections give them: a few channels carry more
    gain = 1.0 + 2.0 * (torch.rand(d, generator=gen, device=dev) > 0.95).float()
    st["q"] = (normal(T, Hq, d) * gain).bfloat16()
    if case["kind"] == "append":
        st["k"] = (normal(T, Hkv, d) * gain).bfloat16()
        st["v"] = normal(T, Hkv, d).bfloat16()
        st["q_out"] = torch.empty_like(st["q"])
        if case["bits"] == 4:
            st["k_held"], st["v_held"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        n_pos = max(n + c for n, c in zip(lens, ctx))
        st["angles"] = _angle_table(n_pos, case["rot"], dev)
    if case["bits"] == 16:
        st["k_cache"] = normal(num_pages, page, Hkv, d).bfloat16()
        st["v_cache"] = normal(num_pages, page, Hkv, d).bfloat16()
    else:
        for n in ("k", "v"):
            codes = torch.empty((num_pages, Hkv, page, d // 2), dtype=torch.uint8, device=dev)
            scales = torch.empty((num_pages, Hkv, page, d // 16), dtype=torch.uint8, device=dev)
            for i in range(0, num_pages, 4096):  # in pieces: the spread-out codes are wide
                j = min(num_pages, i + 4096)
                codes[i:j], scales[i:j] = _pack4(normal(j - i, Hkv, page, d))
            st[n + "_codes"], st[n + "_scales"] = codes, scales
    if case["kind"] == "attend":
        st["out"] = torch.empty_like(st["q"])
    if own:
        from speculative_decoding_draft_depth_gb300 import ddt
        st["handle"] = ddt.Context(ddt.make_config(
            R_max=R, L=4, V=32, B=8, Hq=Hq, Hkv=Hkv, d=d, page_size=page, max_pages_per_req=max_pages,
            num_pages=num_pages))
        if case["kind"] == "append":
            st["rotary"] = ddt.Rotary(st["angles"], case["rot"], case["inter"])
        if case["bits"] == 4:
            st["kv4"] = ddt.Kv4Cache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"])
    return st


def _angle_table(n_pos, rot, dev):
    """cos and sin of position * 10000^(-2j/rot), [n_pos, rot] fp32: rot/2 cosines, then rot/2 sines."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), -1).float()


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return _append(st, case) if case["kind"] == "append" else _attend(st, case)


def _run_own(st, case):
    h, R = st["handle"], case["R"]
    if case["kind"] == "append" and case["bits"] == 16:
        h.ddt_append_kv(st["q"], st["k"], st["v"], st["q_start"], st["ctx_lens"], st["table"], R, st["k_cache"],
                        st["v_cache"], q_out=st["q_out"], rotary=st["rotary"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if case["kind"] == "append":
        h.ddt_append_kvq(st["q"], st["k"], st["v"], st["q_start"], st["ctx_lens"], st["table"], R, st["kv4"],
                         q_out=st["q_out"], rotary=st["rotary"], k_held=st["k_held"], v_held=st["v_held"])
        return st["q_out"], st["k_held"], st["v_held"], st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"]
    if case["bits"] == 16:
        h.ddt_prompt_attention(st["q"], st["q_start"], st["ctx_lens"], st["table"], R, st["k_cache"], st["v_cache"],
                               st["out"])
    else:
        h.ddt_prompt_attention_kvq(st["q"], st["q_start"], st["ctx_lens"], st["table"], R, st["kv4"], st["out"])
    return st["out"]


def _rotate(x, row, rot, inter):
    """x [T, H, d] rotated in fp32 by the table rows [T, rot]."""
    x = x.float()
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if inter else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _slots(st, case):
    """Of every new token: its position, its page and its row in the page."""
    start = st["q_start"].long()
    t = torch.arange(st["T"], device=start.device)
    r = torch.searchsorted(start, t, right=True) - 1
    pos = st["ctx_lens"].long()[r] + t - start[r]
    return pos, st["table"][r, pos // case["page"]].long(), pos % case["page"]


def _append(st, case):
    pos, pg, at = _slots(st, case)
    row = st["angles"][pos]
    st["q_out"].copy_(_rotate(st["q"], row, case["rot"], case["inter"]))
    k, v = _rotate(st["k"], row, case["rot"], case["inter"]), st["v"].float()
    if case["bits"] == 16:
        st["k_cache"][pg, at] = k.bfloat16()
        st["v_cache"][pg, at] = v.bfloat16()
        return st["q_out"], st["k_cache"], st["v_cache"]
    for n, x in (("k", k), ("v", v)):
        codes, scales = _pack4(x)
        st[n + "_codes"][pg, :, at] = codes
        st[n + "_scales"][pg, :, at] = scales
        st[n + "_held"].copy_(_unpack4(codes, scales))
    return st["q_out"], st["k_held"], st["v_held"], st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"]


def _rows_of(st, case, r, n):
    """Keys and values of request r's first n positions, [Hkv, n, d] fp32."""
    page = case["page"]
    pg = st["table"][r, :(n + page - 1) // page].long()
    if case["bits"] == 16:
        return tuple(st[x][pg].flatten(0, 1)[:n].transpose(0, 1).float() for x in ("k_cache", "v_cache"))
    return tuple(_unpack4(st[x + "_codes"][pg], st[x + "_scales"][pg]).transpose(0, 1).flatten(1, 2)[:, :n]
                 for x in ("k", "v"))


def _attend(st, case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    G, t0 = Hq // Hkv, 0
    for r, (n, c) in enumerate(zip(st["lens"], st["ctx"])):
        k, v = _rows_of(st, case, r, c + n)
        step = max(1, (1 << 29) // (Hq * (c + n)))  # rows at a time, for the scores' memory
        for i in range(0, n, step):
            m = min(step, n - i)
            last = c + i + m  # keys up to the chunk's last token
            q = st["q"][t0 + i:t0 + i + m].float().reshape(m, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * m, d)
            s = (q @ k[:, :last].transpose(1, 2) / math.sqrt(d)).view(Hkv, G, m, last)
            if m > 1:
                own_pos = torch.arange(c + i, last, device=s.device)
                s.masked_fill_(torch.arange(last, device=s.device)[None, :] > own_pos[:, None], -math.inf)
            p = (s - s.amax(-1, keepdim=True)).exp()
            p = (p / p.sum(-1, keepdim=True)).view(Hkv, G * m, last)
            o = (p @ v[:, :last]).view(Hkv, G, m, d).permute(2, 0, 1, 3).reshape(m, Hq, d)
            st["out"][t0 + i:t0 + i + m] = o
        t0 += n
    return st["out"]


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st, case) if case["kind"] == "append" else _exact_attend(st, case)


def _exact_append(st, case):
    d, rot, page, dev = case["d"], case["rot"], case["page"], st["q"].device
    where = [(r, c + i) for r, (n, c) in enumerate(zip(st["lens"], st["ctx"])) for i in range(n)]
    req = torch.tensor([w[0] for w in where], device=dev)
    pos = torch.tensor([w[1] for w in where], device=dev)
    # each pair as a complex number, turned by its angle
    j = torch.arange(rot // 2, device=dev)
    first, second = (2 * j, 2 * j + 1) if case["inter"] else (j, j + rot // 2)
    phase = pos.double()[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev), -2.0 * j / rot)
    turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]

    def rotated(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = rotated(st["q"]), rotated(st["k"]), st["v"].double()
    pg = st["table"][req, pos // page].long()
    if case["bits"] == 16:
        caches = [st["k_cache"].double(), st["v_cache"].double()]
        for cache, x in zip(caches, (k, v)):
            cache[pg, pos % page] = x
        return [q] + caches
    grid = torch.tensor(MAG, dtype=torch.float64, device=dev)
    held = []
    for x in (k, v):
        b = x.unflatten(-1, (d // 16, 16))
        sig = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double()
        y = b.abs() / sig.clamp(min=1e-30)
        hi = torch.searchsorted(grid, y.contiguous()).clamp(1, 7)
        low, high = grid[hi - 1], grid[hi]
        up = (y - low > high - y) | ((y - low == high - y) & (hi % 2 == 0))
        held.append((torch.where(up, high, low) * sig * b.sign()).flatten(-2))
    return [q] + held + [None] * 4


def _exact_attend(st, case):
    if work(case)["flops"] > 3e12:
        return None
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    G, out, t0 = Hq // Hkv, torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device), 0
    for r in range(case["R"]):
        n, c = st["lens"][r], st["ctx"][r]
        at = torch.arange(c + n, device=out.device)
        pg, row = st["table"][r, at // page].long(), at % page
        for h in range(Hkv):
            if case["bits"] == 16:
                k, v = st["k_cache"][pg, row, h].double(), st["v_cache"][pg, row, h].double()
            else:
                k, v = (_unpack4(st[x + "_codes"][pg, h, row], st[x + "_scales"][pg, h, row], torch.float64)
                        for x in ("k", "v"))
            for i in range(0, n, 512):
                m = min(512, n - i)
                last = c + i + m
                q = st["q"][t0 + i:t0 + i + m, h * G:(h + 1) * G].double()
                s = torch.einsum("mgd,nd->mgn", q, k[:last]) * d ** -0.5
                ahead = at[None, None, :last] > at[c + i:last][:, None, None]
                p = torch.softmax(s.masked_fill(ahead, -math.inf), -1)
                out[t0 + i:t0 + i + m, h * G:(h + 1) * G] = torch.einsum("mgn,nd->mgd", p, v[:last])
        t0 += n
    return out
