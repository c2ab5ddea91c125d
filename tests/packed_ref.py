"""Plain forms of the packed-sequence operators for their tests: the append
(rotation and 4-bit blocks) in fp32 exactly as the header defines it, and
causal attention in fp64; shared layouts and tolerances."""
import numpy as np
import torch

from speculative_decoding_draft_depth_gb300 import ddt

MAGS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
SENTINEL = -7.0


class Packed:
    """R requests' packed tokens over a paged pool: lens new tokens each behind
    ctx cached ones, `lead` rows before the first request and `tail` behind the
    last. Pages are shuffled; slots that no request has reached hold `stale`."""

    def __init__(self, lens, ctx, Hq=8, Hkv=2, d=64, page=16, bits=16, seed=0, lead=0, tail=0,
                 stale=float("nan"), R_max=None, k_scale=1.0, v_scale=1.0, extra_pages=5, v_gain=1.0):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.lens, self.ctx, self.R = list(lens), list(ctx), len(lens)
        self.Hq, self.Hkv, self.d, self.page, self.bits = Hq, Hkv, d, page, bits
        self.starts = np.concatenate(([0], np.cumsum(lens))).astype(np.int32) + lead
        self.T = int(self.starts[-1]) + tail
        need = [-(-(n + c) // page) for n, c in zip(lens, ctx)]
        self.max_pages, self.num_pages = max(need + [1]) + 1, sum(need) + extra_pages
        perm = torch.randperm(self.num_pages, generator=g)
        table = torch.full((self.R, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = perm[at:at + n].int()
            at += n
        self.table = table.cuda()
        self.q_start = torch.from_numpy(self.starts).cuda()
        self.ctx_lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        cg = torch.Generator(device="cuda")
        cg.manual_seed(seed + 1)

        def normal(*s):
            return torch.randn(*s, generator=cg, device="cuda")

        self.q, self.k = normal(self.T, Hq, d).bfloat16(), normal(self.T, Hkv, d).bfloat16()
        self.v = (normal(self.T, Hkv, d) * v_gain).bfloat16()
        self.h = ddt.Context(ddt.make_config(R_max=R_max or max(1, self.R), L=4, V=32, B=8, Hq=Hq, Hkv=Hkv, d=d,
                                             page_size=page, max_pages_per_req=self.max_pages,
                                             num_pages=self.num_pages))
        pool = (self.num_pages, page, Hkv, d)
        if bits == 16:
            self.k_cache = torch.full(pool, stale, device="cuda").bfloat16()
            self.v_cache = torch.full(pool, stale, device="cuda").bfloat16()
        else:
            self.kv4 = self.h.alloc_kv4(k_scale, v_scale)
            if stale != stale:  # NaN scales and the largest codes where nothing was appended
                for t in (self.kv4.k_codes, self.kv4.v_codes):
                    t.fill_(0x77)
                for t in (self.kv4.k_scales, self.kv4.v_scales):
                    t.fill_(0x7f)
        self._normal = normal

    # -- the pool as plain rows
    def slots(self, r, a, b):
        """Page and row of request r's slots a .. b - 1."""
        p = torch.arange(a, b, device="cuda")
        return self.table[r, p // self.page].long(), p % self.page

    def fill_context(self):
        """Random keys and values into every request's cached slots."""
        for r, c in enumerate(self.ctx):
            if c:
                self.put(r, 0, c, self._normal(c, self.Hkv, self.d).bfloat16(),
                         self._normal(c, self.Hkv, self.d).bfloat16())

    def fill_new(self):
        """The packed k and v into their slots, unturned."""
        for r, (n, c) in enumerate(zip(self.lens, self.ctx)):
            s = int(self.starts[r])
            if n:
                self.put(r, c, c + n, self.k[s:s + n], self.v[s:s + n])

    def put(self, r, a, b, k, v):
        pg, row = self.slots(r, a, b)
        if self.bits == 16:
            self.k_cache[pg, row], self.v_cache[pg, row] = k, v
            return
        for n, x, g in (("k", k, self.kv4.k_scale), ("v", v, self.kv4.v_scale)):
            codes, scales, _ = quantise(x.float().cpu().numpy(), g)
            getattr(self.kv4, n + "_codes")[pg, :, row] = torch.from_numpy(codes).cuda()
            getattr(self.kv4, n + "_scales")[pg, :, row] = torch.from_numpy(scales).cuda()

    def rows(self, r, n):
        """Request r's first n keys and values, [n, Hkv, d] fp64."""
        pg, row = self.slots(r, 0, n)
        if self.bits == 16:
            return self.k_cache[pg, row].double(), self.v_cache[pg, row].double()
        return tuple(values4(getattr(self.kv4, x + "_codes")[pg, :, row],
                             getattr(self.kv4, x + "_scales")[pg, :, row], g)
                     for x, g in (("k", self.kv4.k_scale), ("v", self.kv4.v_scale)))

    # -- calls
    def attend(self, q=None, out=None, stream=None):
        q = self.q if q is None else q
        out = torch.full((self.T, self.Hq, self.d), SENTINEL, device="cuda").bfloat16() if out is None else out
        if self.bits == 16:
            self.h.ddt_prompt_attention(q, self.q_start, self.ctx_lens, self.table, self.R, self.k_cache,
                                        self.v_cache, out, stream=stream)
        else:
            self.h.ddt_prompt_attention_kvq(q, self.q_start, self.ctx_lens, self.table, self.R, self.kv4, out,
                                            stream=stream)
        return out

    def append(self, rotary=None, **kw):
        q_out = kw.pop("q_out", torch.full_like(self.q, SENTINEL))
        q, k, v = kw.pop("q", self.q), kw.pop("k", self.k), kw.pop("v", self.v)
        if self.bits == 16:
            self.h.ddt_append_kv(q, k, v, self.q_start, self.ctx_lens, self.table, self.R, self.k_cache,
                                 self.v_cache, q_out=q_out, rotary=rotary, **kw)
        else:
            self.h.ddt_append_kvq(q, k, v, self.q_start, self.ctx_lens, self.table, self.R, self.kv4,
                                  q_out=q_out, rotary=rotary, **kw)
        return q_out

    # -- what attention has to give
    def attention64(self, q=None):
        """out and the tolerance of every element, [T, Hq, d] fp64; rows of no
        request hold SENTINEL with tolerance 0.

        Tolerance: the result is rounded to bf16 (2^-8 |o|); each probability is
        rounded to bf16 (2^-8 of it), which moves the result by at most 2^-8 A,
        A = sum_j p_j |v_j|; a score s = q.k/sqrt(d) summed in fp32 is off by at
        most e = 2^-22 (d/16) sum |q_i k_i| / sqrt(d) (the products are exact, a
        partial sum of 16 is rounded each time, to two bits less than fp32 has),
        plus 2^-22 |s| for its scaling, which moves p_j by a factor within
        exp(+-2e) through numerator and sum; exp2 and the fp32 sums add 2^-20.
        Over the 4-bit cache a probability is an fp16 number: the weight
        w = 2^7 2^(s - m), with m no more than the row's largest score, is rounded
        to 11 bits or, below 2^-14, to a multiple of 2^-24. The second error is at
        most 2^-25, so 2^-32 of a weight at m, and the sum of weights is at least
        one weight at the row's largest score: it moves the result by at most
        2^-32 sum_j |v_j| over the row's keys."""
        q = self.q if q is None else q
        out = torch.full((self.T, self.Hq, self.d), SENTINEL, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        G = self.Hq // self.Hkv
        for r, (n, c) in enumerate(zip(self.lens, self.ctx)):
            if n == 0:
                continue
            s0 = int(self.starts[r])
            k, v = self.rows(r, c + n)
            qq = q[s0:s0 + n].double().view(n, self.Hkv, G, self.d)
            sc = self.d ** -0.5
            s = torch.einsum("mhgd,nhd->hgmn", qq, k) * sc
            mag = torch.einsum("mhgd,nhd->hgmn", qq.abs(), k.abs()) * sc
            ahead = torch.arange(c + n, device="cuda")[None, :] > torch.arange(c, c + n, device="cuda")[:, None]
            s.masked_fill_(ahead, -float("inf"))
            p = torch.softmax(s, -1)
            e = torch.where(p > 0, mag * (2.0 ** -22 * (self.d // 16 + 1)), 0.0).amax(-1)  # [Hkv, G, n]
            o = torch.einsum("hgmn,nhd->mhgd", p, v)
            A = torch.einsum("hgmn,nhd->mhgd", p, v.abs())
            rel = 2.0 ** -8 + 2.0 ** -20 + 2.01 * e.permute(2, 0, 1)[..., None]
            out[s0:s0 + n] = o.reshape(n, self.Hq, self.d)
            # 1.01: products of two of these errors
            tol[s0:s0 + n] = (1.01 * (2.0 ** -8 * o.abs() + rel * A)).reshape(n, self.Hq, self.d)
            if self.bits == 4:
                seen = torch.einsum("mn,nhd->mhd", (~ahead).double(), v.abs())
                tol[s0:s0 + n] += (1.01 * 2.0 ** -32 * seen).repeat_interleave(self.Hq // self.Hkv, 1)
        return out, tol


def check_close(got, want, tol):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError("%d of %d differ, first at %s: got %r, want %r +- %r" % (
            int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(tol[i])))


# ---------------------------------------------------------------- the append in fp32
def turn(x, pos, table, rot, interleaved):
    """x [T, H, d] fp32 turned by table rows [., rot] of positions pos."""
    x = x.astype(np.float32).copy()
    c, s = table[pos][:, None, :rot // 2], table[pos][:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2].copy(), x[..., 1:rot:2].copy()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2].copy(), x[..., rot // 2:rot].copy()
        x[..., :rot // 2], x[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return x


def e4m3(x):
    """fp32 (at most 448) to e4m3 bits, to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_value(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).float().numpy()


def quantise(x, g):
    """fp32 [..., d] -> codes [..., d/2] u8, scales [..., d/16] u8, values fp32."""
    d = x.shape[-1]
    g = np.float32(g)
    b = x.astype(np.float32).reshape(x.shape[:-1] + (d // 16, 16))
    amax = np.max(np.abs(b), -1)  # NaN if the block has one
    inv6 = np.float32(1) / (np.float32(6) * g)
    sc = e4m3(np.minimum(amax * inv6, np.float32(448)))
    s = (e4m3_value(sc) * g)[..., None]
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        a = np.abs(b / s)  # rounded to nearest
        m = ((a > .25).astype(np.uint8) + (a >= .75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
        m = np.where(s > 0, m, 0).astype(np.uint8)
    val = MAGS[m] * s
    val = np.where(np.signbit(b), -val, val).reshape(x.shape)
    code = (m | (np.signbit(b).astype(np.uint8) << 3)).reshape(x.shape[:-1] + (d // 8, 8))
    byts = np.stack((code[..., 0] | code[..., 2] << 4, code[..., 4] | code[..., 6] << 4,
                     code[..., 1] | code[..., 3] << 4, code[..., 5] | code[..., 7] << 4), -1)
    return byts.reshape(x.shape[:-1] + (d // 2,)).astype(np.uint8), sc, val


def values4(codes, scales, g):
    """Codes [..., d/2] and scales [..., d/16] (CUDA u8) -> values fp64."""
    c = codes.cpu().numpy().reshape(codes.shape[:-1] + (-1, 4))
    ch = np.stack((c[..., 0] & 15, c[..., 2] & 15, c[..., 0] >> 4, c[..., 2] >> 4,
                   c[..., 1] & 15, c[..., 3] & 15, c[..., 1] >> 4, c[..., 3] >> 4), -1)
    v = np.where(ch & 8, -MAGS[ch & 7], MAGS[ch & 7]).astype(np.float64)
    s = e4m3_value(scales.cpu().numpy()).astype(np.float64) * float(np.float32(g))
    v = v.reshape(scales.shape + (16,)) * s[..., None]
    return torch.from_numpy(v.reshape(codes.shape[:-1] + (-1,))).cuda()
