"""Thin ctypes binding over libddt.so (include/ddt.h).

Argument marshalling only: every step of the round runs in the library's
sm_103a kernels. Tensors are torch CUDA tensors (torch supplies device
memory and streams); bf16 tensors may be torch.bfloat16 or int16/uint16
views of the same bits. There is no fallback: if the library is missing or
fails to load, loading raises.
"""
import collections
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libddt.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, ENOMEM = 0, 1, 2, 3, 4
BF16, F32 = 0, 1
DEV_NAN_LOGITS, DEV_BAD_PAGE, DEV_BAD_TREE, DEV_TIMEOUT, DEV_BAD_LENGTH = 0x1, 0x2, 0x4, 0x8, 0x10

EXPORTS = ("ddt_create", "ddt_destroy", "ddt_workspace_bytes", "ddt_topk_logprobs",
           "ddt_build_tree", "ddt_build_tree_conditioned", "ddt_build_mask", "ddt_tree_attention", "ddt_target_argmax",
           "ddt_walk", "ddt_compact", "ddt_accept", "ddt_round", "ddt_round_conditioned",
           "ddt_markov_table", "ddt_build_tree_markov", "ddt_round_markov",
           "ddt_accept_stochastic", "ddt_schedule_prefix", "ddt_append_kv", "ddt_append_kvq",
           "ddt_prompt_attention", "ddt_prompt_attention_kvq", "ddt_device_status", "ddt_strerror",
           "ddt_last_cuda_error", "ddt_debug_arm_attention_timeout", "ddt_debug_arm_prompt_timeout")


class DdtError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib.ddt_strerror(status).decode() if _lib is not None else str(status)
        extra = ""
        if status == ECUDA and _lib is not None:
            extra = " (cudaError %d)" % _lib.ddt_last_cuda_error()
        super().__init__("%s: %s%s" % (where, msg, extra))


class Config(ctypes.Structure):
    _fields_ = [("R_max", ctypes.c_int32), ("L", ctypes.c_int32), ("V", ctypes.c_int32),
                ("B", ctypes.c_int32), ("K", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_req", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("draft_dtype", ctypes.c_int32), ("target_dtype", ctypes.c_int32),
                ("markov_dim", ctypes.c_int32), ("frontier", ctypes.c_int32),
                ("prefilter", ctypes.c_int32)]


_P = ctypes.c_void_p


class RoundArgs(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32)] + [(n, _P) for n in (
        "draft_logits", "target_logits", "q", "k_tree", "v_tree", "k_cache", "v_cache",
        "block_table", "ctx_lens", "top_lp", "top_ids", "tree_tokens", "parents", "depths",
        "n_nodes", "mask", "attn_out", "target_argmax", "acc_len", "acc_nodes", "acc_tokens",
        "bonus", "att_event_begin", "att_event_end")]


class AppendArgs(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("T", ctypes.c_int32), ("q", _P), ("k", _P), ("v", _P),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_start", _P), ("ctx_lens", _P),
                ("block_table", _P), ("cos_sin", _P), ("rotary_dim", ctypes.c_int32),
                ("max_pos", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("q_out", _P),
                ("new_lens", _P)]


class Kv4(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_scales", _P), ("v_scales", _P),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Rotary:
    """The position rotation of an append: a [max_pos, dim] f32 CUDA table of
    dim / 2 cosines and dim / 2 sines per position (rotary_table makes one);
    dim leading channels are turned, in pairs (j, j + dim / 2) or, interleaved,
    (2j, 2j + 1)."""

    def __init__(self, table, dim, interleaved=False):
        if table.dtype != torch.float32 or table.dim() != 2 or table.shape[1] != dim:
            raise ValueError("expected a [max_pos, %d] float32 table" % dim)
        self.table, self.dim, self.interleaved = table, dim, bool(interleaved)


def rotary_table(max_pos, dim, base=10000.0, inv_freq=None, device="cuda"):
    """[max_pos, dim] f32: cos and sin of position * inv_freq[j], j < dim / 2
    (default base ** (-2j / dim)); angles in fp64, since a far position's
    angle has no fraction left in fp32."""
    if inv_freq is None:
        inv_freq = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64).to(device)
    if inv_freq.shape != (dim // 2,):
        raise ValueError("expected %d inverse frequencies" % (dim // 2))
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv_freq
    return torch.cat((ang.cos(), ang.sin()), dim=1).float().contiguous()


class Kv4Cache:
    """A KV cache held in 4 bits (ddt_kv4): uint8 CUDA tensors k_codes, v_codes
    [num_pages, Hkv, page_size, d / 2], k_scales, v_scales [num_pages, Hkv,
    page_size, d / 16] and the two global scales. Context.alloc_kv4 makes one."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales, k_scale=1.0, v_scale=1.0):
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)

    def check(self, cfg):
        p, h, s, d = cfg.num_pages, cfg.Hkv, cfg.page_size, cfg.d
        for t, n in ((self.k_codes, "k_codes"), (self.v_codes, "v_codes")):
            _shaped(t, n, _U8, (p, h, s, d // 2))
        for t, n in ((self.k_scales, "k_scales"), (self.v_scales, "v_scales")):
            _shaped(t, n, _U8, (p, h, s, d // 16))


# what the packed-sequence calls look at, as plain values (a ctypes field is slow to read)
Dims = collections.namedtuple("Dims", "R_max Hq Hkv d page_size max_pages_per_req num_pages")

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)


def _shaped(t, name, dtypes, shape):
    """Raise unless t has one of the types and the shape."""
    if t.dtype not in dtypes:
        raise ValueError("%s: expected %s, got %s" % (name, dtypes[0], t.dtype))
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(t.shape)))


def _rows(t, name, T, heads, d):
    """The token stride of packed rows [T, heads, d], each row dense."""
    _shaped(t, name, _BF16, (T, heads, d))
    if t.is_contiguous():
        return 0
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError("%s: expected each token's heads and channels dense" % name)
    if T <= 1:  # (a single row has no next one)
        return 0
    if t.stride(0) < heads * d:  # (an expanded or unfolded tensor: its rows share memory)
        raise ValueError("%s: expected tokens that do not overlap" % name)
    return t.stride(0)


def check_append(cfg, q, k, v, q_start, ctx_lens, block_table, R, q_out, rotary, new_lens):
    """Types and shapes of an append's tensors; the token strides of q, k, v."""
    T = k.shape[0]
    ks, vs = _rows(k, "k", T, cfg.Hkv, cfg.d), _rows(v, "v", T, cfg.Hkv, cfg.d)
    qs = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        qs = _rows(q, "q", T, cfg.Hq, cfg.d)
        _shaped(q_out, "q_out", _BF16, (T, cfg.Hq, cfg.d))
    check_packed(cfg, q_start, ctx_lens, block_table, R)
    if rotary is not None and (rotary.dim % 32 or not 32 <= rotary.dim <= cfg.d):
        raise ValueError("rotary: expected a multiple of 32 channels up to %d" % cfg.d)
    if new_lens is not None:
        _shaped(new_lens, "new_lens", _I32, (R,))
    return qs, ks, vs


def check_packed(cfg, q_start, ctx_lens, block_table, R):
    if not 0 <= R <= cfg.R_max:
        raise ValueError("R: expected 0..%d" % cfg.R_max)
    _shaped(q_start, "q_start", _I32, (R + 1,))
    _shaped(ctx_lens, "ctx_lens", _I32, (R,))
    _shaped(block_table, "block_table", _I32, (R, cfg.max_pages_per_req))


def check_prompt(cfg, q, q_start, ctx_lens, block_table, R, out):
    """Types and shapes of a prompt attention's tensors; q's token stride."""
    T = q.shape[0]
    qs = _rows(q, "q", T, cfg.Hq, cfg.d)
    _shaped(out, "out", _BF16, (T, cfg.Hq, cfg.d))
    check_packed(cfg, q_start, ctx_lens, block_table, R)
    return qs


def _cache_shapes(cfg, k_cache, v_cache):
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _shaped(t, n, _BF16, (cfg.num_pages, cfg.page_size, cfg.Hkv, cfg.d))


_lib = None


def load(path=LIB_PATH):
    """Load libddt.so and declare its signatures; raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libddt.so not built at %s (run __graft_entry__.build())" % path)
    L = ctypes.CDLL(path)
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "ddt_create": ([ctypes.POINTER(Config), ctypes.POINTER(_P)], i32),
        "ddt_destroy": ([_P], None),
        "ddt_workspace_bytes": ([ctypes.POINTER(Config)], sz),
        "ddt_topk_logprobs": ([_P, _P, i32, _P, _P, _P], i32),
        "ddt_build_tree": ([_P, _P, _P, i32, _P, _P, _P, _P, _P, _P], i32),
        "ddt_build_mask": ([_P, _P, _P, i32, _P, _P], i32),
        "ddt_build_tree_conditioned": ([_P, _P, _P, _P, _P, i32, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P], i32),
        "ddt_tree_attention": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, i32, _P, _P], i32),
        "ddt_target_argmax": ([_P, _P, i32, _P, _P], i32),
        "ddt_walk": ([_P, _P, _P, _P, _P, i32, _P, _P, _P, _P, _P], i32),
        "ddt_compact": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, i32, _P], i32),
        "ddt_accept": ([_P, _P, _P, _P, _P, i32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P],
                       i32),
        "ddt_round": ([_P, ctypes.POINTER(RoundArgs), _P], i32),
        "ddt_round_conditioned": ([_P, ctypes.POINTER(RoundArgs), _P, _P, _P, _P], i32),
        "ddt_markov_table": ([_P, _P, _P, _P, _P, i32, _P, _P, _P], i32),
        "ddt_build_tree_markov": ([_P, _P, _P, i32, _P, _P, _P, _P, _P, _P], i32),
        "ddt_round_markov": ([_P, ctypes.POINTER(RoundArgs), _P, _P, _P, _P], i32),
        "ddt_accept_stochastic": ([_P, _P, _P, _P, _P, _P, i32, _P, _P, _P, _P], i32),
        "ddt_schedule_prefix": ([_P, _P, i32, _P, _P, _P, _P, _P], i32),
        "ddt_append_kv": ([_P, ctypes.POINTER(AppendArgs), _P, _P, _P], i32),
        "ddt_append_kvq": ([_P, ctypes.POINTER(AppendArgs), ctypes.POINTER(Kv4), _P, _P, _P], i32),
        "ddt_prompt_attention": ([_P, _P, i64, _P, _P, i32, i32, _P, _P, _P, _P, _P], i32),
        "ddt_prompt_attention_kvq": ([_P, _P, i64, _P, _P, i32, i32, ctypes.POINTER(Kv4), _P, _P,
                                      _P], i32),
        "ddt_device_status": ([_P, ctypes.POINTER(i32)], i32),
        "ddt_debug_arm_attention_timeout": ([_P, i64], i32),
        "ddt_debug_arm_prompt_timeout": ([_P, i64], i32),
        "ddt_strerror": ([i32], ctypes.c_char_p),
        "ddt_last_cuda_error": ([], i32),
    }
    for name, (argt, rest) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = argt
        fn.restype = rest
    _lib = L
    return L


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status, where):
    if status != OK:
        raise DdtError(status, where)


def make_config(R_max, L, V, B, Hq, Hkv, d, page_size, max_pages_per_req, num_pages, K=0,
                draft_dtype=BF16, target_dtype=BF16, markov_dim=0, frontier=0, prefilter=0):
    return Config(R_max, L, V, B, K, Hq, Hkv, d, page_size, max_pages_per_req, num_pages,
                  draft_dtype, target_dtype, markov_dim, frontier, prefilter)


def workspace_bytes(cfg):
    return int(load().ddt_workspace_bytes(ctypes.byref(cfg)))


class Context:
    """One ddt_ctx (and its device workspace) on the current CUDA device."""

    def __init__(self, cfg):
        lib = load()
        self.cfg = cfg
        h = _P()
        _check(lib.ddt_create(ctypes.byref(cfg), ctypes.byref(h)), "ddt_create")
        self._h = h
        self.device = torch.cuda.current_device()
        self.dims = Dims(cfg.R_max, cfg.Hq, cfg.Hkv, cfg.d, cfg.page_size, cfg.max_pages_per_req,
                         cfg.num_pages)
        self.K = cfg.K if cfg.K else min(cfg.B, cfg.V)
        self.P = cfg.B + 1
        self.W = (self.P + 31) // 32

    def close(self):
        if getattr(self, "_h", None):
            _lib.ddt_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- one call per C entry point -----------------------------------------
    def ddt_topk_logprobs(self, draft_logits, R, top_lp, top_ids, stream=None):
        _check(_lib.ddt_topk_logprobs(self._h, _ptr(draft_logits), R, _ptr(top_lp), _ptr(top_ids),
                                      _stream(stream)), "ddt_topk_logprobs")

    def ddt_build_tree(self, top_lp, top_ids, R, tree_tokens, parents, depths, n_nodes, mask=None,
                       stream=None):
        _check(_lib.ddt_build_tree(self._h, _ptr(top_lp), _ptr(top_ids), R, _ptr(tree_tokens),
                                   _ptr(parents), _ptr(depths), _ptr(n_nodes), _ptr(mask),
                                   _stream(stream)), "ddt_build_tree")

    def ddt_build_tree_conditioned(self, draft_logits, W, E, anchors, R, tree_tokens, parents,
                                   depths, n_nodes, mask=None, cand_lp=None, cand_ids=None,
                                   frontier_tok=None, stream=None):
        _check(_lib.ddt_build_tree_conditioned(
            self._h, _ptr(draft_logits), _ptr(W), _ptr(E), _ptr(anchors), R, _ptr(cand_lp),
            _ptr(cand_ids), _ptr(frontier_tok), _ptr(tree_tokens), _ptr(parents), _ptr(depths),
            _ptr(n_nodes), _ptr(mask), _stream(stream)), "ddt_build_tree_conditioned")

    def ddt_build_mask(self, parents, n_nodes, R, mask, stream=None):
        _check(_lib.ddt_build_mask(self._h, _ptr(parents), _ptr(n_nodes), R, _ptr(mask),
                                   _stream(stream)), "ddt_build_mask")

    def ddt_tree_attention(self, q, k_tree, v_tree, k_cache, v_cache, block_table, ctx_lens, mask,
                           R, out, stream=None):
        _check(_lib.ddt_tree_attention(self._h, _ptr(q), _ptr(k_tree), _ptr(v_tree), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), _ptr(mask),
                                       R, _ptr(out), _stream(stream)), "ddt_tree_attention")

    def ddt_target_argmax(self, target_logits, R, argmax_out, stream=None):
        _check(_lib.ddt_target_argmax(self._h, _ptr(target_logits), R, _ptr(argmax_out),
                                      _stream(stream)), "ddt_target_argmax")

    def ddt_walk(self, argmax, tree_tokens, parents, n_nodes, R, acc_len, acc_nodes, acc_tokens,
                 bonus, stream=None):
        _check(_lib.ddt_walk(self._h, _ptr(argmax), _ptr(tree_tokens), _ptr(parents),
                             _ptr(n_nodes), R, _ptr(acc_len), _ptr(acc_nodes), _ptr(acc_tokens),
                             _ptr(bonus), _stream(stream)), "ddt_walk")

    def ddt_compact(self, k_cache, v_cache, block_table, ctx_lens, k_tree, v_tree, acc_nodes,
                    acc_len, R, stream=None):
        _check(_lib.ddt_compact(self._h, _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                _ptr(ctx_lens), _ptr(k_tree), _ptr(v_tree), _ptr(acc_nodes),
                                _ptr(acc_len), R, _stream(stream)), "ddt_compact")

    def ddt_accept(self, target_logits, tree_tokens, parents, n_nodes, R, argmax_out, acc_len,
                   acc_nodes, acc_tokens, bonus, k_cache, v_cache, block_table, k_tree, v_tree,
                   ctx_lens, stream=None):
        _check(_lib.ddt_accept(self._h, _ptr(target_logits), _ptr(tree_tokens), _ptr(parents),
                               _ptr(n_nodes), R, _ptr(argmax_out), _ptr(acc_len), _ptr(acc_nodes),
                               _ptr(acc_tokens), _ptr(bonus), _ptr(k_cache), _ptr(v_cache),
                               _ptr(block_table), _ptr(k_tree), _ptr(v_tree), _ptr(ctx_lens),
                               _stream(stream)), "ddt_accept")

    def ddt_accept_stochastic(self, draft_logits, target_logits, draft_tokens, u, r, R, acc_len,
                              acc_tokens, n_guess=None, stream=None):
        """Temperature-1 verification of R drafted chains of L guesses.
        n_guess: None (every guess), or an int32 [R] CUDA tensor of the
        guesses each request verifies, e.g. ddt_schedule_prefix's n_keep."""
        _check(_lib.ddt_accept_stochastic(self._h, _ptr(draft_logits), _ptr(target_logits),
                                          _ptr(draft_tokens), _ptr(u), _ptr(r), R, _ptr(acc_len),
                                          _ptr(acc_tokens), _ptr(n_guess), _stream(stream)),
               "ddt_accept_stochastic")

    def ddt_schedule_prefix(self, conf, R, cost_ms, n_keep, n_total=None, stats=None,
                            stream=None):
        """The guesses each of R requests verifies: conf [R, L] f32,
        cost_ms [R*L + 1] f32, n_keep [R] i32 out; n_total [1] i32 and
        stats [2] f64 (tokens per ms, expected tokens) optional."""
        _check(_lib.ddt_schedule_prefix(self._h, _ptr(conf), R, _ptr(cost_ms), _ptr(n_keep),
                                        _ptr(n_total), _ptr(stats), _stream(stream)),
               "ddt_schedule_prefix")

    # -- packed sequences over the paged cache --------------------------------
    # (a decoding step makes these calls once a layer: their checks are kept short)
    def _at(self, t, dense=True):
        """Device address of a tensor on this context's device (None: NULL)."""
        if t is None:
            return None
        if t.get_device() != self.device:
            raise ValueError("expected a tensor on CUDA device %d" % self.device)
        if dense and not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return t.data_ptr()

    def _own_stream(self, stream):
        """The given stream, or the current one of this context's device."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream

    def _kv4(self, cache):
        cache.check(self.dims)
        at = self._at
        return Kv4(at(cache.k_codes), at(cache.v_codes), at(cache.k_scales), at(cache.v_scales),
                   cache.k_scale, cache.v_scale)

    def _append_args(self, q, k, v, q_start, ctx_lens, block_table, R, q_out, rotary, new_lens):
        qs, ks, vs = check_append(self.dims, q, k, v, q_start, ctx_lens, block_table, R, q_out,
                                  rotary, new_lens)
        at = self._at
        table, dim, rows, inter = None, 0, 0, 0
        if rotary is not None:
            table, dim, rows = at(rotary.table), rotary.dim, rotary.table.shape[0]
            inter = int(rotary.interleaved)
        return AppendArgs(R, k.shape[0], at(q, False), at(k, False), at(v, False), qs, ks, vs,
                          at(q_start), at(ctx_lens), at(block_table), table, dim, rows, inter,
                          at(q_out), at(new_lens))

    def ddt_append_kv(self, q, k, v, q_start, ctx_lens, block_table, R, k_cache, v_cache,
                      q_out=None, rotary=None, new_lens=None, stream=None):
        """Append R requests' packed new tokens to the paged cache: k, v
        [T, Hkv, d] (and q [T, Hq, d] to q_out) bf16, turned by `rotary` (a
        Rotary, or None). q, k and v may be views of one projection's rows;
        q_out may be q itself when q is dense. new_lens [R] i32 (optional):
        the lengths after the append; ctx_lens stays as it is."""
        a = self._append_args(q, k, v, q_start, ctx_lens, block_table, R, q_out, rotary, new_lens)
        _cache_shapes(self.dims, k_cache, v_cache)
        _check(_lib.ddt_append_kv(self._h, ctypes.byref(a), self._at(k_cache), self._at(v_cache),
                                  self._own_stream(stream)), "ddt_append_kv")

    def ddt_append_kvq(self, q, k, v, q_start, ctx_lens, block_table, R, cache, q_out=None,
                       rotary=None, new_lens=None, k_held=None, v_held=None, stream=None):
        """The same into a Kv4Cache; k_held, v_held [T, Hkv, d] bf16 (optional):
        the values that the cache now holds for the new tokens."""
        a = self._append_args(q, k, v, q_start, ctx_lens, block_table, R, q_out, rotary, new_lens)
        for t, n in ((k_held, "k_held"), (v_held, "v_held")):
            if t is not None:
                _shaped(t, n, _BF16, (k.shape[0], self.dims.Hkv, self.dims.d))
        c = self._kv4(cache)
        _check(_lib.ddt_append_kvq(self._h, ctypes.byref(a), ctypes.byref(c), self._at(k_held),
                                   self._at(v_held), self._own_stream(stream)), "ddt_append_kvq")

    def ddt_prompt_attention(self, q, q_start, ctx_lens, block_table, R, k_cache, v_cache, out,
                             stream=None):
        """Causal attention of R requests' packed queries q [T, Hq, d] bf16 over
        the paged cache that holds their keys and values (ctx_lens [R]: the
        lengths before these tokens) into out [T, Hq, d] bf16."""
        qs = check_prompt(self.dims, q, q_start, ctx_lens, block_table, R, out)
        _cache_shapes(self.dims, k_cache, v_cache)
        at = self._at
        _check(_lib.ddt_prompt_attention(self._h, at(q, False), qs, at(q_start), at(ctx_lens), R,
                                         q.shape[0], at(k_cache), at(v_cache), at(block_table),
                                         at(out), self._own_stream(stream)), "ddt_prompt_attention")

    def ddt_prompt_attention_kvq(self, q, q_start, ctx_lens, block_table, R, cache, out,
                                 stream=None):
        """The same over a Kv4Cache."""
        qs = check_prompt(self.dims, q, q_start, ctx_lens, block_table, R, out)
        c = self._kv4(cache)
        at = self._at
        _check(_lib.ddt_prompt_attention_kvq(self._h, at(q, False), qs, at(q_start), at(ctx_lens), R,
                                             q.shape[0], ctypes.byref(c), at(block_table), at(out),
                                             self._own_stream(stream)), "ddt_prompt_attention_kvq")

    def alloc_kv4(self, k_scale=1.0, v_scale=1.0, device="cuda"):
        """An empty (all zero) Kv4Cache of this context's page pool."""
        c = self.cfg
        t = [torch.zeros((c.num_pages, c.Hkv, c.page_size, n), dtype=torch.uint8, device=device)
             for n in (c.d // 2, c.d // 2, c.d // 16, c.d // 16)]
        return Kv4Cache(*t, k_scale=k_scale, v_scale=v_scale)

    def ddt_round(self, R, bufs, stream=None, att_events=None):
        """bufs: dict of tensors named like the fields of ddt_round_args.
        att_events: optional (begin, end) torch.cuda.Event pair, recorded by
        the library around the attention launch (each already created, e.g.
        by one earlier record())."""
        a = self._round_args(R, bufs, att_events)
        _check(_lib.ddt_round(self._h, ctypes.byref(a), _stream(stream)), "ddt_round")

    def ddt_markov_table(self, draft_logits, W, E, anchors, R, cand_ids, tab_lp, stream=None):
        _check(_lib.ddt_markov_table(self._h, _ptr(draft_logits), _ptr(W), _ptr(E), _ptr(anchors),
                                     R, _ptr(cand_ids), _ptr(tab_lp), _stream(stream)),
               "ddt_markov_table")

    def ddt_build_tree_markov(self, cand_ids, tab_lp, R, tree_tokens, parents, depths, n_nodes,
                              mask=None, stream=None):
        _check(_lib.ddt_build_tree_markov(self._h, _ptr(cand_ids), _ptr(tab_lp), R,
                                          _ptr(tree_tokens), _ptr(parents), _ptr(depths),
                                          _ptr(n_nodes), _ptr(mask), _stream(stream)),
               "ddt_build_tree_markov")

    def ddt_round_markov(self, R, bufs, W, E, anchors, stream=None, att_events=None):
        """The SparklingTree round: bufs as for ddt_round (top_lp / top_ids
        unused), W, E [V, H] bf16 and anchors [R] int32."""
        a = self._round_args(R, bufs, att_events)
        _check(_lib.ddt_round_markov(self._h, ctypes.byref(a), _ptr(W), _ptr(E), _ptr(anchors),
                                     _stream(stream)), "ddt_round_markov")

    def _round_args(self, R, bufs, att_events):
        """ddt_round_args from a dict of tensors named like its fields (absent
        ones are NULL) and the optional attention event pair."""
        a = RoundArgs()
        a.R = R
        for name, _ in RoundArgs._fields_[1:]:
            if name.startswith("att_event"):
                continue
            setattr(a, name, _ptr(bufs.get(name)))
        if att_events is not None:
            a.att_event_begin = ctypes.c_void_p(att_events[0].cuda_event)
            a.att_event_end = ctypes.c_void_p(att_events[1].cuda_event)
        return a

    def ddt_round_conditioned(self, R, bufs, W, E, anchors, stream=None, att_events=None):
        """The parent-conditioned round: bufs as for ddt_round (draft_logits are
        the backbone's per-depth logits; top_lp / top_ids unused), W, E [V, H]
        bf16 and anchors [R] int32."""
        a = self._round_args(R, bufs, att_events)
        _check(_lib.ddt_round_conditioned(self._h, ctypes.byref(a), _ptr(W), _ptr(E), _ptr(anchors),
                                          _stream(stream)), "ddt_round_conditioned")

    def ddt_device_status(self):
        out = ctypes.c_int32(0)
        _check(_lib.ddt_device_status(self._h, ctypes.byref(out)), "ddt_device_status")
        return out.value

    def ddt_debug_arm_attention_timeout(self, wait_cycles):
        """Test only: the next a4 launch starts with a bounded wait that runs
        out after wait_cycles SM cycles (see include/ddt.h)."""
        _check(_lib.ddt_debug_arm_attention_timeout(self._h, int(wait_cycles)),
               "ddt_debug_arm_attention_timeout")

    def ddt_debug_arm_prompt_timeout(self, wait_cycles):
        """Test only: the next tensor-core prompt attention starts with a bounded
        wait that runs out after wait_cycles SM cycles (see include/ddt.h)."""
        _check(_lib.ddt_debug_arm_prompt_timeout(self._h, int(wait_cycles)), "ddt_debug_arm_prompt_timeout")

    # -- allocation helper (plumbing) ----------------------------------------
    def alloc_outputs(self, R, device="cuda"):
        """Output buffers of one round for R requests, named as in ddt_round_args."""
        c, K, P, W = self.cfg, self.K, self.P, self.W
        i32 = dict(dtype=torch.int32, device=device)
        return dict(
            top_lp=torch.empty((R, c.L, K), dtype=torch.float32, device=device),
            top_ids=torch.empty((R, c.L, K), **i32),
            tree_tokens=torch.empty((R, c.B), **i32),
            parents=torch.empty((R, P), **i32),
            depths=torch.empty((R, P), **i32),
            n_nodes=torch.empty((R,), **i32),
            mask=torch.empty((R, P, W), **i32),
            attn_out=torch.empty((R, P, c.Hq, c.d), dtype=torch.float32, device=device),
            target_argmax=torch.empty((R, P), **i32),
            acc_len=torch.empty((R,), **i32),
            acc_nodes=torch.empty((R, c.L), **i32),
            acc_tokens=torch.empty((R, c.L + 1), **i32),
            bonus=torch.empty((R,), **i32),
        )
