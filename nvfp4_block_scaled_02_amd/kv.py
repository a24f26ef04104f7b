"""Torch-facing wrappers over the key/value-cache calls of libnvfp4.so
(include/nvfp4.h): planning a step's pages, the norm and rotation of query and
key heads, writing and reading the paged NVFP4 cache, attention over it.

Argument marshalling only, as in api.py: every tensor is checked against the
extent the kernels index, every call goes to the current stream of its
device, and ``prepare(fn, ...)`` turns any of them into a ``Launch``.
Projections (q, k, v, their gradients) may be views: their heads must be
dense, their tokens may be any multiple of 4 values apart (8 for
``kv_attention``).
"""
import ctypes
import threading
from dataclasses import dataclass, field
from typing import Optional

import torch

from . import _native as N
from .api import _invoke, _need, _preparing, _SELECT, _stream, default_global_max

_PAIRS = {"halves": N.PAIRS_HALVES, "neighbours": N.PAIRS_NEIGHBOURS}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _check(t, dtype, name, numel=None):
    """_need, with its answer first where nothing is wrong (these calls are
    made every token: the checks' own time counts)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous()
            and (numel is None or t.numel() == numel)):
        _need(t, dtype, name, numel)


def _heads(x, name, tokens=None, heads=None, dim=None, granule=4):
    """[tokens, heads, D] bf16 on a GPU with dense heads: (tokens, heads, D,
    elements from token to token)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must live on a GPU device, got {x.device}")
    if x.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {x.dtype}")
    if x.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head_dim]")
    t, h, d = x.shape
    if (tokens is not None and t != tokens) or (heads is not None and h != heads) or \
            (dim is not None and d != dim):
        raise ValueError(f"{name} must be [{tokens}, {heads if heads is not None else 'heads'}, "
                         f"{dim if dim is not None else 'head_dim'}], got {tuple(x.shape)}")
    st, sh, sd = x.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"the heads of {name} must be dense (strides {x.stride()})")
    if t <= 1:
        st = h * d
    elif st < h * d or st % granule:
        raise ValueError(f"the tokens of {name} must be a multiple of {granule} values and at "
                         f"least a token apart (strides {x.stride()})")
    if x.data_ptr() % (2 * granule):
        raise ValueError(f"{name} must be {2 * granule}-byte aligned")
    return t, h, d, st


# ---------------------------------------------------------------- cache
@dataclass(frozen=True, eq=False)
class KVCache:
    """The paged NVFP4 cache of one layer: k_codes [P, H, S, D/2], k_scales
    [P, H, S, D/16], v_codes [P, H, S/8, D/2, 8], v_scales [P, H, S/8, D/16, 8]
    (uint8), the calibrated outer amaxes k_amax and v_amax [H] (float32) and
    S_g.  Slot page * S + i is token i of a page.  The tensors' addresses are
    taken once: a cache with other ones is another KVCache."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_amax: torch.Tensor
    v_amax: torch.Tensor
    global_max: float
    num_pages: int = field(init=False)
    kv_heads: int = field(init=False)
    page_size: int = field(init=False)
    head_dim: int = field(init=False)

    def __post_init__(self):
        _need(self.k_codes, torch.uint8, "k_codes")
        if self.k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page_size, head_dim / 2]")
        p, h, s, half = self.k_codes.shape
        d = 2 * half
        if d % 16:
            raise ValueError(f"head_dim must be a multiple of 16, got {d}")
        _need(self.k_scales, torch.uint8, "k_scales", p * h * s * (d // 16))
        _need(self.v_codes, torch.uint8, "v_codes", p * h * s * half)
        _need(self.v_scales, torch.uint8, "v_scales", p * h * s * (d // 16))
        _need(self.k_amax, torch.float32, "k_amax", h)
        _need(self.v_amax, torch.float32, "v_amax", h)
        sg = float(self.global_max)
        args = N.KVCacheArgs(
            k_codes=_ptr(self.k_codes), k_scales=_ptr(self.k_scales), v_codes=_ptr(self.v_codes),
            v_scales=_ptr(self.v_scales), k_amax=_ptr(self.k_amax), v_amax=_ptr(self.v_amax),
            num_pages=p, kv_heads=h, page_size=s, head_dim=d, global_fp8_max=sg)
        for name, value in (("num_pages", p), ("kv_heads", h), ("page_size", s), ("head_dim", d),
                            ("global_max", sg), ("_args", args)):
            object.__setattr__(self, name, value)

    @property
    def device(self):
        return self.k_codes.device


def kv_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, k_amax: torch.Tensor,
             v_amax: torch.Tensor, *, global_max: float = 0.0, select: str = "4over6") -> KVCache:
    """A new cache on the device of k_amax.  global_max 0: the default of the
    selection rule it will be written with."""
    dev = k_amax.device
    z = lambda *n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
    return KVCache(z(num_pages, kv_heads, page_size, head_dim // 2),
                   z(num_pages, kv_heads, page_size, head_dim // 16),
                   z(num_pages, kv_heads, page_size // 8, head_dim // 2, 8),
                   z(num_pages, kv_heads, page_size // 8, head_dim // 16, 8), k_amax, v_amax,
                   float(global_max) or default_global_max("e4m3", select))


# ---------------------------------------------------------------- plan
@dataclass
class KVPlan:
    """What kv_plan returns: see nvfp4_kv_plan of include/nvfp4.h."""
    cu_new: torch.Tensor
    seq_lens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    free_count: torch.Tensor
    refused: torch.Tensor


def _span(t):
    """Addresses [first, last) of a contiguous tensor."""
    at = t.data_ptr()
    return at, at + t.numel() * t.element_size()


def kv_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
            free_pages: torch.Tensor, free_count: torch.Tensor, *, page_size: int, num_pages: int,
            tokens: int, out: Optional[KVPlan] = None) -> KVPlan:
    """The pages, slots and positions of a step's new tokens from the
    requests' lengths; the new pages are written into block_table [batch,
    width] (int32).  free_pages [num_pages] and free_count [1] (int32) are the
    stack of free pages; the result's free_count is the count after the step.
    tokens: at least the sum of new_lens (the rest is padding; a request that
    does not fit into it is refused).  out: a KVPlan to write, which shares
    no memory with the inputs."""
    _check(ctx_lens, _I32, "ctx_lens")
    batch = ctx_lens.numel()
    _check(new_lens, _I32, "new_lens", batch)
    _check(block_table, _I32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, width], got {tuple(block_table.shape)}")
    _check(free_pages, _I32, "free_pages", num_pages)
    _check(free_count, _I32, "free_count", 1)
    dev = ctx_lens.device
    if out is None:
        # one allocation: the 32-bit outputs one after another
        words = ctx_lens.new_empty(2 * batch + tokens + 3)
        cu, lens, pos, count, refused = words.split((batch + 1, batch, tokens, 1, 1))
        out = KVPlan(cu, lens, pos, ctx_lens.new_empty(tokens, dtype=_I64), count, refused)
    else:
        _check(out.cu_new, _I32, "cu_new", batch + 1)
        _check(out.seq_lens, _I32, "seq_lens", batch)
        _check(out.positions, _I32, "positions", tokens)
        _check(out.slots, _I64, "slots", tokens)
        _check(out.free_count, _I32, "free_count", 1)
        _check(out.refused, _I32, "refused", 1)
        inputs = dict(ctx_lens=ctx_lens, new_lens=new_lens, block_table=block_table,
                      free_pages=free_pages, free_count=free_count)
        for name in ("cu_new", "seq_lens", "positions", "slots", "free_count", "refused"):
            a, b = _span(getattr(out, name))
            for of, t in inputs.items():
                c, d = _span(t)
                if a < d and c < b:
                    raise ValueError(f"out.{name} and {of} share memory: the call reads its "
                                     "inputs while it writes its outputs")
    args = N.KVPlanArgs(
        ctx_lens.data_ptr(), new_lens.data_ptr(), batch, block_table.data_ptr(),
        block_table.shape[1], free_pages.data_ptr(), free_count.data_ptr(), num_pages, page_size,
        tokens, out.cu_new.data_ptr(), out.seq_lens.data_ptr(), out.positions.data_ptr(),
        out.slots.data_ptr(), out.free_count.data_ptr(), out.refused.data_ptr())
    _invoke("nvfp4_kv_plan", (ctypes.byref(args),), dev,
            (ctx_lens, new_lens, block_table, free_pages, free_count, out, args))
    return out


# ---------------------------------------------------------------- norm and rotation
def rope_table(positions: int, rot_dim: int, *, base: float = 10000.0, device="cuda"):
    """(cos, sin) float32 [positions, rot_dim / 2] of position * base^(-2j /
    rot_dim), the angles in 64 bits."""
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _side(x, w, n, t, d):
    """(pointer, tokens, heads, D, stride, weight pointer) of queries or keys."""
    if x is None:
        if w is not None:
            raise ValueError(f"{n}_weight without {n}")
        return 0, t, 0, d, 0, 0
    t, h, d, st = _heads(x, n, t, None, d)
    if w is not None:
        _check(w, _BF16, n + "_weight", d)
        return x.data_ptr(), t, h, d, st, w.data_ptr()
    return x.data_ptr(), t, h, d, st, 0


def _out_of(x, given, n):
    """Output of side n like x, given or new and dense: (tensor, pointer, stride)."""
    if x is None:
        return None, 0, 0
    if given is None:
        given = x.new_empty(x.shape)
        return given, given.data_ptr(), x.shape[1] * x.shape[2]
    return given, given.data_ptr(), _heads(given, n + "_out", *x.shape)[3]


def _qk(q, k, positions, cos, sin, q_weight, k_weight, eps, pairs, q_out, k_out, want_k=True):
    """nvfp4_qk_args and its outputs; q or k may be None."""
    if q is None and k is None:
        raise ValueError("pass q, k or both")
    pr = _choice(_PAIRS, pairs, "pairs")
    qp, t, hq, d, qs, qw = _side(q, q_weight, "q", None, None)
    kp, t, hk, d, ks, kw = _side(k, k_weight, "k", t, d)
    pp = cp = sp = top = rot = 0
    if cos is not None and sin is not None and positions is not None:
        _check(cos, _F32, "cos")
        if cos.dim() != 2 or cos.shape[1] * 2 > d:
            raise ValueError(f"cos must be [positions, rot_dim / 2] with rot_dim <= {d}, "
                             f"got {tuple(cos.shape)}")
        _check(sin, _F32, "sin", cos.numel())
        _check(positions, _I32, "positions", t)
        pp, cp, sp = positions.data_ptr(), cos.data_ptr(), sin.data_ptr()
        top, rot = cos.shape
        rot *= 2
    elif not (cos is None and sin is None and positions is None):
        raise ValueError("pass positions, cos and sin, or none of them")
    qo, qop, qos = _out_of(q, q_out, "q")
    ko, kop, kos = _out_of(k, k_out, "k") if want_k else (None, 0, 0)
    return N.QKArgs(qp, kp, t, hq, hk, d, qs, ks, pp, cp, sp, top, rot, pr, qw, kw, eps, qop, kop,
                    qos, kos), qo, ko


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                 sin: Optional[torch.Tensor] = None, *, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, pairs: str = "halves",
                 out: Optional[tuple] = None):
    """RMS norm of every head of q and k [tokens, heads, D] (where it has a
    weight [D]) and rotation of its first 2 * cos.shape[1] values by the
    angles of positions [tokens] (int32): (q_out, k_out).  out: (q_out,
    k_out), which may be q and k."""
    qo, ko = out if out is not None else (None, None)
    a, qo, ko = _qk(q, k, positions, cos, sin, q_weight, k_weight, eps, pairs, qo, ko)
    _invoke("nvfp4_qk_norm_rope", (ctypes.byref(a),), (q if q is not None else k).device,
            (q, k, positions, cos, sin, q_weight, k_weight, qo, ko, a))
    return qo, ko


_BWD_WORKSPACES = {}


def _capturing():
    return torch.cuda.is_current_stream_capturing()


def _place(dev):
    """Whose workspaces a call uses: those of its (device, stream); None where
    it gets new ones: under graph capture (the graph's) and inside prepare()
    (the Launch's, which may run on any stream, beside any other call)."""
    return None if _preparing() or _capturing() else (dev.index, _stream(dev))


def _cached_workspace(table, key, dev, nbytes, zeroed):
    """A workspace of at least nbytes whose first `zeroed` bytes were zero
    before its first use: one per place, made larger when needed; a new one
    each call without a place."""
    if nbytes == 0:
        return None
    ws = table.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws[:zeroed].zero_()
        if key is not None:
            table[key] = ws
    return ws


def qk_norm_rope_bwd(dq_out: Optional[torch.Tensor], dk_out: Optional[torch.Tensor],
                     q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                     positions: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                     sin: Optional[torch.Tensor] = None, *,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     pairs: str = "halves", out: Optional[dict] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Gradient of qk_norm_rope at (q, k) for the gradients dq_out and dk_out
    of its results: (dq, dk, dq_weight, dk_weight), the last two float32 [D]
    or None.  out: optional {"dq", "dk", "dq_weight", "dk_weight"}.
    workspace: a uint8 tensor of the size the library asks for, zeroed before
    its first use; without one a call uses its stream's, a prepared Launch its
    own (for runs that do not overlap)."""
    out = out or {}
    a, dq, dk = _qk(q, k, positions, cos, sin, q_weight, k_weight, eps, pairs, out.get("dq"),
                    out.get("dk"))
    dev = (q if q is not None else k).device
    strides, dws = [], []
    for n, x, g, w in (("q", q, dq_out, q_weight), ("k", k, dk_out, k_weight)):
        if (x is None) != (g is None):
            raise ValueError(f"pass {n} and d{n}_out, or neither")
        strides.append(_heads(g, f"d{n}_out", *x.shape)[3] if g is not None else 0)
        dw = None
        if w is not None:
            dw = out.get(f"d{n}_weight")
            if dw is None:
                dw = w.new_empty(a.head_dim, dtype=_F32)
            else:
                _check(dw, _F32, f"d{n}_weight", a.head_dim)
        dws.append(dw)
    ws = None
    if q_weight is not None or k_weight is not None:
        n = N.lib().nvfp4_qk_norm_rope_bwd_workspace_bytes(a.head_dim)
        if workspace is not None:
            _need(workspace, torch.uint8, "workspace", n)
            ws = workspace
        else:
            ws = _cached_workspace(_BWD_WORKSPACES, _place(dev), dev, n, n)
    _invoke("nvfp4_qk_norm_rope_bwd",
            (ctypes.byref(a), _ptr(dq_out), strides[0], _ptr(dk_out), strides[1], _ptr(dws[0]),
             _ptr(dws[1]), _ptr(ws)), dev,
            (q, k, positions, cos, sin, q_weight, k_weight, dq_out, dk_out, dq, dk, dws, ws, a))
    return dq, dk, dws[0], dws[1]


# ---------------------------------------------------------------- write and read
def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
              q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
              eps: float = 1e-6, pairs: str = "halves", select: str = "4over6",
              q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Quantizes k (after its norm and rotation, as qk_norm_rope) and v
    [tokens, kv_heads, D] into the cache at slots [tokens] (int64; a slot
    outside the cache is skipped), and returns q after its norm and rotation
    (None without q).  select: "6" or "4over6"."""
    a, qo, _ = _qk(q, k, positions, cos, sin, q_weight, k_weight, eps, pairs, q_out, None, False)
    t = a.tokens
    if a.k_heads != cache.kv_heads or a.head_dim != cache.head_dim:
        raise ValueError(f"k must be [tokens, {cache.kv_heads}, {cache.head_dim}], got {tuple(k.shape)}")
    st = _heads(v, "v", t, cache.kv_heads, cache.head_dim)[3]
    _check(slots, _I64, "slots", t)
    args = N.KVAppendArgs(a, v.data_ptr(), st, slots.data_ptr(), cache._args,
                          _choice(_SELECT, select, "select"))
    _invoke("nvfp4_kv_append", (ctypes.byref(args),), k.device,
            (cache, q, k, v, slots, positions, cos, sin, q_weight, k_weight, qo, args))
    return qo


def kv_read(cache: KVCache, slots: torch.Tensor, *, out: Optional[tuple] = None):
    """(k, v) bf16 [tokens, kv_heads, D]: what the cache holds at slots
    (int64); 0 for a slot outside the cache."""
    _check(slots, _I64, "slots")
    n = slots.numel()
    h, d = cache.kv_heads, cache.head_dim
    if out is None:
        out = tuple(slots.new_empty((2, n, h, d), dtype=_BF16).unbind(0))
    else:
        for o, name in zip(out, ("k_out", "v_out")):
            _check(o, _BF16, name, n * h * d)
    _invoke("nvfp4_kv_read", (ctypes.byref(cache._args), _ptr(slots), n, _ptr(out[0]), _ptr(out[1])),
            slots.device, (cache, slots, out))
    return out


# ---------------------------------------------------------------- attention
_ATTENTION_WORKSPACES, _COUNTERS = {}, {}
KV_COUNTER_BYTES = N.KV_COUNTER_BYTES
# An attention call may be two launches with one workspace between them, and
# the library call lets other threads run: none may issue its own in between
# on the same stream, and so with the same workspace.
_ISSUE = threading.RLock()


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, cu_q: Optional[torch.Tensor] = None, *,
                 max_seq_len: Optional[int] = None, scale: Optional[float] = None,
                 causal: bool = True, window: int = 0, want_lse: bool = False,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 counters: Optional[torch.Tensor] = None):
    """Attention of q [tokens, q_heads, D] over the cache: request b's queries
    are rows cu_q[b] .. cu_q[b+1] (int32; None: one each) and the last of its
    seq_lens[b] tokens (int32), whose pages block_table [batch, width] (int32)
    names.  max_seq_len: an upper bound of seq_lens (default: the table's
    width); scale: default D^-1/2; window: attend the last `window` tokens only
    (0: all).  Returns out [tokens, q_heads, D] bf16, or (out, lse) with
    want_lse.  workspace: a uint8 tensor of at least the size the library asks
    for (a stream's own grows to the largest asked for and is kept).  counters: a uint8 tensor of KV_COUNTER_BYTES zeros, which every call
    leaves zero; with it few pieces of a split sequence are joined in the same
    launch.  Without them a call uses its stream's (a prepared Launch its own,
    for runs that do not overlap), and under graph capture a new workspace and
    no counters (a graph that is to have them brings its own)."""
    t, h, d, st = _heads(q, "q", None, None, cache.head_dim, 8)
    _check(seq_lens, _I32, "seq_lens")
    batch = seq_lens.numel()
    _check(block_table, _I32, "block_table")
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be [{batch}, width], got {tuple(block_table.shape)}")
    if cu_q is not None:
        _check(cu_q, _I32, "cu_q", batch + 1)
    elif t != batch:
        raise ValueError(f"without cu_q every request has one query: {t} rows, {batch} requests")
    dev = q.device
    if out is None:
        out = q.new_empty((t, h, d))
    else:
        _check(out, _BF16, "out", t * h * d)
    if lse is None and want_lse:
        lse = torch.empty((t, h), dtype=_F32, device=dev)
    elif lse is not None:
        _check(lse, _F32, "lse", t * h)
    width = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = width * cache.page_size
    args = N.KVAttentionArgs(q.data_ptr(), t, st, h, cache._args, block_table.data_ptr(), batch,
                             width, seq_lens.data_ptr(), _ptr(cu_q), max_seq_len,
                             d ** -0.5 if scale is None else scale, int(causal), window,
                             out.data_ptr(), _ptr(lse), 0, 0)
    place = _place(dev) if workspace is None or counters is None else None
    if counters is not None:
        _check(counters, _U8, "counters", KV_COUNTER_BYTES)
    elif place is not None or not _capturing():
        counters = _cached_workspace(_COUNTERS, place, dev, KV_COUNTER_BYTES, KV_COUNTER_BYTES)
    args.counters = _ptr(counters)
    n = N.lib().nvfp4_kv_attention_workspace_bytes(ctypes.byref(args))
    if workspace is not None:
        _check(workspace, _U8, "workspace")
        if workspace.numel() < n:
            raise ValueError(f"workspace must hold {n} bytes, got {workspace.numel()}")
    with _ISSUE:
        if workspace is None:
            workspace = _cached_workspace(_ATTENTION_WORKSPACES, place, dev, n, 0)
        args.workspace = _ptr(workspace)
        _invoke("nvfp4_kv_attention", (ctypes.byref(args),), dev,
                (q, cache, block_table, seq_lens, cu_q, out, lse, workspace, counters, args))
    return (out, lse) if lse is not None else out
