"""Serving operators beside the MoE layer: block tables and slot maps, the
8-bit KV cache and its attention, expert routing from logits.

Argument marshalling only: every call checks its tensors, then makes one call
of the C ABI (include/moe_decode.h states the formulas and the rules).  All of
it is asynchronous on `stream` (default: the current stream); tensors made
here are allocated on that stream.
"""
from typing import NamedTuple

import torch

from ._binding import DTYPE_BF16, DTYPE_F16, DTYPE_F32, KV_ATTENTION, KV_CACHE, ROUTE, check, lib

_CODES = (torch.float8_e4m3fn, torch.uint8)
_SCALES = (torch.float8_e8m0fnu, torch.uint8)
_DTYPE = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
_SCORING = {"sigmoid": 0, "softmax": 1}


def _raw_stream(stream, device):
    """cudaStream_t of `stream` or of the device's current stream; the calls
    launch on the current device, so the tensors must live there."""
    index = device.index
    if index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    return stream.cuda_stream


def _empty(stream, dtype, device, *shape):
    """A new tensor whose memory belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _want(ok, name, what, t):
    if not ok:
        got = (f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}"
               if isinstance(t, torch.Tensor) else repr(t))
        raise ValueError(f"{name}: want {what}, got {got}")


def _vector(t, n, dtype, name, device):
    """A contiguous 1-D tensor of n elements (n None: any)."""
    if (t.dtype != dtype or t.device != device or not t.is_contiguous()
            or (t.dim() != 1 if n is None else t.shape != (n,))):
        _want(False, name, f"{dtype} [{'n' if n is None else n}] contiguous on {device}", t)


def _table(t, rows, device):
    if (t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != rows or t.device != device
            or (t.shape[1] > 1 and t.stride(1) != 1)
            or (rows > 1 and t.stride(0) < t.shape[1])):
        _want(False, "block_table", f"torch.int32 [{rows}, max_blocks] with contiguous rows on "
              f"{device}", t)
    return t.stride(0) if rows > 1 else t.shape[1]


class KVPlan(NamedTuple):
    """What kv_plan writes (see moe_kv_plan)."""
    seq_lens: torch.Tensor     # int32 [rows]: cached tokens with this step's
    q_start: torch.Tensor      # int32 [rows + 1]: first new token of each row
    slot_map: torch.Tensor     # int32 [n_slots]: cache slot of each new token, or -1
    n_free: torch.Tensor       # int32 [1]: blocks left on the free stack
    n_unserved: torch.Tensor   # int32 [1]: rows that got no blocks


def kv_plan(ctx_lens, q_lens, block_table, free_list, n_free, block_size, n_slots, stream=None):
    """Block tables and slot maps of one step from request lengths (moe_kv_plan):
    extends block_table in place and returns a KVPlan.  ctx_lens, q_lens int32
    [rows]; block_table int32 [rows, max_blocks]; free_list int32 [n], n_free
    int32 [1]: a stack of free block ids and its height; n_slots: entries of
    the slot map, at least the new tokens the step may have.  A row is taken
    to hold the blocks of its ctx_lens: one that got shorter gives the others
    back by kv_release's keep_lens first."""
    dev = ctx_lens.device
    _want(ctx_lens.is_cuda, "ctx_lens", "a CUDA tensor", ctx_lens)
    rows = ctx_lens.shape[0]
    _vector(ctx_lens, rows, torch.int32, "ctx_lens", dev)
    _vector(q_lens, rows, torch.int32, "q_lens", dev)
    _vector(free_list, None, torch.int32, "free_list", dev)
    _vector(n_free, 1, torch.int32, "n_free", dev)
    stride = _table(block_table, rows, dev)
    n_slots = int(n_slots)
    _want(n_slots >= 0, "n_slots", "a number of slots >= 0", n_slots)
    raw = _raw_stream(stream, dev)
    # one allocation, cut in one operation (no gradients: the form that keeps no record)
    buf = _empty(stream, torch.int32, dev, n_slots + 2 * rows + 3)
    slots, lens, start, left, unserved = torch.unsafe_split_with_sizes(
        buf, [n_slots, rows, rows + 1, 1, 1])
    at = buf.data_ptr()
    at_lens = at + 4 * n_slots
    at_left = at_lens + 8 * rows + 4
    rc = lib().moe_kv_plan(raw, ctx_lens.data_ptr(), q_lens.data_ptr(), rows,
                           block_table.data_ptr(), stride, block_table.shape[1],
                           free_list.data_ptr(), free_list.shape[0], n_free.data_ptr(),
                           int(block_size), at_lens, at_lens + 4 * rows, at, n_slots, at_left,
                           at_left + 4)
    check(rc, "moe_kv_plan")
    return KVPlan(lens, start, slots, left, unserved)


def kv_release(finished, seq_lens, block_table, free_list, n_free, block_size, stream=None,
               keep_lens=None):
    """Give the finished rows' blocks back (moe_kv_release): finished bool or
    uint8 [rows]; pushes onto free_list, zeroes their seq_lens and updates
    n_free, all in place.  With keep_lens (int32 [rows]) the other rows give
    back what lies past that many tokens, and it becomes their length
    (moe_kv_release_past): a row whose drafts were rejected is shortened this
    way before the next kv_plan."""
    dev = seq_lens.device
    _want(seq_lens.is_cuda, "seq_lens", "a CUDA tensor", seq_lens)
    rows = seq_lens.shape[0]
    _vector(seq_lens, rows, torch.int32, "seq_lens", dev)
    _vector(finished, rows, torch.bool if finished.dtype == torch.bool else torch.uint8,
            "finished", dev)
    if keep_lens is not None:
        _vector(keep_lens, rows, torch.int32, "keep_lens", dev)
    _vector(free_list, None, torch.int32, "free_list", dev)
    _vector(n_free, 1, torch.int32, "n_free", dev)
    stride = _table(block_table, rows, dev)
    check(lib().moe_kv_release_past(_raw_stream(stream, dev), finished.data_ptr(),
                                    None if keep_lens is None else keep_lens.data_ptr(), rows,
                                    seq_lens.data_ptr(), block_table.data_ptr(), stride,
                                    block_table.shape[1], free_list.data_ptr(), free_list.shape[0],
                                    n_free.data_ptr(), int(block_size), n_free.data_ptr()),
          "moe_kv_release")


class KVCache:
    """A paged KV cache in 8 bits over borrowed tensors (moe_kv_cache_t).

    k, v: E4M3 codes (float8_e4m3fn or uint8) [n_blocks, n_kv_heads, block_size,
    head_dim], alike in strides, the last dimension contiguous, the other
    strides multiples of 16: a token-major cache is passed as a transposed
    view.  k_scale, v_scale: E8M0 (float8_e8m0fnu or uint8) [n_blocks,
    n_kv_heads], heads contiguous.
    """

    def __init__(self, k, v, k_scale, v_scale):
        _want(k.is_cuda and k.dim() == 4 and k.dtype in _CODES, "k",
              "CUDA E4M3 codes [n_blocks, n_kv_heads, block_size, head_dim]", k)
        _want(v.dtype in _CODES and v.shape == k.shape and v.stride() == k.stride()
              and v.device == k.device, "v", "the same shape and strides as k", v)
        self.n_blocks, self.n_kv_heads, self.block_size, self.head_dim = k.shape
        _want(k.stride(3) == 1, "k", "a contiguous last dimension", k)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _want(t.dtype in _SCALES and tuple(t.shape) == tuple(k.shape[:2])
                  and t.device == k.device and (t.shape[1] == 1 or t.stride(1) == 1)
                  and t.stride() == k_scale.stride(), name,
                  "E8M0 scales [n_blocks, n_kv_heads], heads contiguous, both alike", t)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self._struct = KV_CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                     v_scale.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                                     k_scale.stride(0), *k.shape)
        self._workspace = lib().moe_kv_attention_workspace(self.head_dim)

    @classmethod
    def empty(cls, n_blocks, n_kv_heads, block_size, head_dim, device="cuda"):
        """A new head-major cache; its contents do not matter until written."""
        shape = (n_blocks, n_kv_heads, block_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.full(shape[:2], 127, dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn),
                   ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu))

    def _new(self, t, name):
        if (t.dim() != 3 or t.shape[1] != self.n_kv_heads or t.shape[2] != self.head_dim
                or t.stride(2) != 1 or t.device != self.device):
            _want(False, name, f"[tokens, {self.n_kv_heads}, {self.head_dim}] with a contiguous "
                  f"last dimension on {self.device}", t)

    def append(self, k, v, slot_map, stream=None):
        """Write the new tokens' keys and values (bfloat16 or float16 [tokens,
        n_kv_heads, head_dim]) to the slots of slot_map (int32 [tokens], or longer: a plan's
        padded map) (moe_kv_append)."""
        self._new(k, "k")
        self._new(v, "v")
        _want(k.dtype == v.dtype and k.dtype in (torch.bfloat16, torch.float16), "k, v",
              "bfloat16 or float16, both alike", k)
        n = k.shape[0]
        _want(v.shape[0] == n, "v", f"{n} tokens, as k", v)
        _vector(slot_map, None, torch.int32, "slot_map", self.device)
        _want(slot_map.shape[0] >= n, "slot_map", f"at least {n} entries", slot_map)
        rc = lib().moe_kv_append(_raw_stream(stream, self.device), self._struct, k.data_ptr(),
                                 v.data_ptr(), _DTYPE[k.dtype], k.stride(0), k.stride(1),
                                 v.stride(0), v.stride(1), slot_map.data_ptr(), n)
        check(rc, "moe_kv_append")

    def attention(self, q, block_table, seq_lens, q_start, max_q, scale=None, causal=True,
                  window=0, out=None, return_lse=False, stream=None):
        """Attention of the rows' new tokens over the cache (moe_kv_attention):
        q bfloat16 or float16 [tokens, n_heads, head_dim], packed by q_start
        (int32 [rows + 1]); block_table int32 [rows, max_blocks]; seq_lens
        int32 [rows].  max_q: the longest row's queries (picks the kernel
        only).  scale defaults to 1 / sqrt(head_dim).  Returns out, or (out,
        lse) with lse float32 [tokens, n_heads]."""
        d, dev = self.head_dim, self.device
        if (q.dim() != 3 or q.shape[2] != d or q.stride(2) != 1 or q.device != dev
                or q.dtype not in (torch.bfloat16, torch.float16)):
            _want(False, "q", f"bfloat16 or float16 [tokens, heads, {d}] with a contiguous last "
                  f"dimension on {dev}", q)
        tokens, heads = q.shape[0], q.shape[1]
        rows = seq_lens.shape[0]
        _vector(seq_lens, rows, torch.int32, "seq_lens", dev)
        _vector(q_start, rows + 1, torch.int32, "q_start", dev)
        table_stride = _table(block_table, rows, dev)
        raw = _raw_stream(stream, dev)
        if out is None:
            out = _empty(stream, q.dtype, dev, tokens, heads, d)
        elif (out.shape != q.shape or out.dtype != q.dtype or out.device != dev
                or out.stride(2) != 1):
            _want(False, "out", "the shape and type of q, last dimension contiguous", out)
        lse = _empty(stream, torch.float32, dev, tokens, heads) if return_lse else None
        ws = _empty(stream, torch.uint8, dev, self._workspace)
        qs, os = q.stride(), out.stride()
        args = KV_ATTENTION.pack(
            q.data_ptr(), qs[0], qs[1], out.data_ptr(), os[0], os[1],
            lse.data_ptr() if return_lse else 0, block_table.data_ptr(), table_stride,
            seq_lens.data_ptr(), q_start.data_ptr(), ws.data_ptr(), self._workspace,
            _DTYPE[q.dtype], rows, tokens, heads, block_table.shape[1], int(max_q), int(causal),
            int(window), d ** -0.5 if scale is None else scale)
        check(lib().moe_kv_attention(raw, self._struct, args), "moe_kv_attention")
        return (out, lse) if return_lse else out


def moe_route(logits, top_k, bias=None, scoring="sigmoid", n_groups=1, topk_groups=1,
              group_top=2, renormalize=True, routed_scale=1.0, idx=None, w=None, stream=None):
    """Expert routing from logits (moe_route): logits float32, bfloat16 or
    float16 [rows, experts] with contiguous rows -> idx int32, w float32
    [rows, top_k], in descending order of score + bias."""
    if (logits.dim() != 2 or logits.dtype not in _DTYPE or not logits.is_cuda
            or (logits.shape[1] > 1 and logits.stride(1) != 1)):
        _want(False, "logits", "float32, bfloat16 or float16 [rows, experts] with contiguous rows "
              "on a CUDA device", logits)
    rows, experts = logits.shape
    dev = logits.device
    if bias is not None:
        _vector(bias, experts, torch.float32, "bias", dev)
    _want(scoring in _SCORING, "scoring", "'sigmoid' or 'softmax'", scoring)
    raw = _raw_stream(stream, dev)
    top_k = int(top_k)
    shape = (rows, top_k)
    if idx is None:
        _want(top_k >= 1, "top_k", "at least 1", top_k)
        idx = _empty(stream, torch.int32, dev, rows, top_k)
    elif (idx.dtype != torch.int32 or tuple(idx.shape) != shape or idx.device != dev
            or not idx.is_contiguous()):
        _want(False, "idx", f"torch.int32 {shape} contiguous on {dev}", idx)
    if w is None:
        w = _empty(stream, torch.float32, dev, rows, top_k)
    elif (w.dtype != torch.float32 or tuple(w.shape) != shape or w.device != dev
            or not w.is_contiguous()):
        _want(False, "w", f"torch.float32 {shape} contiguous on {dev}", w)
    cfg = ROUTE.pack(experts, top_k, _SCORING[scoring], int(n_groups), int(topk_groups),
                     int(group_top), int(bool(renormalize)), routed_scale)
    check(lib().moe_route(raw, cfg, logits.data_ptr(), _DTYPE[logits.dtype], logits.stride(0),
                          rows, bias.data_ptr() if bias is not None else None, idx.data_ptr(),
                          w.data_ptr()), "moe_route")
    return idx, w
