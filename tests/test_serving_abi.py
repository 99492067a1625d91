"""The serving operators' C ABI without a GPU: struct layouts, argument checks
that come before any CUDA call, and the 64-bit restatements' own pins."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M
from moe_decode_step_gb300 import _binding as b

import _serving as ref

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_decode_step_gb300 import build
    build.build()


class Cache(ctypes.Structure):
    _fields_ = [(n, P) for n in ("k", "v", "k_scale", "v_scale")] + \
        [(n, ctypes.c_int64) for n in ("block_stride", "head_stride", "token_stride",
                                       "scale_stride")] + \
        [(n, ctypes.c_int32) for n in ("n_blocks", "n_kv_heads", "block_size", "head_dim")]


class Attention(ctypes.Structure):
    _fields_ = [("q", P), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out", P), ("out_token_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64), ("lse", P), ("block_table", P),
                ("table_stride", ctypes.c_int64), ("seq_lens", P), ("q_start", P),
                ("workspace", P), ("workspace_bytes", ctypes.c_size_t)] + \
        [(n, ctypes.c_int32) for n in ("dtype", "n_rows", "n_tokens", "n_heads", "max_blocks",
                                       "max_q", "causal", "window")] + [("scale", ctypes.c_float)]


class Route(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_experts", "top_k", "scoring", "n_groups",
                                              "topk_groups", "group_top", "renormalize")] + \
        [("routed_scale", ctypes.c_float)]


def test_packed_formats_have_the_structs_layout():
    for fmt, st in ((b.KV_CACHE, Cache), (b.KV_ATTENTION, Attention), (b.ROUTE, Route)):
        assert fmt.size == ctypes.sizeof(st)
        values = list(range(1, len(st._fields_) + 1))
        got = st.from_buffer_copy(fmt.pack(*values))
        assert [getattr(got, n) for n, _ in st._fields_] == values


def _cache(**kw):
    good = dict(k=4096, v=8192, k_scale=64, v_scale=128, block_stride=2 * 16 * 128,
                head_stride=16 * 128, token_stride=128, scale_stride=2, n_blocks=4, n_kv_heads=2,
                block_size=16, head_dim=128)
    return Cache(**{**good, **kw})


def _append(c, k=4096, v=4096, dtype=0, strides=(256, 128, 256, 128), slots=64, n=3):
    return M.lib().moe_kv_append(None, ctypes.byref(c) if c else None, k, v, dtype, *strides,
                                 slots, n)


def test_cache_and_append_checks():
    bad, no = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    assert _append(None) == bad
    for kw in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None),
               dict(block_size=8), dict(block_size=48), dict(block_size=256), dict(n_blocks=0),
               dict(n_kv_heads=0)):
        assert _append(_cache(**kw)) == bad, kw
    for kw in (dict(head_dim=96), dict(head_dim=256), dict(k=4104), dict(v=8), dict(token_stride=136),
               dict(block_stride=100), dict(head_stride=8), dict(n_blocks=2 ** 27)):
        assert _append(_cache(**kw)) == no, kw
    assert _append(_cache(), dtype=2) == bad and _append(_cache(), dtype=-1) == bad
    assert _append(_cache(), n=-1) == bad and _append(_cache(), n=0) == M.MOE_OK
    assert _append(_cache(), k=None) == bad and _append(_cache(), slots=None) == bad
    assert _append(_cache(), v=8) == no and _append(_cache(), strides=(256, 128, 256, 4)) == no


def _attention(c=None, **kw):
    good = dict(q=4096, q_token_stride=512, q_head_stride=128, out=8192, out_token_stride=512,
                out_head_stride=128, lse=None, block_table=64, table_stride=4, seq_lens=64,
                q_start=64, workspace=4096, workspace_bytes=1 << 30, dtype=0, n_rows=1, n_tokens=1,
                n_heads=4, max_blocks=4, max_q=1, causal=1, window=0, scale=1.0)
    a = Attention(**{**good, **kw})
    return M.lib().moe_kv_attention(None, ctypes.byref(c or _cache()), ctypes.byref(a))


def test_attention_checks():
    bad, no = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    assert M.lib().moe_kv_attention(None, ctypes.byref(_cache()), None) == bad
    for kw in (dict(dtype=2), dict(dtype=-1), dict(n_rows=-1), dict(n_tokens=-1), dict(n_heads=3),
               dict(n_heads=0), dict(max_blocks=0), dict(table_stride=3), dict(window=-1),
               dict(scale=float("nan")), dict(q=None), dict(out=None), dict(block_table=None),
               dict(seq_lens=None), dict(q_start=None), dict(workspace=None)):
        assert _attention(**kw) == bad, kw
    for kw in (dict(q=4104), dict(out=8), dict(q_token_stride=4), dict(out_head_stride=12),
               dict(workspace=128), dict(n_rows=16385), dict(max_blocks=2 ** 27, table_stride=2 ** 27)):
        assert _attention(**kw) == no, kw
    assert _attention(n_rows=0) == M.MOE_OK and _attention(n_tokens=0) == M.MOE_OK
    assert M.lib().moe_kv_attention_workspace(96) == 0


def _plan(**kw):
    good = dict(ctx=64, q=64, rows=2, table=64, stride=4, mb=4, free=64, cap=4, n_free=64, bs=16,
                seq=64, qs=64, slot=64, slots=4, out=128, un=64)
    return M.lib().moe_kv_plan(None, *{**good, **kw}.values())


def test_plan_and_release_checks():
    bad = M.MOE_ERR_INVALID_ARG
    for name in ("ctx", "q", "table", "free", "n_free", "seq", "qs", "slot", "out", "un"):
        assert _plan(**{name: None}) == bad, name
    for kw in (dict(rows=0), dict(stride=3), dict(mb=0, stride=0), dict(cap=-1), dict(bs=24),
               dict(bs=0), dict(slots=-1), dict(out=64)):
        assert _plan(**kw) == bad, kw
    assert _plan(rows=16385) == M.MOE_ERR_UNSUPPORTED
    good = [64, 2, 64, 64, 4, 4, 64, 4, 64, 16, 64]
    for i, v in itertools.chain(((i, None) for i in (0, 2, 3, 6, 8, 10)),
                                ((1, 0), (4, 3), (7, -1), (9, 8))):
        args = list(good)
        args[i] = v
        assert M.lib().moe_kv_release(None, *args) == bad, (i, v)


def _route(logits=64, dtype=2, stride=64, rows=1, idx=64, w=64, **kw):
    good = dict(n_experts=64, top_k=4, scoring=0, n_groups=1, topk_groups=1, group_top=1,
                renormalize=1, routed_scale=1.0)
    cfg = Route(**{**good, **kw})
    return M.lib().moe_route(None, ctypes.byref(cfg), logits, dtype, stride, rows, None, idx, w)


def test_route_checks():
    bad, no = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED
    assert M.lib().moe_route(None, None, 64, 2, 64, 1, None, 64, 64) == bad
    for kw in (dict(n_experts=0), dict(top_k=0), dict(top_k=65), dict(n_groups=0), dict(n_groups=3),
               dict(topk_groups=0), dict(topk_groups=2), dict(n_groups=32, top_k=4),
               dict(group_top=0), dict(group_top=3), dict(scoring=2), dict(scoring=-1),
               dict(routed_scale=float("nan")), dict(rows=-1), dict(stride=-1), dict(dtype=3),
               dict(logits=None), dict(idx=None), dict(w=None)):
        assert _route(**kw) == bad, kw
    for kw in (dict(n_experts=2048), dict(top_k=33), dict(n_groups=64, topk_groups=8)):
        assert _route(**kw) == no, kw
    assert _route(rows=0) == M.MOE_OK


def test_python_checks_refuse_host_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="ctx_lens"):
        M.kv_plan(t, t, t.view(1, 4), t, t[:1], 16, 4)
    with pytest.raises(ValueError, match="logits"):
        M.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="k:"):
        c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
        M.KVCache(c, c, c[..., 0, 0], c[..., 0, 0])


# -- the restatements themselves ------------------------------------------------
def test_e4m3_table_and_rounding():
    tab = ref.e4m3_table()
    assert tab[126] == 448.0 and tab[8] == 2.0 ** -6 and tab[1] == 2.0 ** -9 and np.isnan(tab[127])
    t8 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(tab, nan=-1), np.nan_to_num(t8, nan=-1))
    rng = np.random.default_rng(0)
    x = rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000)
    x = np.clip(np.concatenate([x, tab[:127], (tab[:126] + tab[1:127]) / 2, -tab[:127]]), -448, 448)
    want = torch.from_numpy(x).to(torch.float32)
    keep = want.double().numpy() == x          # float32 values: one rounding on either side
    got = ref.e4m3_round(x)[keep]
    assert np.array_equal(got, want.to(torch.float8_e4m3fn).view(torch.uint8).numpy()[keep])


def test_block_exponent():
    for amax, e in ((0.0, -60), (448.0, 0), (448.5, 1), (1.0, -8), (1.75, -8), (1.76, -7),
                    (2.0 ** 100, 60), (1e-30, -60)):
        assert ref.block_exp(amax) == e


def test_plan_restatement_by_hand():
    table = np.full((3, 4), -1)
    table[1, 0] = 50
    seq, qs, slot, left, unserved, t = ref.plan([0, 15, 3], [17, 2, 1], table, np.arange(100, 110),
                                                4, 16, 22)
    # row 2's block is not in the table (entry -1): its slot lies in "block -1"
    assert seq.tolist() == [17, 17, 4] and qs.tolist() == [0, 17, 19, 20]
    assert t[0, :2].tolist() == [103, 102] and t[1, :2].tolist() == [50, 101]
    assert left == 1 and unserved == 0
    assert slot[:3].tolist() == [1648, 1649, 1650] and slot[16] == 1632
    assert slot[17:19].tolist() == [815, 1616] and slot[20:].tolist() == [-1, -1]


def test_route_restatement_by_hand():
    x = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    idx, w = ref.route(x, None, 2, "softmax", 1, 1, 1, False, 2.0)
    assert idx.tolist() == [[1, 3]] and np.allclose(w, [[0.8, 0.6]])
    idx, w = ref.route(x, None, 2, "softmax", 2, 1, 1, True, 1.0)
    assert idx.tolist() == [[1, 0]] and np.allclose(w, [[0.8, 0.2]])
    idx, w = ref.route(x, np.array([0, 0, 1.0, 0]), 1, "softmax", 2, 1, 2, False, 1.0)
    assert idx.tolist() == [[2]] and np.allclose(w, [[0.2]])
