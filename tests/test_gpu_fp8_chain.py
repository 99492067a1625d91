"""The 8-bit operators as they are used together: norm, routing, dispatch, experts up and
down, combine.  Every stage is held to its own bound (_fp8.py) on what the stage before
it gave; then the whole chain in a CUDA graph, on another stream, twice in a row, and the
MoE layer of the example against MoELayer."""
import importlib.util
import os

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import moe_decode_step_gb300 as M
from gen.configs import CONFIGS

import _fp8 as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decode_block.py")
spec = importlib.util.spec_from_file_location("decode_block", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _u8(t):
    return t.view(torch.uint8).cpu().numpy()


class Chain:
    def __init__(self, tokens, d, f, experts, k, mx, seed=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.experts, self.k, self.mx = experts, k, mx
        up, ups = zip(*(ref.random_w(rng, 2 * f, d, mx) for _ in range(experts)))
        down, downs = zip(*(ref.random_w(rng, d, f, mx) for _ in range(experts)))
        self.up, self.ups, self.down, self.downs = (
            torch.from_numpy(np.stack(t)).to(DEV) for t in (up, ups, down, downs))
        if not mx:
            self.up, self.down = (t.view(torch.float8_e4m3fn) for t in (self.up, self.down))
        self.router = torch.randn(experts, d, generator=g, device=DEV).to(torch.bfloat16)
        self.router *= d ** -0.5
        self.gamma = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
        self.x = torch.randn(tokens, d, generator=g, device=DEV).to(torch.bfloat16)
        self.residual = torch.randn(tokens, d, generator=g, device=DEV).to(torch.bfloat16)

    def run(self, x, residual, stream=None):
        """Everything between the attention and the next layer; residual is updated."""
        n = M.rms_norm(x, self.gamma, residual=residual, eps=1e-6, quantize=True, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            logits = F.linear(n.out, self.router)
        idx, w = M.moe_route(logits, self.k, stream=stream)
        by = M.moe_dispatch(idx, self.experts, stream=stream)
        h = M.expert_linear(n.codes, n.scales, self.up, self.ups, by.offsets, rows=by.rows,
                            activation="swiglu", quantize=True, stream=stream)
        y = M.expert_linear(h.codes, h.scales, self.down, self.downs, by.offsets, stream=stream)
        out = M.moe_combine(y, w, by.slots, residual=residual, stream=stream)
        return n, idx, w, by, h, y, out

    def flat(self, x, residual, stream=None):
        n, idx, w, by, h, y, out = self.run(x, residual, stream)
        return [*n, idx, w, *by, *h, y, out, residual]


CASES = [(1, 256, 128, 8, 2, True), (70, 512, 256, 16, 4, True), (70, 512, 384, 16, 4, False),
         (600, 256, 128, 8, 2, False), (33, 1024, 256, 64, 4, True)]


@pytest.mark.parametrize("tokens,d,f,experts,k,mx", CASES)
def test_every_stage(tokens, d, f, experts, k, mx):
    c = Chain(tokens, d, f, experts, k, mx)
    x, r0 = c.x.clone(), c.residual.clone()
    r = r0.clone()
    n, idx, w, by, h, y, out = c.run(x, r)
    z = _np(x) + _np(r0)
    size = np.abs(_np(x)) + np.abs(_np(r0))
    scale = 1.0 / np.sqrt((z * z).mean(axis=1, keepdims=True) + 1e-6)
    v = z * scale * _np(c.gamma)
    tol = 64 * 2.0 ** -24 * np.abs(v) + 2.0 ** -24 * size * scale * np.abs(_np(c.gamma))
    ref.check_values(n.out, v, tol, torch.bfloat16, "norm")
    ref.check_codes(n.codes, n.scales, v, tol, "norm")
    ref.check_values(r, z, 2.0 ** -24 * size, torch.bfloat16, "residual")
    for got, want in zip(by, ref.dispatch(idx.cpu().numpy(), experts)):
        assert np.array_equal(got.cpu().numpy(), want)
    off, rows = by.offsets.tolist(), by.rows.cpu().numpy()
    xv = ref.row_values(_u8(n.codes), _u8(n.scales))[rows]
    hv = ref.row_values(_u8(h.codes), _u8(h.scales))
    for e in range(experts):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        p, t = ref.swiglu(*ref.product(
            xv[a:b], ref.weight_values(_u8(c.up[e]), _u8(c.ups[e]), mx)))
        ref.check_codes(h.codes[a:b], h.scales[a:b], p, t, ("up", e))
        p, t = ref.product(hv[a:b], ref.weight_values(_u8(c.down[e]), _u8(c.downs[e]), mx))
        ref.check_values(y[a:b], p, t, torch.bfloat16, ("down", e))
    terms = _np(w)[..., None] * _np(y)[by.slots.cpu().numpy()]
    tol = (k + 1) * 2.0 ** -24 * (np.abs(terms).sum(axis=1) + np.abs(_np(r)))
    ref.check_values(out, terms.sum(axis=1) + _np(r), tol, torch.bfloat16, "combine")


def _equal(a, b):
    return all(torch.equal(s.contiguous().view(torch.uint8), t.contiguous().view(torch.uint8))
               for s, t in zip(a, b))


def test_graph_replays_follow_new_inputs():
    c = Chain(70, 512, 256, 16, 4, True, seed=3)
    x, r = c.x.clone(), c.residual.clone()
    c.flat(x, r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = c.flat(x, r)
    for seed in range(3):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        r.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        x1, r1 = x.clone(), r.clone()
        g.replay()
        torch.cuda.synchronize()
        assert _equal(got, c.flat(x1, r1))


def test_another_stream_and_calls_in_a_row():
    """The same bits on another stream, called again and again without waiting, and from
    two streams at once."""
    c = Chain(300, 512, 256, 16, 4, False, seed=4)
    want = c.flat(c.x, c.residual.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    copies = [c.residual.clone() for _ in range(12)]
    torch.cuda.synchronize()
    got = [c.flat(c.x, r, streams[i % 2]) for i, r in enumerate(copies)]
    torch.cuda.synchronize()
    assert all(_equal(want, o) for o in got)


def test_calls_from_threads():
    import threading
    c = Chain(40, 256, 128, 8, 2, True, seed=5)
    want = c.flat(c.x, c.residual.clone())
    torch.cuda.synchronize()
    results, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            rs = [c.residual.clone() for _ in range(20)]
            torch.cuda.synchronize()
            results[i] = [c.flat(c.x, r, s) for r in rs]
            s.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert all(_equal(want, o) for r in results.values() for o in r)


def test_prompt_layer_is_the_moe_layer():
    """The example's layer for any number of rows against MoELayer on the same rows and
    weights.  Bound: rounding a value to E4M3 moves it by at most 2^-4 of itself, so a
    product with random weights by 2^-4 of its rms: x once before the gates and ups (a
    gate counts 1.1 times, the slope of silu), the results once before the way down, the
    shared expert's weights at both: 2.1 + 1 + 2 times 2^-4 of the sum's rms."""
    cfg = CONFIGS["tiny_b1"]
    layer = example.synthetic.make_layer(cfg, max_batch=64)
    prompt = example.PromptLayer(cfg)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(64, cfg.d, generator=g, device=DEV).to(torch.bfloat16)
    zero = torch.zeros_like(x)
    dbg = layer.forward_debug(x, zero.clone())
    z = (dbg["y_routed"] + dbg["y_shared"]).double()
    r = zero.clone()
    out = prompt.forward(x, r)
    idx, _ = layer.router_topk(x)
    logits = F.linear(x, prompt.weights["router_w"])
    mine, _ = M.moe_route(logits, cfg.top_k, bias=prompt.weights["router_bias"],
                          routed_scale=cfg.routed_scale)
    same = (idx.sort(1).values == mine.sort(1).values).all(1)   # (16-bit logits may swap a pair)
    assert int(same.sum()) >= 48
    off = (r.double() - z)[same]
    assert off.square().mean().sqrt() <= 5.1 * 2.0 ** -4 * z[same].square().mean().sqrt()
    want = r.double() * torch.rsqrt(r.double().square().mean(1, keepdim=True) + cfg.rms_eps)
    want *= prompt.weights["rms_gamma"].double()
    # (r is the rounded sum: 2^-8 of it, and the output's own rounding)
    assert (out.double() - want).abs().max() <= 3 * 2.0 ** -8 * want.abs().max()
    layer.close()


def test_prompt_layer_is_alike_for_any_number_of_rows():
    """Rows do not depend on one another: 700 rows at once and 50 at a time agree but
    for the order of split sums."""
    prompt = example.PromptLayer(CONFIGS["tiny_b1"])
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(700, 1024, generator=g, device=DEV).to(torch.bfloat16)
    r = torch.zeros_like(x)
    all_at_once = prompt.forward(x, r)
    parts = []
    for a in range(0, 700, 50):
        parts.append(prompt.forward(x[a:a + 50].contiguous(), torch.zeros_like(x[a:a + 50])))
    a, b = all_at_once.double(), torch.cat(parts).double()
    # a code or an output may round the other way where sums are added in another order;
    # router logits too, so that a row may choose another expert: rows are compared
    off = (a - b).square().mean(1).sqrt() / a.square().mean(1).sqrt()
    assert float(off.median()) <= 2.0 ** -8 and int((off > 2.0 ** -4).sum()) <= 7
