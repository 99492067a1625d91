"""The example's MoE layer for any number of rows: the experts it chooses and their
weights against MoELayer and 64 bits, its result against a 64-bit restatement on the
same 8-bit operands."""
import numpy as np
import pytest
import torch

from gen.configs import CONFIGS

import _fp8 as ref
from test_gpu_fp8_chain import example

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _np(t):
    return t.detach().double().cpu().numpy()


def _u8(t):
    return t.view(torch.uint8).cpu().numpy()


def _choices(monkeypatch, prompt, x, residual):
    """forward's result, and the idx and weights it went by."""
    seen = []
    route = example.M.moe_route

    def watched(*a, **k):
        seen.append(route(*a, **k))
        return seen[-1]
    monkeypatch.setattr(example.M, "moe_route", watched)
    out = prompt.forward(x, residual)
    monkeypatch.undo()
    return out, seen[0][0].cpu().numpy(), _np(seen[0][1])


def test_chooses_the_layers_experts(monkeypatch):
    """All 64 rows, but those whose k-th and next score are less than 1e-5 apart."""
    cfg = CONFIGS["tiny_b1"]
    layer = example.synthetic.make_layer(cfg, max_batch=64)
    prompt = example.PromptLayer(cfg)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(64, cfg.d, generator=g, device=DEV).to(torch.bfloat16)
    _, idx, mix = _choices(monkeypatch, prompt, x, torch.zeros_like(x))
    want_idx, want_mix = layer.router_topk(x)
    want_idx, want_mix = want_idx.cpu().numpy(), _np(want_mix)
    layer.close()
    score = 1 / (1 + np.exp(-_np(x) @ _np(prompt.weights["router_w"]).T))
    biased = np.sort(score + _np(prompt.weights["router_bias"]), axis=1)[:, ::-1]
    clear = biased[:, cfg.top_k - 1] - biased[:, cfg.top_k] >= 1e-5
    assert clear.sum() >= 60
    for b in np.flatnonzero(clear):
        assert sorted(idx[b]) == sorted(want_idx[b]), b
        at = {int(e): j for j, e in enumerate(want_idx[b])}
        s = score[b, idx[b]]
        for j, e in enumerate(idx[b]):
            assert abs(mix[b, j] - want_mix[b, at[int(e)]]) <= 2e-6
            assert abs(mix[b, j] - cfg.routed_scale * s[j] / s.sum()) <= 2e-6


def test_result_on_the_same_operands(monkeypatch):
    """Bounds: an expert's result, the shared expert's, their sum and the residual are each
    rounded to 16 bits, by 2^-8 of themselves at most: three times 2^-8 of the sum of
    absolute terms, in rms.  (The restatement rounds h to 8 bits from 64-bit sums: the few
    codes in 10^5 that turn move a row by less than 2^-8 / 8 of it.)"""
    cfg = CONFIGS["tiny_b1"]
    prompt = example.PromptLayer(cfg)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(40, cfg.d, generator=g, device=DEV).to(torch.bfloat16)
    r0 = torch.randn(40, cfg.d, generator=g, device=DEV).to(torch.bfloat16)
    r = r0.clone()
    out, idx, mix = _choices(monkeypatch, prompt, x, r)
    w = prompt.weights
    xv = ref.row_values(*ref.quantize(_np(x)))

    def expert(rows, up, down):
        h, _ = ref.swiglu(*ref.product(rows, up))
        return ref.row_values(*ref.quantize(h)) @ down.T

    shared = [ref.weight_values(_u8(q.codes), _u8(q.scales), False)
              for q in (prompt.shared_gu, prompt.shared_d)]
    z = expert(xv, *shared)
    size = np.abs(z)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        y = mix[t, j][:, None] * expert(
            xv[t], ref.weight_values(_u8(w["w_gu_q"][e]), _u8(w["w_gu_s"][e]), True),
            ref.weight_values(_u8(w["w_d_q"][e]), _u8(w["w_d_s"][e]), True))
        z[t] += y          # (a token chooses an expert once)
        size[t] += np.abs(y)
    z += _np(r0)
    size += np.abs(_np(r0))
    off = _np(r) - z
    assert np.sqrt((off ** 2).mean()) <= 3 * 2.0 ** -8 * np.sqrt((size ** 2).mean())
    assert (np.sqrt((off ** 2).mean(1)) <= 3.5 * 2.0 ** -8 * np.sqrt((size ** 2).mean(1))).all()
    # the norm is of the unrounded sum, each value of r within 2^-8 of it and so their
    # rms, and is rounded itself
    rv = _np(r)
    want = rv / np.sqrt((rv ** 2).mean(1, keepdims=True) + cfg.rms_eps) * _np(w["rms_gamma"])
    assert (np.abs(_np(out) - want) <= 3.1 * 2.0 ** -8 * np.abs(want)).all()
