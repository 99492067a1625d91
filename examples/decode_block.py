"""A decoder block served with the library: paged 8-bit KV cache, attention,
routing statistics and the MoE layer, over requests of different lengths.

    python examples/decode_block.py

One step is kv_plan (blocks and slots for this step's tokens), the projections
(torch), KVCache.append, KVCache.attention and MoELayer.forward.  Lengths,
tables and the free stack stay on the device, so the decode step is captured
into a CUDA graph once and replayed for every token; kv_release gives a
finished request's blocks back.  PromptLayer is the MoE layer for any number of
rows, with 8-bit activations.  Its products read the experts' canonical layout,
MoELayer the tcgen05 path's, so each has the weights once.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_decode_step_gb300 as M  # noqa: E402
from gen.configs import CONFIGS  # noqa: E402
from moe_decode_step_gb300 import synthetic  # noqa: E402


class DecoderBlock:
    """Attention with random projections in front of a synthetic MoE layer."""

    def __init__(self, cfg, rows, n_heads=16, n_kv_heads=2, head_dim=64, block_size=16,
                 n_blocks=256, max_blocks=32, seed=0):
        dev = torch.device("cuda", torch.cuda.current_device())
        g = torch.Generator(device=dev).manual_seed(seed)
        self.cfg, self.rows, self.heads, self.d = cfg, rows, n_heads, cfg.d
        self.kv_heads, self.head_dim = n_kv_heads, head_dim
        self.weights = synthetic.make_weights(cfg)
        self.moe = synthetic.make_layer(cfg, max_batch=rows, weights=self.weights)

        def matrix(n, k):
            w = torch.randn(n, k, generator=g, device=dev) * k ** -0.5
            return w.to(torch.bfloat16)

        self.w_qkv = matrix((n_heads + 2 * n_kv_heads) * head_dim, cfg.d)
        self.w_o = matrix(cfg.d, n_heads * head_dim)
        self.cache = M.KVCache.empty(n_blocks, n_kv_heads, block_size, head_dim, dev)

        def ints(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=dev)

        self.table, self.ctx_lens = ints(rows, max_blocks), ints(rows)
        self.free_list = torch.arange(n_blocks, dtype=torch.int32, device=dev)
        self.n_free = torch.full((1,), n_blocks, dtype=torch.int32, device=dev)
        self.unserved = ints(1)
        self.one_each = torch.ones(rows, dtype=torch.int32, device=dev)

    def attend(self, x, q_lens, max_q):
        """Blocks and slots for this step's tokens, their keys and values into
        the cache, and their attention: x bf16 [tokens, d], packed by row."""
        plan = M.kv_plan(self.ctx_lens, q_lens, self.table, self.free_list, self.n_free,
                         self.cache.block_size, x.shape[0])
        qkv = F.linear(x, self.w_qkv).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        self.cache.append(k, v, plan.slot_map)
        out = self.cache.attention(q, self.table, plan.seq_lens, plan.q_start, max_q)
        self.ctx_lens.copy_(plan.seq_lens)
        self.n_free.copy_(plan.n_free)
        self.unserved += plan.n_unserved
        return out

    def prefill(self, prompts):
        """Prompts (a list of bf16 [n, d]) into the cache; each row's last
        attention output [rows, d], and how often the prompts' tokens choose
        each expert (what a placement of the experts is decided from)."""
        x = torch.cat(prompts)
        lens = torch.tensor([p.shape[0] for p in prompts], dtype=torch.int32, device=x.device)
        out = self.attend(x, lens, max(p.shape[0] for p in prompts))
        y = F.linear(out.flatten(1), self.w_o)
        logits = F.linear(x.float(), self.weights["router_w"].float())
        idx, _ = M.moe_route(logits, self.cfg.top_k, bias=self.weights["router_bias"],
                             routed_scale=self.cfg.routed_scale)
        load = torch.bincount(idx.flatten(), minlength=self.cfg.n_experts)
        return y[torch.cumsum(lens, 0) - 1], load

    def decode(self, x, residual):
        """One token per row: x and residual bf16 [rows, d], residual updated;
        returns the layer's normalised output."""
        out = self.attend(x, self.one_each, 1)
        residual += F.linear(out.flatten(1), self.w_o)
        h = F.rms_norm(residual.float(), (self.d,)).to(torch.bfloat16)
        return self.moe.forward(h, residual)

    def release(self, finished):
        """finished: bool [rows]."""
        M.kv_release(finished, self.ctx_lens, self.table, self.free_list, self.n_free,
                     self.cache.block_size)


class PromptLayer:
    """The MoE layer for any number of rows: its experts' MXFP4 weights in the canonical
    layout, the shared expert's in 8 bits, 8-bit activations."""

    def __init__(self, cfg):
        self.cfg = cfg
        self.weights = synthetic.make_weights(cfg, layout=0)
        self.router_w = self.weights["router_w"].float()
        self.shared_gu = M.fp8_pack(self.weights["shared_gu"])
        self.shared_d = M.fp8_pack(self.weights["shared_d"])

    def forward(self, x, residual):
        """x and residual bf16 [tokens, d], residual updated; returns the normalised
        output, as MoELayer.forward."""
        c, w = self.cfg, self.weights
        # (in 32 bits, as MoELayer has them: rounded to 16 they choose other experts)
        logits = F.linear(x.float(), self.router_w)
        idx, mix = M.moe_route(logits, c.top_k, bias=w["router_bias"], routed_scale=c.routed_scale)
        by = M.moe_dispatch(idx, c.n_experts)
        x8 = M.fp8_quantize(x)
        h = M.expert_linear(*x8, w["w_gu_q"], w["w_gu_s"], by.offsets, rows=by.rows,
                            activation="swiglu", quantize=True)
        y = M.expert_linear(*h, w["w_d_q"], w["w_d_s"], by.offsets)
        hs = M.fp8_linear(*x8, *self.shared_gu, activation="swiglu", quantize=True)
        z = M.moe_combine(y, mix, by.slots, residual=M.fp8_linear(*hs, *self.shared_d))
        return M.rms_norm(z, w["rms_gamma"], residual=residual, eps=c.rms_eps).out


def generate(block, prompts, steps, graph=True):
    """Prefill, then `steps` decode steps; the outputs [steps, rows, d] and the
    prompts' expert load."""
    last, load = block.prefill(prompts)
    x = last.clone()
    residual = torch.zeros_like(x)
    outs = [block.decode(x, residual).clone()]   # (also warms the capture up)
    x.copy_(outs[0])
    g = None
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = block.decode(x, residual)
            x.copy_(out)
    for _ in range(steps - 1):
        if g is not None:
            g.replay()
        else:
            x.copy_(block.decode(x, residual))
        outs.append(x.clone())
    return torch.stack(outs), load


def main():
    cfg = CONFIGS["tiny_b1"]
    rows, steps = 4, 24
    block = DecoderBlock(cfg, rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randn(n, cfg.d, generator=g, device="cuda").to(torch.bfloat16)
               for n in (70, 1, 33, 200)]
    out, load = generate(block, prompts, steps)
    used = block.free_list.shape[0] - int(block.n_free)
    print(f"{rows} requests, prompts of {[p.shape[0] for p in prompts]} tokens, {steps} steps: "
          f"contexts {block.ctx_lens.tolist()}, {used} blocks in use")
    print(f"output rms {out.float().square().mean().sqrt():.3f}; the prompts' busiest experts "
          f"{torch.topk(load, 4).indices.tolist()}")
    tokens = torch.cat(prompts)
    out = PromptLayer(cfg).forward(tokens, torch.zeros_like(tokens))
    print(f"all {tokens.shape[0]} prompt tokens through the MoE layer: output rms "
          f"{out.float().square().mean().sqrt():.3f}")
    block.release(torch.ones(rows, dtype=torch.bool, device="cuda"))
    print(f"released: {int(block.n_free)} of {block.free_list.shape[0]} blocks free, "
          f"{int(block.unserved)} unserved rows")


if __name__ == "__main__":
    main()
