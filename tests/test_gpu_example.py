"""The serving operators and the MoE layer together, as examples/decode_block.py
runs them.

Tolerance, fixed before the first run: keys and values are E4M3 codes, each
within 2^-4 of its value (a block's largest value sets the scale, and values of
the same order are normal codes), so scores and values each move the result by
at most about 2^-4 of its rms: 2 * 2^-4 together."""
import importlib.util
import os

import pytest
import torch

from gen.configs import CONFIGS

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decode_block.py")
spec = importlib.util.spec_from_file_location("decode_block", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

LENS = (70, 1, 33, 200)


def _block(seed=0):
    return example.DecoderBlock(CONFIGS["tiny_b1"], len(LENS), seed=seed)


def _prompts():
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.randn(n, CONFIGS["tiny_b1"].d, generator=g, device="cuda").to(torch.bfloat16)
            for n in LENS]


def test_graph_replay_equals_eager_and_blocks_balance():
    steps = 20
    results = []
    for graph in (False, True):
        block = _block()
        out, load = example.generate(block, _prompts(), steps, graph)
        torch.cuda.synchronize()
        assert torch.isfinite(out).all()
        assert block.moe.status() == 0
        # the capture itself runs nothing: both have decoded `steps` tokens
        assert block.ctx_lens.tolist() == [n + steps for n in LENS]
        used = sum(-(-(n + steps) // block.cache.block_size) for n in LENS)
        total = block.free_list.shape[0]
        assert int(block.n_free) == total - used and int(block.unserved) == 0
        assert int(load.sum()) == sum(LENS) * block.cfg.top_k
        block.release(torch.ones(len(LENS), dtype=torch.bool, device="cuda"))
        assert int(block.n_free) == total and block.ctx_lens.tolist() == [0] * len(LENS)
        assert sorted(block.free_list.tolist()) == list(range(total))
        results.append(out)
    assert torch.equal(results[0], results[1])


def test_prefill_matches_attention_over_the_unrounded_values():
    block = _block()
    prompts = _prompts()
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    out = block.attend(torch.cat(prompts), lens, max(LENS)).double()
    at = 0
    for p in prompts:
        n, d = p.shape[0], block.head_dim
        qkv = (p.double() @ block.w_qkv.double().T).view(n, -1, d).transpose(0, 1)
        q, k, v = qkv.split([block.heads, block.kv_heads, block.kv_heads])
        group = block.heads // block.kv_heads
        k, v = (t.repeat_interleave(group, 0) for t in (k, v))
        s = q @ k.transpose(1, 2) * d ** -0.5
        s.masked_fill_(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
        want = (s.softmax(-1) @ v).transpose(0, 1)
        got = out[at:at + n]
        at += n
        rms = want.square().mean().sqrt()
        assert (got - want).square().mean().sqrt() <= 2 * 2 ** -4 * rms
