"""Prompts that fill a small part of their cache: every state that is joined was written by the call itself."""
import math

import numpy as np
import pytest
import torch

from _gpu_util import cuda_i32, lib, model_pair
from synthetic import ModelShape, make_tokens
from test_gpu_attend import Case, _rows
from test_gpu_shared_prompt import SHAPES, TOL, _round

pytestmark = pytest.mark.gpu


def _in_a_long_cache(c, seed, n, cap, q8, page, seqs=1, seq=0):
    """Gives the sequences of `c` a prompt of n slots at the start of a full cache of `cap` slots; returns the cache."""
    from _attend_util import rows8
    from speculative_decoding_verify_04_gb300 import spec
    pre = spec.KVCache(c.model, seqs, cap, page=page, q8=q8)
    g = torch.Generator().manual_seed(seed)
    k, v = _rows(g, n, c.Hkv, c.hd), _rows(g, n, c.Hkv, c.hd)
    gd = torch.Generator(device="cuda").manual_seed(seed + 1)
    full = [torch.randn(cap, c.Hkv, c.hd, generator=gd, device="cuda").to(torch.bfloat16) for _ in range(2)]
    for x, y in zip(full, (k, v)):
        x[:n] = y.cuda()
    pre.import_rows(seq, 0, full[0][None], full[1][None])
    held = (lambda x: torch.from_numpy(rows8(x.double().numpy())[2])) if q8 else (lambda x: x.double())
    c.pk, c.pv, c.prompt, c.pseq = held(k), held(v), pre, seq
    c.kv.set_prefix(pre, seq)
    return pre


# head layouts and batches whose lists go to the tile kernel: 256 vectors a KV head, 160, 20 and 384
LAYOUTS = {"32 heads over 8": (32, 8, 128, 8, 8), "16 over 4": (16, 4, 64, 8, 5), "8 full": (8, 8, 128, 4, 5),
           "16 over 2": (16, 2, 64, 6, 8)}


@pytest.mark.parametrize("layout,q8,page", [("32 heads over 8", False, None), ("32 heads over 8", True, 64),
                                            ("16 over 4", False, 128), ("16 over 4", True, None),
                                            ("8 full", False, None), ("16 over 2", True, 64)])
@pytest.mark.parametrize("cap", [4096, 32768])
@pytest.mark.parametrize("n", [129, 200, 300, 1000, 2000])
def test_a_short_prompt_in_a_long_cache(layout, q8, page, cap, n):
    """After calls over the whole cache, of the same rows and of fewer, a prompt of n slots gives what 64 bits say
    and the same bits again."""
    heads, kv_heads, dim, B, rows = LAYOUTS[layout]
    c = Case(50, heads, kv_heads, dim, [7 * b for b in range(B)], [rows] * B, prompt=1)
    pre = _in_a_long_cache(c, 51, n, cap, q8, page, seqs=2, seq=1)
    from speculative_decoding_verify_04_gb300 import spec
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    few = torch.empty_like(q)
    outs = []
    for fewer in (False, True):
        # the workspace as calls of other layouts leave it
        pre.set_lengths([0, cap])
        if fewer:
            spec.spec_attend(c.kv, 0, [rows - 1] * B, q, few, k=k, v=v)
        else:
            c.run(100 * q, k, v)
        pre.set_lengths([0, n])
        outs.append(c.run(q, k, v))
    c.check(outs[0])
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("n", [0, 1, 128, 129, 257, 1100])
def test_lengths_that_move_between_replays(n):
    """A captured call over a long prompt, replayed where the prompt has n slots."""
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(52, 16, 4, 64, [3 * b for b in range(8)], [4] * 8, prompt=1)
    pre = _in_a_long_cache(c, 53, n, 8192, False, None)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    pre.set_lengths([8192])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(q, k, v, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            spec.spec_attend(c.kv, 0, c.counts, q, out, k=k, v=v)
        graph.replay()
    torch.cuda.synchronize()
    pre.set_lengths([n])
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


@pytest.mark.parametrize("name", ["hd64", "hd128"])
@pytest.mark.parametrize("q8", [False, True])
def test_forward_calls_over_a_short_prompt_in_a_long_cache(name, q8):
    """Prefill, draft and verification: the logits over a part-filled prompt cache, after rounds over a long prompt,
    are those over a prompt cache of the prompt's length."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES[name], seed=60, max_rows=64, max_batch=8, max_position=8192)
    B, n = 7, 300
    prompt = make_tokens(n, shape.vocab, seed=61)
    suffixes = [make_tokens(1 + 9 * b, shape.vocab, seed=62 + b) for b in range(B)]
    tight, roomy = spec.KVCache(model, 1, n, q8=q8), spec.KVCache(model, 1, 6000, q8=q8)
    spec.spec_prefill(model, tight, 0, cuda_i32(prompt))
    rows = tight.export_rows(0, 0, shape.n_layers, 0, n)
    g = torch.Generator(device="cuda").manual_seed(63)
    noise = [torch.randn(shape.n_layers, 6000, shape.n_kv_heads, shape.head_dim, generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    for x, y in zip(noise, rows):
        x[:, :n] = y
    roomy.import_rows(0, 0, *noise)
    got = []
    for pre in (tight, roomy):
        # rounds over the whole long cache leave their states behind
        roomy.set_lengths([6000])
        other = spec.KVCache(model, B, 64, q8=q8)
        other.set_prefix(roomy)
        t0 = cuda_i32(list(range(B)))
        _round(model, shape, other, t0, 4)
        roomy.set_lengths([n])
        kv = spec.KVCache(model, B, 160, q8=q8)
        kv.set_prefix(pre)
        first = torch.empty(B, shape.vocab, device="cuda")
        for b, s in enumerate(suffixes):
            spec.spec_prefill(model, kv, b, cuda_i32(s), last_logits=first[b])
        # the same tokens for both: no draft of its own
        cand = cuda_i32(np.stack([make_tokens(5, shape.vocab, seed=80 + b) for b in range(B)]))
        logits = torch.empty(B, 5, shape.vocab, device="cuda")
        spec.spec_verify(model, kv, [5] * B, cand, 5, logits=logits)
        r = _round(model, shape, kv, t0, 4)
        got.append([first, logits, r["hL"][:, 0]])       # (later rows follow the tokens that were drafted)
    for a, b in zip(*got):
        assert (a - b).abs().max() < TOL
    assert model.device_error() == 0
