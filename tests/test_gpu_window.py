"""Attention over a window with sinks against the plain form in 64 bits, alone and in the forward calls."""
import math

import numpy as np
import pytest
import torch

from oracle.decoder import Decoder
from test_gpu_attend import Case

pytestmark = pytest.mark.gpu

TREE = [-1, 0, 0, 1, 1, 2, 3, 6, 7]


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def window_sees(P, n, c, parents, window, sinks):
    """[c, P + n + c]: what row j sees of the prompt, its sequence's slots and the call's rows."""
    from _attend_util import chain_mask, tree_mask
    d = np.array(depths(parents[:c]) if parents else range(c))
    index = np.concatenate([np.arange(P + n), P + n + d])
    sees = np.ones((c, P + n + c), dtype=bool)
    sees[:, P + n:] = tree_mask(parents) if parents else chain_mask(c)
    near = (P + n + d)[:, None] - index[None] < window
    return sees & (near | (index < sinks)[None])


class WindowCase(Case):
    def __init__(self, seed, *args, window, sinks=0, **kw):
        super().__init__(seed, *args, **kw)
        self.window, self.sinks = window, sinks
        self.kv.set_window(window, sinks)

    def check(self, out):
        from _attend_util import attend64, attend_tol
        out = out.double().cpu()
        r0 = 0
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            rows = slice(r0, r0 + c)
            r0 += c
            if not c:
                continue
            keys, vals, P = [self.keys[b], self.nk[rows]], [self.vals[b], self.nv[rows]], 0
            if self.prompt is not None:
                keys, vals, P = [self.pk] + keys, [self.pv] + vals, self.pk.shape[0]
            sees = window_sees(P, n, c, self.parents, self.window, self.sinks)
            ref, mass, big = attend64(self.q[rows].double(), torch.cat(keys), torch.cat(vals), 1.0 / math.sqrt(self.hd), sees)
            tol = attend_tol(ref, mass, big, self.hd) + sees.shape[1] * 2.0 ** -126
            assert not torch.isnan(out[rows]).any(), f"sequence {b}: NaN"
            off = (out[rows] - ref).abs() - tol
            assert off.max() <= 0, f"sequence {b}: {off.max()} over the bound"
        assert self.model.device_error() == 0


LAYOUTS = [(64, 4, 4), (64, 16, 4), (128, 8, 2), (128, 6, 2), (64, 5, 1), (128, 32, 32)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", LAYOUTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (17, 4), (40, 20), (1000, 4)])
def test_chains(dim, heads, kv_heads, window, sinks, q8):
    c = WindowCase(1, heads, kv_heads, dim, [70, 0, 16, 133], [5, 3, 1, 4], window=window, sinks=sinks, q8=q8)
    c.check(c.run())


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 255, 256, 700])
@pytest.mark.parametrize("window,sinks", [(1, 0), (15, 1), (16, 16), (33, 17), (64, 40), (300, 64)])
@pytest.mark.parametrize("q8,rows", [(False, 1), (True, 1), (False, 9), (True, 9), (False, 64)])
def test_lengths(n, window, sinks, q8, rows):
    c = WindowCase(2, 8, 2, 64, [n, 3], [rows, 1], window=window, sinks=sinks, q8=q8, dirty=True)
    c.check(c.run())


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (3, 1), (5, 80), (70, 4), (500, 2)])
def test_paged_trees(page, q8, dim, window, sinks):
    """Windows shorter than the trees are deep, sinks among the trees' own rows, pages that end inside a window."""
    c = WindowCase(3, 8, 2, dim, [0, 60, 130, 64], [9] * 4, window=window, sinks=sinks, q8=q8, page=page, parents=TREE)
    c.check(c.run())


@pytest.mark.parametrize("prompt", [0, 1, 15, 16, 63, 64, 65, 200])
@pytest.mark.parametrize("q8,prompt_q8", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (8, 3), (40, 70), (100, 4), (90, 300)])
def test_windows_that_reach_into_a_prompt(prompt, q8, prompt_q8, window, sinks):
    c = WindowCase(4, 8, 2, 64, [17, 0, 64, 150], [5, 3, 1, 4], prompt=prompt, window=window, sinks=sinks, q8=q8,
                   prompt_q8=prompt_q8, page=64 if q8 and prompt_q8 else None, dirty=True)
    c.check(c.run())


@pytest.mark.parametrize("heads,kv_heads,rows", [(32, 8, 29), (16, 2, 13), (4, 4, 64), (8, 1, 33)])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("prompt", [None, 700])
def test_many_query_vectors(heads, kv_heads, rows, q8, prompt):
    parents = [-1] + [(i - 1) // 2 for i in range(1, rows)]
    c = WindowCase(5, heads, kv_heads, 128, [900, 0, 333, 64, 1500], [rows] * 5, window=800, sinks=5, q8=q8,
                   prompt=prompt, parents=parents, max_rows=5 * rows)
    c.check(c.run())


@pytest.mark.parametrize("q8", [False, True])
def test_64_rows_and_sequences_without_rows(q8):
    c = WindowCase(6, 4, 1, 64, [5, 9, 0, 333], [64, 0, 1, 0], window=30, sinks=4, q8=q8)
    c.check(c.run())
    c = WindowCase(6, 2, 1, 128, [40, 2], [64, 64], window=30, sinks=4, q8=q8, parents=[-1] + list(range(63)))
    c.check(c.run())


@pytest.mark.parametrize("rows", [1, 4, 20])
@pytest.mark.parametrize("q8", [False, True])
def test_what_a_row_does_not_see_has_no_influence(rows, q8):
    """NaN and infinities in the slots before the windows, between sinks and window, in those that only the first
    rows see, and behind the sequence."""
    window, sinks, n = 37, 3, 150
    c = WindowCase(7, 8, 2, 64, [n, 90], [rows, rows], window=window, sinks=sinks, q8=q8)
    clean = c.run()
    c.check(clean)
    for bad in (math.nan, math.inf, -math.inf):
        for b, n_b in enumerate(c.lens):
            lo = n_b - window + 1                            # the first slot that the first row sees
            x = torch.full((1, lo - sinks, 2, 64), bad, dtype=torch.bfloat16, device="cuda")
            c.kv.import_rows(b, 0, x, x, slot0=sinks)
        assert torch.equal(c.run(), clean)
        if rows > 1 and not (q8 and math.isinf(bad)):       # (an 8-bit cache holds infinities as numbers)
            # row 0 alone sees slot lo: its result shows it, the others' do not
            x = torch.full((1, 1, 2, 64), bad, dtype=torch.bfloat16, device="cuda")
            c.kv.import_rows(1, 0, x, x, slot0=c.lens[1] - window + 1)
            got = c.run()
            assert not torch.isfinite(got[rows].float()).any()
            assert torch.equal(got[:rows], clean[:rows]) and torch.equal(got[rows + 1:], clean[rows + 1:])
            x = c.keys[1][c.lens[1] - window + 1].to(torch.bfloat16).cuda()[None, None]
            y = c.vals[1][c.lens[1] - window + 1].to(torch.bfloat16).cuda()[None, None]
            c.kv.import_rows(1, 0, x.contiguous(), y.contiguous(), slot0=c.lens[1] - window + 1)


def test_a_row_without_finite_scores_is_nan():
    c = WindowCase(8, 4, 2, 64, [50], [2], window=10, sinks=2)
    k = c.k.clone()
    k[:, 0] = math.inf                                       # +inf scores in KV head 0
    q = torch.ones_like(c.q)
    out = c.run(q=q.cuda(), k=k.cuda())
    assert torch.isnan(out[:, :2].float()).all() and torch.isfinite(out[:, 2:].float()).all()


def test_layers_differ_and_windows_go_away():
    """A window for the middle layer of three; the others see everything, bit for bit as before; then none."""
    full = Case(9, 8, 2, 64, [200, 31], [5, 5], layers=3, layer=1)
    before = full.run()
    full.check(before)
    full.kv.set_window(20, 2, layer0=0, n_layers=1)
    assert torch.equal(full.run(), before)
    full.kv.set_window(20, 2, layer0=1, n_layers=1)
    windowed = full.run()
    assert not torch.equal(windowed, before)
    c = WindowCase(9, 8, 2, 64, [200, 31], [5, 5], layers=3, layer=1, window=20, sinks=2)
    assert torch.equal(c.run(), windowed)
    c.check(windowed)
    full.kv.set_window(0)
    assert torch.equal(full.run(), before)


def test_lengths_move_under_a_captured_call():
    c = WindowCase(10, 8, 2, 64, [100, 40], [3, 3], window=30, sinks=4)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    c.run(q, k, v, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(q, k, v, out)
    for lens in ([100, 40], [17, 0], [60, 39]):
        c.kv.set_lengths(lens)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        again = torch.empty_like(out)
        c.run(q, k, v, again)
        assert torch.equal(out, again)


def test_slots_past_32_bits():
    """A cache of more than 2^31 values a layer: the window lies behind them."""
    from _attend_util import head_model, attend64, attend_tol
    from speculative_decoding_verify_04_gb300 import spec
    model = head_model(8, 8, 128, max_rows=4, max_batch=2)
    n, W = (1 << 20) + 77, 500
    kv = spec.KVCache(model, 2, n + 8)                       # 2 x 8 x 2^20 x 128 values
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(W + 3, 8, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kv.import_rows(1, 0, k[None, :W], v[None, :W], slot0=n - W)
    kv.set_lengths([0, n])
    kv.set_window(W)
    q = torch.randn(3, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    spec.spec_attend(kv, 0, [0, 3], q, out, k=k[W:], v=v[W:])
    sees = window_sees(0, W, 3, None, W, 0)
    ref, mass, big = attend64(q.double().cpu(), k.double().cpu(), v.double().cpu(), 128 ** -0.5, sees)
    assert ((out.double().cpu() - ref).abs() - attend_tol(ref, mass, big, 128)).max() <= 0


# ---------------------------------------------------------------------------
# the forward calls

class WindowDecoder(Decoder):
    """The oracle's decoder with windows (window, sinks) by layer."""

    def __init__(self, dec, windows):
        super().__init__(dec.shape, dec.w)
        self.windows = windows

    def layer(self, l, h, pos, slots, visible, cache):
        if l in self.windows:
            window, sinks = self.windows[l]
            at = {int(s): int(p) for s, p in zip(slots, pos)}
            visible = [np.array([s for s in vis if (i := at.get(int(s), int(s))) < sinks or int(p) - i < window])
                       for p, vis in zip(pos, visible)]
        return super().layer(l, h, pos, slots, visible, cache)

    def _attend_causal_block(self, q, kc, vc, pos, slots, visible):
        return np.stack([self._attend(q[t], kc, vc, visible[t]) for t in range(q.shape[0])])


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hd,B,page,windows", [
    (64, 1, None, {0: (20, 4), 1: (20, 4), 2: (20, 4)}), (128, 3, 64, {0: (20, 4), 1: (20, 4), 2: (20, 4)}),
    (64, 3, 64, {1: (7, 0)}), (64, 7, None, {0: (3, 1), 2: (33, 2)})])
def test_rounds_match_the_oracle(hd, B, page, windows):
    """Prefill, layer-skip draft, verification and commit over windows, in all layers or in some."""
    from _gpu_util import cuda_i32, lib, model_pair, top_gap
    from oracle import spec as OS
    from oracle.accept import accept_greedy_chain, argmax_lowest
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens
    lib()
    sh = ModelShape(3, 256, 8 if hd == 64 else 4, 2, hd, 512, 2048, 1, "bf16")
    model, dec, shape = model_pair(sh, seed=3, max_rows=64, max_batch=8, max_position=512)
    dec = WindowDecoder(dec, windows)
    prompts = [make_tokens(70 + 9 * b, shape.vocab, seed=5 + b) for b in range(B)]
    kv = spec.KVCache(model, B, 200, page=page)
    for l, (w, s) in windows.items():
        kv.set_window(w, s, layer0=l, n_layers=1)
    t0, k = _i32(B), 4
    for b, p in enumerate(prompts):
        spec.spec_prefill(model, kv, b, cuda_i32(p), next_tok=t0[b:b + 1])
    cand, acc, nxt = _i32(B, k + 1), _i32(B), _i32(B)
    hL = torch.empty(B, k + 1, shape.d_model, device="cuda")
    logits = torch.empty(B, k + 1, shape.vocab, device="cuda")
    spec.spec_draft(model, kv, t0, k, cand, hL)
    spec.spec_verify(model, kv, [k + 1] * B, cand, k + 1, h_in=hL, h_stride=k + 1, logits=logits, acc_len=acc, next_tok=nxt)
    spec.kv_commit(kv, acc)
    for b, p in enumerate(prompts):
        cache = dec.new_cache(len(p) + 16)
        first = dec.prefill(cache, p)
        if top_gap(first) >= 2e-2:
            assert int(t0[b]) == argmax_lowest(first)
        c, got = cand[b].cpu().numpy(), logits[b].cpu().numpy()
        want = OS.verify(dec, cache, len(p), dec.embed(c), 0)
        assert np.abs(got - want).max() < 2e-2, b
        assert (int(acc[b]), int(nxt[b])) == accept_greedy_chain(list(c[1:]), got)
    assert kv.get_lengths() == [len(p) + int(a) + 1 for p, a in zip(prompts, acc.cpu())]
    assert model.device_error() == 0


@pytest.mark.parametrize("own_trees", [False, True])
def test_token_trees_match_the_oracle(own_trees):
    from _gpu_util import cuda_i32, lib, model_pair
    from oracle import spec as OS
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens, tree_parents
    lib()
    model, dec, shape = model_pair(ModelShape(3, 256, 8, 2, 64, 512, 2048, 1, "bf16"), seed=6, max_rows=64, max_batch=4,
                                   max_position=512)
    windows = {0: (2, 1), 1: (30, 0), 2: (3, 5)}
    dec = WindowDecoder(dec, windows)
    par = [int(p) for p in tree_parents([2, 2, 1])]
    N, B = len(par), 3
    kv = spec.KVCache(model, B, 120, page=64)
    for l, (w, s) in windows.items():
        kv.set_window(w, s, layer0=l, n_layers=1)
    prompts = [make_tokens(40 + 13 * b, shape.vocab, seed=8 + b) for b in range(B)]
    for b, p in enumerate(prompts):
        spec.spec_prefill(model, kv, b, cuda_i32(p))
    toks = np.stack([make_tokens(N, shape.vocab, seed=20 + b) for b in range(B)])
    logits, tk = torch.empty(B * N, shape.vocab, device="cuda"), cuda_i32(toks)
    if own_trees:
        spec.spec_verify_trees(model, kv, [N] * B, tk, N, cuda_i32(np.tile(par, (B, 1))), N, logits=logits)
    else:
        spec.spec_verify(model, kv, [N] * B, tk, N, tree_parent=par, logits=logits)
    got = logits.view(B, N, -1).cpu().numpy()
    for b, p in enumerate(prompts):
        cache = dec.new_cache(len(p) + 32)
        dec.prefill(cache, p)
        want = OS.verify(dec, cache, len(p), dec.embed(toks[b]), 0, par)
        assert np.abs(got[b] - want).max() < 2e-2
    assert model.device_error() == 0


def test_noalloc_verify_has_the_same_bits():
    from _gpu_util import cuda_i32, lib, model_pair
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens
    lib()
    model, _, shape = model_pair(ModelShape(3, 256, 8, 2, 64, 512, 2048, 1, "bf16"), seed=6, max_rows=64, max_batch=4,
                                 max_position=512)
    kv = spec.KVCache(model, 2, 120)
    kv.set_window(25, 3)
    for b in range(2):
        spec.spec_prefill(model, kv, b, cuda_i32(make_tokens(60 + b, shape.vocab, seed=b)))
    tk = cuda_i32(np.stack([make_tokens(5, shape.vocab, seed=30 + b) for b in range(2)]))
    out = []
    for f in (spec.spec_verify, spec.spec_verify_noalloc):
        logits = torch.empty(10, shape.vocab, device="cuda")
        f(model, kv, [5, 5], tk, 5, logits=logits)
        out.append(logits)
    assert torch.equal(*out)
