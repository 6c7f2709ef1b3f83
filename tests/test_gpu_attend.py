"""Attention over a cache and a shared prompt against the plain form in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TREE = [-1, 0, 0, 1, 1, 2, 3]


def _rows(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(torch.bfloat16)


class Case:
    """A batch of sequences with `lens` committed slots and `counts` new rows that continue `prompt` slots."""

    def __init__(self, seed, heads, kv_heads, dim, lens, counts, prompt=None, q8=False, prompt_q8=False, page=None,
                 parents=None, cap=None, dirty=False, layers=1, layer=0, max_rows=256, max_batch=None):
        from _attend_util import head_model, rows8
        from speculative_decoding_verify_04_gb300 import spec
        g = torch.Generator().manual_seed(seed)
        self.lens, self.counts, self.parents, self.layer = lens, counts, parents, layer
        self.H, self.Hkv, self.hd = heads, kv_heads, dim
        B, T = len(lens), sum(counts)
        self.model = head_model(heads, kv_heads, dim, layers=layers, max_rows=max_rows, max_batch=max_batch or B)
        cap = cap or max(n + c for n, c in zip(lens, counts)) + 3
        self.kv = spec.KVCache(self.model, B, cap, page=page, q8=q8)
        held = (lambda x: torch.from_numpy(rows8(x.double().numpy())[2])) if q8 else (lambda x: x.double())
        held_p = (lambda x: torch.from_numpy(rows8(x.double().numpy())[2])) if prompt_q8 else (lambda x: x.double())
        if dirty:
            # every slot of every layer holds NaN or an infinity before the real rows come
            for b in range(B):
                bad = torch.full((layers, cap, kv_heads, dim), math.nan)
                bad[:, ::2] = math.inf
                bad = bad.to(torch.bfloat16).cuda()
                if page is None:
                    self.kv.import_rows(b, 0, bad, bad)
        self.keys, self.vals = [], []
        for b, n in enumerate(lens):
            k, v = _rows(g, n, kv_heads, dim), _rows(g, n, kv_heads, dim)
            if n:
                self.kv.import_rows(b, layer, k[None].cuda(), v[None].cuda())
            self.keys.append(held(k))
            self.vals.append(held(v))
        self.kv.set_lengths(lens)
        self.prompt = None
        if prompt is not None:
            cap_p = prompt + 5
            self.prompt = spec.KVCache(self.model, 2 if (max_batch or B) > 1 else 1, cap_p, page=page, q8=prompt_q8)
            self.pseq = self.prompt.batch - 1
            if dirty and page is None:
                bad = torch.full((layers, cap_p, kv_heads, dim), math.nan, dtype=torch.bfloat16).cuda()
                for b in range(self.prompt.batch):
                    self.prompt.import_rows(b, 0, bad, bad)
            k, v = _rows(g, prompt, kv_heads, dim), _rows(g, prompt, kv_heads, dim)
            if prompt:
                self.prompt.import_rows(self.pseq, layer, k[None].cuda(), v[None].cuda())
            self.prompt.set_lengths([0] * self.pseq + [prompt])
            self.kv.set_prefix(self.prompt, self.pseq)
            self.pk, self.pv = held_p(k), held_p(v)
        self.q = _rows(g, T, heads, dim, scale=2.0)
        self.k, self.v = _rows(g, T, kv_heads, dim), _rows(g, T, kv_heads, dim)
        self.nk, self.nv = held(self.k), held(self.v)

    def run(self, q=None, k=None, v=None, out=None):
        from speculative_decoding_verify_04_gb300 import spec
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        spec.spec_attend(self.kv, self.layer, self.counts, q, out, k=self.k.cuda() if k is None else k,
                         v=self.v.cuda() if v is None else v, tree_parent=self.parents)
        return out

    def check(self, out, floor=0.0):
        from _attend_util import attend64, attend_tol, chain_mask, tree_mask
        out = out.double().cpu()
        r0 = 0
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            rows = slice(r0, r0 + c)
            r0 += c
            if not c:
                continue
            keys, vals = [self.keys[b], self.nk[rows]], [self.vals[b], self.nv[rows]]
            P = 0
            if self.prompt is not None:
                keys, vals = [self.pk] + keys, [self.pv] + vals
                P = self.pk.shape[0]
            sees = np.ones((c, P + n + c), dtype=bool)
            sees[:, P + n:] = tree_mask(self.parents) if self.parents else chain_mask(c)
            ref, mass, big = attend64(self.q[rows].double(), torch.cat(keys), torch.cat(vals),
                                      1.0 / math.sqrt(self.hd), sees)
            tol = attend_tol(ref, mass, big, self.hd)
            # f32 sums of values far below the largest lose what lies 2^-24 under it; and each of a row's n products
            # p v (p at most 1 before the division by a sum of at least 1) may be flushed to zero below 2^-126
            tol = tol + sees.shape[1] * 2.0 ** -126 + floor + 2.0 ** -22 * torch.cat(vals).abs().amax() * (floor > 0)
            off = (out[rows] - ref).abs() - tol
            assert not torch.isnan(out[rows]).any(), f"sequence {b}: NaN"
            assert off.max() <= 0, f"sequence {b}: {off.max()} over the bound"
        assert self.model.device_error() == 0


@pytest.mark.parametrize("q8,prompt_q8", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 4), (64, 16, 4), (128, 8, 2), (128, 6, 2), (64, 5, 1), (128, 32, 32)])
def test_chains_over_a_prompt(dim, heads, kv_heads, q8, prompt_q8):
    c = Case(1, heads, kv_heads, dim, [17, 0, 64, 1], [5, 3, 1, 4], prompt=129, q8=q8, prompt_q8=prompt_q8)
    c.check(c.run())


@pytest.mark.parametrize("prompt", [0, 1, 15, 16, 63, 64, 65, 127, 128, 255, 257, 1000])
@pytest.mark.parametrize("q8", [False, True])
def test_prompt_lengths(prompt, q8):
    c = Case(2, 8, 2, 128, [3, 70], [2, 5], prompt=prompt, q8=q8, prompt_q8=q8)
    c.check(c.run())


@pytest.mark.parametrize("prompt", [0, 1, 15, 63, 64, 65, 127, 128, 129, 255, 257, 700])
@pytest.mark.parametrize("q8,dim,page", [(False, 64, None), (True, 128, None), (False, 128, 64), (True, 64, 128)])
def test_prompt_lengths_under_many_vectors(prompt, q8, dim, page):
    """More than 64 query vectors a KV head; what lies behind the lengths is NaN or an infinity."""
    c = Case(9, 16, 2, dim, [3, 70, 0], [6, 5, 1], prompt=prompt, q8=q8, prompt_q8=q8, page=page, dirty=True)
    c.check(c.run())


@pytest.mark.parametrize("T,prompt", [(4, 300), (5, 300), (8, 1000), (15, 1000), (16, 1000), (17, 300)])
@pytest.mark.parametrize("q8,prompt_q8", [(False, True), (True, False), (True, True)])
def test_prompts_under_up_to_68_vectors(T, prompt, q8, prompt_q8):
    """One to five blocks of 16 query vectors over a short prompt, and the first size past them."""
    c = Case(10, 8, 2, 128, [20, 300], [T - 1, 1], prompt=prompt, q8=q8, prompt_q8=prompt_q8)
    c.check(c.run())


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 700])
@pytest.mark.parametrize("q8", [False, True])
def test_own_lengths_without_a_prompt(n, q8):
    c = Case(3, 4, 2, 64, [n, 0], [1, 4], q8=q8)
    c.check(c.run())


@pytest.mark.parametrize("page", [64, 128])
@pytest.mark.parametrize("q8,prompt_q8", [(False, False), (True, True)])
@pytest.mark.parametrize("dim", [64, 128])
def test_paged_trees(page, q8, prompt_q8, dim):
    c = Case(4, 8, 2, dim, [0, 60, 130, 64], [7] * 4, prompt=200, q8=q8, prompt_q8=prompt_q8, page=page, parents=TREE)
    c.check(c.run())


def test_64_rows_and_sequences_without_rows():
    c = Case(5, 4, 1, 64, [5, 9, 0, 33], [64, 0, 1, 0], prompt=100)
    c.check(c.run())


@pytest.mark.parametrize("q8", [False, True])
def test_a_long_chain_of_64_tree_rows(q8):
    parents = [-1] + list(range(63))
    c = Case(6, 2, 1, 128, [40], [64], prompt=300, q8=q8, parents=parents)
    c.check(c.run())


@pytest.mark.parametrize("rows,prompt", [(1, 2500), (3, 1500), (9, 900), (40, 600)])
@pytest.mark.parametrize("q8", [False, True])
def test_many_query_vectors(rows, prompt, q8):
    """From a few to several tiles of query vectors a KV head, over several ranges of the prompt."""
    B = 6
    c = Case(7, 16, 4, 128, [11 * b for b in range(B)], [max(1, rows - b) for b in range(B)], prompt=prompt,
             q8=q8, prompt_q8=q8)
    c.check(c.run())


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads,B,rows,prompt", [(128, 32, 8, 64, 8, 6001), (64, 16, 4, 40, 7, 5000),
                                                              (128, 8, 8, 3, 40, 9000), (64, 32, 1, 64, 4, 3000)])
def test_long_prompts_and_many_tiles(dim, heads, kv_heads, B, rows, prompt, q8):
    """Enough key tiles and tiles of query vectors that every SM works through several; ten calls, each against 64
    bits (computed on the GPU), all of the same bits."""
    from _attend_util import attend_tol, rows8
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(20, heads, kv_heads, dim, [0] * B, [rows] * B, prompt=1, max_rows=B * rows, max_batch=B)
    g = torch.Generator(device="cuda").manual_seed(21)
    k, v = (torch.randn(prompt, kv_heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pre = spec.KVCache(c.model, 1, prompt + 3, q8=q8)
    pre.import_rows(0, 0, k[None], v[None])
    pre.set_lengths([prompt])
    c.kv.set_prefix(pre, 0)
    held = pre.export_rows(0, 0, 1, 0, prompt) if q8 else (k[None], v[None])
    if q8:                                                  # a stretch of it against the definition
        assert torch.equal(held[0][0, :50].double().cpu(), torch.from_numpy(rows8(k[:50].double().cpu().numpy())[2]))
    G, T = heads // kv_heads, B * rows
    scale = 1.0 / math.sqrt(dim)
    q = c.q.cuda().double().view(B, rows, kv_heads, G, dim)
    pk, pv = (x[0].double() for x in held)
    nk, nv = (x.cuda().double().view(B, rows, kv_heads, dim) for x in (c.k, c.v))
    hide = ~torch.ones(rows, rows, dtype=torch.bool, device="cuda").tril()
    ref, mass, big = (torch.empty(T, heads, d, dtype=torch.float64, device="cuda") for d in (dim, dim, 1))
    for h in range(kv_heads):
        qh = q[:, :, h]
        s = torch.cat([torch.einsum("brgd,kd->brgk", qh, pk[:, h]),
                       torch.einsum("brgd,bkd->brgk", qh, nk[:, :, h]).masked_fill(hide[None, :, None], -math.inf)], -1) * scale
        p = torch.softmax(s, -1)
        hs = slice(h * G, (h + 1) * G)
        for out, vals, new in ((ref, pv[:, h], nv[:, :, h]), (mass, pv[:, h].abs(), nv[:, :, h].abs())):
            o = torch.einsum("brgk,kd->brgd", p[..., :prompt], vals) + torch.einsum("brgk,bkd->brgd", p[..., prompt:], new)
            out[:, hs] = o.reshape(T, G, dim)
        top = torch.maximum(torch.einsum("brgd,kd->brgk", qh.abs(), pk[:, h].abs()).amax(-1),
                            torch.einsum("brgd,bkd->brgk", qh.abs(), nk[:, :, h].abs()).amax(-1)) * scale
        big[:, hs, 0] = top.reshape(T, G)
        del s, p
    tol = attend_tol(ref, mass, big[..., 0], dim)
    first = None
    for _ in range(10):
        out = c.run()
        assert ((out.double() - ref).abs() <= tol).all()
        first = out if first is None else first
        assert torch.equal(first, out)
    assert c.model.device_error() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q8", [False, True])
def test_what_lies_behind_the_lengths_does_not_show(q8, dim):
    """Slots past the committed lengths hold NaN and infinities; so do the other sequences of the prompt's cache."""
    c = Case(8, 8, 4, dim, [0, 5, 70], [2, 3, 1], prompt=133, q8=q8, prompt_q8=q8, dirty=True, layers=2, layer=1)
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scales", ["small", "large", "wide", "zeros", "tiny"])
@pytest.mark.parametrize("rows", [1, 12])
def test_8_bit_rows_of_all_magnitudes(dim, scales, rows):
    """Exponents inside and outside of what half precision holds, rows of zeros among others and alone: the
    prompt's tiles change their operands' type, the row kernel its references."""
    from _attend_util import rows8
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(30, 8, 2, dim, [9, 40, 100], [rows] * 3, prompt=300, q8=True, prompt_q8=True)
    g = torch.Generator().manual_seed(31)

    def f(n):
        e = {"small": lambda: torch.randint(-16, -9, (n, 2, 1), generator=g), "large": lambda: torch.randint(0, 5, (n, 2, 1), generator=g),
             "wide": lambda: torch.randint(-30, 14, (n, 2, 1), generator=g), "zeros": lambda: torch.randint(-200, 2, (n, 2, 1), generator=g),
             "tiny": lambda: torch.full((n, 2, 1), -124)}[scales]()
        x = torch.randn(n, 2, dim, generator=g).double() * torch.exp2(e.double())
        return x.float().to(torch.bfloat16)

    # keys of ordinary size (the scores must not saturate), values of all sizes
    k, v = _rows(g, 300, 2, dim), f(300)
    c.prompt.import_rows(c.pseq, 0, k[None].cuda(), v[None].cuda())
    c.pk, c.pv = (torch.from_numpy(rows8(x.double().numpy())[2]) for x in (k, v))
    for b, n in enumerate(c.lens):
        v = f(n)
        c.kv.import_rows(b, 0, (c.keys[b].to(torch.bfloat16))[None].cuda(), v[None].cuda())
        c.keys[b] = torch.from_numpy(rows8(c.keys[b].numpy())[2])
        c.vals[b] = torch.from_numpy(rows8(v.double().numpy())[2])
    c.v = f(3 * rows)
    c.nv = torch.from_numpy(rows8(c.v.double().numpy())[2])
    c.check(c.run(), floor=2.0 ** -100 if scales in ("zeros", "wide") else 0.0)


def test_rows_of_a_fused_projection():
    """q, k and v as column ranges of one [T, (H + 2 Hkv) hd] buffer, at an odd element offset (no 16-byte alignment)."""
    for q8 in (False, True):
        for shift in (0, 1):
            c = Case(9, 4, 2, 64, [20, 3], [3, 2], prompt=50, q8=q8)
            T, w = 5, 8 * 64
            flat = torch.zeros(T * (w + 3) + shift, dtype=torch.bfloat16, device="cuda")
            buf = flat[shift:].view(T, w + 3)
            q, k, v = (buf[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 256), (256, 384), (384, 512)))
            q.copy_(c.q)
            k.copy_(c.k)
            v.copy_(c.v)
            big = torch.full((T + 2, 4 * 64 + 5), 3.0, dtype=torch.bfloat16, device="cuda")
            out = big[:T, 1:257].unflatten(1, (4, 64))
            c.run(q, k, v, out)
            c.check(out)
            # nothing around the rows is touched
            assert (big[T:] == 3).all() and (big[:, 0] == 3).all() and (big[:, 257:] == 3).all()


def test_rows_written_once_and_read_again():
    """k and v given: written; not given: the slots are read as they are.  Equal bits."""
    from speculative_decoding_verify_04_gb300 import spec
    for q8 in (False, True):
        c = Case(10, 4, 2, 64, [20, 3], [3, 2], prompt=50, q8=q8)
        a = c.run()
        b = torch.empty_like(a)
        spec.spec_attend(c.kv, 0, c.counts, c.q.cuda(), b)
        assert torch.equal(a, b)
        spec.kv_commit(c.kv, torch.tensor([2, 1], dtype=torch.int32, device="cuda"))
        assert c.kv.get_lengths() == [23, 5]
        k, _ = c.kv.export_rows(0, 0, 1, 20, 3)
        assert torch.equal(k[0].double().cpu(), c.nk[:3])


def test_repeats_give_the_same_bits():
    c = Case(11, 16, 4, 128, [100, 30, 0], [5, 4, 3], prompt=1000, q8=True)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())


def test_captured_and_replayed_after_the_lengths_moved():
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(12, 8, 2, 64, [10, 40], [2, 2], prompt=90, cap=80)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(q, k, v, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            spec.spec_attend(c.kv, 0, c.counts, q, out, k=k, v=v)
    torch.cuda.synchronize()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)
    # the sequences grow by their two rows; the next replay writes and sees the slots behind them
    c.kv.set_lengths([12, 42])
    c.keys = [torch.cat([x, c.nk[2 * b:2 * b + 2]]) for b, x in enumerate(c.keys)]
    c.vals = [torch.cat([x, c.nv[2 * b:2 * b + 2]]) for b, x in enumerate(c.vals)]
    c.lens = [12, 42]
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


@pytest.mark.parametrize("prompt_q8", [False, True])
def test_calls_in_a_row_over_two_caches(prompt_q8):
    """Two caches of one model behind one prompt, called in turn without a wait, eagerly and in a graph: the kernels
    of neighbouring calls overlap and share the workspace, and every output has the bits of a call on its own."""
    from speculative_decoding_verify_04_gb300 import spec
    B, rows = 12, 6
    c = Case(41, 16, 2, 128, [37 * b for b in range(B)], [rows] * B, prompt=3001, q8=True, prompt_q8=prompt_q8)
    g = torch.Generator(device="cuda").manual_seed(42)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    other = spec.KVCache(c.model, B, 700)
    for b in range(B):
        other.import_rows(b, 0, r(1, 600 - 50 * b, 2, 128), r(1, 600 - 50 * b, 2, 128))
    other.set_lengths([600 - 50 * b for b in range(B)])
    other.set_prefix(c.prompt, c.pseq)
    T = B * rows
    calls = [(c.kv, c.q.cuda(), c.k.cuda(), c.v.cuda()), (other, r(T, 16, 128), r(T, 2, 128), r(T, 2, 128))]

    def run(i):
        kv, q, k, v = calls[i]
        out = torch.full_like(q, 7.0)
        spec.spec_attend(kv, 0, [rows] * B, q, out, k=k, v=v)
        return out

    want = []
    for i in range(2):
        want.append(run(i))
        torch.cuda.synchronize()
    c.check(want[0])
    outs = [(i & 1, run(i & 1)) for i in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(want[i], o) for i, o in outs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = [(i & 1, run(i & 1)) for i in range(5)]
        for _ in range(10):
            for _, o in outs:
                o.fill_(3.0)
            graph.replay()
            assert all(torch.equal(want[i], o) for i, o in outs)
    torch.cuda.synchronize()
    assert c.model.device_error() == 0


def test_on_another_stream():
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(13, 8, 2, 64, [10, 40], [2, 2], prompt=90, q8=True)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    spec.spec_attend(c.kv, 0, c.counts, q, out, k=k, v=v, stream=s)
    s.synchronize()
    c.check(out)


def test_no_room_is_reported():
    """Rows past the capacity are dropped, the device error word says so, the rows that fit are right."""
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(14, 4, 2, 64, [10, 3], [1, 3], cap=13)
    c.check(c.run())
    c.kv.set_lengths([12, 12])
    out = c.run()
    torch.cuda.synchronize()
    assert c.model.device_error() & spec.DEVERR_CAPACITY
    assert out.shape[0] == 4


def test_minus_infinity_keys_and_nan_rows():
    """A key with -inf scores has no weight; a row whose every key has, or that meets a NaN key, is NaN."""
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(15, 2, 1, 64, [0], [3])
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0] = -math.inf
    k[2, 0, 5] = math.nan
    v = torch.arange(1, 4, device="cuda")[:, None, None].expand(3, 1, 64).to(torch.bfloat16)
    out = torch.empty_like(q)
    spec.spec_attend(c.kv, 0, [3], q, out, k=k, v=v.contiguous())
    out = out.float().cpu()
    assert torch.isnan(out[0]).all() and (out[1] == 2).all() and torch.isnan(out[2]).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 64), (2, 128), (8, 128)])
def test_a_new_rows_nan_stays_with_the_rows_that_see_it(q8, heads, dim):
    """A tree whose nodes 2 and 5 hold NaN and infinities in k and v: their descendants are NaN, the others are as
    if those rows were zeros (one and several query heads a KV head: both forms of the row kernel)."""
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(40, heads, 2, dim, [21], [7], prompt=30, q8=q8, parents=TREE)
    clean_k, clean_v = c.k.clone(), c.v.clone()
    clean_k[[2, 5]] = 0
    clean_v[[2, 5]] = 0
    want = c.run(k=clean_k.cuda(), v=clean_v.cuda())
    k, v = c.k.clone(), c.v.clone()
    k[2], v[2], v[5, 0, 3], v[5, 1, 7] = math.nan, math.nan, math.nan, math.nan
    if not q8:
        v[2, :, ::2] = math.inf
    got = c.run(k=k.cuda(), v=v.cuda())
    assert torch.isnan(got[[2, 5]].float()).all()
    assert torch.equal(got[[0, 1, 3, 4, 6]], want[[0, 1, 3, 4, 6]])
    assert c.model.device_error() == 0


@pytest.mark.parametrize("own_page,prompt_page", [(None, 64), (128, None), (64, 256)])
@pytest.mark.parametrize("q8,prompt_q8", [(False, True), (True, False)])
def test_caches_of_different_kinds(own_page, prompt_page, q8, prompt_q8):
    from _attend_util import rows8
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(41, 8, 2, 64, [70, 3], [6, 5], prompt=300, q8=q8, page=own_page)
    pre = spec.KVCache(c.model, 1, 320, page=prompt_page, q8=prompt_q8)
    g = torch.Generator().manual_seed(42)
    k, v = _rows(g, 300, 2, 64), _rows(g, 300, 2, 64)
    pre.import_rows(0, 0, k[None].cuda(), v[None].cuda())
    pre.set_lengths([300])
    c.kv.set_prefix(pre)
    f = (lambda x: torch.from_numpy(rows8(x.double().numpy())[2])) if prompt_q8 else (lambda x: x.double())
    c.pk, c.pv = f(k), f(v)
    c.check(c.run())


def test_refusals():
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    c = Case(16, 4, 2, 64, [3, 3], [2, 2], prompt=10)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)

    def bad(match, *a, **kw):
        with pytest.raises(spec.SpecError, match=match):
            spec.spec_attend(*a, **kw)

    bad("go together", c.kv, 0, [2, 2], q, out, k=k)
    bad("layer", c.kv, 1, [2, 2], q, out)
    bad("batch", c.kv, 0, [1, 1, 1], q, out)
    bad(r"\[0, 64\]", c.kv, 0, [65, 1], q.repeat(20, 1, 1), out.repeat(20, 1, 1))
    bad(r"\[0, 64\]", c.kv, 0, [-1, 3], q, out)
    bad("need a CUDA", c.kv, 0, [2, 2], q.float(), out)
    bad("need a CUDA", c.kv, 0, [2, 2], q[:3], out)
    bad("need a CUDA", c.kv, 0, [2, 2], q.transpose(1, 2), out)
    bad("tree_parent", c.kv, 0, [2, 2], q, out, tree_parent=[-1])
    bad("tree_parent", c.kv, 0, [2, 2], q, out, tree_parent=[0, 0])
    bad("tree_parent", c.kv, 0, [2, 2], q, out, tree_parent=[-1, 1])
    bad("node count", c.kv, 0, [2, 1], q, out, tree_parent=[-1, 0])
    spec.spec_attend(c.kv, 0, [0, 0], q, out)            # nothing to do
    for kv, pre, seq, match in ((c.kv, c.kv, 0, "its own prefix"), (c.kv, c.prompt, 9, "out of range"),
                                (c.prompt, spec.KVCache(c.model, 1, 8), 0, "is a prefix itself")):
        with pytest.raises(spec.SpecError, match=match):
            kv.set_prefix(pre, seq)
    third = spec.KVCache(c.model, 1, 8)
    with pytest.raises(spec.SpecError, match="prefix of its own"):
        third.set_prefix(c.kv)
    other = head_model(4, 2, 64)
    with pytest.raises(spec.SpecError, match="another model"):
        third.set_prefix(spec.KVCache(other, 1, 8))
    f32 = head_model(4, 2, 64, dtype="f32")
    with pytest.raises(spec.SpecError, match="bf16 models only"):
        spec.KVCache(f32, 1, 8, q8=True)
    a, b = spec.KVCache(f32, 1, 8), spec.KVCache(f32, 1, 8)
    with pytest.raises(spec.SpecError, match="bf16 models only"):
        a.set_prefix(b)
    # a destroyed prompt stops the calls until another one, or none, is set
    c.check(c.run())
    c.prompt.close()
    bad("prefix was destroyed", c.kv, 0, [2, 2], q, out)
    c.kv.set_prefix(None)
    c.prompt = None
    c.check(c.run())
