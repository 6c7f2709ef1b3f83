"""Rotary positions of rows against the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TREE = [-1, 0, 0, 1, 1, 2, 3, 6]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from _gpu_util import lib
    lib()


def pair_axes(sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a] > 0:
                out.append(a)
                left[a] -= 1
    return out


def rope64(x, pos, sections, interleaved, theta):
    """x [T, H, hd] float64 numpy, pos [axes, T]."""
    n = sum(sections)
    axes = pair_axes(sections, interleaved)
    y = x.copy()
    for i in range(n):
        a = pos[axes[i]].astype(np.float64) * theta ** (-i / n)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y[..., i] = x[..., i] * c - x[..., i + n] * s
        y[..., i + n] = x[..., i + n] * c + x[..., i] * s
    return y


def bound(x, y, n, bf16):
    """An angle is off by 2^-28 and by 2^-52 of itself in either form (below 2^-21 here, at 2^31), cosine and sine by 2^-23
    each, the two products and their sum by three roundings of 2^-24 of |x_i| + |x_{i+n}|; then one rounding."""
    pair = np.abs(x[..., :n]) + np.abs(x[..., n:2 * n])
    err = np.zeros_like(x)
    err[..., :n] = err[..., n:2 * n] = pair * (2.0 ** -28 + 2.0 ** -21 + 2.0 ** -23 + 3 * 2.0 ** -24)
    return err + np.abs(y) * (2.0 ** -8 if bf16 else 0.0)


def run(q, k, sections=None, pos=None, interleaved=False, theta=10000.0, in_place=False, **kw):
    from speculative_decoding_verify_04_gb300 import spec
    qo = q if in_place else torch.full_like(q, 7.0)
    ko = None if k is None else (k if in_place else torch.full_like(k, 7.0))
    spec.spec_rope(q, qo, k, ko, theta=theta, positions=pos, sections=sections, interleaved=interleaved, **kw)
    return qo, ko


def check(x, y, pos, sections, interleaved, theta):
    a = x.double().cpu().numpy()
    want = rope64(a, pos, sections, interleaved, theta)
    off = np.abs(y.double().cpu().numpy() - want) - bound(a, want, sum(sections), x.dtype == torch.bfloat16)
    assert off.max() <= 0, off.max()
    n2 = 2 * sum(sections)
    assert torch.equal(x[..., n2:], y[..., n2:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 3, 64, 1025, 4097])
@pytest.mark.parametrize("hd,sections,interleaved", [
    (64, [32], False), (128, [64], False), (128, [16, 24, 24], False), (128, [24, 20, 20], True), (64, [11, 8, 5], True),
    (64, [11, 8, 5], False), (64, [0, 16, 0, 8], True), (128, [7], False), (80, [40], False), (6, [1, 1], False),
    (256, [128], False)])
def test_rows_by_positions(dtype, T, hd, sections, interleaved):
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, 5, hd, generator=g, device="cuda").to(dtype)
    k = torch.randn(T, 2, hd, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 200000, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = run(q, k, sections, pos, interleaved)
    for x, y in ((q, qo), (k, ko)):
        check(x, y, pos.cpu().numpy(), sections, interleaved, 10000.0)


@pytest.mark.parametrize("pos", [0, 1, -1, -77777, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("theta", [1.0, 10000.0, 1e6, 5e8])
def test_positions_of_any_size(pos, theta):
    q = torch.randn(2, 3, 128, generator=torch.Generator().manual_seed(2)).cuda()
    p = torch.tensor([pos, max(pos - 1, -2 ** 31)], dtype=torch.int32, device="cuda")
    qo, _ = run(q, None, pos=p, theta=theta)
    check(q, qo, p.cpu().numpy()[None], [64], False, theta)
    if pos == 0:
        assert torch.equal(qo[0], q[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_results_in_place(dtype):
    """Rows of a fused projection (q | k | v side by side), an odd start, results over their inputs: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, Hkv, hd = 37, 6, 2, 64
    flat = torch.randn(T, (H + 2 * Hkv) * hd + 3, generator=g, device="cuda").to(dtype)
    for start in (0, 1):
        rows = flat[:, start:]
        q = rows[:, :H * hd].unflatten(1, (H, hd))
        k = rows[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd))
        pos = torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
        want = run(q.contiguous(), k.contiguous(), pos=pos)
        got = run(q, k, pos=pos)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        kept = flat.clone()
        held = flat.clone()[:, start:]
        q2, k2 = held[:, :H * hd].unflatten(1, (H, hd)), held[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd))
        run(q2, k2, pos=pos, in_place=True)
        assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
        assert torch.equal(held[:, (H + Hkv) * hd:], kept[:, start:][:, (H + Hkv) * hd:])      # what lies beside the rows


def test_partial_heads_in_place_keep_the_rest():
    x = torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(4)).cuda()
    y = x.clone()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    run(y, None, [5, 4], torch.stack([pos, pos + 3]), in_place=True)
    check(x, y, torch.stack([pos, pos + 3]).cpu().numpy(), [5, 4], False, 10000.0)


@pytest.mark.parametrize("prompt", [None, 100])
@pytest.mark.parametrize("parents", [None, TREE])
def test_positions_of_a_cache(prompt, parents):
    """The rows of a call: behind the committed slots (and the prompt), by depth in a tree; the lengths as they stand
    when a captured call is replayed."""
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    model = head_model(4, 2, 64, max_batch=4)
    kv = spec.KVCache(model, 4, 5000)
    if prompt:
        pre = spec.KVCache(model, 2, 300)
        pre.set_lengths([7, prompt])
        kv.set_prefix(pre, 1)
    counts = [len(TREE)] * 3 if parents else [5, 0, 64, 1]
    T = sum(counts)
    q = torch.randn(T, 4, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    depth = []
    for p in TREE:
        depth.append(0 if p < 0 else depth[p] + 1)

    def rows(lens):
        return np.concatenate([(prompt or 0) + n + (np.array(depth) if parents else np.arange(c))
                               for n, c in zip(lens, counts)])[None].astype(np.int32)

    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kv.set_lengths([900, 3, 4000, 0])
    spec.spec_rope(q, qo, k, ko, kv=kv, n_rows=counts, tree_parent=parents)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spec.spec_rope(q, qo, k, ko, kv=kv, n_rows=counts, tree_parent=parents)
    for lens in ([900, 3, 4000, 0], [0, 0, 0, 0], [4999, 4, 31, 17]):
        kv.set_lengths(lens)
        qo.zero_()
        graph.replay()
        for x, y in ((q, qo), (k, ko)):
            check(x, y, rows(lens), [32], False, 10000.0)
        assert torch.equal(qo, run(q, None, pos=torch.from_numpy(rows(lens)[0]).cuda())[0])


def test_the_model_turns_its_rows_alike():
    """Layer 0's K rows of a prefill are the projections turned by spec_rope (to the cache's rounding)."""
    from _gpu_util import cuda_i32, model_pair
    from oracle.decoder import linear, rms_norm
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens
    shape = ModelShape(2, 256, 8, 2, 64, 512, 2048, 1, "bf16")
    model, dec, shape = model_pair(shape, seed=3, max_rows=64, max_batch=1, max_position=512)
    kv = spec.KVCache(model, 1, 100)
    toks = make_tokens(50, shape.vocab, seed=1)
    spec.spec_prefill(model, kv, 0, cuda_i32(toks))
    W = dec.w["layers"][0]
    k = linear(rms_norm(dec.embed(toks), W["attn_norm"], shape.rms_eps), W["wk"]).reshape(50, 2, 64)
    kv.set_lengths([0])
    x = torch.from_numpy(k).float().cuda()
    y = torch.empty_like(x)
    spec.spec_rope(x, y, kv=kv, n_rows=[50], theta=shape.rope_theta)
    held, _ = kv.export_rows(0, 0, 1, 0, 50)
    # the cache rounds to bf16 (2^-8 of the value), the projection is f32 sums of bf16 pairs
    assert ((held[0].float() - y).abs() - (2.0 ** -8 * y.abs() + 1e-4 * y.abs().max())).max() <= 0


def test_streams_and_empty_calls():
    from speculative_decoding_verify_04_gb300 import spec
    e = torch.empty(0, 4, 64, device="cuda")
    spec.spec_rope(e, e, positions=torch.empty(0, dtype=torch.int32, device="cuda"))
    q = torch.randn(1000, 8, 128, device="cuda")
    pos = torch.arange(1000, dtype=torch.int32, device="cuda")
    want, _ = run(q, None, pos=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(q)
    with torch.cuda.stream(s):
        spec.spec_rope(q, out, positions=pos)
    s.synchronize()
    assert torch.equal(out, want)


def test_refused_tensors():
    from speculative_decoding_verify_04_gb300 import spec
    q = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad, word in ((dict(positions=pos[:3]), "positions"), (dict(positions=pos.long()), "positions"),
                      (dict(positions=pos.cpu()), "positions"), (dict(), "positions or a cache"),
                      (dict(positions=pos, sections=[20, 20]), "positions"), (dict(positions=pos, sections=[33]), "sections"),
                      (dict(positions=pos, sections=[0]), "sections"), (dict(positions=pos, sections=[]), "sections"),
                      (dict(positions=pos, sections=[-1]), "sections"), (dict(positions=pos, theta=0.5), "theta"),
                      (dict(positions=pos, theta=math.nan), "theta"), (dict(positions=pos, k_out=q), "k_out"),
                      (dict(positions=pos, k=q), "k_out"), (dict(positions=pos, k=q.half(), k_out=q.half()), "k:")):
        with pytest.raises(spec.SpecError, match=word):
            spec.spec_rope(q, q, **bad)
    for bad in (q[:3], q.half(), q.transpose(0, 1), q[:, :, ::2], q.cpu(), None):
        with pytest.raises(spec.SpecError, match="q"):
            spec.spec_rope(q, bad, positions=pos)
        if bad is not q[:3]:
            with pytest.raises(spec.SpecError):
                spec.spec_rope(bad, q, positions=pos)
