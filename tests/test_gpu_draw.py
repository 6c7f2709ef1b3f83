"""Draws from logits rows (temperature, top-k, top-p, min-p) against the definition in 64 bits, token for token."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from _gpu_util import lib
    lib()


def draw64(x, u, T, k, p, mp):
    """(token, log probability, kept ids, their probabilities, ids at the nucleus' border) of one row x (float64 numpy) for
    float32 settings.  Weights are exact to 2^-35 of themselves and to a unit, 2^-49 of the best token's 1 or, in rows whose
    weights add up to much, V 2^-61 rounded up to a power of two: the mass before a token and p of the whole are each off by
    2^-35 of the whole and n units at most, so a token may count to either side of the border only where the two lie within
    twice that."""
    T, p, mp, u = (float(np.float32(v)) for v in (T, p, mp, u))
    if T == 0:
        return int(np.argmax(x)), 0.0, np.array([np.argmax(x)]), np.ones(1), []
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if k:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    border = []
    if p < 1:
        before, all_ = np.concatenate([[0.0], np.cumsum(w)[:-1]]), math.fsum(w)
        keep = before < p * all_
        unit = max(2.0 ** -49, 2.0 ** (math.ceil(math.log2(max(2, x.size))) - 61))
        border = order[np.abs(before - p * all_) <= 2 * (2.0 ** -35 * all_ + w.size * unit)]
        keep[0] = True
        order, w = order[keep], w[keep]
    order, w = order[w >= mp], w[w >= mp]
    by_id = np.argsort(order)
    order, w = order[by_id], w[by_id]
    upto = np.cumsum(w)
    at = min(int(np.searchsorted(upto, u * upto[-1], side="right")), w.size - 1)
    return int(order[at]), math.log(w[at] / upto[-1]), order, w / upto[-1], border


def rows_of(seed, R, V, dtype=torch.float32, fall=(1.1, 2.0)):
    """Rows whose probabilities fall with a power of the rank, as a language model's do."""
    g = torch.Generator().manual_seed(seed)
    a = fall[0] + (fall[1] - fall[0]) * torch.rand(R, 1, generator=g)
    return (15.0 - a * torch.log1p(V * torch.rand(R, V, generator=g)) + 0.2 * torch.randn(R, V, generator=g)).to(dtype)


def uniforms(seed, R):
    return torch.rand(R, generator=torch.Generator().manual_seed(seed))


def check(x, u, T=1.0, k=0, p=1.0, mp=0.0, probs=True, strided=None):
    """x [R, V] on the CPU; settings are numbers or lists by row."""
    from speculative_decoding_verify_04_gb300 import spec
    R, V = x.shape
    xc = x.cuda() if strided is None else strided
    uc = u.cuda()
    arg = {}
    for name, v, dt in (("temperature", T, torch.float32), ("top_k", k, torch.int32), ("top_p", p, torch.float32),
                        ("min_p", mp, torch.float32)):
        arg[name] = torch.tensor(v, dtype=dt, device="cuda") if isinstance(v, (list, tuple)) else v
    tok = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((R,), 7.0, device="cuda")
    pr = torch.full((R, V), 7.0, device="cuda") if probs else None
    spec.spec_sample_logits(xc, uc, tok, logprob=lp, probs=pr, **arg)
    bare = torch.empty_like(tok)
    spec.spec_sample_logits(xc, uc, bare, **arg)
    assert torch.equal(tok, bare)
    row = lambda v, r: v[r] if isinstance(v, (list, tuple)) else v                      # noqa: E731
    for r in range(R):
        want, logp, ids, q, border = draw64(x[r].double().numpy(), u[r].item(), row(T, r), row(k, r), row(p, r), row(mp, r))
        assert int(tok[r]) == want, (r, int(tok[r]), want, ids.size)
        # log p = (x - m) / T - log S, each to a few roundings of 2^-24 of itself
        z = abs(logp) + (0 if row(T, r) == 0 else math.log(max(1.0, ids.size)))
        assert abs(float(lp[r]) - logp) <= 8 * 2.0 ** -24 * (z + 1e-3), (r, float(lp[r]), logp)
        if probs:
            got = pr[r].double().cpu().numpy()
            full = np.zeros(V)
            full[ids] = q
            got[border] = full[border] = 0.0
            # 2^-35 of a weight, two roundings of it, the sum's and the quotient's; weights below 2^-41 of the best are zero
            assert np.abs(got - full).max() <= 1e-12 + 2.0 ** -21 * full.max()
            assert (np.abs(got - full) <= 2.0 ** -21 * full + 2.0 ** -41).all()
            assert not got[np.setdiff1d(np.arange(V), ids)].any()


SETTINGS = [dict(), dict(T=0.0), dict(k=1), dict(k=7), dict(k=50, T=0.7), dict(p=0.9), dict(p=0.5, T=1.4), dict(mp=0.05),
            dict(k=40, p=0.95), dict(k=300, p=0.8, mp=0.02, T=0.8), dict(p=0.95, mp=0.001), dict(p=0.0), dict(mp=1.0),
            dict(T=0.05), dict(T=30.0, p=0.3), dict(T=1e-30), dict(T=1e30)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s", range(len(SETTINGS)))
@pytest.mark.parametrize("V", [1, 2, 9, 255, 257, 1000, 1024, 1025, 5003, 32000])
def test_settings_and_sizes(V, s, dtype):
    R = 6
    check(rows_of(V + s, R, V, dtype), uniforms(100 * s + V, R), probs=V <= 5003, **SETTINGS[s])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(1, 50257), (3, 131072), (200, 20011), (2, 262145), (1, 1048576), (500, 4000)])
@pytest.mark.parametrize("s", [0, 4, 5, 7, 9, 10])
def test_many_rows_and_large_vocabularies(R, V, s, dtype):
    check(rows_of(7 * V + s, R, V, dtype), uniforms(s + R, R), probs=R * V <= 600000, **SETTINGS[s])


@pytest.mark.parametrize("k", [1, 2, 100, 1000, 2000, 2047, 2048, 2049, 9000, 39999, 40000, 50000])
@pytest.mark.parametrize("p", [1.0, 0.9])
def test_large_top_k(k, p):
    """Lists that fit and lists that do not."""
    R, V = 4, 40000
    check(rows_of(k, R, V, fall=(0.2, 1.2)), uniforms(k + 1, R), k=k, p=p, T=1.3)


@pytest.mark.parametrize("p", [0.01, 0.5, 0.9, 0.999, 0.9999999])
@pytest.mark.parametrize("fall", [(0.0, 0.3), (0.8, 1.1), (1.0, 3.0)])
def test_nuclei_of_any_size(p, fall):
    R, V = 6, 70001
    check(rows_of(int(1000 * p), R, V, fall=fall), uniforms(3, R), p=p)


@pytest.mark.parametrize("values", [1, 2, 5, 40])
@pytest.mark.parametrize("kw", [dict(), dict(k=13), dict(k=3000), dict(p=0.7), dict(p=0.25, k=5000), dict(mp=0.3)])
@pytest.mark.parametrize("V", [300, 9000])
def test_ties_go_to_the_lower_id(values, kw, V):
    R = 5
    g = torch.Generator().manual_seed(values)
    x = torch.randint(0, values, (R, V), generator=g).float() * 0.5
    x[:, 5] = -0.0                                           # equal to 0.0
    check(x, uniforms(values, R), **kw)


@pytest.mark.parametrize("kw", [dict(), dict(k=50), dict(k=3000), dict(p=0.9), dict(mp=0.1), dict(T=0.0)])
@pytest.mark.parametrize("mask", [-math.inf, torch.finfo(torch.float32).min, -1e30])
def test_masked_rows(kw, mask):
    """Few tokens left, one left, and rows masked by the type's lowest value."""
    R, V = 6, 30000
    x = rows_of(11, R, V)
    keep = torch.rand(R, V, generator=torch.Generator().manual_seed(12)) < 0.01
    keep[0] = False
    keep[0, 29999] = True
    keep[1] = False
    keep[1, :3] = True
    x = torch.where(keep, x, torch.full_like(x, mask))
    check(x, uniforms(13, R), **kw)


@pytest.mark.parametrize("scale,shift", [(1.0, 1e4), (1.0, -3e4), (1e-3, 0.0), (1e4, 0.0), (1e30, 0.0), (1.0, 3e38)])
def test_logits_of_any_size(scale, shift):
    R, V = 5, 3000
    x = rows_of(14, R, V) * scale + shift
    for kw in (dict(), dict(p=0.9), dict(k=20, p=0.5), dict(mp=0.2)):
        check(x, uniforms(15, R), T=max(scale, 1e-3), **kw)


def test_settings_by_row():
    R, V = 64, 12345
    rng = np.random.default_rng(16)
    T = [float(np.float32(v)) for v in rng.choice([0.0, 0.5, 1.0, 1.7], R)]
    k = [int(v) for v in rng.choice([0, 1, 20, 500, 5000, 20000], R)]
    p = [float(np.float32(v)) for v in rng.choice([1.0, 0.9, 0.3, 2.0], R)]
    mp = [float(np.float32(v)) for v in rng.choice([0.0, 0.05, 0.5], R)]
    for dtype in (torch.float32, torch.bfloat16):
        check(rows_of(17, R, V, dtype), uniforms(18, R), T=T, k=k, p=p, mp=mp, probs=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    R, V = 9, 2049
    x = rows_of(19, R, V, dtype)
    for start in range(0, 9):
        wide = torch.full((R, V + 20), math.nan, dtype=dtype, device="cuda")
        wide[:, start:start + V] = x.cuda()
        for kw in (dict(), dict(k=30, p=0.9), dict(p=0.95)):
            check(x, uniforms(20, R), strided=wide[:, start:start + V], **kw)


def test_a_probability_row_may_be_a_slice():
    from speculative_decoding_verify_04_gb300 import spec
    R, V = 3, 1003
    x, u = rows_of(21, R, V).cuda(), uniforms(22, R).cuda()
    wide = torch.full((R, V + 13), 5.0, device="cuda")
    tok, tok2 = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
    want = torch.empty(R, V, device="cuda")
    spec.spec_sample_logits(x, u, tok, probs=wide[:, 6:6 + V], top_k=50)
    spec.spec_sample_logits(x, u, tok2, probs=want, top_k=50)
    assert torch.equal(wide[:, 6:6 + V], want) and torch.equal(tok, tok2)
    assert (wide[:, :6] == 5).all() and (wide[:, 6 + V:] == 5).all()


@pytest.mark.parametrize("kw", [dict(), dict(k=20), dict(p=0.6)])
def test_the_whole_range_of_u(kw):
    """Many u on one row, the least and the greatest among them."""
    V = 777
    x = rows_of(23, 1, V, fall=(0.5, 0.5))
    u = torch.cat([torch.tensor([0.0, 2.0 ** -149, 2.0 ** -126, 1e-30, 2.0 ** -24, 1 - 2.0 ** -24, 0.5]), uniforms(24, 1000)])
    check(x.expand(u.numel(), V).contiguous(), u, probs=False, **kw)


def test_rows_without_a_distribution_and_settings_out_of_range():
    from speculative_decoding_verify_04_gb300 import spec
    R, V = 15, 2000
    x = rows_of(25, R, V)
    T, p, mp, k = [1.0] * R, [0.9] * R, [0.01] * R, [30] * R
    u = uniforms(26, R)
    x[0, 7] = math.nan
    x[1, 1999] = math.inf
    x[2] = -math.inf
    T[3], T[4], T[5], T[6] = -1.0, math.nan, math.inf, 1e-38
    p[7], p[8] = -0.1, math.nan
    mp[9], mp[10] = 1.5, math.nan
    k[11] = -1
    u[12], u[13] = 1.0, math.nan
    f = lambda v: torch.tensor(v, device="cuda")             # noqa: E731
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    lp, pr = torch.zeros(R, device="cuda"), torch.zeros(R, V, device="cuda")
    spec.spec_sample_logits(x.cuda(), u.cuda(), tok, temperature=f(T), top_p=f(p), min_p=f(mp),
                            top_k=torch.tensor(k, dtype=torch.int32, device="cuda"), logprob=lp, probs=pr)
    assert (tok[:14] == -1).all() and torch.isnan(lp[:14]).all() and torch.isnan(pr[:14]).all()
    want = draw64(x[14].double().numpy(), u[14].item(), 1.0, 30, 0.9, 0.01)
    assert int(tok[14]) == want[0]


def test_calls_of_any_number_of_rows_give_the_same_bits():
    from speculative_decoding_verify_04_gb300 import spec
    V = 30011
    x, u = rows_of(27, 700, V, torch.bfloat16).cuda(), uniforms(28, 700).cuda()
    for kw in (dict(top_k=100, top_p=0.9), dict(top_p=0.97), dict()):
        out = []
        for n in (1, 3, 60, 700):
            tok = torch.empty(n, dtype=torch.int32, device="cuda")
            lp, pr = torch.empty(n, device="cuda"), torch.empty(n, V, device="cuda")
            spec.spec_sample_logits(x[:n], u[:n], tok, logprob=lp, probs=pr, **kw)
            out.append((tok, lp, pr))
        for got in out[:-1]:
            assert all(torch.equal(a, b[:a.shape[0]]) for a, b in zip(got, out[-1]))


def test_streams_captured_calls_and_empty_ones():
    from speculative_decoding_verify_04_gb300 import spec
    R, V = 20, 32000
    x, u = rows_of(29, R, V).cuda(), uniforms(30, R).cuda()
    tok, lp = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    spec.spec_sample_logits(x[:0], u[:0], tok[:0])
    call = lambda: spec.spec_sample_logits(x, u, tok, top_k=50, top_p=0.9, logprob=lp)      # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (31, 32):
        x.copy_(rows_of(seed, R, V))
        u.copy_(uniforms(seed, R))
        g.replay()
        torch.cuda.synchronize()
        got = tok.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            call()
        s.synchronize()
        assert torch.equal(tok, got)
        assert got.tolist() == [draw64(x[r].double().cpu().numpy(), u[r].item(), 1.0, 50, 0.9, 0.0)[0] for r in range(R)]


def test_refusals():
    from speculative_decoding_verify_04_gb300 import spec
    x = torch.zeros(2, 100, device="cuda")
    u, tok = torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad, word in ((dict(temperature=-1.0), "temperature"), (dict(temperature=math.nan), "temperature"),
                      (dict(temperature=math.inf), "temperature"), (dict(temperature=1e-39), "temperature"),
                      (dict(top_k=-1), "top_k"), (dict(top_p=-0.5), "top_p"), (dict(top_p=math.nan), "top_p"),
                      (dict(min_p=1.5), "min_p"), (dict(min_p=-0.1), "min_p"), (dict(top_k=tok.long()), "top_k"),
                      (dict(temperature=u.double()), "temperature"), (dict(top_p=u[:1]), "top_p"),
                      (dict(min_p=u.cpu()), "min_p"), (dict(probs=torch.zeros(2, 99, device="cuda")), "probs"),
                      (dict(probs=torch.zeros(1, 100, device="cuda")), "probs"), (dict(logprob=u[:1]), "logprob")):
        with pytest.raises(spec.SpecError, match=word):
            spec.spec_sample_logits(x, u, tok, **bad)
    for bad in ((x.half(), u, tok), (x[:, ::2], u, tok), (x[0], u, tok), (x.cpu(), u, tok), (None, u, tok), (x, u[:1], tok),
                (x, u.double(), tok), (x, u, tok[:1]), (x, u, tok.long()), (x, None, tok), (x, u, None)):
        with pytest.raises(spec.SpecError):
            spec.spec_sample_logits(*bad)


@pytest.mark.parametrize("order", ["down", "up", "blocks"])
@pytest.mark.parametrize("kw", [dict(), dict(k=700), dict(k=1900), dict(k=6000), dict(p=0.9), dict(p=0.99), dict(k=3000, p=0.8),
                                dict(mp=0.001), dict(p=0.999, mp=1e-4)])
def test_rows_whose_order_is_unlike_chance(order, kw):
    """Sorted rows, and rows whose likely tokens all lie in one segment of four: what holds on average does not."""
    R, V = 4, 60000
    x = rows_of(33, R, V, fall=(0.7, 1.4))
    if order == "blocks":
        away = (torch.arange(V) // 256) % 4 != (torch.arange(V) // 1024) % 4
        x = torch.where(away, x - 6.0, x)
    else:
        x = torch.sort(x, 1, descending=order == "down")[0]
    check(x, uniforms(34, R), **kw)


@pytest.mark.parametrize("kw", [dict(), dict(k=5000), dict(k=69999), dict(p=0.5), dict(p=0.25, k=20000), dict(mp=0.5), dict(p=0.7, mp=1.0)])
@pytest.mark.parametrize("values", [1, 2, 3])
def test_large_rows_of_few_values(kw, values):
    R, V = 3, 70001
    x = torch.randint(0, values, (R, V), generator=torch.Generator().manual_seed(values)).float() * 0.3
    check(x, uniforms(35, R), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(p=0.95), dict(k=1500, p=0.9), dict()])
def test_two_calls_at_once(dtype, kw):
    """Calls on two streams at a time, many times over: the tokens of the calls on their own."""
    from speculative_decoding_verify_04_gb300 import spec
    R, V = 60, 50257
    x = [rows_of(36 + i, R, V, dtype).cuda() for i in range(2)]
    u = [uniforms(38 + i, R).cuda() for i in range(2)]
    args = dict(top_k=kw.get("k", 0), top_p=kw.get("p", 1.0))
    want = []
    for a, b in zip(x, u):
        t = torch.empty(R, dtype=torch.int32, device="cuda")
        spec.spec_sample_logits(a, b, t, **args)
        want.append(t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(20)] for _ in range(2)]
    for n in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                spec.spec_sample_logits(x[i], u[i], got[i][n], **args)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in got[i])


def test_a_k_past_32_bits_is_every_token():
    from speculative_decoding_verify_04_gb300 import spec
    x, u = rows_of(44, 4, 5000, torch.float32).cuda(), uniforms(44, 4).cuda()
    got = [torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(3)]
    for t, k in zip(got, (0, 2 ** 31 - 1, 2 ** 32 + 1)):
        spec.spec_sample_logits(x, u, t, top_k=k)
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])
    with pytest.raises(spec.SpecError):
        spec.spec_sample_logits(x, u, got[0], top_k=1 - 2 ** 32)
