"""Log probabilities, entropy and best tokens of logits rows against 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _ref(x, T, tokens, n):
    """(log p, entropy, ids, log p of the ids) in 64 bits from the rows' values."""
    z = x.double() / T
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    ids = torch.sort(x.double(), dim=1, descending=True, stable=True)[1][:, :n]
    return lp.gather(1, tokens.long()[:, None])[:, 0], ent, ids, lp.gather(1, ids)


def _tol(x, T, lp):
    """Bound of a log probability's error.  d = log2e (x - max x) / T carries the rounding of log2e / T and
    of one multiply-add, 2^-23 of its size; 2^d then 2^-22 and, for the terms that count (d above -32),
    32 ln2 2^-23; a thread's sum of V / 512 terms and the joins of 32 + 16 + 8 states 2^-24 a step; the
    final logarithm, product and difference 3 2^-24 of their size.  Twice that, for the sum of products."""
    V = x.shape[1]
    size = torch.where(torch.isfinite(lp), lp.abs(), torch.zeros_like(lp))
    S = math.log(V)
    return 2 * ((size + S) * (2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -22 + 32 * 2.0 ** -23 + (V / 512 + 56) * 2.0 ** -24)


def _call(x, tokens, n, T=1.0, what=("lp", "ent", "top")):
    from _gpu_util import lib
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    R = x.shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    lp = torch.full((R,), 5.0, **f) if "lp" in what else None
    ent = torch.full((R,), 5.0, **f) if "ent" in what else None
    ids = torch.full((R, n), -7, dtype=torch.int32, device="cuda") if "top" in what and n else None
    tlp = torch.full((R, n), 5.0, **f) if ids is not None else None
    spec.spec_logprobs(x, tokens if "lp" in what else None, lp, ent, ids, tlp, temperature=T)
    return lp, ent, ids, tlp


def _check(x, tokens, n, T=1.0):
    lp, ent, ids, tlp = _call(x, tokens, n, T)
    xc = x.detach().cpu()
    wl, we, wi, wt = _ref(xc, T, tokens.cpu(), n)

    def near(got, want, tol):
        got, want = got.double().cpu(), want.double()
        inf = torch.isinf(want)
        assert torch.equal(got[inf], want[inf])
        assert ((got - want).abs()[~inf] <= tol[~inf]).all(), ((got - want).abs()[~inf] - tol[~inf]).max()

    near(lp, wl, _tol(xc, T, wl))
    # the entropy is a mean of -log p: the same bound at its own size plus one per weight error (|d| <= 32 counts)
    near(ent, we, 34 * _tol(xc, T, we))
    if n:
        assert torch.equal(ids.cpu().long(), wi)
        near(tlp, wt, _tol(xc, T, wt))


def _logits(seed, R, V, dtype=torch.float32, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, V, generator=g) * scale).to(dtype)
    t = torch.randint(0, V, (R,), generator=g).to(torch.int32)
    return x.cuda(), t.cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 255, 256, 257, 1000, 4099, 32000, 100003])
@pytest.mark.parametrize("R", [1, 3])
def test_vocabularies(dtype, V, R):
    x, t = _logits(V, R, V, dtype)
    _check(x, t, min(5, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [0, 1, 2, 20, 32])
@pytest.mark.parametrize("R,V", [(2, 20001), (30, 20001), (70, 9001), (400, 3001)])
def test_alternatives(dtype, n, R, V):
    """Rows over 8, 4, 2 and 1 CTAs; bf16 logits tie often."""
    x, t = _logits(n + R, R, V, dtype)
    _check(x, t, n)


@pytest.mark.parametrize("T", [0.05, 0.7, 1.0, 3.0])
def test_temperatures(T):
    x, t = _logits(5, 9, 5003)
    _check(x, t, 4, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lower_id(dtype):
    V = 3001
    flat = torch.zeros(4, V, dtype=dtype)
    flat[1, 7::10] = 2.0                                   # 300 equal best
    flat[2, ::256] = 1.0                                   # one in every segment
    flat[3, 2990:] = 1.0                                   # all in the last
    t = torch.tensor([0, 17, 1, 3000], dtype=torch.int32)
    _check(flat.cuda(), t.cuda(), 32)
    big = torch.zeros(2, 70000, dtype=dtype).cuda()
    _check(big, torch.tensor([69999, 0], dtype=torch.int32).cuda(), 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 20, 32])
@pytest.mark.parametrize("V", [9001, 131072])
def test_long_runs_of_equal_logits(dtype, n, V):
    """A mask that leaves fewer tokens than asked for, equal rows, zeros of both signs, ties at the last place."""
    x = torch.full((6, V), -math.inf, dtype=dtype)
    x[0, V - 3] = 1.0
    x[1, [5, 600, V - 1]] = torch.tensor([0.5, -2.0, 0.5], dtype=dtype)
    x[2] = 0.25
    x[3] = 0.0
    x[3, 1::2] = -0.0
    x[4] = -1.0
    x[4, 300:300 + n - 1] = 2.0                             # one place is left to the equal ones
    x[5] = -1.0
    x[5, V // 2:V // 2 + 700] = 3.0
    t = torch.tensor([V - 3, 600, V - 1, 1, 300, V - 1], dtype=torch.int32)
    _check(x.cuda(), t.cuda(), n)


def test_one_segment_holds_every_best_token():
    x = torch.linspace(0, 1, 5000).repeat(2, 1)
    x[0, 512:768] = torch.linspace(5, 9, 256)
    x[1, 300:400] = 20 - torch.arange(100) * 0.01
    _check(x.cuda(), torch.tensor([600, 300], dtype=torch.int32).cuda(), 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [700, 33000])
def test_masks(dtype, V):
    """-inf logits: few tokens left, fewer than asked for, one, none."""
    x, t = _logits(8, 6, V, dtype)
    x[0, torch.randperm(V)[:V - 40].cuda()] = -math.inf
    x[1, 3:] = -math.inf
    x[2] = -math.inf
    x[2, V - 1] = -4.0
    x[3, :V // 2] = -math.inf
    x[4, 256:512] = -math.inf
    t[1], t[2] = 1, V - 1
    _check(x, t, 8)
    t[1], t[2] = 5, 0                                       # masked tokens: -inf
    _check(x, t, 8)


def test_lowest_finite_logits():
    """A mask of the type's lowest value instead of -inf: no overflow, no weight."""
    for dtype in (torch.float32, torch.bfloat16):
        x, t = _logits(9, 3, 5000, dtype)
        x[0, 10:] = torch.finfo(dtype).min
        x[1, :] = torch.finfo(dtype).min
        x[1, 77] = 0.0
        t[0], t[1] = 3, 77
        _check(x, t, 2)


def test_rows_without_a_distribution():
    x, t = _logits(10, 5, 3000)
    x[0] = -math.inf
    x[1, 1234] = math.nan
    x[2, 5] = math.inf
    x[3] = math.nan
    lp, ent, ids, tlp = _call(x, t, 3)
    for r in range(4):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and (ids[r] == -1).all() and torch.isnan(tlp[r]).all(), r
    _check(x[4:], t[4:], 3)


def test_tokens_outside_the_vocabulary():
    x, t = _logits(11, 4, 500)
    t[0], t[1] = -1, 500
    lp, ent, _, _ = _call(x, t, 2)
    assert torch.isnan(lp[:2]).all() and torch.isfinite(lp[2:]).all() and torch.isfinite(ent).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (3, 5), (7, 1)])
def test_strides_and_addresses(dtype, shift, pad):
    R, V = 5, 4097
    x, t = _logits(12, R, V, dtype)
    flat = torch.full((shift + R * (V + pad),), 50.0, dtype=dtype, device="cuda")
    view = flat[shift:].view(R, V + pad)[:, :V]
    view.copy_(x)
    _check(view, t, 6)


def test_each_output_alone_and_untouched_rows():
    from speculative_decoding_verify_04_gb300 import spec
    x, t = _logits(13, 3, 2000)
    full = _call(x, t, 4)
    for what in ("lp", "ent", "top"):
        got = _call(x, t, 4, what=(what,))
        for a, b in zip(got, full):
            assert a is None or torch.equal(a, b)
    lp = torch.full((5,), 9.0, device="cuda")
    spec.spec_logprobs(x, t, lp)
    assert (lp[3:] == 9).all()
    spec.spec_logprobs(x[:0], t, lp)                       # no rows


def test_captured_and_on_another_stream():
    from speculative_decoding_verify_04_gb300 import spec
    x, t = _logits(14, 7, 9000)
    want = _call(x, t, 5)
    got = [torch.empty_like(o) for o in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        spec.spec_logprobs(x, t, *got)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for o in got:
        o.zero_()
    torch.cuda.synchronize()
    spec.spec_logprobs(x, t, *got, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    from _gpu_util import lib
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    x, t = _logits(15, 2, 100)
    f = torch.empty(2, device="cuda")
    i33, f33 = torch.empty(2, 33, dtype=torch.int32, device="cuda"), torch.empty(2, 33, device="cuda")

    def bad(match, *a, **kw):
        with pytest.raises(spec.SpecError, match=match):
            spec.spec_logprobs(*a, **kw)

    bad("temperature", x, t, f, temperature=0.0)
    bad("temperature", x, t, f, temperature=math.nan)
    bad("temperature", x, t, f, temperature=math.inf)
    bad("go together", x, t, None)
    bad("go together", x, None, f)
    bad("no output", x, None, None)
    bad("n_top", x, t, f, None, i33, f33)
    bad("top_ids", x, t, f, None, i33[:, :2].contiguous(), None)
    bad("2-D", x.half(), t, f)
    bad("2-D", x.t(), t, f)
    bad("tokens", x, t.long(), f)
    bad("logprob", x, t, f[:1])
    bad("bad sizes", x[:1].expand(2, 100), t, f)
