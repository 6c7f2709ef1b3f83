"""A layer of a caller's own over a windowed cache, step by step: rotary positions, attention, the draw of the next
token and of a verified chain."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

H, HKV, HD, V, D = 8, 2, 64, 3001, 128


def _weights(g):
    w = {n: torch.randn(*s, generator=g, device="cuda") * c for n, s, c in (
        ("embed", (V, D), 1.0), ("q", (D, H * HD), 0.15), ("k", (D, HKV * HD), 0.15), ("v", (D, HKV * HD), 0.15),
        ("o", (H * HD, D), 0.1), ("head", (D, V), 0.3))}
    return {n: x.to(torch.bfloat16).float() for n, x in w.items()}


def _logits64(w, tokens, window, sinks, theta):
    """[n, V]: the layer over a whole sequence in 64 bits (keys and values rounded to bf16, as the cache holds them)."""
    w = {n: x.double().cpu() for n, x in w.items()}
    n = len(tokens)
    x = w["embed"][tokens]
    bf = lambda t: t.float().to(torch.bfloat16).double()                  # noqa: E731
    q, k, v = bf(x @ w["q"]).view(n, H, HD), bf(x @ w["k"]).view(n, HKV, HD), bf(x @ w["v"]).view(n, HKV, HD)
    i = torch.arange(HD // 2, dtype=torch.float64)
    a = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2 * i / HD)
    c, s = a.cos()[:, None], a.sin()[:, None]

    def turn(t):
        lo, hi = t[..., :HD // 2], t[..., HD // 2:]
        return bf(torch.cat([lo * c - hi * s, hi * c + lo * s], -1))

    q, k = turn(q), turn(k)
    sc = torch.einsum("rhd,nhd->rhn", q, k.repeat_interleave(H // HKV, 1)) / math.sqrt(HD)
    t = torch.arange(n)
    sees = (t[None] <= t[:, None]) & ((t[:, None] - t[None] < window) | (t[None] < sinks))
    p = torch.softmax(sc.masked_fill(~sees[:, None], -math.inf), -1)
    y = torch.einsum("rhn,nhd->rhd", p, v.repeat_interleave(H // HKV, 1)).reshape(n, H * HD)
    return (x + y @ w["o"]) @ w["head"]


@pytest.mark.parametrize("q8", [False, True])
def test_steps_of_a_layer(q8):
    from _attend_util import head_model
    from speculative_decoding_verify_04_gb300 import spec
    g = torch.Generator(device="cuda").manual_seed(1)
    w = _weights(g)
    B, window, sinks, theta = 3, 24, 3, 10000.0
    model = head_model(H, HKV, HD, max_rows=64 * B, max_batch=B)
    kv = spec.KVCache(model, B, 160, page=64, q8=q8)
    kv.set_window(window, sinks)
    seqs = [[7, 11], [5], [3, 2, 1]]
    settings = dict(temperature=torch.tensor([0.0, 0.8, 1.0], device="cuda"), top_k=torch.tensor([0, 20, 0], dtype=torch.int32, device="cuda"),
                    top_p=torch.tensor([1.0, 0.9, 1.0], device="cuda"), min_p=torch.tensor([0.0, 0.0, 0.1], device="cuda"))

    def layer(rows):
        """Logits of the new rows of each sequence (lists of tokens) behind its committed slots."""
        counts = [len(r) for r in rows]
        x = w["embed"][torch.tensor(sum(rows, []), device="cuda")]
        q, k, v = ((x @ w[n]).to(torch.bfloat16).view(-1, h, HD) for n, h in (("q", H), ("k", HKV), ("v", HKV)))
        spec.spec_rope(q, q, k, k, theta=theta, kv=kv, n_rows=counts)
        out = torch.empty_like(q)
        spec.spec_attend(kv, 0, counts, q, out, k=k, v=v)
        return (x + out.float().reshape(-1, H * HD) @ w["o"]) @ w["head"], counts

    todo = [list(s) for s in seqs]
    for step in range(40):
        logits, counts = layer(todo)
        spec.kv_commit(kv, torch.tensor([c - 1 for c in counts], dtype=torch.int32, device="cuda"))
        last = logits[torch.tensor(np.cumsum(counts) - 1, device="cuda")]
        u = torch.rand(B, generator=g, device="cuda")
        tok, lp = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, device="cuda")
        spec.spec_sample_logits(last.contiguous(), u, tok, logprob=lp, **settings)
        assert (tok >= 0).all() and (lp <= 0).all()
        assert int(tok[0]) == int(last[0].argmax())
        todo = [[int(t)] for t in tok]
        for s, t in zip(seqs, todo):
            s += t
    # every logit of the last rows against the whole sequences in 64 bits: outputs of the attention are bf16 (2^-8), its
    # probabilities one bf16 number (2^-8), projections f32 sums that are rounded to bf16 and may round to the other
    # side (2^-8 each of q, k and v): five such steps on a layer output of |y| <= max |v|, through o and the head.
    # An 8-bit cache's values are off by 2^-4 of themselves
    logits, _ = layer(todo)
    for b, s in enumerate(seqs):
        want = _logits64(w, s, window, sinks, theta)
        scale = (want - want.mean()).abs().max()
        off = (logits[b].double().cpu() - want[-1]).abs().max()
        assert off <= scale * (0.25 if q8 else 5 * 2.0 ** -8), (b, float(off), float(scale))
    assert kv.get_lengths() == [len(s) - 1 for s in seqs] and model.device_error() == 0


def test_distributions_for_the_rejection_test():
    """p and q rows cut by top-k and min-p into spec_accept: chains drawn from q are kept as the ratio says, and tokens
    outside p's cut never leave."""
    from speculative_decoding_verify_04_gb300 import spec
    g = torch.Generator(device="cuda").manual_seed(2)
    B, k, V_ = 200, 4, 1000
    target = 3.0 * torch.randn(B, k + 1, V_, generator=g, device="cuda")
    draft = target[:, :k] + torch.randn(B, k, V_, generator=g, device="cuda")
    p, q = torch.empty(B, k + 1, V_, device="cuda"), torch.empty(B, k, V_, device="cuda")
    drafted = torch.empty(B, k, dtype=torch.int32, device="cuda")
    u1 = torch.randint(0, 1 << 24, (B * k,), generator=g, device="cuda").float() * 2.0 ** -24
    spec.spec_sample_logits(draft.reshape(B * k, V_), u1, drafted.view(-1), temperature=0.8, probs=q.view(B * k, V_))
    bonus = torch.empty(B * (k + 1), dtype=torch.int32, device="cuda")
    spec.spec_sample_logits(target.reshape(-1, V_), torch.zeros(B * (k + 1), device="cuda"), bonus, temperature=0.8, top_k=40,
                            min_p=0.02, probs=p.view(-1, V_))
    u = torch.randint(0, 1 << 24, (B, k + 1), generator=g, device="cuda").float() * 2.0 ** -24
    acc, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    spec.spec_accept(p, q, drafted, u, acc, nxt)
    a, n = acc.tolist(), nxt.tolist()
    ratio = (p[:, :k].gather(2, drafted.long()[..., None])[..., 0].double() /
             q.gather(2, drafted.long()[..., None])[..., 0].double())
    kept = (u[:, :k].double() < ratio).cpu()
    for b in range(B):
        want = 0
        while want < k and kept[b, want]:
            want += 1
        assert a[b] == want and p[b, a[b], n[b]] > 0
        assert all(p[b, j, drafted[b, j]] > 0 for j in range(a[b]))
    assert 0 < sum(a) < B * k
