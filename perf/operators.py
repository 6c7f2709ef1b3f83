"""Cases of the operators for many continuations of one prompt.

Three operators, each in its plain form (elementary torch operations in 32
bits) and as calls of the library:

``cache8``    K/V rows written into an 8-bit cache (a power-of-two scale for
              every slot and KV head, e4m3 values) and read back.
``attend``    one layer's attention of the candidate rows of a batch whose
              sequences continue one long prompt: the new K/V rows go into
              each sequence's own cache, then every row sees the shared prompt,
              its sequence's committed slots and its own ancestors.
``logprobs``  log probabilities of given tokens under rows of logits, with
              the rows' entropy and best alternatives.

``listed`` gives the cases, ``draw`` one more of the same ranges, ``prepare``
a case's inputs, ``run`` one pass, ``work`` its least bytes and operations and
``exact`` its outputs from the definitions in 64 bits.
"""
import math

import torch

own = False


def listed():
    return [
        # one speculative chain of an 8-layer GQA decoder put into a cache and looked at again: latency
        dict(name="cache8 chain", op="cache8", layers=8, slots=5, kv_heads=4, dim=64, page=0),
        # an odd stretch of a context parked in a paged cache, GQA with 8 KV heads
        dict(name="cache8 paged odd", op="cache8", layers=16, slots=777, kv_heads=8, dim=128, page=64),
        # a whole 2048-token context of the 32-layer 4096-wide decoder parked and restored
        dict(name="cache8 context", op="cache8", layers=32, slots=2048, kv_heads=32, dim=128, page=0),
        # one sequence, one token, a short prompt: the smallest decode step
        dict(name="attend one token", op="attend", batch=1, rows=1, branching="", ragged=False, heads=16, kv_heads=4,
             dim=64, prefix=500, own_len=37, prefix_bits=16, own_bits=16, page=0),
        # eight samples of a 4096-token prompt verifying ragged chains of up to 5 candidates, 32 full heads
        dict(name="attend chains", op="attend", batch=8, rows=5, branching="", ragged=True, heads=32, kv_heads=32,
             dim=128, prefix=4096, own_len=300, prefix_bits=16, own_bits=8, page=0),
        # sixteen samples verifying 29-node token trees over a 2048-token prompt, paged caches
        dict(name="attend trees", op="attend", batch=16, rows=29, branching="4,2,2", ragged=False, heads=16,
             kv_heads=4, dim=64, prefix=2048, own_len=200, prefix_bits=16, own_bits=16, page=64),
        # plain decoding of 64 samples of a long prompt, everything held in 8 bits
        dict(name="attend decode", op="attend", batch=64, rows=1, branching="", ragged=False, heads=32, kv_heads=8,
             dim=128, prefix=16384, own_len=1024, prefix_bits=8, own_bits=8, page=64),
        # 64 samples of a 32768-token document verifying 8 candidates each: the largest
        dict(name="attend document", op="attend", batch=64, rows=8, branching="", ragged=False, heads=32, kv_heads=8,
             dim=128, prefix=32768, own_len=512, prefix_bits=16, own_bits=8, page=0),
        # the emitted token of one decode step: latency
        dict(name="logprobs one", op="logprobs", rows=1, vocab=32000, bits=32, top=0, temperature=1.0, masked=False),
        # the verified rows of eight chains of 5, five alternatives a position
        dict(name="logprobs chains", op="logprobs", rows=40, vocab=32000, bits=32, top=5, temperature=1.0,
             masked=False),
        # rows under a grammar mask that leaves a tenth of an odd vocabulary, half-precision logits
        dict(name="logprobs masked", op="logprobs", rows=333, vocab=100003, bits=16, top=1, temperature=0.7,
             masked=True),
        # scoring the samples for a ranking: many rows of a large vocabulary, twenty alternatives
        dict(name="logprobs ranking", op="logprobs", rows=512, vocab=131072, bits=32, top=20, temperature=1.0,
             masked=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache8", "attend", "attend", "logprobs"])
    if op == "cache8":
        dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 32])
        layers = _log_int(rng, 1, 32)
        most = 32 * 2048 * 32 * 128 // (layers * kv_heads * dim)
        return dict(op=op, layers=layers, slots=_log_int(rng, 1, min(8192, most)), kv_heads=kv_heads, dim=dim,
                    page=rng.choice([0, 64, 128]))
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 160000)
        return dict(op=op, rows=_log_int(rng, 1, min(2000, 512 * 131072 // vocab)), vocab=vocab,
                    bits=rng.choice([16, 32]), top=rng.choice([0, 1, 5, 20]),
                    temperature=rng.choice([0.6, 1.0, 1.3]), masked=rng.random() < 0.3)
    heads, kv_heads = rng.choice([(4, 4), (16, 4), (32, 32), (32, 8), (24, 8), (20, 4)])
    branching = rng.choice(["", "", "4,2,2", "3,2", "2,2,2,2"])
    rows = _tree_size(branching) if branching else _log_int(rng, 1, 16)
    batch = _log_int(rng, 1, max(1, 512 // rows))
    dim = rng.choice([64, 128])
    # no more score elements than the largest listed case
    most = 64 * 8 * 32 * 32768 // (batch * rows * heads)
    case = dict(op=op, batch=batch, rows=rows, branching=branching, ragged=not branching and rng.random() < 0.5,
                heads=heads, kv_heads=kv_heads, dim=dim, prefix=_log_int(rng, 16, min(32768, most)),
                own_len=_log_int(rng, 1, 1024), prefix_bits=rng.choice([8, 16]), own_bits=rng.choice([8, 16]),
                page=rng.choice([0, 64]))
    while case["own_len"] > 1 and case["batch"] * case["own_len"] * kv_heads * dim > 64 * 1024 * 8 * 128:
        case["own_len"] //= 2
    return case


def _tree_size(branching):
    n = w = 1
    for b in branching.split(","):
        w *= int(b)
        n += w
    return n


def _tree_parents(branching):
    """Parents of a level-order tree whose nodes of level l have branching[l] children."""
    parents, level = [-1], [0]
    for b in branching.split(","):
        nxt = []
        for node in level:
            for _ in range(int(b)):
                nxt.append(len(parents))
                parents.append(node)
        level = nxt
    return parents


def _own_lens(case):
    """Committed slots of the sequences: from own_len down to none."""
    B, n = case["batch"], case["own_len"]
    return [n] if B == 1 else [n * (B - 1 - b) // (B - 1) for b in range(B)]


def _row_counts(case):
    B, r = case["batch"], case["rows"]
    return [1 + (5 * b + r - 1) % r if case["ragged"] else r for b in range(B)]


def _kv_values(gen, shape):
    """K or V rows as a decoder makes them: a scale of its own for every head, a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[-2], 1, generator=gen, device="cuda"))
    loud = torch.rand(shape[-2], shape[-1], generator=gen, device="cuda") < 0.03
    return torch.where(loud, 6.0 * x, x).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return {"cache8": _prepare_cache8, "attend": _prepare_attend, "logprobs": _prepare_logprobs}[case["op"]](case, gen)


def run(state):
    return {"cache8": _run_cache8, "attend": _run_attend, "logprobs": _run_logprobs}[state["op"]](state)


def work(case):
    if case["op"] == "cache8":
        n = case["layers"] * case["slots"] * case["kv_heads"]
        held = n * (case["dim"] + 1)                    # e4m3 values and one exponent
        return {"bytes": 2 * (2 * n * case["dim"] * 2 + 2 * held), "flops": 2 * n * case["dim"] * 4}
    if case["op"] == "logprobs":
        n, R = case["rows"] * case["vocab"], case["rows"]
        return {"bytes": n * case["bits"] // 8 + R * (4 + 4 + 4 + 8 * case["top"]), "flops": 6 * n}
    lens, counts = _own_lens(case), _row_counts(case)
    T, H, Hkv, hd = sum(counts), case["heads"], case["kv_heads"], case["dim"]
    slot = {16: 4 * hd, 8: 2 * (hd + 1)}                # K and V of one slot and KV head
    held = case["prefix"] * slot[case["prefix_bits"]] + (sum(lens) + T) * slot[case["own_bits"]]
    seen = T * case["prefix"] + sum(n * (s + n) for s, n in zip(lens, counts))
    return {"bytes": Hkv * (held + T * 4 * hd) + 2 * T * H * hd * 2, "flops": 4 * seen * H * hd}


# ---------------------------------------------------------------------------
# the 8-bit form: x = value * 2^exponent, the exponent the least that holds the
# row's largest magnitude within e4m3's 448 (in [-124, 119], so that every value
# is a bf16 number)

def _quantise(x):
    """(e4m3 values, exponents) of rows x[..., dim]."""
    x = x.float()
    m, p = torch.frexp(x.abs().amax(-1))                # amax = m * 2^p, m in [0.5, 1)
    e = torch.where(m > 0.875, p - 8, p - 9).clamp(-124, 119)
    e = torch.where(m == 0, torch.full_like(e, -124), e)
    y = (x * _two_to(-e).unsqueeze(-1)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), e.to(torch.int8)


def _two_to(e):
    """2^e in 32 bits, from the exponent's bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _values(y, e):
    return y.float() * _two_to(e).unsqueeze(-1)


def _quantised_64(x):
    """The 64-bit values that rows x[..., dim] have in the 8-bit form."""
    x = x.double()
    big = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((big / 448.0).clamp_min(2.0 ** -200)))
    e = torch.where(torch.exp2(e - 1) * 448.0 >= big, e - 1, e)      # log2's last bit
    e = torch.where(torch.exp2(e) * 448.0 < big, e + 1, e).clamp(-124.0, 119.0)
    y = x / torch.exp2(e)
    # spacing of e4m3 at |y|: 2^(binade - 3), binades from -6 up
    binade = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6)))
    binade = torch.where(torch.exp2(binade) > y.abs().clamp_min(2.0 ** -6), binade - 1, binade)
    binade = torch.where(torch.exp2(binade + 1) <= y.abs(), binade + 1, binade)
    step = torch.exp2(binade - 3.0)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0) * torch.exp2(e)


def _library_model(heads, kv_heads, dim, layers, max_rows, max_batch):
    """A model handle of the given head layout (the operators need no more of it)."""
    from types import SimpleNamespace

    from speculative_decoding_verify_04_gb300 import spec
    shape = SimpleNamespace(n_layers=layers, d_model=64, n_heads=heads, n_kv_heads=kv_heads, head_dim=dim, d_ff=64,
                            vocab=128, exit_layer=0, dtype="bf16", rms_eps=1e-5, rope_theta=10000.0)

    def z(*s):
        return torch.zeros(s, dtype=torch.bfloat16, device="cuda")

    layer = {"attn_norm": z(64), "wq": z(heads * dim, 64), "wk": z(kv_heads * dim, 64), "wv": z(kv_heads * dim, 64),
             "wo": z(64, heads * dim), "ffn_norm": z(64), "w_gate": z(64, 64), "w_up": z(64, 64), "w_down": z(64, 64)}
    w = {"embed": z(128, 64), "lm_head": z(128, 64), "final_norm": z(64), "layers": [layer] * layers}
    return spec.Model(shape, w, max_rows=max_rows, max_batch=max_batch, max_position=1)


# ---------------------------------------------------------------------------
# cache8

def _prepare_cache8(case, gen):
    s = (case["layers"], case["slots"], case["kv_heads"], case["dim"])
    state = dict(op="cache8", k=_kv_values(gen, s), v=_kv_values(gen, s))
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        model = _library_model(case["kv_heads"], case["kv_heads"], case["dim"], case["layers"], 1, 1)
        state["kv"] = spec.KVCache(model, 1, case["slots"], page=case["page"] or None, q8=True)
    return state


def _run_cache8(state):
    k, v = state["k"], state["v"]
    if own:
        kv = state["kv"]
        kv.import_rows(0, 0, k, v)
        return kv.export_rows(0, 0, k.shape[0], 0, k.shape[1])
    return tuple(_values(*_quantise(x)).to(torch.bfloat16) for x in (k, v))


# ---------------------------------------------------------------------------
# attend

def _prepare_attend(case, gen):
    B, R, H, Hkv, hd = case["batch"], case["rows"], case["heads"], case["kv_heads"], case["dim"]
    P, lens, counts = case["prefix"], _own_lens(case), _row_counts(case)
    S, T = max(lens), sum(counts)
    parents = _tree_parents(case["branching"]) if case["branching"] else None
    dev = dict(device="cuda")
    state = dict(op="attend", counts=counts, parents=parents)
    state["q"] = (2.0 * torch.randn(T, H, hd, generator=gen, **dev)).to(torch.bfloat16)
    state["k"], state["v"] = _kv_values(gen, (T, Hkv, hd)), _kv_values(gen, (T, Hkv, hd))
    pk, pv = _kv_values(gen, (P, Hkv, hd)), _kv_values(gen, (P, Hkv, hd))
    ok, ov = _kv_values(gen, (B, S, Hkv, hd)), _kv_values(gen, (B, S, Hkv, hd))
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        model = _library_model(H, Hkv, hd, 1, T, B)
        page = case["page"] or None
        prompt = spec.KVCache(model, 1, P, page=page, q8=case["prefix_bits"] == 8)
        prompt.import_rows(0, 0, pk[None], pv[None])
        prompt.set_lengths([P])
        kv = spec.KVCache(model, B, S + R, page=page, q8=case["own_bits"] == 8)
        for b, n in enumerate(lens):
            if n:
                kv.import_rows(b, 0, ok[b, :n].contiguous()[None], ov[b, :n].contiguous()[None])
        kv.set_lengths(lens)
        kv.set_prefix(prompt, 0)
        state["kv"] = kv
        state["out"] = torch.empty_like(state["q"])
        return state
    # the same caches as tensors: bf16, or e4m3 values with their exponents
    state["prefix"] = [_quantise(x) if case["prefix_bits"] == 8 else x for x in (pk, pv)]
    state["owned"] = [_quantise(x) if case["own_bits"] == 8 else x for x in (ok, ov)]
    state["own_bits"] = case["own_bits"]
    # (sequence, row) of the rows back to back, and what each may see of its sequence's slots and rows
    n, s = torch.tensor(counts, **dev), torch.tensor(lens, **dev)
    j = torch.arange(R, **dev)
    state["at"] = torch.nonzero(j[None] < n[:, None], as_tuple=True)
    tree = torch.ones(R, R, dtype=torch.bool).tril()
    if parents:
        tree = torch.eye(R, dtype=torch.bool)
        for i in range(1, R):
            tree[i] |= tree[parents[i]]
    slots = (torch.arange(S, **dev)[None] < s[:, None])[:, None].expand(B, R, S)
    rows = (tree.cuda()[None] & (j[None, None] < n[:, None, None])).expand(B, R, R)
    state["sees"] = torch.cat([slots, rows], 2)
    return state


def _run_attend(state):
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        spec.spec_attend(state["kv"], 0, state["counts"], state["q"], state["out"], k=state["k"], v=state["v"],
                         tree_parent=state["parents"])
        return state["out"]
    b, j = state["at"]
    sees = state["sees"]
    B, R, N = sees.shape
    T, H, hd = state["q"].shape
    pk, pv = (_values(*x) if isinstance(x, tuple) else x.float() for x in state["prefix"])
    ok, ov = (_values(*x) if isinstance(x, tuple) else x.float() for x in state["owned"])
    nk, nv = (_values(*_quantise(x)) if state["own_bits"] == 8 else x.float() for x in (state["k"], state["v"]))
    Hkv = pk.shape[1]
    G = H // Hkv
    # the rows padded to (sequence, row), each sequence's new rows behind its slots
    q = torch.zeros(B, R, Hkv, G, hd, device="cuda")
    q[b, j] = state["q"].float().view(T, Hkv, G, hd) / math.sqrt(hd)
    new = torch.zeros(2, B, R, Hkv, hd, device="cuda")
    new[0, b, j], new[1, b, j] = nk, nv
    ok, ov = torch.cat([ok, new[0]], 1), torch.cat([ov, new[1]], 1)
    # scores over the prompt, one product a KV head, and over the sequence's own keys
    qp = q.permute(2, 0, 1, 3, 4).reshape(Hkv, B * R * G, hd)
    sp = qp @ pk.permute(1, 2, 0)
    so = torch.einsum("brhgd,bnhd->hbrgn", q, ok)
    so = so.masked_fill(~sees[None, :, :, None], -math.inf).reshape(Hkv, B * R * G, N)
    top = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    sp, so = (sp - top).exp_(), (so - top).exp_()
    total = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    out = sp @ pv.permute(1, 0, 2)
    out += torch.einsum("hbrgn,bnhd->hbrgd", so.view(Hkv, B, R, G, N), ov).reshape(Hkv, B * R * G, hd)
    out = (out / total).view(Hkv, B, R, G, hd).permute(1, 2, 0, 3, 4)
    return out[b, j].reshape(T, H, hd).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# logprobs

def _prepare_logprobs(case, gen):
    R, V = case["rows"], case["vocab"]
    x = 2.5 * torch.randn(R, V, generator=gen, device="cuda")
    # what the model expects: one to eight tokens well above the rest, by row
    for _ in range(8):
        at = torch.randint(0, V, (R, 1), generator=gen, device="cuda")
        x.scatter_(1, at, 9.0 + 4.0 * torch.randn(R, 1, generator=gen, device="cuda"))
    tokens = torch.where(torch.rand(R, generator=gen, device="cuda") < 0.7, x.argmax(1),
                         torch.randint(0, V, (R,), generator=gen, device="cuda"))
    if case["masked"]:
        keep = torch.rand(R, V, generator=gen, device="cuda") < 0.1
        keep[torch.arange(R, device="cuda"), tokens] = True
        x = torch.where(keep, x, -math.inf)
    return dict(op="logprobs", x=x.to(torch.float32 if case["bits"] == 32 else torch.bfloat16),
                tokens=tokens.to(torch.int32), top=case["top"], temperature=case["temperature"])


def _run_logprobs(state):
    x, tokens, n = state["x"], state["tokens"], state["top"]
    R = x.shape[0]
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        out = [torch.empty(R, dtype=torch.float32, device="cuda") for _ in range(2)]
        if n:
            out += [torch.empty(R, n, dtype=torch.int32, device="cuda"),
                    torch.empty(R, n, dtype=torch.float32, device="cuda")]
        spec.spec_logprobs(x, tokens, *out, temperature=state["temperature"])
        return out
    z = x.float() / state["temperature"]
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    logp = z - total.log()
    # 0 * log 0 = 0: a masked token adds nothing to the entropy
    out = [logp.gather(1, tokens.long()[:, None])[:, 0],
           -torch.where(e > 0, e * logp, torch.zeros_like(e)).sum(1) / total[:, 0]]
    if n:
        # the n best by value, ties to the lower id
        ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :n]
        out += [ids.to(torch.int32), logp.gather(1, ids)]
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "cache8":
        return tuple(_quantised_64(x) for x in (state["k"], state["v"]))
    if case["op"] == "logprobs":
        return _exact_logprobs(state)
    return _exact_attend(case, state)


def _exact_logprobs(state):
    x, n = state["x"].double(), state["top"]
    tokens = state["tokens"].long()
    rows = []
    for r in range(x.shape[0]):
        z = x[r] / state["temperature"]
        lse = torch.logsumexp(z, 0)
        lp = z - lse
        p = lp.exp()
        kept = p > 0
        row = [lp[tokens[r]], -(p[kept] * lp[kept]).sum()]
        if n:
            # ids by decreasing logit, equal logits by increasing id
            best = torch.topk(x[r], n).values[-1]
            near = torch.nonzero(x[r] >= best)[:, 0]
            near = near[torch.sort(-x[r][near], stable=True)[1]][:n]
            row += [near.to(torch.int32), lp[near]]
        rows.append(row)
    return [torch.stack([r[i] for r in rows]) for i in range(len(rows[0]))]


def _exact_attend(case, state):
    H, Hkv, hd = case["heads"], case["kv_heads"], case["dim"]
    lens, counts = _own_lens(case), state["counts"]

    def held(x):
        return x[0].double() * torch.exp2(x[1].double()).unsqueeze(-1) if isinstance(x, tuple) else x.double()

    pk, pv = (held(x) for x in state["prefix"])
    ok, ov = (held(x) for x in state["owned"])
    nk, nv = (_quantised_64(x) if case["own_bits"] == 8 else x.double() for x in (state["k"], state["v"]))
    out = torch.empty(sum(counts), H, hd, dtype=torch.float64, device="cuda")
    first = 0
    for b, (s, n) in enumerate(zip(lens, counts)):
        rows = slice(first, first + n)
        first += n
        sees = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        if state["parents"]:
            sees.fill_(False)
            for i in range(n):
                x = i
                while x >= 0:
                    sees[i, x] = True
                    x = state["parents"][x]
        for g in range(Hkv):
            heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            keys = torch.cat([pk[:, g], ok[b, :s, g], nk[rows, g]])
            vals = torch.cat([pv[:, g], ov[b, :s, g], nv[rows, g]])
            score = state["q"][rows, heads].double() @ keys.T / math.sqrt(hd)
            score[:, :, -n:].masked_fill_(~sees[:, None], -math.inf)
            out[rows, heads] = torch.softmax(score, -1) @ vals
    return out
