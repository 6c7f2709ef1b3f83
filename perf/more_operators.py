"""Cases of the operators of one decoding step over a window: rotary positions,
attention and the draw of the next token.

Three operators, each in its plain form (elementary torch operations in 32 bits,
in 64 where 32 lose what matters) and as calls of the library:

``rope``    query and key rows turned by their positions, which may have several
            axes (time, height, width), each with its share of the frequencies.
``window``  one layer's attention of a batch's candidate rows over a cache whose
            rows see the last tokens of their sequence and its first few (sinks).
``sample``  one token a row of logits, drawn from given random numbers after
            temperature, top-k, top-p and min-p.

``listed`` gives the cases, ``draw`` one more of the same ranges, ``prepare``
a case's inputs, ``run`` one pass, ``work`` its least bytes and operations and
``exact`` its outputs from the definitions in 64 bits.
"""
import math

import torch

own = False


def listed():
    return [
        # the one row of a decode step: latency
        dict(name="rope one token", op="rope", rows=1, heads=16, kv_heads=4, dim=64, sections="32", interleaved=False,
             far=2000, tree="", bits=16),
        # eight 29-node token trees behind long contexts, positions from the cache's lengths
        dict(name="rope trees", op="rope", rows=232, heads=32, kv_heads=8, dim=128, sections="64", interleaved=False,
             far=120000, tree="4,2,2", bits=16),
        # an odd number of patches of a picture, the axes' frequencies in turn, part of a head turned, 32-bit rows
        dict(name="rope patches odd", op="rope", rows=1333, heads=20, kv_heads=4, dim=64, sections="11,8,5",
             interleaved=True, far=5000, tree="", bits=32),
        # a video's patches in one prompt: the largest
        dict(name="rope video", op="rope", rows=16384, heads=32, kv_heads=8, dim=128, sections="16,24,24",
             interleaved=False, far=30000, tree="", bits=16),
        # one sequence, one token, a short window: the smallest decode step
        dict(name="window one token", op="window", batch=1, rows=1, branching="", ragged=False, heads=16, kv_heads=4,
             dim=64, prefix=0, own_len=700, window=256, sinks=4, prefix_bits=16, own_bits=16, page=0),
        # sixteen ragged chains over 8-bit pages, an odd window that reaches into the prompt they share
        dict(name="window chains", op="window", batch=16, rows=5, branching="", ragged=True, heads=32, kv_heads=8,
             dim=128, prefix=777, own_len=1500, window=1000, sinks=7, prefix_bits=8, own_bits=8, page=64),
        # sixteen 29-node token trees
        dict(name="window trees", op="window", batch=16, rows=29, branching="4,2,2", ragged=False, heads=16,
             kv_heads=4, dim=64, prefix=0, own_len=5000, window=2048, sinks=4, prefix_bits=16, own_bits=16, page=64),
        # plain decoding of 64 long sequences
        dict(name="window decode", op="window", batch=64, rows=1, branching="", ragged=False, heads=32, kv_heads=8,
             dim=128, prefix=0, own_len=16384, window=4096, sinks=4, prefix_bits=16, own_bits=16, page=0),
        # 32 long sequences verifying 8 candidates each: the largest
        dict(name="window document", op="window", batch=32, rows=8, branching="", ragged=False, heads=32, kv_heads=8,
             dim=128, prefix=0, own_len=24000, window=8192, sinks=128, prefix_bits=16, own_bits=16, page=0),
        # the draw of one decode step: latency
        dict(name="sample one", op="sample", rows=1, vocab=32000, bits=32, temperature=0.8, top_k=50, top_p=0.95,
             min_p=0.0, mixed=False, masked=False, probs=False),
        # a batch whose requests bring settings of their own (greedy ones among them), half-precision logits of an
        # odd vocabulary under a grammar mask, the distributions kept for the rejection test
        dict(name="sample batch", op="sample", rows=100, vocab=50257, bits=16, temperature=1.0, top_k=0, top_p=0.9,
             min_p=0.05, mixed=True, masked=True, probs=True),
        # many samples of a large vocabulary cut to the nucleus
        dict(name="sample nucleus", op="sample", rows=512, vocab=131072, bits=32, temperature=1.0, top_k=0, top_p=0.95,
             min_p=0.0, mixed=False, masked=False, probs=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "window", "window", "sample"])
    if op == "rope":
        heads, kv_heads = rng.choice([(4, 4), (16, 4), (32, 32), (32, 8), (24, 8), (20, 4)])
        dim, tree = rng.choice([64, 128]), rng.choice(["", "", "4,2,2", "3,2"])
        sections = rng.choice([[32], [16, 16], [8, 12, 12], [11, 8, 5]])
        sections = [dim // 64 * n for n in sections] if not tree else [dim // 2]
        bits = rng.choice([16, 16, 32])
        most = 16384 * 40 * 128 * 16 // ((heads + kv_heads) * dim * bits)
        rows = _log_int(rng, 1, 64) * _tree_size(tree) if tree else _log_int(rng, 1, min(16384, most))
        return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim,
                    sections=",".join(str(n) for n in sections), interleaved=len(sections) > 1 and rng.random() < 0.5,
                    far=_log_int(rng, 100, 120000 if tree else 1000000), tree=tree, bits=bits)
    if op == "sample":
        vocab = _log_int(rng, 1000, 160000)
        probs = rng.random() < 0.3
        return dict(op=op, rows=_log_int(rng, 1, min(2000, 512 * 131072 // (vocab * (2 if probs else 1)))), vocab=vocab,
                    bits=rng.choice([16, 32]), temperature=rng.choice([0.3, 0.8, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 1, 40, _log_int(rng, 2, 2000)]), top_p=rng.choice([1.0, 1.0, 0.95, 0.8]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.3, masked=rng.random() < 0.3,
                    probs=probs)
    heads, kv_heads = rng.choice([(4, 4), (16, 4), (32, 32), (32, 8), (24, 8), (20, 4)])
    branching = rng.choice(["", "", "4,2,2", "3,2", "2,2,2,2"])
    rows = _tree_size(branching) if branching else _log_int(rng, 1, 16)
    batch = _log_int(rng, 1, max(1, min(64, 512 // rows)))
    dim, window = rng.choice([64, 128]), _log_int(rng, 16, 8192)
    prefix = rng.choice([0, 0, _log_int(rng, 16, 8192)])
    # no more cache and no more score elements than the largest listed case
    cache = 32 * 24000 * 8 * 128 // (batch * kv_heads * dim)
    window = min(window, 32 * 8 * 32 * 8192 // (batch * rows * heads), cache)
    return dict(op=op, batch=batch, rows=rows, branching=branching, ragged=not branching and rng.random() < 0.5,
                heads=heads, kv_heads=kv_heads, dim=dim, prefix=prefix, own_len=_log_int(rng, 1, min(24000, cache)),
                window=window, sinks=rng.choice([0, 1, 4, 4, 64, 100]), prefix_bits=rng.choice([8, 16]),
                own_bits=rng.choice([8, 16, 16]), page=rng.choice([0, 64]))


def _tree_size(branching):
    n = w = 1
    for b in branching.split(",") if branching else []:
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


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _own_lens(case):
    """Committed slots of the sequences: from own_len down to none."""
    B, n = case["batch"], case["own_len"]
    return [n] if B == 1 else [n * (B - 1 - b) // (B - 1) for b in range(B)]


def _row_counts(case):
    B, r = case["batch"], case["rows"]
    return [1 + (5 * b + r - 1) % r if case["ragged"] else r for b in range(B)]


def _row_depths(case):
    return _depths(_tree_parents(case["branching"])) if case["branching"] else list(range(case["rows"]))


def _kv_values(gen, shape):
    """K or V rows as a decoder makes them: a scale of its own for every head, a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    scale = torch.exp(0.5 * torch.randn(shape[-2], 1, generator=gen, device="cuda"))
    loud = torch.rand(shape[-2], shape[-1], generator=gen, device="cuda") < 0.03
    return x.mul_(torch.where(loud, 6.0 * scale, scale).to(torch.bfloat16))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return {"rope": _prepare_rope, "window": _prepare_window, "sample": _prepare_sample}[case["op"]](case, gen)


def run(state):
    return {"rope": _run_rope, "window": _run_window, "sample": _run_sample}[state["op"]](state)


def work(case):
    if case["op"] == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        axes = len(case["sections"].split(","))
        return {"bytes": 2 * n * case["bits"] // 8 + 4 * axes * case["rows"], "flops": 3 * n}
    if case["op"] == "sample":
        n, R = case["rows"] * case["vocab"], case["rows"]
        return {"bytes": n * (case["bits"] // 8 + (4 if case["probs"] else 0)) + 12 * R, "flops": 4 * n}
    H, Hkv, hd, W, K, P = (case[x] for x in ("heads", "kv_heads", "dim", "window", "sinks", "prefix"))
    slot = {16: 4 * hd, 8: 2 * (hd + 1)}                # K and V of one slot and KV head
    depths, seen, held, prompt = _row_depths(case), 0, 0, set()
    T = sum(_row_counts(case))
    for s, n in zip(_own_lens(case), _row_counts(case)):
        lo = max(0, P + s - W + 1)                      # the first key of the first row's window
        prompt.update(((0, min(K, P)), (lo, P)))
        held += min(K, P + s, lo) - min(K, P, lo) + s - max(0, lo - P) + n
        for d in depths[:n]:
            first = max(0, P + s + d - W + 1)
            seen += P + s + d + 1 - first + min(K, first)
    read = torch.zeros(P + 1, dtype=torch.bool)
    for a, b in prompt:
        read[a:b] = True
    held = held * slot[case["own_bits"]] + int(read.sum()) * slot[case["prefix_bits"]]
    return {"bytes": Hkv * (held + T * 4 * hd) + 2 * T * H * hd * 2, "flops": 4 * seen * H * hd}


def _library_model(heads, kv_heads, dim, max_rows, max_batch):
    """A model handle of the given head layout (the operators need no more of it)."""
    from types import SimpleNamespace

    from speculative_decoding_verify_04_gb300 import spec
    shape = SimpleNamespace(n_layers=1, d_model=64, n_heads=heads, n_kv_heads=kv_heads, head_dim=dim, d_ff=64,
                            vocab=128, exit_layer=0, dtype="bf16", rms_eps=1e-5, rope_theta=10000.0)

    def z(*s):
        return torch.zeros(s, dtype=torch.bfloat16, device="cuda")

    layer = {"attn_norm": z(64), "wq": z(heads * dim, 64), "wk": z(kv_heads * dim, 64), "wv": z(kv_heads * dim, 64),
             "wo": z(64, heads * dim), "ffn_norm": z(64), "w_gate": z(64, 64), "w_up": z(64, 64), "w_down": z(64, 64)}
    w = {"embed": z(128, 64), "lm_head": z(128, 64), "final_norm": z(64), "layers": [layer]}
    return spec.Model(shape, w, max_rows=max_rows, max_batch=max_batch, max_position=1)


# ---------------------------------------------------------------------------
# rope: pair i of a row's first 2 n dims, (x_i, x_{i+n}), turned by the angle
# position[axis of i] * theta^(-i / n); the other dims pass

_THETA = 10000.0


def _pair_axes(sections, interleaved):
    """Axis of every frequency pair: the sections one after another, or the axes in turn while they last."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, axes = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


def _prepare_rope(case, gen):
    T, H, Hkv, hd = (case[x] for x in ("rows", "heads", "kv_heads", "dim"))
    sections = [int(n) for n in case["sections"].split(",")]
    dtype = torch.bfloat16 if case["bits"] == 16 else torch.float32
    state = dict(op="rope", sections=sections, interleaved=case["interleaved"])
    state["q"] = torch.randn(T, H, hd, generator=gen, device="cuda").to(dtype)
    state["k"] = torch.randn(T, Hkv, hd, generator=gen, device="cuda").to(dtype)
    if case["tree"]:
        # one tree a sequence behind its committed slots
        n = _tree_size(case["tree"])
        parents = _tree_parents(case["tree"])
        lens = torch.randint(0, case["far"], (T // n,), generator=gen, device="cuda", dtype=torch.int32)
        state["pos"] = (lens[:, None] + torch.tensor(_depths(parents), dtype=torch.int32, device="cuda")).reshape(1, T)
        if own:
            from speculative_decoding_verify_04_gb300 import spec
            # the cache whose lengths count; of its rows the operator needs none
            kv = spec.KVCache(_library_model(1, 1, 64, 1, T // n), T // n, case["far"] + n)
            kv.set_lengths(lens.tolist())
            state.update(kv=kv, counts=[n] * (T // n), parents=parents)
    else:
        # an image's or a video's grid behind a text: time from `far` on, height and width within 64
        t = torch.arange(T, device="cuda")
        first = int(torch.randint(0, case["far"], (1,), generator=gen, device="cuda"))
        grid = [first + t // 1024, first + t // 32 % 32, first + t % 32] if len(sections) > 1 else [first + t]
        state["pos"] = torch.stack(grid[:len(sections)]).to(torch.int32).contiguous()
    if own:
        state["q_out"], state["k_out"] = torch.empty_like(state["q"]), torch.empty_like(state["k"])
    return state


def _run_rope(state):
    q, k = state["q"], state["k"]
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        if "kv" in state:
            spec.spec_rope(q, state["q_out"], k, state["k_out"], theta=_THETA, kv=state["kv"], n_rows=state["counts"],
                           tree_parent=state["parents"])
        else:
            spec.spec_rope(q, state["q_out"], k, state["k_out"], theta=_THETA, positions=state["pos"],
                           sections=state["sections"], interleaved=state["interleaved"])
        return state["q_out"], state["k_out"]
    n = sum(state["sections"])
    axes = torch.tensor(_pair_axes(state["sections"], state["interleaved"]), device="cuda")
    # angles of far positions need 64 bits
    freq = torch.pow(torch.tensor(_THETA, dtype=torch.float64, device="cuda"),
                     -torch.arange(n, device="cuda").double() / n)
    angle = state["pos"].double()[axes].T * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x in (q, k):
        y = x.float()
        a, b = y[..., :n], y[..., n:2 * n]
        out.append(torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * n:]], -1).to(x.dtype))
    return tuple(out)


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


# ---------------------------------------------------------------------------
# window: the row of index i = prompt + committed + depth sees the key of index t
# of its sequence (and of its own chain or tree path) where t < sinks or i - t < window

def _prepare_window(case, gen):
    B, R, H, Hkv, hd = (case[x] for x in ("batch", "rows", "heads", "kv_heads", "dim"))
    P, W, K, lens, counts = case["prefix"], case["window"], case["sinks"], _own_lens(case), _row_counts(case)
    S, T = max(lens), sum(counts)
    parents = _tree_parents(case["branching"]) if case["branching"] else None
    dev = dict(device="cuda")
    state = dict(op="window", counts=counts, parents=parents, prefix_len=P)
    state["q"] = (2.0 * torch.randn(T, H, hd, generator=gen, **dev)).to(torch.bfloat16)
    state["k"], state["v"] = _kv_values(gen, (T, Hkv, hd)), _kv_values(gen, (T, Hkv, hd))
    pk, pv = _kv_values(gen, (P, Hkv, hd)), _kv_values(gen, (P, Hkv, hd))
    ok, ov = _kv_values(gen, (B, S, Hkv, hd)), _kv_values(gen, (B, S, Hkv, hd))
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        model = _library_model(H, Hkv, hd, T, B)
        page = case["page"] or None
        kv = spec.KVCache(model, B, S + R, page=page, q8=case["own_bits"] == 8)
        for b, n in enumerate(lens):
            if n:
                kv.import_rows(b, 0, ok[b, :n].contiguous()[None], ov[b, :n].contiguous()[None])
        kv.set_lengths(lens)
        if P:
            prompt = spec.KVCache(model, 1, P, page=page, q8=case["prefix_bits"] == 8)
            prompt.import_rows(0, 0, pk[None], pv[None])
            prompt.set_lengths([P])
            kv.set_prefix(prompt, 0)
        kv.set_window(W, sinks=K)
        state["kv"] = kv
        state["out"] = torch.empty_like(state["q"])
        return state
    # the same caches as tensors: bf16, or e4m3 values with their exponents
    state["prefix"] = [_quantise(x) if case["prefix_bits"] == 8 else x for x in (pk, pv)] if P else None
    state["owned"] = [_quantise(x) if case["own_bits"] == 8 else x for x in (ok, ov)]
    state["own_bits"] = case["own_bits"]
    # (sequence, row) of the rows back to back; every sequence's keys of index below its committed end that a
    # row of it may see (-1: none), and which of them and of the new rows each row sees
    n, s = torch.tensor(counts, **dev), torch.tensor(lens, **dev) + P
    j, d = torch.arange(R, **dev), torch.tensor(_row_depths(case), **dev)
    state["at"] = torch.nonzero(j[None] < n[:, None], as_tuple=True)
    lo = (s - W + 1).clamp_min(0)
    N = int((s - lo + torch.minimum(lo, torch.full_like(lo, K))).max())
    x = torch.arange(max(N, 1), **dev)[None]
    sink = torch.minimum(lo, torch.full_like(lo, K))[:, None]
    t = torch.where(x < sink, x, lo[:, None] + x - sink)
    t = torch.where(t < s[:, None], t, torch.full_like(t, -1))
    state["index"] = t
    i = s[:, None, None] + d[None, :, None]
    slots = (t[:, None] >= 0) & ((t[:, None] < K) | (i - t[:, None] < W))
    tree = torch.ones(R, R, dtype=torch.bool).tril()
    if parents:
        tree = torch.eye(R, dtype=torch.bool)
        for r in range(1, R):
            tree[r] |= tree[parents[r]]
    near = (d[:, None] - d[None] < W)[None] | (s[:, None, None] + d[None, None] < K)
    rows = tree.cuda()[None] & near & (j[None, None] < n[:, None, None])
    state["sees"] = torch.cat([slots, rows], 2)
    return state


def _run_window(state):
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        spec.spec_attend(state["kv"], 0, state["counts"], state["q"], state["out"], k=state["k"], v=state["v"],
                         tree_parent=state["parents"])
        return state["out"]
    b, j = state["at"]
    sees, t, P = state["sees"], state["index"], state["prefix_len"]
    B, R, N = sees.shape
    T, H, hd = state["q"].shape
    Hkv = state["k"].shape[1]
    G = H // Hkv
    keys = []
    for which, new in enumerate((state["k"], state["v"])):
        # the visible slots of every sequence, from the prompt and from its own cache
        x = state["owned"][which]
        here = (torch.arange(B, device="cuda")[:, None], (t - P).clamp_min(0).clamp_max(_first(x).shape[1] - 1))
        x = _values(x[0][here], x[1][here]) if isinstance(x, tuple) else x[here].float()
        if P:
            y, there = state["prefix"][which], t.clamp(0, P - 1)
            y = _values(y[0][there], y[1][there]) if isinstance(y, tuple) else y[there].float()
            x = torch.where((t < P)[:, :, None, None], y, x)
        rows = torch.zeros(B, R, Hkv, hd, device="cuda")
        rows[b, j] = _values(*_quantise(new)) if state["own_bits"] == 8 else new.float()
        keys.append(torch.cat([x, rows], 1))
    q = torch.zeros(B, R, Hkv, G, hd, device="cuda")
    q[b, j] = state["q"].float().view(T, Hkv, G, hd) / math.sqrt(hd)
    s = torch.einsum("brhgd,bnhd->brhgn", q, keys[0])
    s = s.masked_fill(~sees[:, :, None, None], -math.inf)
    s = (s - s.amax(-1, keepdim=True)).exp()
    out = torch.einsum("brhgn,bnhd->brhgd", s, keys[1]) / s.sum(-1, keepdim=True)
    return out[b, j].reshape(T, H, hd).to(torch.bfloat16)


def _first(x):
    return x[0] if isinstance(x, tuple) else x


# ---------------------------------------------------------------------------
# sample: w = exp((x - max x) / temperature).  Kept are the top_k largest logits
# (ties to the lower id), of those the shortest run by decreasing logit whose w
# reach top_p of theirs, of those the w of at least min_p; the token is the first by id
# at which the sum of the kept w passes u times their sum.  Temperature 0: the best token.

def _prepare_sample(case, gen):
    R, V, dev = case["rows"], case["vocab"], dict(device="cuda")
    # a language model's rows: probabilities that fall with a power of the rank, steeper or flatter by row
    fall = 1.1 + 0.9 * torch.rand(R, 1, generator=gen, **dev)
    x = 15.0 - fall * torch.log1p(V * torch.rand(R, V, generator=gen, **dev))
    x += 0.2 * torch.randn(R, V, generator=gen, **dev)
    if case["masked"]:
        keep = torch.rand(R, V, generator=gen, **dev) < 0.1
        keep[torch.arange(R, **dev), torch.randint(0, V, (R,), generator=gen, **dev)] = True
        x = torch.where(keep, x, -math.inf)
    state = dict(op="sample", x=x.to(torch.float32 if case["bits"] == 32 else torch.bfloat16), probs=case["probs"])
    state["u"] = torch.rand(R, generator=gen, **dev)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        state[name] = case[name]
    if case["mixed"]:
        # settings by request: greedy, top-k, nucleus, min-p and combinations of them
        kind = torch.randint(0, 6, (R,), generator=gen, **dev)

        def by_kind(dtype, *values):
            return torch.tensor(values, dtype=dtype, **dev)[kind]

        t, p, m = case["temperature"], case["top_p"], case["min_p"]
        state["temperature"] = by_kind(torch.float32, 0.0, t, t, 0.7, t, 1.2)
        state["top_k"] = by_kind(torch.int32, 0, 50, 0, 1000, 0, 0)
        state["top_p"] = by_kind(torch.float32, 1.0, 1.0, p, 0.95, 1.0, 1.0)
        state["min_p"] = by_kind(torch.float32, 0.0, 0.0, 0.0, 0.0, m, 0.0)
    return state


def _by_row(state, name, dtype):
    """A setting as [rows, 1]: a tensor of the rows, or one number as the library takes it (32 bits)."""
    v, R = state[name], state["x"].shape[0]
    if not isinstance(v, torch.Tensor):
        v = torch.full((R,), v, dtype=torch.int32 if name == "top_k" else torch.float32, device="cuda")
    return v.to(dtype)[:, None]


def _run_sample(state):
    x, u = state["x"], state["u"]
    R, V = x.shape
    if own:
        from speculative_decoding_verify_04_gb300 import spec
        tokens = torch.empty(R, dtype=torch.int32, device="cuda")
        logprob = torch.empty(R, dtype=torch.float32, device="cuda")
        probs = torch.empty(R, V, dtype=torch.float32, device="cuda") if state["probs"] else None
        spec.spec_sample_logits(x, u, tokens, temperature=state["temperature"], top_k=state["top_k"],
                                top_p=state["top_p"], min_p=state["min_p"], logprob=logprob, probs=probs)
        return [tokens, logprob] + ([probs] if state["probs"] else [])
    # 64 bits: which token's interval u meets, and which one ends the nucleus, are matters of the last bits
    temp = _by_row(state, "temperature", torch.float64)
    top_k, top_p, min_p = _by_row(state, "top_k", torch.int64), _by_row(state, "top_p", torch.float64), \
        _by_row(state, "min_p", torch.float64)
    top_k = torch.where(temp == 0, torch.ones_like(top_k), torch.where(top_k == 0, torch.full_like(top_k, V), top_k))
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    z = x.gather(1, order).double()
    w = ((z - z[:, :1]) / torch.where(temp == 0, torch.ones_like(temp), temp)).exp()
    at = torch.arange(V, device="cuda")[None]
    kept = torch.where(at < top_k, w, torch.zeros_like(w))
    before = kept.cumsum(1) - kept
    cut = (before >= top_p * kept.sum(1, keepdim=True)) & (top_p < 1) & (at > 0)
    kept = torch.where(cut | (w < min_p), torch.zeros_like(w), kept)
    # back to the order of the ids
    by_id = torch.zeros_like(w).scatter_(1, order, kept)
    upto = by_id.cumsum(1)
    total = upto[:, -1:]
    past = (upto > u.double()[:, None] * total) & (by_id > 0)
    tokens = torch.where(past, at, torch.full_like(at, V)).amin(1)
    p = by_id / total
    logprob = p.gather(1, tokens[:, None])[:, 0].log()
    return [tokens.to(torch.int32), logprob.float()] + ([p.float()] if state["probs"] else [])


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "window": _exact_window, "sample": _exact_sample}[case["op"]](case, state)


def _exact_rope(case, state):
    n = sum(state["sections"])
    out = [state["q"].double(), state["k"].double()]
    src = [x.clone() for x in out]
    axes = _pair_axes(state["sections"], state["interleaved"])
    for i in range(n):
        angle = state["pos"][axes[i]].double() * _THETA ** (-i / n)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for x, y in zip(src, out):
            z = torch.complex(x[..., i], x[..., i + n]) * turn
            y[..., i], y[..., i + n] = z.real, z.imag
    return tuple(out)


def _exact_window(case, state):
    H, Hkv, hd = case["heads"], case["kv_heads"], case["dim"]
    P, W, K, lens, counts = case["prefix"], case["window"], case["sinks"], _own_lens(case), state["counts"]
    depths = _row_depths(case)

    def held(x, *at):
        x = tuple(y[at] for y in x) if isinstance(x, tuple) else x[at]
        return x[0].double() * torch.exp2(x[1].double()).unsqueeze(-1) if isinstance(x, tuple) else x.double()

    new = [_quantised_64(x) if case["own_bits"] == 8 else x.double() for x in (state["k"], state["v"])]
    out = torch.empty(sum(counts), H, hd, dtype=torch.float64, device="cuda")
    first = 0
    for b, (s, n) in enumerate(zip(lens, counts)):
        rows = slice(first, first + n)
        first += n
        # every key of the sequence that any row may see, with its index
        lo = max(0, P + s - W + 1)
        t = torch.tensor(sorted(set(range(min(K, P + s))) | set(range(lo, P + s))), dtype=torch.long, device="cuda")
        parts = []
        for w in range(2):
            x = [held(state["prefix"][w], t[t < P])] if P else []
            parts.append(torch.cat(x + [held(state["owned"][w], b, t[t >= P] - P), new[w][rows]]))
        sees = torch.zeros(n, t.numel() + n, dtype=torch.bool, device="cuda")
        for r in range(n):
            i = P + s + depths[r]
            sees[r, :t.numel()] = (t < K) | (t > i - W)
            x = r
            while x >= 0:
                if depths[r] - depths[x] < W or P + s + depths[x] < K:
                    sees[r, t.numel() + x] = True
                x = state["parents"][x] if state["parents"] else x - 1
        for g in range(Hkv):
            heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            score = state["q"][rows, heads].double() @ parts[0][:, g].T / math.sqrt(hd)
            score.masked_fill_(~sees[:, None], -math.inf)
            out[rows, heads] = torch.softmax(score, -1) @ parts[1][:, g]
    return out


def _exact_sample(case, state):
    x, u = state["x"].double(), state["u"].double()
    R, V = x.shape
    temp, top_k, top_p, min_p = (_by_row(state, name, torch.float64)[:, 0].tolist()
                                 for name in ("temperature", "top_k", "top_p", "min_p"))
    tokens, logprob = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.float64, device="cuda")
    probs = torch.zeros(R, V, dtype=torch.float64, device="cuda") if state["probs"] else None
    for r in range(R):
        if temp[r] == 0:
            ids = torch.nonzero(x[r] == x[r].max())[:1, 0]
            w = torch.ones(1, dtype=torch.float64, device="cuda")
        else:
            ids = torch.nonzero(x[r] > -math.inf)[:, 0]
            ids = ids[torch.sort(-x[r, ids], stable=True)[1]]
            if top_k[r]:
                ids = ids[:int(top_k[r])]
            w = torch.exp((x[r, ids] - x[r, ids[0]]) / temp[r])
            if top_p[r] < 1:
                upto = torch.cumsum(w, 0)
                n = int((upto < top_p[r] * upto[-1]).sum()) + 1
                ids, w = ids[:n], w[:n]
            ids, w = ids[w >= min_p[r]], w[w >= min_p[r]]
            ids, by_id = torch.sort(ids)
            w = w[by_id]
        upto = torch.cumsum(w, 0)
        at = min(int((upto <= u[r] * upto[-1]).sum()), ids.numel() - 1)
        tokens[r] = ids[at]
        logprob[r] = torch.log(w[at] / upto[-1])
        if probs is not None:
            probs[r, ids] = w / upto[-1]
    return [tokens, logprob] + ([probs] if probs is not None else [])
