"""Many continuations of one prompt through the forward calls: a prompt that is held once, 8-bit caches, and a
whole best-of-n run (draft, verify, commit, log probabilities)."""
import numpy as np
import pytest
import torch

from _gpu_util import cuda_i32, lib, model_pair, top_gap
from oracle import spec as OS
from oracle.accept import accept_greedy_chain, accept_greedy_tree, argmax_lowest
from synthetic import ModelShape, make_tokens, tree_parents

pytestmark = pytest.mark.gpu

TOL = 2e-2                  # the bound of the bf16 path's logits against the oracle
SHAPES = {"hd64": ModelShape(3, 256, 8, 2, 64, 512, 2048, 1, "bf16"),
          "hd128": ModelShape(3, 256, 4, 2, 128, 512, 2048, 1, "bf16")}


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _continuations(model, prompt, suffixes, page=None, q8=False, prompt_q8=False, cap=160):
    """A cache of the continuations `suffixes` of `prompt`, the prompt prefilled once into a cache of its own."""
    from speculative_decoding_verify_04_gb300 import spec
    pre = spec.KVCache(model, 2, len(prompt) + 7, page=page, q8=prompt_q8)
    spec.spec_prefill(model, pre, 1, cuda_i32(prompt))
    kv = spec.KVCache(model, len(suffixes), cap, page=page, q8=q8)
    kv.set_prefix(pre, 1)
    t0 = _i32(len(suffixes))
    for b, s in enumerate(suffixes):
        spec.spec_prefill(model, kv, b, cuda_i32(s), next_tok=t0[b:b + 1])
    return kv, t0


def _round(model, shape, kv, t0, k):
    from speculative_decoding_verify_04_gb300 import spec
    B = t0.numel()
    r = dict(cand=_i32(B, k + 1), hL=torch.empty(B, k + 1, shape.d_model, device="cuda"),
             logits=torch.empty(B, k + 1, shape.vocab, device="cuda"), acc=_i32(B), nxt=_i32(B))
    spec.spec_draft(model, kv, t0, k, r["cand"], r["hL"])
    spec.spec_verify(model, kv, [k + 1] * B, r["cand"], k + 1, h_in=r["hL"], h_stride=k + 1, logits=r["logits"],
                     acc_len=r["acc"], next_tok=r["nxt"])
    return r


@pytest.mark.parametrize("name", ["hd64", "hd128"])
@pytest.mark.parametrize("B,page", [(1, None), (3, 64), (7, None)])
def test_rounds_over_a_shared_prompt_match_the_oracle(name, B, page):
    """Prefill, layer-skip draft and verification with the prompt held once, against the oracle with all of it
    in one context.  One sequence's 5 rows take the row kernel (f32 queries in two parts), the others the tile
    kernel (queries rounded to bf16)."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, dec, shape = model_pair(SHAPES[name], seed=3, max_rows=64, max_batch=8, max_position=512)
    prompt = make_tokens(150, shape.vocab, seed=4)
    suffixes = [make_tokens(1 + 9 * b, shape.vocab, seed=5 + b) for b in range(B)]
    kv, t0 = _continuations(model, prompt, suffixes, page=page)
    assert kv.get_lengths() == [len(s) for s in suffixes]
    r = _round(model, shape, kv, t0, 4)
    spec.kv_commit(kv, r["acc"])
    for b, s in enumerate(suffixes):
        n = len(prompt) + len(s)
        cache = dec.new_cache(n + 16)
        first = dec.prefill(cache, np.concatenate([prompt, s]))
        if top_gap(first) >= TOL:
            assert int(t0[b]) == argmax_lowest(first)
        cand, got = r["cand"][b].cpu().numpy(), r["logits"][b].cpu().numpy()
        want = OS.verify(dec, cache, n, dec.embed(cand), 0)
        assert np.abs(got - want).max() < TOL, b
        assert (int(r["acc"][b]), int(r["nxt"][b])) == accept_greedy_chain(list(cand[1:]), got)
    assert kv.get_lengths() == [len(s) + int(a) + 1 for s, a in zip(suffixes, r["acc"].cpu())]
    assert model.device_error() == 0


@pytest.mark.parametrize("own_trees", [False, True])
def test_token_trees_over_a_shared_prompt(own_trees):
    """One tree for the batch and one tree a sequence; the accepted path is compacted in the sequences' own slots."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, dec, shape = model_pair(SHAPES["hd64"], seed=6, max_rows=64, max_batch=4, max_position=512)
    prompt = make_tokens(70, shape.vocab, seed=7)
    suffixes = [make_tokens(3 + 5 * b, shape.vocab, seed=8 + b) for b in range(3)]
    kv, t0 = _continuations(model, prompt, suffixes, page=64)
    par = [int(p) for p in tree_parents([2, 2, 1])]
    N, B = len(par), 3
    toks = np.stack([make_tokens(N, shape.vocab, seed=20 + b) for b in range(B)])
    want = []
    for b, s in enumerate(suffixes):
        n = len(prompt) + len(s)
        cache = dec.new_cache(n + 32)
        first = dec.prefill(cache, np.concatenate([prompt, s]))
        # a greedy path through nodes 2, 5 and 9 of the tree
        g = OS.generate_greedy_ar(dec, np.concatenate([prompt, s]), 4)
        toks[b, 0], toks[b, 2], toks[b, 5], toks[b, 9] = argmax_lowest(first), g[1], g[2], g[3]
        want.append(OS.verify(dec, cache, n, dec.embed(toks[b]), 0, par))
    logits, acc, nxt, path = torch.empty(B * N, shape.vocab, device="cuda"), _i32(B), _i32(B), _i32(B, 64)
    tk = cuda_i32(toks)
    if own_trees:
        spec.spec_verify_trees(model, kv, [N] * B, tk, N, cuda_i32(np.tile(par, (B, 1))), N, logits=logits, acc_len=acc,
                               next_tok=nxt, path=path)
    else:
        spec.spec_verify(model, kv, [N] * B, tk, N, tree_parent=par, logits=logits, acc_len=acc, next_tok=nxt, path=path)
    got = logits.view(B, N, -1).cpu().numpy()
    before = [kv.export_rows(b, 0, shape.n_layers, 0, len(s) + N) for b, s in enumerate(suffixes)]
    spec.kv_commit(kv, acc, path)
    for b, s in enumerate(suffixes):
        assert np.abs(got[b] - want[b]).max() < TOL
        d, _, p, x = accept_greedy_tree([int(t) for t in toks[b]], par, got[b])
        assert (int(acc[b]), int(nxt[b])) == (d, x) and path[b, :d + 1].tolist() == [int(i) for i in p]
        at = list(range(len(s))) + [len(s) + int(i) for i in p]
        k, _ = kv.export_rows(b, 0, shape.n_layers, 0, len(at))
        assert torch.equal(k, before[b][0][:, at])
    assert model.device_error() == 0


@pytest.mark.parametrize("name", ["hd64", "hd128"])
def test_forward_calls_write_8_bit_rows(name):
    """The first layer's K and V rows do not depend on any cache: in an 8-bit cache they are the quantised rows of
    a bf16 cache, exactly; and a whole round's results follow from its own logits."""
    from _attend_util import rows8
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES[name], seed=9, max_rows=64, max_batch=4, max_position=512)
    seqs = [make_tokens(n, shape.vocab, seed=30 + n) for n in (1, 64, 83)]
    rows, rounds = [], []
    for q8, page in ((False, None), (True, None), (True, 64)):
        kv = spec.KVCache(model, 3, 140, page=page, q8=q8)
        t0 = _i32(3)
        for b, s in enumerate(seqs):
            spec.spec_prefill(model, kv, b, cuda_i32(s), next_tok=t0[b:b + 1])
        assert kv.get_lengths() == [1, 64, 83]
        rows.append([[x.double().cpu().numpy() for x in kv.export_rows(b, 0, 1, 0, len(s))] for b, s in enumerate(seqs)])
        r = _round(model, shape, kv, t0, 3)
        spec.kv_commit(kv, r["acc"])
        for b in range(3):
            got = (int(r["acc"][b]), int(r["nxt"][b]))
            assert got == accept_greedy_chain(r["cand"][b, 1:].tolist(), r["logits"][b].cpu().numpy())
        assert kv.get_lengths() == [len(s) + int(a) + 1 for s, a in zip(seqs, r["acc"].cpu())]
        rounds.append(r)
        assert model.device_error() == 0
    for b in range(3):
        for which in range(2):
            assert np.array_equal(rows[1][b][which], rows8(rows[0][b][which])[2])
            assert np.array_equal(rows[1][b][which], rows[2][b][which])
    # contiguous and paged: the same bits
    assert torch.equal(rounds[1]["logits"], rounds[2]["logits"]) and torch.equal(rounds[1]["cand"], rounds[2]["cand"])


def test_an_8_bit_cache_and_a_bf16_cache_of_its_values():
    """The rows that a verification wrote into an 8-bit cache are the quantised rows of a bf16 cache of the same
    context; and attention over an 8-bit cache equals attention over a bf16 cache of the values it stands for."""
    from _attend_util import rows8
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    shape = ModelShape(1, 256, 4, 2, 64, 512, 2048, 0, "bf16")
    model, _, _ = model_pair(shape, seed=10, max_rows=16, max_batch=1, max_position=256)
    ctx, tok = make_tokens(100, shape.vocab, seed=11), cuda_i32(make_tokens(1, shape.vocab, seed=12))
    q8, bf = spec.KVCache(model, 1, 128, q8=True), spec.KVCache(model, 1, 128)
    logits = torch.empty(1, shape.vocab, device="cuda")
    spec.spec_prefill(model, q8, 0, cuda_i32(ctx))
    spec.spec_verify(model, q8, [1], tok, 1, logits=logits)
    k, v = q8.export_rows(0, 0, 1, 0, 101)
    bf.import_rows(0, 0, k[:, :100].contiguous(), v[:, :100].contiguous())
    bf.set_lengths([100])
    spec.spec_verify(model, bf, [1], tok, 1, logits=logits)
    k2, v2 = bf.export_rows(0, 0, 1, 100, 1)
    for held, plain in ((k, k2), (v, v2)):
        assert np.array_equal(held[:, 100:].double().cpu().numpy(), rows8(plain.double().cpu().numpy())[2])
    q8.set_lengths([101])
    bf.import_rows(0, 0, k[:, 100:].contiguous(), v[:, 100:].contiguous(), slot0=100)
    bf.set_lengths([101])
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(14)).to(torch.bfloat16).cuda()
    new_k, new_v = (torch.full((1, 2, 64), x, dtype=torch.bfloat16, device="cuda") for x in (0.5, -0.25))   # exact in 8 bits
    out = []
    for kv in (q8, bf):
        out.append(torch.empty_like(q))
        spec.spec_attend(kv, 0, [1], q, out[-1], k=new_k, v=new_v)
    a, b = (x.double() for x in out)
    # each is off by half a bf16 step of itself, 2^-8, and by far less inside: two halves, of the larger value
    assert ((a - b).abs() <= (2.0 ** -7 + 2.0 ** -10) * torch.maximum(a.abs(), b.abs()).amax()).all()
    assert model.device_error() == 0


def test_best_of_n():
    """Five samples of one prompt, 8-bit caches over a bf16 prompt: draft, verify, commit, and the tokens scored; the
    scores are those of the verifications' logits, the lengths those of the accepted tokens."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES["hd64"], seed=15, max_rows=64, max_batch=5, max_position=512)
    prompt = make_tokens(200, shape.vocab, seed=16)
    B, k = 5, 3
    kv, t0 = _continuations(model, prompt, [make_tokens(2, shape.vocab, seed=40 + b) for b in range(B)], page=64, q8=True)
    lens, score, want = [2] * B, torch.zeros(B, dtype=torch.float64), np.zeros(B)
    for _ in range(4):
        r = _round(model, shape, kv, t0, k)
        spec.kv_commit(kv, r["acc"])
        # the emitted tokens: the accepted candidates, then the next token, each under the row before it
        emitted = torch.cat([r["cand"][:, 1:], torch.zeros_like(r["nxt"])[:, None]], 1).contiguous()
        rows = torch.arange(B, device="cuda")
        emitted[rows, r["acc"].long()] = r["nxt"]
        lp, ent = torch.empty(B, k + 1, device="cuda"), torch.empty(B, k + 1, device="cuda")
        ids, tlp = _i32(B * (k + 1), 3), torch.empty(B * (k + 1), 3, device="cuda")
        spec.spec_logprobs(r["logits"].view(B * (k + 1), -1), emitted.view(-1), lp.view(-1), ent.view(-1), ids, tlp)
        ref = torch.log_softmax(r["logits"].double(), -1).cpu()
        assert (ids[:, 0].cpu() == ref.view(B * (k + 1), -1).argmax(-1)).all()
        for b in range(B):
            a = int(r["acc"][b])
            lens[b] += a + 1
            score[b] += lp[b, :a + 1].double().sum().cpu()
            want[b] += sum(float(ref[b, j, int(emitted[b, j])]) for j in range(a + 1))
            # greedy emission: every emitted token is its row's best
            assert ids.view(B, k + 1, 3)[b, :a + 1, 0].tolist() == emitted[b, :a + 1].tolist()
        assert kv.get_lengths() == lens
        t0 = r["nxt"].clone()
    assert np.allclose(score.numpy(), want, atol=1e-4)
    assert model.device_error() == 0


def test_tree_drafts_and_the_call_without_allocations():
    """The tree drafts propose over a shared prompt what they propose over the whole context; spec_verify_noalloc gives
    the bits of spec_verify over 8-bit and shared caches."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES["hd64"], seed=23, max_rows=64, max_batch=2, max_position=512)
    prompt = make_tokens(90, shape.vocab, seed=24)
    suffixes = [make_tokens(5, shape.vocab, seed=25), make_tokens(17, shape.vocab, seed=26)]
    par = [int(p) for p in tree_parents([2, 2])]
    n = len(par)
    whole = spec.KVCache(model, 2, 160)
    t1 = _i32(2)
    for b, s in enumerate(suffixes):
        spec.spec_prefill(model, whole, b, cuda_i32(np.concatenate([prompt, s])), next_tok=t1[b:b + 1])
    scratch = torch.empty(2 * n, shape.vocab, device="cuda")
    ref, refL = _i32(2, n), torch.empty(2, n, shape.d_model, device="cuda")
    spec.spec_draft_tree(model, whole, t1, par, ref, refL, scratch)
    for q8 in (False, True):
        kv, t0 = _continuations(model, prompt, suffixes, q8=q8, prompt_q8=q8)
        tok, hL = _i32(2, n), torch.empty(2, n, shape.d_model, device="cuda")
        spec.spec_draft_tree(model, kv, t1, par, tok, hL, scratch)
        par_d, n_d, tok_d = _i32(2, n), _i32(2), _i32(2, n)
        spec.spec_draft_tree_dynamic(model, kv, t1, [2, 2], 1.5, tok_d, par_d, n_d, hL.clone(), scratch)
        assert n_d.tolist() == [n, n] and torch.equal(tok_d, tok)
        if not q8:
            # the states differ by the queries' rounding only
            assert torch.equal(t0, t1) and torch.equal(tok, ref)
            assert (hL - refL).abs().max() < TOL
        a, b = (torch.empty(2 * n, shape.vocab, device="cuda") for _ in range(2))
        spec.spec_verify(model, kv, [n, n], tok, n, h_in=hL, h_stride=n, tree_parent=par, logits=a)
        spec.spec_verify_noalloc(model, kv, [n, n], tok, n, h_in=hL, h_stride=n, tree_parent=par, logits=b)
        assert torch.equal(a, b)
    assert model.device_error() == 0


def test_without_a_prefix_nothing_changes():
    """A cache that had a prefix and lost it gives the bits of one that never had; a cache that serves as prefix too."""
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES["hd64"], seed=17, max_rows=16, max_batch=2, max_position=256)
    toks = cuda_i32(make_tokens(40, shape.vocab, seed=18))
    cand = cuda_i32(make_tokens(4, shape.vocab, seed=19))
    a, b = (torch.empty(4, shape.vocab, device="cuda") for _ in range(2))
    kv, other = spec.KVCache(model, 1, 64), spec.KVCache(model, 1, 64)
    spec.spec_prefill(model, kv, 0, toks)
    spec.spec_prefill(model, other, 0, toks)
    spec.spec_verify(model, kv, [4], cand, 4, logits=a)
    other.set_prefix(kv)
    spec.spec_verify(model, other, [4], cand, 4, logits=b)
    assert not torch.equal(a, b)
    other.set_prefix(None)
    spec.spec_verify(model, other, [4], cand, 4, logits=b)
    assert torch.equal(a, b)
    spec.spec_verify(model, kv, [4], cand, 4, logits=b)
    assert torch.equal(a, b) and model.device_error() == 0


def test_the_model_calls_stop_at_a_destroyed_prompt():
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES["hd64"], seed=20, max_rows=16, max_batch=2, max_position=256)
    kv, t0 = _continuations(model, make_tokens(9, shape.vocab, seed=21), [make_tokens(2, shape.vocab, seed=22)])
    kv.prefix.close()
    cand, hL = _i32(1, 3), torch.empty(1, 3, shape.d_model, device="cuda")
    with pytest.raises(spec.SpecError, match="prefix was destroyed"):
        spec.spec_draft(model, kv, t0, 2, cand, hL)
    with pytest.raises(spec.SpecError, match="prefix was destroyed"):
        spec.spec_prefill(model, kv, 0, t0)
    with pytest.raises(spec.SpecError, match="prefix was destroyed"):
        spec.spec_verify(model, kv, [1], t0, 1)
