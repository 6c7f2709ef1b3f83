"""Weights far below a row's largest one, values far below the others, and queries in 32 bits: what the attention's
operands of 16 bits must not lose."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


class Keys:
    """One KV head of `dim`, `rows` query vectors (1, ..) a sequence, `n` keys of given first elements and values."""

    def __init__(self, dim, rows, scores, values, prompt, q8, own_q8=True):
        from _attend_util import head_model
        from speculative_decoding_verify_04_gb300 import spec
        self.model = head_model(1, 1, dim, max_rows=256, max_batch=4)
        # q = 8 e0, so that a key's score is k0 8 / sqrt(dim); dim 1 keeps the rows of K from being zeros
        n = scores.numel()
        k = torch.zeros(n, 1, dim)
        k[:, 0, 0] = scores
        k[:, 0, 1] = 1.0
        self.k, self.v = k.to(torch.bfloat16), values[:, None].to(torch.bfloat16)
        self.kv = spec.KVCache(self.model, 4, 64 if prompt else n + 16, q8=own_q8)
        self.q = torch.zeros(4 * rows, 1, dim, dtype=torch.bfloat16)
        self.q[:, 0, 0] = 8.0
        self.rows, self.dim = rows, dim
        if prompt:
            self.pre = spec.KVCache(self.model, 1, n, q8=q8)
            self.pre.import_rows(0, 0, self.k[None].cuda(), self.v[None].cuda())
            self.pre.set_lengths([n])
            self.kv.set_prefix(self.pre)
        else:
            for b in range(4):
                self.kv.import_rows(b, 0, self.k[None].cuda(), self.v[None].cuda())
            self.kv.set_lengths([n] * 4)

    def run(self):
        """The sequences' new rows have scores so low that they count for nothing, and values of zero."""
        from speculative_decoding_verify_04_gb300 import spec
        T = self.q.shape[0]
        k, v = torch.zeros(2, T, 1, self.dim, dtype=torch.bfloat16, device="cuda")
        k[:, 0, 0] = -448.0
        out = torch.empty(T, 1, self.dim, dtype=torch.bfloat16, device="cuda")
        spec.spec_attend(self.kv, 0, [self.rows] * 4, self.q.cuda(), out, k=k.contiguous(), v=v.contiguous())
        assert self.model.device_error() == 0
        return out.double().cpu()

    def want(self):
        from _attend_util import attend64, attend_tol
        n = self.k.shape[0]
        ref, mass, big = attend64(self.q[:1].double(), self.k.double(), self.v.double(), 1.0 / math.sqrt(self.dim),
                                  np.ones((1, n), dtype=bool))
        return ref, attend_tol(ref, mass, big, self.dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,prompt", [(1, False), (5, False), (12, False), (1, True), (32, True)])
def test_many_weights_far_below_the_largest(dim, rows, prompt):
    """In every 16 keys one has weight 1 and shows in dim 0, the others weigh 2^-26 and alone show in dim 1."""
    n = 16 * 80
    # 2^-26 or somewhat less: -18 at 64 dims, -26 * 8 / sqrt(128) = -18.4 at 128; both are e4m3 numbers
    scores = torch.full((n,), -18.0 if dim == 64 else -26.0)
    scores[::16] = 0.0
    values = torch.zeros(n, dim)
    values[:, 1] = 1.0
    values[::16] = 0.0
    values[::16, 0] = 1.0
    c = Keys(dim, rows, scores, values, prompt, True)
    out, (ref, tol) = c.run(), c.want()
    # half-precision operands under a prompt: each weight off by at most 2^-32 of the row's largest, whose weight
    # is 1 / 80 of the sum; elsewhere by 2^-40 of it
    tol = tol + n * (2.0 ** -32 if prompt and rows > 16 else 2.0 ** -40) / 80
    assert 10 * tol[0, 0, 1] < ref[0, 0, 1]
    assert ((out - ref).abs() <= tol).all(), ((out - ref).abs() / tol).amax()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 12, 32])
def test_a_value_far_below_the_others(dim, rows):
    """One key has all of the weight, its value is far below the smallest that half precision holds; the others'
    values are ordinary."""
    n = 40
    g = torch.Generator().manual_seed(3)
    scores = torch.full((n,), -240.0)                    # weights below 2^-170
    scores[17] = 0.0
    values = torch.randn(n, dim, generator=g)
    values[17] = values[17].sign() * torch.linspace(1.0, 1.75, dim) * 2.0 ** -116
    c = Keys(dim, rows, scores, values, True, True)
    from _attend_util import rows8
    c.v = torch.from_numpy(rows8(c.v.double().numpy())[2])
    out, (ref, tol) = c.run(), c.want()
    # weights below 2^-126 may be flushed to zero; the reference's are below 2^-170
    assert (ref.abs() > 2.0 ** -117).all()
    assert ((out - ref).abs() <= tol).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_forward_calls_keep_queries_of_32_bits_under_any_dispatch(dim, q8):
    """A verification over a prompt held in a short and in a long cache: one goes to the row kernel, one to the tile
    kernel, everything else is the same.  One layer with an identity O projection, no MLP and an identity LM head, so
    that a logit is an element of (embedding + attention) / rms."""
    from _attend_util import attend64
    from _gpu_util import cuda_i32, lib, to_cuda
    from oracle.decoder import linear, rms_norm, rope
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens, make_weights, weights_to_numpy
    lib()
    H, Hkv, n, B, R = 512 // dim, 128 // dim, 300, 4, 4
    shape = ModelShape(1, 512, H, Hkv, dim, 512, 512, 0, "bf16")
    w = make_weights(shape, 70)
    lw = w["layers"][0]
    for name, std in (("wq", 5.0), ("wk", 1.0), ("wv", 1.0)):
        lw[name] = (lw[name].float() * (std / 0.02 / math.sqrt(512))).to(torch.bfloat16)
    lw["wo"], w["lm_head"] = torch.eye(512).to(torch.bfloat16), torch.eye(512).to(torch.bfloat16)
    lw["w_down"].zero_()
    wn = weights_to_numpy(w)
    model = spec.Model(shape, to_cuda(w), max_rows=64, max_batch=B, max_position=512)
    g = torch.Generator(device="cuda").manual_seed(71)
    k, v = (torch.randn(1, n, Hkv, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    toks = np.stack([make_tokens(R, 512, seed=72 + b) for b in range(B)])
    got = []
    # 16 rows of 4 heads a KV head are 64 vectors: the tile kernel takes them where the cache is long
    for cap in (n, 40000):
        pre, kv = spec.KVCache(model, 1, cap, q8=q8), spec.KVCache(model, B, 64, q8=q8)
        pre.import_rows(0, 0, k, v)
        pre.set_lengths([n])
        kv.set_prefix(pre)
        logits = torch.empty(B, R, 512, device="cuda")
        launches = model.launch_count()
        spec.spec_verify(model, kv, [R] * B, cuda_i32(toks), R, logits=logits)
        got.append((logits.double().cpu(), model.launch_count() - launches))
    (a, la), (b, lb) = got
    assert lb == la + 1                                  # the tile kernel is one launch more
    pk, pv = (x[0].double().cpu() for x in pre.export_rows(0, 0, 1, 0, n))
    for s in range(B):
        h = np.asarray(wn["embed"][toks[s]], dtype=np.float64)
        q = linear(rms_norm(h, wn["layers"][0]["attn_norm"], shape.rms_eps), wn["layers"][0]["wq"]).reshape(R, H, dim)
        q = torch.from_numpy(np.stack([rope(q[t], n + t, shape.rope_theta) for t in range(R)]))
        nk, nv = (x[0].double().cpu() for x in kv.export_rows(s, 0, 1, 0, R))
        sees = np.concatenate([np.ones((R, n), dtype=bool), np.tril(np.ones((R, R), dtype=bool))], 1)
        out, mass, big = attend64(q, torch.cat([pk, nk]), torch.cat([pv, nv]), 1.0 / math.sqrt(dim), sees)
        # a path's error: queries in two bf16 parts, each off by 2^-8 of what it holds (together 2^-16), and f32 sums of
        # two products a dim; weights off by d move the mean by 2 d mass; a weight's operand is off by 2^-16 (bf16 pair)
        # or 2^-11 (f16, 8-bit caches; 2^-32 of the row's largest below 2^-24 of it); f32 sums over the keys
        d = (2.0 ** -16 + 2 * dim * 2.0 ** -24) * big[..., None] + 2.0 ** -21
        e = (2 * d + (2.0 ** -11 if q8 else 2.0 ** -16) + (n + R) * 2.0 ** -24) * mass
        if q8:
            e = e + (n + R) * 2.0 ** -32 * torch.cat([pv, nv]).abs().amax()
        e = (2 * e + 2 * 2.0 ** -16 * out.abs()).reshape(R, 512)       # two paths, each output as a bf16 pair
        y = torch.from_numpy(h) + out.reshape(R, 512)
        rms = (y.square().mean(-1, keepdim=True) + shape.rms_eps).sqrt()
        y = y / rms
        # the logits: the same norm of both, its input a bf16 pair
        tol = e / rms + y.abs() * (e.amax(-1, keepdim=True) / rms + 2.0 ** -14)
        off = (a[s] - b[s]).abs()
        assert ((a[s] - y).abs() < 0.05).all()           # (the formula is the model's)
        assert (off <= tol).all(), (off / tol).amax()
    assert model.device_error() == 0


@pytest.mark.parametrize("q8", [False, True])
def test_32_layers_over_a_shared_prompt(q8):
    """A deep model's verification over a prompt in the tile kernel: against the oracle within the bound of the bf16
    path, and (8-bit prompts, whose values the oracle does not round) against the row kernel's."""
    from _gpu_util import cuda_i32, lib, model_pair
    from oracle import spec as OS
    from speculative_decoding_verify_04_gb300 import spec
    from synthetic import ModelShape, make_tokens
    from test_gpu_shared_prompt import TOL
    lib()
    B, R, n = 6, 4, 150
    model, dec, shape = model_pair(ModelShape(32, 256, 8, 2, 64, 512, 2048, 1, "bf16"), seed=75, max_rows=64, max_batch=B,
                                   max_position=512)
    prompt = make_tokens(n, shape.vocab, seed=76)
    toks = np.stack([make_tokens(R, shape.vocab, seed=77 + b) for b in range(B)])
    pre, kv = spec.KVCache(model, 1, n, q8=q8), spec.KVCache(model, B, 64, q8=q8)
    spec.spec_prefill(model, pre, 0, cuda_i32(prompt))
    kv.set_prefix(pre)
    got = torch.empty(B, R, shape.vocab, device="cuda")
    spec.spec_verify(model, kv, [R] * B, cuda_i32(toks), R, logits=got)     # 96 vectors a KV head
    for b in range(B):
        if q8:
            # one sequence's 16 vectors
            want = torch.empty(R, shape.vocab, device="cuda")
            spec.spec_verify(model, kv, [R], cuda_i32(toks[b]), R, logits=want)
            want = want.cpu().numpy()
        else:
            cache = dec.new_cache(n + R)
            dec.prefill(cache, prompt)
            want = OS.verify(dec, cache, n, dec.embed(toks[b]), 0)
        assert np.abs(got[b].cpu().numpy() - want).max() < TOL, b
    assert model.device_error() == 0
