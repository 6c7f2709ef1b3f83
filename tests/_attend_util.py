"""Plain 64-bit forms of the 8-bit cache rows, the attention over a shared prompt and
the log probabilities, and model handles of a given head layout (test infrastructure)."""
from __future__ import annotations

import math
from types import SimpleNamespace

import numpy as np
import torch


def head_model(heads, kv_heads, dim, layers=1, max_rows=256, max_batch=16, dtype="bf16"):
    """A library model whose weights are zero: the cache and attention calls need only its shape."""
    from _gpu_util import lib
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = SimpleNamespace(n_layers=layers, d_model=64, n_heads=heads, n_kv_heads=kv_heads, head_dim=dim, d_ff=64,
                            vocab=128, exit_layer=0, dtype=dtype, rms_eps=1e-5, rope_theta=10000.0)

    def z(*s):
        return torch.zeros(s, dtype=t, device="cuda")

    layer = {"attn_norm": z(64), "wq": z(heads * dim, 64), "wk": z(kv_heads * dim, 64), "wv": z(kv_heads * dim, 64),
             "wo": z(64, heads * dim), "ffn_norm": z(64), "w_gate": z(64, 64), "w_up": z(64, 64), "w_down": z(64, 64)}
    w = {"embed": z(128, 64), "lm_head": z(128, 64), "final_norm": z(64), "layers": [layer] * layers}
    return spec.Model(shape, w, max_rows=max_rows, max_batch=max_batch, max_position=1)


def rows8(x):
    """(bytes, exponents + 127, values) of rows x[..., dim] (float64 in, numpy out) in the 8-bit form."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    _, p = np.frexp(mag / 448.0)                        # mag / 448 = m 2^p, m in [0.5, 1): 2^(p-1) is too small unless m = 0.5
    e = np.where(mag == np.ldexp(448.0, p - 1), p - 1, p)
    e = np.where(mag == 0, -124, np.clip(e, -124, 119)).astype(int)
    y = x / np.ldexp(1.0, e)[..., None]
    a = np.minimum(np.where(np.isnan(y), 0.0, np.abs(y)), 448.0)
    binade = np.maximum(np.frexp(a)[1] - 1, -6)
    n = np.rint(np.ldexp(a, 3 - binade))                # in units of the binade's spacing, ties to even
    a = np.ldexp(n, binade - 3)
    # the value's code: exponent field binade + 7 with 3 bits of mantissa, or a subnormal
    b2 = np.maximum(np.frexp(a)[1] - 1, -6)
    m = np.ldexp(a, 3 - b2).astype(int)
    code = np.where(a < 2.0 ** -6, np.ldexp(a, 9).astype(int), ((b2 + 7) << 3) | (m & 7))
    code = np.where(np.isnan(x), 0x7F, code) | np.where(np.signbit(x), 0x80, 0)
    val = np.where(np.isnan(x), np.nan, np.copysign(a, x)) * np.ldexp(1.0, e)[..., None]
    return code.astype(np.uint8), (e + 127).astype(np.uint8), val


def chain_mask(n):
    return np.tril(np.ones((n, n), dtype=bool))


def tree_mask(parents):
    n = len(parents)
    m = np.eye(n, dtype=bool)
    for i in range(1, n):
        m[i] |= m[parents[i]]
    return m


def attend64(q, keys, vals, scale, sees):
    """out[R, H, hd] and the bound's two sums for one sequence: q [R, H, hd], keys and vals
    [N, Hkv, hd] (float64 tensors), sees [R, N] bool.  Also sum p |v| and max |q|.|k| scale."""
    R, H, hd = q.shape
    Hkv = keys.shape[1]
    G = H // Hkv
    kk = keys.repeat_interleave(G, 1)
    vv = vals.repeat_interleave(G, 1)
    hide = ~torch.as_tensor(sees)[:, None]
    clean_k = torch.where(torch.as_tensor(sees).any(0)[:, None, None], kk, torch.zeros_like(kk))
    clean_v = torch.where(torch.as_tensor(sees).any(0)[:, None, None], vv, torch.zeros_like(vv))
    s = (torch.einsum("rhd,nhd->rhn", q, clean_k) * scale).masked_fill(hide, -math.inf)
    p = torch.softmax(s, -1)
    big = (torch.einsum("rhd,nhd->rhn", q.abs(), clean_k.abs()) * scale).masked_fill(hide, 0).amax(-1)
    return torch.einsum("rhn,nhd->rhd", p, clean_v), torch.einsum("rhn,nhd->rhd", p, clean_v.abs()), big


def attend_tol(out, mass, big, hd):
    """Elementwise bound of the kernels' error.  The result is rounded to bf16 once: 2^-8 |out|.
    Every probability may be rounded to bf16 before its product: 2^-8 sum p |v| = 2^-8 mass.  A score
    is off by the f32 sum of hd products, hd 2^-24 sum |q k| scale, and its 2^x by 2^-21; a relative
    error d of the weights moves the mean by at most 2 d mass (numerator and denominator)."""
    d = hd * 2.0 ** -24 * big[..., None] + 2.0 ** -21
    return 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2 * d + 2.0 ** -16) * mass
