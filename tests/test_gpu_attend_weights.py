"""Weights far below a row's largest one and values far below the others: what the attention's operands of 16 bits must
not lose."""
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
