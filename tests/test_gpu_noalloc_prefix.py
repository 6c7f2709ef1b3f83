"""spec_verify_noalloc checks a cache's prefix before it enqueues anything."""
import pytest
import torch

from _gpu_util import cuda_i32, lib, model_pair
from synthetic import make_tokens
from test_gpu_shared_prompt import SHAPES, _continuations

pytestmark = pytest.mark.gpu


def test_a_destroyed_prefix_is_refused_before_anything_is_enqueued():
    from speculative_decoding_verify_04_gb300 import spec
    lib()
    model, _, shape = model_pair(SHAPES["hd64"], seed=20, max_rows=16, max_batch=2, max_position=256)
    kv, t0 = _continuations(model, make_tokens(9, shape.vocab, seed=21), [make_tokens(2, shape.vocab, seed=22)])
    logits = torch.empty(1, shape.vocab, device="cuda")
    spec.spec_verify_noalloc(model, kv, [1], cuda_i32([3]), 1, logits=logits)
    kv.prefix.close()
    # its own check, ahead of the clearing of its counters, not the one of the call that it ends in
    with pytest.raises(spec.SpecError, match="spec_verify_noalloc: the cache's prefix was destroyed"):
        spec.spec_verify_noalloc(model, kv, [1], cuda_i32([3]), 1, logits=logits)
    kv.set_prefix(None)
    spec.spec_verify_noalloc(model, kv, [1], cuda_i32([3]), 1, logits=logits)
    assert model.device_error() == 0
