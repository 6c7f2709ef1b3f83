"""Argument checks of the cache, attention and log-probability calls that need no GPU."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verify_04_gb300 import build, spec
    build.build()
    return spec.load()


def _err(lib):
    return lib.spec_last_error().decode()


def test_logprobs_arguments(lib):
    p, f = P(4096), ctypes.c_float

    def call(logits=p, dtype=0, stride=100, rows=2, vocab=100, T=1.0, tok=p, lp=p, ent=None, n=0, ids=None, tlp=None):
        return lib.spec_logprobs(logits, dtype, stride, rows, vocab, f(T), tok, lp, ent, n, ids, tlp, None)

    for kw, code, word in ((dict(logits=None), -1, "null"), (dict(dtype=2), -1, "dtype"), (dict(stride=99), -1, "sizes"),
                           (dict(rows=-1), -1, "sizes"), (dict(vocab=0), -1, "sizes"), (dict(T=0.0), -1, "temperature"),
                           (dict(T=-1.0), -1, "temperature"), (dict(T=1e-39), -1, "temperature"),
                           (dict(T=float("nan")), -1, "temperature"), (dict(T=float("inf")), -1, "temperature"),
                           (dict(lp=None), -1, "together"), (dict(tok=None), -1, "together"),
                           (dict(n=33, ids=p, tlp=p), -1, "n_top"), (dict(n=-1), -1, "n_top"),
                           (dict(n=5, vocab=4, ids=p, tlp=p), -1, "n_top"), (dict(n=5, ids=p), -1, "n_top"),
                           (dict(n=0, ids=p, tlp=p), -1, "n_top"), (dict(tok=None, lp=None), -1, "no output"),
                           (dict(logits=P(4098)), -1, "aligned"), (dict(logits=P(4097), dtype=1), -1, "aligned"),
                           (dict(vocab=(1 << 20) + 1, stride=1 << 21), -5, "1048576")):
        assert call(**kw) == code and word in _err(lib), kw
    assert call(rows=0) == 0


def test_attend_and_caches_without_handles(lib):
    n = ctypes.cast((ctypes.c_int32 * 1)(1), P)
    out = P()
    p = P(4096)
    assert lib.spec_attend(None, 0, 1, n, p, 64, None, 0, None, 0, None, p, 64, None) == -1 and "null" in _err(lib)
    assert lib.spec_kv_create_q8(None, 1, 1, 0, 0, ctypes.byref(out)) == -1 and "null" in _err(lib)
    assert lib.spec_kv_set_prefix(None, None, 0) == -1 and "null" in _err(lib)


def test_binding_refuses_host_tensors(lib):
    import torch
    from speculative_decoding_verify_04_gb300 import spec
    with pytest.raises(spec.SpecError, match="logits"):
        spec.spec_logprobs(torch.zeros(2, 10), None, torch.zeros(2))
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for bad in (q, q.float(), q[0], None):
        with pytest.raises(spec.SpecError, match="q: need a CUDA"):
            spec._rows3d(bad, "q", 2, 64, 1, torch.bfloat16, 0)
