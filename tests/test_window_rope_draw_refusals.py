"""Argument checks of the window, rotary and draw calls that need no GPU."""
import ctypes
import math

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verify_04_gb300 import build, spec
    build.build()
    return spec.load()


def _err(lib):
    return lib.spec_last_error().decode()


def test_window_without_a_cache(lib):
    assert lib.spec_kv_set_window(None, 0, 1, 10, 0) == -1 and "null" in _err(lib)


def test_rope_arguments(lib):
    from speculative_decoding_verify_04_gb300 import spec
    p, q = P(4096), P(8192)

    def call(H=4, Hkv=2, hd=64, dtype=0, axes=1, sections=(32, 0, 0, 0), inter=0, theta=1e4, rows=3, src=p, dst=q, stride=256,
             k=p, ko=q, ks=128, pos=p, ps=3, kv=None, batch=0, n=None, no_cfg=False):
        cfg = spec.RopeConfig(H, Hkv, hd, dtype, axes, (ctypes.c_int32 * 4)(*sections), inter, theta)
        return lib.spec_rope(None if no_cfg else ctypes.byref(cfg), rows, src, stride, dst, stride, k, ks, ko, ks, pos, ps, kv,
                             batch, n, None, None)

    for kw, code, word in ((dict(no_cfg=True), -1, "null"), (dict(dtype=2), -1, "dtype"), (dict(H=-1), -1, "sizes"),
                           (dict(H=0, Hkv=0), -1, "sizes"), (dict(rows=-1), -1, "sizes"), (dict(hd=1), -5, "head_dim"),
                           (dict(hd=258), -5, "head_dim"), (dict(H=5000, stride=1 << 20), -5, "heads"),
                           (dict(theta=0.5), -1, "theta"), (dict(theta=math.nan), -1, "theta"), (dict(theta=math.inf), -1, "theta"),
                           (dict(axes=0), -1, "axes"), (dict(axes=5), -1, "axes"), (dict(sections=(33, 0, 0, 0)), -1, "sections"),
                           (dict(sections=(0, 0, 0, 0)), -1, "sections"), (dict(sections=(-1, 0, 0, 0)), -1, "sections"),
                           (dict(axes=2, sections=(20, 20, 0, 0)), -1, "sections"), (dict(pos=None), -1, "positions or a cache"),
                           (dict(axes=2, sections=(16, 16, 0, 0), ps=2), -1, "pos_stride"), (dict(stride=255), -1, "stride"),
                           (dict(ks=127), -1, "stride"), (dict(src=None), -1, "null"), (dict(dst=None), -1, "null"),
                           (dict(k=None), -1, "null"), (dict(src=P(4098)), -1, "aligned"), (dict(ko=P(4097), dtype=1), -1, "aligned")):
        assert call(**kw) == code and word in _err(lib), (kw, _err(lib))
    assert call(rows=0) == 0
    assert call(rows=0, pos=None) == 0


def test_sample_logits_arguments(lib):
    from speculative_decoding_verify_04_gb300 import spec
    p = P(4096)

    def call(logits=p, dtype=0, stride=100, rows=2, vocab=100, u=p, tok=p, lp=None, pr=None, ps=0, no_cfg=False, T=1.0, top_p=1.0,
             min_p=0.0, top_k=0):
        cfg = spec.SampleConfig(T, top_p, min_p, top_k)
        return lib.spec_sample_logits(logits, dtype, stride, rows, vocab, u, None if no_cfg else ctypes.byref(cfg), tok, lp, pr, ps,
                                      None)

    for kw, code, word in ((dict(no_cfg=True), -1, "null"), (dict(dtype=2), -1, "dtype"), (dict(rows=-1), -1, "sizes"),
                           (dict(vocab=0), -1, "sizes"), (dict(stride=99), -1, "sizes"), (dict(pr=p, ps=99), -1, "sizes"),
                           (dict(vocab=(1 << 20) + 1, stride=1 << 21), -5, "1048576"), (dict(rows=1 << 30), -5, "rows"),
                           (dict(T=-1.0), -1, "temperature"), (dict(T=math.nan), -1, "temperature"),
                           (dict(T=math.inf), -1, "temperature"), (dict(T=1e-31), -1, "temperature"),
                           (dict(top_k=-1), -1, "top_k"), (dict(top_p=-0.1), -1, "top_p"), (dict(top_p=math.nan), -1, "top_p"),
                           (dict(min_p=-0.1), -1, "min_p"), (dict(min_p=1.1), -1, "min_p"), (dict(min_p=math.nan), -1, "min_p"),
                           (dict(logits=None), -1, "null"), (dict(u=None), -1, "null"), (dict(tok=None), -1, "null"),
                           (dict(logits=P(4098)), -1, "aligned"), (dict(logits=P(4097), dtype=1), -1, "aligned")):
        assert call(**kw) == code and word in _err(lib), (kw, _err(lib))
    assert call(rows=0) == 0


def test_binding_refuses_host_tensors(lib):
    import torch
    from speculative_decoding_verify_04_gb300 import spec
    if not torch.cuda.is_available():
        pytest.skip("the binding asks for the current device first")
    with pytest.raises(spec.SpecError, match="logits"):
        spec.spec_sample_logits(torch.zeros(2, 10), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(1, 2, 64)
    with pytest.raises(spec.SpecError, match="q: need a CUDA"):
        spec.spec_rope(q, q, positions=torch.zeros(1, dtype=torch.int32))


def test_window_binding_refuses_a_closed_cache():
    from speculative_decoding_verify_04_gb300 import spec
    kv = spec.KVCache.__new__(spec.KVCache)
    kv.handle = None
    with pytest.raises(spec.SpecError, match="closed"):
        kv.set_window(10)
