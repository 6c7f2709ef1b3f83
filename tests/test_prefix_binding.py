"""A cache that is closed cannot become a prefix: its missing handle must not read as "no prefix"."""
import pytest


def test_a_closed_prefix_is_refused(monkeypatch):
    from speculative_decoding_verify_04_gb300 import spec

    class Library:
        """Takes every call as the library does where both handles are caches, or the prefix is null."""
        calls = []

        def spec_kv_set_prefix(self, kv, prefix, seq):
            self.calls.append(prefix)
            return 0

    lib = Library()
    monkeypatch.setattr(spec, "load", lambda: lib)
    kv, closed, other = (object.__new__(spec.KVCache) for _ in range(3))
    kv.handle, closed.handle, other.handle = 1, None, 2
    kv.prefix = None
    try:
        with pytest.raises(spec.SpecError, match="closed"):
            kv.set_prefix(closed)
        assert lib.calls == [] and kv.prefix is None
        kv.set_prefix(other)
        kv.set_prefix(None)
        assert lib.calls == [2, None]
    finally:
        for x in (kv, other):
            x.handle = None                       # nothing for the library to free
