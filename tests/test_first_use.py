"""The first use of the library from several threads: nothing is seen half made. (Watched, not raced.)"""
import sys

import pytest


@pytest.fixture
def kvx(monkeypatch):
    import kv_cache_attention_02_gb300 as k
    k.lib()
    for name, value in (("_lib", None), ("_loaded", None), ("_IN", {}), ("_OUT", {})):
        monkeypatch.setattr(k, name, value)
    return k


def test_the_library_is_published_with_its_signatures(kvx, monkeypatch):
    """A call without them passes 64-bit pointers as 32-bit numbers."""
    class Watched(dict):
        def items(self):
            for x in super().items():
                assert kvx._lib is None
                yield x
    monkeypatch.setattr(kvx, "SIGNATURES", Watched(kvx.SIGNATURES))
    found = kvx.lib()
    assert found is kvx._lib and all(getattr(found, name).argtypes == args for name, (_, args) in dict.items(kvx.SIGNATURES))


def test_torch_is_published_with_its_types(kvx):
    pytest.importorskip("torch")
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is kvx._torch.__code__:
            seen.append(kvx._loaded is None or bool(kvx._IN and kvx._OUT))
            return trace
    old = sys.gettrace()
    sys.settrace(trace)
    try:
        kvx._torch()
    finally:
        sys.settrace(old)
    assert len(seen) > 4 and all(seen)
