"""The library's build does not depend on the extension module's (no GPU needed)."""
import ctypes
import os

import pytest

from paged_kv_cache_311_gb300 import build as b


def test_library_is_linked_where_the_module_does_not_compile(tmp_path, monkeypatch):
    """The C library is there, and the module's failure is still an error."""
    monkeypatch.setattr(b, "SOURCES", ["pkv_usage.cu"])

    def fails(path):
        raise RuntimeError("no such header")

    monkeypatch.setattr(b, "build_torch_module", fails)
    out = str(tmp_path / "libpkv.so")
    with pytest.raises(RuntimeError, match="no such header"):
        b.build(out_path=out)
    assert os.path.exists(out)
    assert ctypes.CDLL(out).pkv_kv_cache_usage
