"""The library is built and loaded without the latent calls' extension; the
extension's file is one of its own torch and Python."""
import os
import sysconfig
from importlib import metadata

import pytest

from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from sparse_attention_indexer_mxfp4_gb300 import build as _build


@pytest.fixture
def no_extension(monkeypatch, tmp_path):
    """No extension on disk or loaded, and a compiler that cannot make one."""
    B.lib()
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(_build, "_calls_command", lambda out: ["false"])
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "_calls", None)
    monkeypatch.delenv("IDX_NO_BUILD", raising=False)


def test_library_without_the_extension(no_extension):
    assert B.version() and B.latent_prefill_workspace_size(4, 999, 2) > 0
    with pytest.raises(RuntimeError, match="bind_latent"):
        B._latent_calls()


def test_build_of_both_tells_of_the_extension(no_extension):
    before = os.path.getmtime(_build.LIB)
    with pytest.raises(RuntimeError, match="bind_latent"):
        _build.build()
    assert os.path.getmtime(_build.LIB) == before  # it was up to date, and stays


def test_library_alone_where_nothing_is_built(no_extension, monkeypatch):
    monkeypatch.setenv("IDX_NO_BUILD", "1")
    assert B.version()
    with pytest.raises(B.IndexerError, match="is missing"):
        B._latent_calls()


def test_extension_is_named_by_what_it_was_built_for():
    name = os.path.basename(_build.CALLS)
    assert metadata.version("torch") in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
