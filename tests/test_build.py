"""The build of the native marshalling module (CPU): it reads torch's C++ objects, so it belongs to one torch."""
import os

import pytest

import paged_kv_cache_kvc_gb300 as kvc
from paged_kv_cache_kvc_gb300 import build


@pytest.fixture
def module(tmp_path, monkeypatch):
    """A module file newer than its sources, stamped as built against what runs now."""
    path = tmp_path / "_kvc_call.so"
    path.write_bytes(b"old")
    (tmp_path / "_kvc_call.so.abi").write_text(build.call_abi())
    monkeypatch.setattr(build, "CALL_PATH", str(path))
    monkeypatch.setattr(build, "CALL_STAMP", str(path) + ".abi")
    return path


def test_another_torch_makes_the_module_stale(module, monkeypatch):
    import torch
    assert not build.call_stale()
    monkeypatch.setattr(torch, "__version__", "2.0.0")
    assert build.call_stale()
    monkeypatch.undo()


def test_a_module_without_a_stamp_or_older_than_its_sources_is_stale(module):
    os.remove(build.CALL_STAMP)
    assert build.call_stale()
    with open(build.CALL_STAMP, "w") as f:
        f.write(build.call_abi())
    assert not build.call_stale()
    os.utime(module, (1, 1))
    assert build.call_stale()


def test_a_module_of_another_torch_is_not_loaded(module, monkeypatch):
    if not os.path.exists(kvc.LIB_PATH):
        pytest.skip("library not built")
    monkeypatch.setattr(kvc, "_call", None)
    monkeypatch.setattr(kvc, "CALL_PATH", str(module))
    with open(build.CALL_STAMP, "w") as f:
        f.write("torch 2.0.0")
    with pytest.raises(RuntimeError, match="another torch"):
        kvc._native()


def test_files_are_replaced_at_once(tmp_path):
    """A failed build leaves the old file and nothing else; a mapped old file is another file than the new one."""
    path = tmp_path / "m.so"
    path.write_bytes(b"old")

    def fail(tmp):
        with open(tmp, "wb") as f:
            f.write(b"half")
        raise RuntimeError("linker")
    with pytest.raises(RuntimeError, match="linker"):
        build._replace(str(path), fail)
    assert path.read_bytes() == b"old" and os.listdir(tmp_path) == ["m.so"]
    with open(path, "rb") as mapped:
        def make(tmp):
            assert path.read_bytes() == b"old" and os.path.dirname(tmp) == str(tmp_path)
            with open(tmp, "wb") as f:
                f.write(b"new")
        build._replace(str(path), make)
        assert mapped.read() == b"old"
    assert path.read_bytes() == b"new" and os.listdir(tmp_path) == ["m.so"]


def test_the_module_is_linked_beside_its_place():
    compile_, link = build.call_commands("/x/y.so.tmp7")
    assert "/x/y.so.tmp7.o" in compile_ and "/x/y.so.tmp7.o" in link and link[link.index("-o") + 1] == "/x/y.so.tmp7"
