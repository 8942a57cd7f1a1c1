"""The marshalling module of the paged wrappers is optional: the library builds and the wrappers work without it."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from flash_attention_backward_gb300 import build as B  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The module goes to a folder of its own; an older one lies there."""
    target = tmp_path / "_fast.so"
    target.write_bytes(b"of an older build")
    os.utime(target, (0, 0))
    monkeypatch.setattr(B, "fast_path", lambda: str(target))
    monkeypatch.setattr(B, "_fast_given_up", False, raising=False)
    return target


def compiler(monkeypatch, folder, text):
    folder.mkdir()
    (folder / "g++").write_text(text)
    (folder / "g++").chmod(0o755)
    monkeypatch.setenv("PATH", str(folder) + os.pathsep + os.environ["PATH"])


def test_a_compiler_that_fails_leaves_the_library_and_a_warning(monkeypatch, tmp_path, elsewhere):
    log = tmp_path / "calls"
    compiler(monkeypatch, tmp_path / "bin", "#!/bin/sh\necho called >> %s\n"
             "while [ $# -gt 0 ]; do [ \"$1\" = -o ] && echo partial > \"$2\"; shift; done\necho no such header; exit 1\n" % log)
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB)
    assert os.listdir(elsewhere.parent) in (["calls", "bin"], ["bin", "calls"])  # neither the older module nor half of a new one
    B.build()  # not tried again in this process
    assert log.read_text().count("called") == 1


def test_no_compiler_and_no_torch(monkeypatch, tmp_path, elsewhere):
    (tmp_path / "empty").mkdir()
    monkeypatch.setenv("PATH", str(tmp_path / "empty"))
    with pytest.warns(RuntimeWarning, match="FileNotFoundError"):
        assert B.build() == B.LIB
    monkeypatch.setattr(B, "_fast_given_up", False, raising=False)
    assert not elsewhere.exists()


def test_without_torch_the_library_is_built(monkeypatch):
    monkeypatch.setattr(B, "_fast_given_up", False)
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert B.fast_path() is None
    with pytest.warns(RuntimeWarning, match="no PyTorch"):
        assert B.build() == B.LIB


def test_a_library_that_fails_stops_the_modules_compiler(monkeypatch, tmp_path, elsewhere):
    compiler(monkeypatch, tmp_path / "bin", "#!/bin/sh\nexec sleep 600\n")
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))

    def fails(verbose):
        raise RuntimeError("nvcc failed")

    monkeypatch.setattr(B, "_build_library", fails)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()
    assert sorted(os.listdir(tmp_path)) == ["bin"]


def test_a_module_of_another_torch_or_interpreter_is_not_taken(monkeypatch):
    from flash_attention_backward_gb300 import paged
    here = B.fast_path()
    assert os.path.exists(here) and paged._load_fast() is not None
    assert torch.__version__ in here and here.endswith(B.sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert B.fast_path() != here and not B.up_to_date() and paged._load_fast() is None


def test_a_module_built_after_the_import_is_taken(monkeypatch, tmp_path):
    """Import, then build in the same process, as from a fresh tree."""
    import shutil

    from flash_attention_backward_gb300 import paged
    fresh = str(tmp_path / os.path.basename(B.fast_path()))
    old = B.fast_path()
    for m in (B, paged):
        monkeypatch.setattr(m, "fast_path", lambda: fresh)
    monkeypatch.setattr(paged, "_fast", None)
    monkeypatch.setattr(paged, "_plain", False)
    assert paged._load_fast() is None
    monkeypatch.setattr(B, "_fast_command", lambda out: ["cp", old, out])  # (its compiler takes a while)
    B.build()
    assert paged._fast is not None and callable(paged._fast.decode) and not paged._plain
    was = paged._fast
    shutil.copy(old, fresh)
    paged.look_for_fast()
    assert paged._fast is was
