"""The compiled form of the Python calls (csrc/calls.cpp) is an addition: where it does not compile or load, the library is
built and loaded all the same, with a warning, and the Python form of the calls runs."""
import pytest

from sequence_sharded_exact_gb300 import binding, build_lib


@pytest.mark.parametrize("compiler", ["false", "/nowhere/a-compiler"])
def test_a_build_without_them(monkeypatch, tmp_path, compiler):
    target = tmp_path / "calls.so"
    target.write_bytes(b"of older sources")
    build_lib.os.utime(target, (1, 1))
    monkeypatch.setattr(build_lib, "calls_path", lambda: str(target))
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(RuntimeWarning, match="calls.cpp"):
        assert build_lib.build() == build_lib.LIB
    assert not target.exists()  # what the sources no longer are is not left to be loaded


@pytest.mark.parametrize("content", [b"", b"no library", b"\x7fELF" + bytes(100)])
def test_a_file_that_does_not_load(monkeypatch, tmp_path, content):
    path = tmp_path / "calls.so"
    path.write_bytes(content)
    lib = binding.library()
    monkeypatch.setattr(build_lib, "calls_path", lambda: str(path))
    monkeypatch.setattr(binding, "_calls", None)
    with pytest.warns(RuntimeWarning, match="compiled calls"):
        binding._load_calls(lib)
    assert binding._calls is None


def test_a_library_without_the_calls_they_need(monkeypatch):
    """An older library beside them: nothing is bound, the library still loads."""
    class Old:
        def __getattr__(self, name):
            raise AttributeError(name)

    binding.library()
    monkeypatch.setattr(binding, "_calls", None)
    with pytest.warns(RuntimeWarning, match="compiled calls"):
        binding._load_calls(Old())
    assert binding._calls is None
