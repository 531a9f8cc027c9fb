"""What is built when: the CUDA library by itself, the native half of the
recurrent layer's calls only for those calls."""
import pytest

from quantized_recurrent_state_lq_b200 import build, lq


def test_the_library_loads_without_the_binding(monkeypatch):
    """A caller of the state's calls needs no host compiler and no headers of
    torch: loading liblq.so neither builds nor loads the binding."""
    def no_compiler(*a, **k):
        raise FileNotFoundError("g++")
    monkeypatch.setattr(build, "bind_stale", lambda: True)
    monkeypatch.setattr(build, "build_bind", no_compiler)
    monkeypatch.setattr(build, "_stale", lambda: False)
    monkeypatch.setattr(lq, "_lib", None)
    monkeypatch.setattr(lq, "_native", None)
    assert lq.strerror(lq.LQ_OK) == "ok"
    assert build.build() == build.OUT
    with pytest.raises(FileNotFoundError):      # and the calls that need it say so
        lq._binding()


def test_a_binding_of_another_torch_or_python_is_not_taken(monkeypatch):
    """The binding holds the layouts of the torch and Python it was compiled
    against: under another of either it counts as missing."""
    import sysconfig

    import torch
    if build.bind_stale():
        build.build_bind()
    here = build.bind_path()
    assert not build.bind_stale()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert build.bind_stale() and build.bind_path() != here
    monkeypatch.undo()
    assert not build.bind_stale()
    var = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else var(n))
    assert build.bind_stale() and build.bind_path() != here
