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
