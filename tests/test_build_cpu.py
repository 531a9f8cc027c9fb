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


def test_builds_at_the_same_time_do_not_share_a_file(monkeypatch, tmp_path):
    """Two builds of the binding, the second while the first one's compiler is
    still at work: each writes a file of its own and puts it in place whole; a
    compiler that fails leaves nothing behind."""
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    written = []

    def compiler(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        written.append(out)
        if len(written) == 1:
            build.build_bind()
        if len(written) == 3:
            raise RuntimeError("compiler failed")
        with open(out, "w") as f:
            f.write("library %d" % written.index(out))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    path = build.build_bind()
    assert len(set(written)) == 2 and path not in written
    assert open(path).read() == "library 0"
    with pytest.raises(RuntimeError):
        build.build_bind()
    assert [str(p) for p in tmp_path.iterdir()] == [path]
