"""Host logic of the runners, with the CUDA calls stood in for."""
import contextlib
from types import SimpleNamespace

import torch

from quantized_recurrent_state_lq_b200 import configs, runner


def test_scan_runner_captures_on_its_own_device(monkeypatch):
    """A runner on cuda:1 while cuda:0 is current: the side stream, the graph and
    the steps under them belong to cuda:1 (a stream of cuda:0 would capture
    nothing of the steps, which run on their tensors' device)."""
    now, used = ["cuda:0"], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], str(d)
        yield
        now[0] = before

    def on_device(what):
        @contextlib.contextmanager
        def ctx(*a, **k):
            used.append((what, now[0]))
            yield
        return ctx

    def stream(*a, **k):
        used.append(("stream", str(k["device"]) if k.get("device") else now[0]))
        return SimpleNamespace(wait_stream=lambda s: None)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "Stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch.cuda, "stream", on_device("under stream"))
    monkeypatch.setattr(torch.cuda, "graph", on_device("under graph"))
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: None)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: SimpleNamespace(device=k["device"]))
    monkeypatch.setattr(torch, "zeros_like", lambda t: t)
    held = SimpleNamespace(device=torch.device("cuda:1"), clone=lambda: None, copy_=lambda t: None)
    r = object.__new__(runner.ScanRunner)
    r.sl, r.B, r.dtype, r.window, r.state = configs.TINY_SCAN, 2, torch.bfloat16, held, held
    r.step = lambda x, res: used.append(("step", now[0]))
    r.capture()
    assert [u[0] for u in used].count("step") == 2 and ("under graph", "cuda:1") in used
    assert all(d == "cuda:1" for _, d in used), used
    assert now[0] == "cuda:0"
