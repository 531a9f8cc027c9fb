"""Refusals of the recurrent layer's calls: every bad argument is reported on
the host before anything is launched (the fake device addresses are never
touched), so these run without a GPU."""
import ctypes as C

import pytest
import torch

from quantized_recurrent_state_lq_b200 import lq

BASE = 0x7f0000000000
GAP = 0x10000000


def at(i, off=0):
    return BASE + i * GAP + off


def conv(cfg=None, **kw):
    cfg = dict(dict(dtype=lq.LQ_BF16, B=2, C=64, K=4, act=lq.LQ_ACT_SILU), **(cfg or {}))
    a = dict(dict(rows=20, cu=None, x=at(0), ldx=64, w=at(1), bias=at(2), s0=at(3), so=at(4), y=at(5), ldy=64), **kw)
    c = lq.lq_conv_config(*[cfg[n] for n in ("dtype", "B", "C", "K", "act")])
    return lq.lib().lq_conv_prefill(C.addressof(c), a["rows"], a["cu"], a["x"], a["ldx"], a["w"], a["bias"], a["s0"],
                                    a["so"], a["y"], a["ldy"], None)


@pytest.mark.parametrize("cfg,kw,code", [
    ({"dtype": 3}, {}, lq.LQ_ERR_INVALID_ARG), ({"act": 2}, {}, lq.LQ_ERR_INVALID_ARG),
    ({"B": 0}, {}, lq.LQ_ERR_SHAPE), ({"C": 0}, {}, lq.LQ_ERR_SHAPE),
    ({"K": 1}, {}, lq.LQ_ERR_UNSUPPORTED), ({"K": 5}, {}, lq.LQ_ERR_UNSUPPORTED),
    ({"B": 3}, {}, lq.LQ_ERR_SHAPE),                                   # 20 rows of 3 sequences
    ({}, {"rows": -2}, lq.LQ_ERR_INVALID_ARG), ({}, {"rows": (1 << 30) + 2}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"cu": at(6, 2)}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"x": None}, lq.LQ_ERR_INVALID_ARG), ({}, {"y": None}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"w": None}, lq.LQ_ERR_INVALID_ARG), ({}, {"x": at(0, 1)}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"ldx": 63}, lq.LQ_ERR_SHAPE), ({}, {"ldy": 0}, lq.LQ_ERR_SHAPE), ({}, {"ldx": 1 << 40}, lq.LQ_ERR_SHAPE),
    ({}, {"cu": at(5)}, lq.LQ_ERR_INVALID_ARG), ({}, {"cu": at(4, 8)}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"y": at(0)}, lq.LQ_ERR_INVALID_ARG),                         # y over x
    ({}, {"y": at(0, 64), "ldx": 96, "ldy": 96}, lq.LQ_ERR_INVALID_ARG),   # columns that meet
    ({}, {"so": at(3, 128)}, lq.LQ_ERR_INVALID_ARG),                   # windows partly over each other
])
def test_conv_prefill_refuses(cfg, kw, code):
    assert conv(cfg, **kw) == code


def conv_step(**kw):
    a = dict(dict(state=at(0), x=at(1), ldx=64, w=at(2), bias=None, y=at(3), ldy=64), **kw)
    c = lq.lq_conv_config(lq.LQ_F32, 2, 64, 4, 0)
    return lq.lib().lq_conv_step(C.addressof(c), a["state"], a["x"], a["ldx"], a["w"], a["bias"], a["y"], a["ldy"], None)


@pytest.mark.parametrize("kw,code", [
    ({"state": None}, lq.LQ_ERR_INVALID_ARG), ({"x": None}, lq.LQ_ERR_INVALID_ARG), ({"y": None}, lq.LQ_ERR_INVALID_ARG),
    ({"w": None}, lq.LQ_ERR_INVALID_ARG), ({"ldx": 10}, lq.LQ_ERR_SHAPE), ({"y": at(0)}, lq.LQ_ERR_INVALID_ARG),
    ({"state": at(1)}, lq.LQ_ERR_INVALID_ARG), ({"y": at(1, 4)}, lq.LQ_ERR_INVALID_ARG),
    ({"x": at(1, 2)}, lq.LQ_ERR_INVALID_ARG), ({"w": at(2, 2)}, lq.LQ_ERR_INVALID_ARG)])
def test_conv_step_refuses(kw, code):
    assert conv_step(**kw) == code


def ssm(step=False, cfg=None, **kw):
    cfg = dict(dict(dtype=lq.LQ_BF16, B=2, H=4, G=2, dk=128, dv=64, softplus=1), **(cfg or {}))
    a = dict(dict(rows=20, cu=None, x=at(0), ldx=256, dt=at(1), lddt=4, A=at(2), Bm=at(3), ldb=256, Cm=at(4), ldc=256,
                  D=None, bias=None, S0=at(5), S=at(6), y=at(7), ldy=256, ws=None, n=0), **kw)
    c = lq.lq_ssm_config(*[cfg[n] for n in ("dtype", "B", "H", "G", "dk", "dv", "softplus")])
    if step:
        return lq.lib().lq_ssm_step(C.addressof(c), a["S"], a["x"], a["ldx"], a["dt"], a["lddt"], a["A"], a["Bm"],
                                    a["ldb"], a["Cm"], a["ldc"], a["D"], a["bias"], a["y"], a["ldy"], None)
    return lq.lib().lq_ssm_prefill(C.addressof(c), a["rows"], a["cu"], a["x"], a["ldx"], a["dt"], a["lddt"], a["A"],
                                   a["Bm"], a["ldb"], a["Cm"], a["ldc"], a["D"], a["bias"], a["S0"], a["S"], a["y"],
                                   a["ldy"], a["ws"], a["n"], None)


BAD_SSM = [
    ({"dtype": -1}, {}, lq.LQ_ERR_INVALID_ARG), ({"softplus": 2}, {}, lq.LQ_ERR_INVALID_ARG),
    ({"B": 0}, {}, lq.LQ_ERR_SHAPE), ({"H": 0}, {}, lq.LQ_ERR_SHAPE), ({"G": 3}, {}, lq.LQ_ERR_SHAPE),
    ({"G": 8}, {}, lq.LQ_ERR_SHAPE), ({"dk": 96}, {}, lq.LQ_ERR_UNSUPPORTED), ({"dv": 256}, {}, lq.LQ_ERR_UNSUPPORTED),
    ({}, {"x": None}, lq.LQ_ERR_INVALID_ARG), ({}, {"A": None}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"S": None}, lq.LQ_ERR_INVALID_ARG), ({}, {"Cm": at(4, 1)}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"S": at(6, 8)}, lq.LQ_ERR_INVALID_ARG), ({}, {"ldx": 255}, lq.LQ_ERR_SHAPE),
    ({}, {"ldb": 128}, lq.LQ_ERR_SHAPE), ({}, {"lddt": 3}, lq.LQ_ERR_SHAPE),
    ({}, {"y": at(0)}, lq.LQ_ERR_INVALID_ARG), ({}, {"S": at(3)}, lq.LQ_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("cfg,kw,code", BAD_SSM)
def test_ssm_refuses(cfg, kw, code, step):
    assert ssm(step, cfg, **kw) == code


@pytest.mark.parametrize("cfg,kw,code", [
    ({"B": 3}, {}, lq.LQ_ERR_SHAPE), ({}, {"rows": -1}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"S0": at(6, 64)}, lq.LQ_ERR_INVALID_ARG), ({}, {"y": at(5)}, lq.LQ_ERR_INVALID_ARG),
    ({}, {"cu": at(6)}, lq.LQ_ERR_INVALID_ARG), ({}, {"cu": at(7, 4)}, lq.LQ_ERR_INVALID_ARG)])
def test_ssm_prefill_refuses(cfg, kw, code):
    assert ssm(False, cfg, **kw) == code


def test_ssm_workspace_is_checked():
    """One long prompt of few heads needs a workspace: missing, misaligned, too
    small or over another array it is refused."""
    c = lq.lq_ssm_config(lq.LQ_BF16, 1, 4, 2, 128, 64, 1)
    need = lq.lib().lq_ssm_workspace_bytes(C.addressof(c), 5000)
    assert need > 0 and need % 256 == 0
    one = {"B": 1}
    assert ssm(False, one, rows=5000) == lq.LQ_ERR_WORKSPACE
    assert ssm(False, one, rows=5000, ws=at(8, 16), n=need) == lq.LQ_ERR_WORKSPACE
    assert ssm(False, one, rows=5000, ws=at(8), n=need - 1) == lq.LQ_ERR_WORKSPACE
    assert ssm(False, one, rows=5000, ws=at(7), n=need) == lq.LQ_ERR_INVALID_ARG
    assert ssm(False, one, rows=5000, ws=at(2), n=need) == lq.LQ_ERR_INVALID_ARG
    assert ssm(False, one, rows=5000, cu=at(8), ws=at(8), n=need) == lq.LQ_ERR_INVALID_ARG
    assert lq.lq_ssm_workspace_bytes(torch.bfloat16, 1, 4, 2, 128, 64, 5000) == need


def norm(inn, cfg=None, **kw):
    cfg = dict(dict(dtype=lq.LQ_BF16, x_dtype=lq.LQ_BF16, rows=5, G=1, D=64, w_groups=0, act=1, gate_first=0,
                    eps=1e-5, scale=1.0), **(cfg or {}))
    a = dict(dict(x=at(0), ldx=64, w=at(1), z=at(2), ldz=64, res=at(3), ldr=64, sc=None, h=at(4), ldh=64, y=at(5),
                  ldy=64), **kw)
    c = lq.lq_norm_config(*[cfg[f[0]] for f in lq.lq_norm_config._fields_])
    if inn:
        return lq.lib().lq_norm_in(C.addressof(c), a["x"], a["ldx"], a["w"], a["res"], a["ldr"], a["sc"], a["h"],
                                   a["ldh"], a["y"], a["ldy"], None)
    return lq.lib().lq_norm_out(C.addressof(c), a["x"], a["ldx"], a["w"], a["z"], a["ldz"], a["res"], a["ldr"], a["sc"],
                                a["y"], a["ldy"], None)


@pytest.mark.parametrize("inn,cfg,kw,code", [
    (True, {"dtype": 7}, {}, lq.LQ_ERR_INVALID_ARG), (True, {"x_dtype": lq.LQ_F32}, {}, lq.LQ_ERR_INVALID_ARG),
    (False, {"x_dtype": lq.LQ_F16}, {}, lq.LQ_ERR_INVALID_ARG), (True, {"eps": 0.0}, {}, lq.LQ_ERR_INVALID_ARG),
    (False, {"eps": float("nan")}, {}, lq.LQ_ERR_INVALID_ARG), (True, {"rows": -1}, {}, lq.LQ_ERR_INVALID_ARG),
    (True, {"G": 2}, {}, lq.LQ_ERR_SHAPE), (False, {"D": 0}, {}, lq.LQ_ERR_SHAPE),
    (False, {"D": lq.LQ_NORM_MAX_D + 1}, {"ldx": 20000, "ldz": 20000, "ldr": 20000, "ldy": 20000}, lq.LQ_ERR_UNSUPPORTED),
    (False, {"act": 0}, {}, lq.LQ_ERR_INVALID_ARG), (False, {"gate_first": 2}, {}, lq.LQ_ERR_INVALID_ARG),
    (True, {}, {"x": None}, lq.LQ_ERR_INVALID_ARG), (True, {}, {"w": None}, lq.LQ_ERR_INVALID_ARG),
    (True, {}, {"ldx": 8}, lq.LQ_ERR_SHAPE), (False, {}, {"ldz": 8}, lq.LQ_ERR_SHAPE),
    (True, {}, {"y": at(4)}, lq.LQ_ERR_INVALID_ARG), (True, {}, {"y": at(0, 32)}, lq.LQ_ERR_INVALID_ARG),
    (False, {"x_dtype": lq.LQ_F32}, {"y": at(0)}, lq.LQ_ERR_INVALID_ARG),
    (False, {}, {"res": at(3, 1)}, lq.LQ_ERR_INVALID_ARG), (False, {}, {"w": at(1, 2)}, lq.LQ_ERR_INVALID_ARG),
    (False, {}, {"y": at(1)}, lq.LQ_ERR_INVALID_ARG),
])
def test_norms_refuse(inn, cfg, kw, code):
    assert norm(inn, cfg, **kw) == code


def test_workspace_of_a_bad_config_is_zero():
    c = lq.lq_ssm_config(lq.LQ_BF16, 1, 4, 3, 128, 64, 1)
    assert lq.lib().lq_ssm_workspace_bytes(C.addressof(c), 1000) == 0
    assert lq.lib().lq_ssm_workspace_bytes(None, 1000) == 0


def test_binding_takes_cuda_tensors_only():
    x, w = torch.zeros(3, 1, 8), torch.zeros(8, 4)
    for call in (lambda: lq.lq_conv_prefill(x, w), lambda: lq.lq_conv_step(x, x[0], w), lambda: lq.lq_norm_in(x, w[:, 0]),
                 lambda: lq.lq_norm_out(x, w[:, 0]), lambda: lq.lq_ssm_prefill(x[..., None], x, w, x, x),
                 lambda: lq.lq_ssm_step(x, x, x, w, x, x)):
        with pytest.raises(TypeError):
            call()
