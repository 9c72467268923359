"""Host validation of moe_forward_few and moe_block_join: bad arguments are refused before any CUDA
call (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

P = 0x10000  # an aligned stand-in address: validation fails before anything dereferences it


def _cfg(**kw):
    base = dict(T=4, d=256, E=16, k=4, I=128, act_dtype=torch.bfloat16)
    base.update(kw)
    return B.make_config(**base)


NAMES = ["x", "W_r", "b", "W13", "W2", "W13_s", "W2_s", "Ws13", "Ws2", "Ws13_s", "Ws2_s", "W_down",
         "W_up", "out"]


def _few(lib, cfg, ws=P, nbytes=None, **override):
    n = B.moe_few_workspace_size(cfg) if nbytes is None else nbytes
    ref = None if cfg is None else ctypes.byref(cfg)
    return lib.moe_forward_few(ref, *[override.get(a, P) for a in NAMES], ws, n, None)


INVALID, UNSUPPORTED = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
FP8 = dict(w_dtype=torch.float8_e4m3fn)
INT4 = dict(w_dtype=torch.uint8, quant_block=32)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INVALID), (dict(T=17), UNSUPPORTED), (dict(d=0), INVALID), (dict(k=0), INVALID),
    (dict(k=17), INVALID), (dict(E=0), INVALID), (dict(I=0), INVALID), (dict(n_shared=2), INVALID),
    (dict(E=1024), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(d=272), UNSUPPORTED),
    (dict(I=136), UNSUPPORTED), (dict(I_shared=256), UNSUPPORTED), (dict(d=65568), UNSUPPORTED),
    (dict(d_latent=-1), INVALID), (dict(d_latent=72), UNSUPPORTED), (dict(flags=1), UNSUPPORTED),
    (dict(d=192, **FP8), UNSUPPORTED), (dict(quant_block=64, **FP8), UNSUPPORTED),
    (dict(d_latent=128, **FP8), UNSUPPORTED), (dict(act_dtype=torch.float32, **FP8), UNSUPPORTED),
    (dict(w_dtype=torch.uint8), UNSUPPORTED), (dict(d=272, **INT4), UNSUPPORTED),
    (dict(w_dtype=torch.float32), UNSUPPORTED)])
def test_few_configs_are_refused(moelib, bad, status):
    cfg = _cfg(**bad)
    assert B.moe_few_workspace_size(cfg) == 0
    assert _few(moelib, cfg, nbytes=1 << 40) == status


def test_few_arguments_are_refused(moelib):
    cfg = _cfg()
    need = B.moe_few_workspace_size(cfg)
    assert need > 0
    assert _few(moelib, None, nbytes=1 << 40) == INVALID
    assert _few(moelib, cfg, nbytes=need - 1) == B.MOE_ERR_WORKSPACE
    assert _few(moelib, cfg, ws=None) == B.MOE_ERR_WORKSPACE
    assert _few(moelib, cfg, ws=P + 8) == INVALID
    for name in ("x", "W_r", "b", "W13", "W2", "Ws13", "Ws2", "out"):
        assert _few(moelib, cfg, **{name: None}) == INVALID, name
        assert _few(moelib, cfg, **{name: P + 2}) == INVALID, name
    lat = _cfg(d_latent=128, latent_norm=1)
    for name in ("W_down", "W_up"):
        assert _few(moelib, lat, **{name: None}) == INVALID, name
    for kind in (FP8, INT4):
        for name in ("W13_s", "W2_s", "Ws13_s", "Ws2_s"):
            assert _few(moelib, _cfg(**kind), **{name: None}) == INVALID, name
            assert _few(moelib, _cfg(**kind), **{name: P + 4}) == INVALID, name
    cfg.reserved_ = 1
    assert _few(moelib, cfg, nbytes=need) == INVALID


def test_few_zero_tokens(moelib):
    cfg = _cfg(T=0)
    need = B.moe_few_workspace_size(cfg)
    assert need >= 256
    st = moelib.moe_forward_few(ctypes.byref(cfg), *[None] * 14, P, need, None)
    assert st == B.MOE_OK


def test_few_binding_refuses_host_tensors(moelib):
    cfg = _cfg()
    with pytest.raises(ValueError):
        B.moe_forward_few(cfg, torch.zeros(4, 256, dtype=torch.bfloat16), *[None] * 12, None,
                          torch.zeros(8, dtype=torch.uint8), stream=0)


def _join(lib, cfg, resid=P, branch=P, post_w=P, gate=None, pre_w=P, resid_out=P, normed=P):
    ref = None if cfg is None else ctypes.byref(cfg)
    return lib.moe_block_join(ref, resid, branch, post_w, gate, pre_w, resid_out, normed, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769), UNSUPPORTED),
    (dict(act_dtype=torch.uint8), INVALID), (dict(resid_dtype=torch.uint8), INVALID),
    (dict(act_dtype=torch.float32, resid_dtype=torch.bfloat16), UNSUPPORTED),
    (dict(ld_resid=63), INVALID), (dict(ld_branch=-64), INVALID), (dict(ld_gate=1), INVALID),
    (dict(ld_resid_out=63), INVALID), (dict(ld_normed=(1 << 20) + 1), INVALID)])
def test_join_configs_are_refused(moelib, bad, status):
    assert _join(moelib, B.make_join_config(**{**dict(T=4, d=64), **bad})) == status


def test_join_arguments_are_refused(moelib):
    cfg = B.make_join_config(4, 64)
    assert _join(moelib, None) == INVALID
    for name in ("resid", "branch", "resid_out", "pre_w", "normed"):
        assert _join(moelib, cfg, **{name: None}) == INVALID, name
    for name in ("resid", "branch", "post_w", "resid_out", "pre_w", "normed"):
        assert _join(moelib, cfg, **{name: P + 1}) == INVALID, name
    assert _join(moelib, cfg, gate=P) == INVALID
    assert _join(moelib, B.make_join_config(4, 64, gate="channel")) == INVALID
    assert _join(moelib, B.make_join_config(4, 64, resid_dtype=torch.float32), resid=P + 2) == INVALID
    for field, value in (("gate", 4), ("gate", -1), ("flags", 2)):
        cfg = B.make_join_config(4, 64)
        setattr(cfg, field, value)
        assert _join(moelib, cfg) == INVALID, field
    assert moelib.moe_block_join(ctypes.byref(B.make_join_config(0, 64)), *[None] * 7, None) == \
        B.MOE_OK


def test_join_struct_size():
    assert ctypes.sizeof(B.moe_join_config_t) == 80
