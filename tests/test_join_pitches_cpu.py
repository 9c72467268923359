"""Host validation of moe_block_join's row pitches (no GPU needed)."""
import ctypes

import pytest

from mixture_experts_ffn_gemm_gb300 import binding as B

P = 0x10000  # an aligned stand-in address: validation fails before anything dereferences it
READ_OR_RESID = ["ld_resid", "ld_branch", "ld_gate", "ld_resid_out"]


def _refused(lib, T, **pitch):
    cfg = B.make_join_config(T, 64, **pitch)
    return lib.moe_block_join(ctypes.byref(cfg), P, P, P, None, P, P, P, None) == \
        B.MOE_ERR_INVALID_ARG


def _taken(lib, **pitch):
    """No rows: the pitches are checked and nothing is launched."""
    cfg = B.make_join_config(0, 64, **pitch)
    return lib.moe_block_join(ctypes.byref(cfg), *[None] * 7, None) == B.MOE_OK


@pytest.mark.parametrize("name", READ_OR_RESID)
def test_offsets_fit_64_bits(moelib, name):
    for T, ld in ((4, (1 << 58) + 1), (1 << 30, (1 << 30) + 1), (4, -64), (4, 63)):
        assert _refused(moelib, T, **{name: ld}), (T, ld)
    for ld in (0, 64, (1 << 20) + 1, 1 << 40):
        assert _taken(moelib, **{name: ld}), ld


def test_normed_pitch(moelib):
    assert _refused(moelib, 4, ld_normed=(1 << 20) + 1)
    assert _taken(moelib, ld_normed=1 << 20)
    assert not _taken(moelib, ld_normed=(1 << 20) + 1)
