"""GPU tests of the block join where a launch's shared memory comes near the 48 KB that need no
attribute, of calls from several host threads, and of wide row pitches.  The formula in 64 bits and the
tolerances are those of the join's other tests."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from conftest import ROOT  # noqa: E402
from test_gpu_join import BF16, F32, TYPES, _check, _make, _reference, _run  # noqa: E402

from mixture_experts_ffn_gemm_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu

GATES = ("none", "channel", "token", "element")
ROWS = 200  # more rows than the device has SMs: the kernel that keeps rows in shared memory


def _row_bytes(act, res, gate):
    """Shared memory a column takes there: branch, residual and an element gate."""
    size = {F32: 4, BF16: 2}
    return size[act] * (2 if gate == "element" else 1) + size[res]


def _one(act, res, gate, d, seed):
    cfg, st = _make(ROWS, d, act, res, gate, gate == "element", True, True, seed=seed)
    ref = _reference(st, gate, gate == "element")
    _run(cfg, st)
    _check(cfg, st, ref)


def _near_48k():
    """Every type and gate at the widths whose rows take the last 256 bytes below 48 KB, in a process that
    has launched no larger row before."""
    for act, res in TYPES:
        for gate in GATES:
            last = 48 * 1024 // _row_bytes(act, res, gate) // 8 * 8
            first = (48 * 1024 - 256) // _row_bytes(act, res, gate) // 8 * 8
            for d in sorted({first, first + 8, last}):
                try:
                    _one(act, res, gate, d, 1)
                except B.MoEError as e:
                    print(f"refused: {act} {res} {gate} {d}: {e}")
                    return 1
    return 0


def test_rows_near_48k_as_first_calls(cuda_device):
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("d", [4096, 6144, 8192, 12288, 16384])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("act,res", TYPES)
def test_usual_widths(cuda_device, act, res, gate, d):
    _one(act, res, gate, d, 2)


def test_wide_odd_rows_from_two_threads(cuda_device):
    """Odd widths beyond 8192 take d x 4 bytes of shared memory each: calls of different widths from two
    threads do not lower each other's limit."""
    lib = B.load_library()
    calls, bad = 5000, []
    buf = {d: [torch.randn(1, d, device="cuda").to(BF16) for _ in range(4)] for d in (8193, 32767)}

    def work(d):
        r, y, ro, n = buf[d]
        w = torch.ones(d, dtype=BF16, device="cuda")
        cfg = B.make_join_config(1, d)
        stream = torch.cuda.Stream().cuda_stream
        for _ in range(calls):
            s = lib.moe_block_join(ctypes.byref(cfg), r.data_ptr(), y.data_ptr(), None, None,
                                   w.data_ptr(), ro.data_ptr(), n.data_ptr(), stream)
            if s != B.MOE_OK:
                bad.append((d, s))
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(d,)) for d in buf]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[0])


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("d,more", [(7168, 0), (1001, 1)])
def test_one_position_of_a_long_buffer(cuda_device, act, res, d, more):
    """Rows more than 2^20 elements apart, as the last position of every sequence is."""
    T, ld = 3, (1 << 20) + 4096 + more
    cfg, st = _make(T, d, act, res, "element", False, True, True, ld - d, seed=3)
    cfg.ld_normed = 0
    st["normed"] = torch.empty(T, d, dtype=act, device="cuda")
    ref = _reference(st, "element", False)
    _run(cfg, st)
    _check(cfg, st, ref)


def test_pitch_past_32_bits(cuda_device):
    """Two rows more than 2^31 elements apart, in place."""
    T, d, ld = 2, 2048, (1 << 31) + 64
    cfg, st = _make(T, d, BF16, BF16, "channel", False, True, True, seed=4)
    ref = _reference(st, "channel", False)
    for name in ("resid", "branch"):
        buf = torch.empty(ld + d, dtype=BF16, device="cuda").as_strided((T, d), (ld, 1))
        buf.copy_(st[name])
        st[name] = buf
    st["resid_out"] = st["resid"]
    cfg.ld_resid = cfg.ld_branch = cfg.ld_resid_out = ld
    _run(cfg, st)
    _check(cfg, st, ref)


if __name__ == "__main__":
    from mixture_experts_ffn_gemm_gb300 import build
    build.build()
    sys.exit(_near_48k())
