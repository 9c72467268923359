"""The products grouped by expert and the microscaled operators without a GPU: the library's host checks
(nothing is launched, no CUDA call is made) and what the binding refuses before any address reaches it
(a stand-in library notes its calls, CPU tensors stand for device ones)."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_gemm_gb300 import binding as B

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
P = 0x10000  # an aligned stand-in address: every call below returns before it is used


class OnDevice(torch.Tensor):
    """A CPU tensor that says that it is on GPU 0."""
    is_cuda = True

    def get_device(self):
        return 0


class OnAnother(OnDevice):
    def get_device(self):
        return 1


def dev(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or B.MOE_OK

    monkeypatch.setattr(B, "load_library", lambda: Library())
    return made


# ----------------------------------------------------------------------------------------------
# The library
# ----------------------------------------------------------------------------------------------
def _product(lib, ptrs=(P,) * 4, ws=P, ws_bytes=256, **kw):
    cfg = B.make_product_config(**{**dict(rows=100, E=4, N=64, K=128), **kw})
    return lib.moe_grouped_product(ctypes.byref(cfg), *ptrs, ws, ws_bytes, None), cfg


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), B.MOE_ERR_INVALID_ARG), (dict(E=0), B.MOE_ERR_INVALID_ARG),
    (dict(N=0), B.MOE_ERR_INVALID_ARG), (dict(K=-8), B.MOE_ERR_INVALID_ARG),
    (dict(ld_x=120), B.MOE_ERR_INVALID_ARG), (dict(ld_x=132), B.MOE_ERR_INVALID_ARG),
    (dict(ld_y=60), B.MOE_ERR_INVALID_ARG), (dict(ld_y=2 ** 32 + 8), B.MOE_ERR_INVALID_ARG),
    (dict(rows=2 ** 26 + 1), B.MOE_ERR_UNSUPPORTED), (dict(E=1024), B.MOE_ERR_UNSUPPORTED),
    (dict(N=60), B.MOE_ERR_UNSUPPORTED), (dict(K=100), B.MOE_ERR_UNSUPPORTED),
    (dict(K=131080), B.MOE_ERR_UNSUPPORTED), (dict(out_dtype=U8), B.MOE_ERR_INVALID_ARG),
    (dict(accumulate=True), B.MOE_ERR_UNSUPPORTED),
    (dict(accumulate=True, kind="grad_w"), B.MOE_ERR_UNSUPPORTED)])
def test_product_configurations_are_refused(moelib, bad, status):
    st, cfg = _product(moelib, **bad)
    assert st == status and B.moe_product_workspace_size(cfg) == 0
    with pytest.raises(B.MoEError):
        B.alloc_product_workspace(cfg, "cpu")


@pytest.mark.parametrize("kind", ["forward", "grad_x", "grad_w"])
def test_product_pointers_are_checked(moelib, kind):
    for i in range(4):
        ptrs = [P] * 4
        ptrs[i] = None
        assert _product(moelib, ptrs, kind=kind)[0] == B.MOE_ERR_INVALID_ARG
        if i:  # offsets need their element's alignment only
            ptrs[i] = P + 8
            assert _product(moelib, ptrs, kind=kind)[0] == B.MOE_ERR_INVALID_ARG
    assert _product(moelib, ws=None)[0] == B.MOE_ERR_WORKSPACE
    assert _product(moelib, ws_bytes=255)[0] == B.MOE_ERR_WORKSPACE
    assert _product(moelib, ws=P + 4)[0] == B.MOE_ERR_INVALID_ARG
    assert moelib.moe_grouped_product(None, P, P, P, P, P, 256, None) == B.MOE_ERR_INVALID_ARG
    cfg = B.make_product_config(4, 1, 8, 8)
    for field, v in (("kind", 3), ("kind", -1), ("flags", 2)):
        c = type(cfg).from_buffer_copy(cfg)
        setattr(c, field, v)
        assert moelib.moe_grouped_product(ctypes.byref(c), P, P, P, P, P, 256, None) == \
            B.MOE_ERR_INVALID_ARG
    if kind != "grad_w":  # no rows: nothing is touched
        assert _product(moelib, (None,) * 4, kind=kind, rows=0)[0] == B.MOE_OK
    else:
        assert _product(moelib, (None,) * 4, kind=kind, rows=0)[0] == B.MOE_ERR_INVALID_ARG
        assert _product(moelib, (None,) * 4, kind=kind, rows=0, accumulate=True,
                        out_dtype=F32)[0] == B.MOE_OK


MICRO_BAD = [
    (dict(rows=-1), B.MOE_ERR_INVALID_ARG), (dict(src_rows=-1), B.MOE_ERR_INVALID_ARG),
    (dict(K=0), B.MOE_ERR_INVALID_ARG), (dict(groups=0), B.MOE_ERR_INVALID_ARG),
    (dict(copies=0), B.MOE_ERR_INVALID_ARG), (dict(ld=100), B.MOE_ERR_INVALID_ARG),
    (dict(ld=132), B.MOE_ERR_INVALID_ARG), (dict(dtype=U8), B.MOE_ERR_INVALID_ARG),
    (dict(K=96), B.MOE_ERR_UNSUPPORTED), (dict(K=131136), B.MOE_ERR_UNSUPPORTED),
    (dict(rows=2 ** 26 + 1), B.MOE_ERR_UNSUPPORTED), (dict(groups=1024), B.MOE_ERR_UNSUPPORTED),
    (dict(copies=33), B.MOE_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", MICRO_BAD)
def test_micro_configurations_are_refused(moelib, bad, status):
    cfg = B.make_micro_config(**{**dict(rows=100, K=128, format="nv", groups=4), **bad})
    assert B.moe_micro_scales_size(cfg) == 0
    assert moelib.moe_micro_quantize(ctypes.byref(cfg), *[P] * 7, 256, None) == status
    assert moelib.moe_micro_dequantize(ctypes.byref(cfg), *[P] * 6, 256, None) == status
    with pytest.raises(B.MoEError):
        B.alloc_micro(cfg, "cpu")


def test_micro_pointers_are_checked(moelib):
    cfg = B.make_micro_config(100, 128, groups=4)
    q = lambda *a: moelib.moe_micro_quantize(ctypes.byref(cfg), *a, None)  # noqa: E731
    # x, dest, offsets, factor, codes, scales, ws, ws_bytes
    good = [P, P, P, None, P, P, P, 256]
    for i in (0, 4, 5):
        for v in (None, P + 8):
            assert q(*good[:i], v, *good[i + 1:]) == B.MOE_ERR_INVALID_ARG
    assert q(*good[:6], None, 256) == B.MOE_ERR_WORKSPACE
    assert q(*good[:7], 128) == B.MOE_ERR_WORKSPACE
    odd = B.make_micro_config(101, 128, groups=4)  # 101 rows are not four equal groups
    assert moelib.moe_micro_quantize(ctypes.byref(odd), P, None, None, None, P, P, P, 256, None) == \
        B.MOE_ERR_INVALID_ARG
    assert moelib.moe_micro_dequantize(ctypes.byref(odd), P, P, None, None, P, P, 256, None) == \
        B.MOE_ERR_INVALID_ARG
    for kw in (dict(copies=2), dict(src_rows=99)):  # without destinations row t is row t
        c = B.make_micro_config(100, 128, groups=4, **kw)
        assert moelib.moe_micro_quantize(ctypes.byref(c), P, None, P, None, P, P, P, 256, None) == \
            B.MOE_ERR_INVALID_ARG
    d = lambda *a: moelib.moe_micro_dequantize(ctypes.byref(cfg), *a, None)  # noqa: E731
    good = [P, P, P, None, P, P, 256]
    for i in (0, 1, 4):
        for v in (None, P + 8):
            assert d(*good[:i], v, *good[i + 1:]) == B.MOE_ERR_INVALID_ARG
    none = B.make_micro_config(0, 128, groups=4)
    assert moelib.moe_micro_quantize(ctypes.byref(none), *[None] * 6, P, 256, None) == B.MOE_OK
    assert moelib.moe_micro_dequantize(ctypes.byref(none), *[None] * 5, P, 256, None) == B.MOE_OK


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), B.MOE_ERR_INVALID_ARG), (dict(E=0), B.MOE_ERR_INVALID_ARG),
    (dict(out_dtype=U8), B.MOE_ERR_INVALID_ARG), (dict(ld_out=100), B.MOE_ERR_INVALID_ARG),
    (dict(ld_out=132), B.MOE_ERR_INVALID_ARG), (dict(N=100), B.MOE_ERR_UNSUPPORTED),
    (dict(K=96), B.MOE_ERR_UNSUPPORTED), (dict(E=1024), B.MOE_ERR_UNSUPPORTED),
    (dict(N=192, swiglu=True), B.MOE_ERR_UNSUPPORTED), (dict(rows=2 ** 26 + 1), B.MOE_ERR_UNSUPPORTED)])
def test_micro_product_configurations_are_refused(moelib, bad, status):
    cfg = B.make_micro_product_config(**{**dict(rows=100, E=4, N=128, K=128), **bad})
    assert B.moe_micro_product_workspace_size(cfg) == 0
    assert moelib.moe_micro_product(ctypes.byref(cfg), *[P] * 9, 256, None) == status


def test_micro_product_pointers_are_checked(moelib):
    cfg = B.make_micro_product_config(100, 4, 128, 128)
    call = lambda *a: moelib.moe_micro_product(ctypes.byref(cfg), *a, None)  # noqa: E731
    # offsets, a, a_scales, a_factor, w, w_scales, w_factor, out, ws, ws_bytes
    good = [P, P, P, None, P, P, None, P, P, 256]
    for i in (0, 1, 2, 4, 5, 7):
        assert call(*good[:i], None, *good[i + 1:]) == B.MOE_ERR_INVALID_ARG
        if i:
            assert call(*good[:i], P + 8, *good[i + 1:]) == B.MOE_ERR_INVALID_ARG
    assert call(*good[:8], P, 255) == B.MOE_ERR_WORKSPACE
    cfg.rows = 0
    assert call(*[None] * 8, P, 256) == B.MOE_OK


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows,K,groups", [(0, 64, 1), (1, 64, 1), (127, 192, 3), (128, 256, 3),
                                           (1000, 7168, 384)])
def test_scale_bytes_of_the_binding_are_the_library_s(moelib, fmt, rows, K, groups):
    cfg = B.make_micro_config(rows, K, fmt, groups)
    assert B.moe_micro_scales_size(cfg) == B._scale_bytes(rows, K, groups, cfg.format)


def test_scale_tiles_of_groups_do_not_meet():
    """A group's first tile is (its first row) / 128 + its number: every tile of every group lies behind
    the group before it and inside the buffer, whatever the sizes."""
    import random
    rng = random.Random(0)
    for _ in range(300):
        counts = [rng.choice([0, 1, 127, 128, 129, rng.randint(0, 600)]) for _ in range(rng.randint(1, 30))]
        start, end = 0, 0
        for g, n in enumerate(counts):
            first = start // 128 + g
            assert first >= end
            end = first + (n + 127) // 128
            start += n
        assert end <= start // 128 + len(counts)


# ----------------------------------------------------------------------------------------------
# The binding
# ----------------------------------------------------------------------------------------------
R, E, N, K = 10, 3, 16, 64


def _operands(kind):
    cfg = B.make_product_config(R, E, N, K, kind)
    x, dy, w = dev(R, K), dev(R, N), dev(E, N, K)
    a, b, out = {"forward": (x, w, dy), "grad_x": (dy, w, x), "grad_w": (dy, x, w)}[kind]
    return cfg, dict(offsets=dev(E + 1, dtype=I32), a=a, b=b, out=out, ws=dev(256, dtype=U8))


@pytest.mark.parametrize("kind", ["forward", "grad_x", "grad_w"])
def test_product_refuses_types_shapes_and_devices(calls, kind):
    cfg, op = _operands(kind)
    B.moe_grouped_product(cfg, *op.values(), stream=0)
    B.moe_grouped_product(cfg, *{**op, "offsets": dev(E + 2, dtype=I32)}.values(), stream=0)
    n = len(calls)
    for name in ("offsets", "a", "b", "out"):
        t = op[name]
        wrong = [dev(*t.shape, dtype=torch.float16), dev(t.shape[0] - 1, *t.shape[1:], dtype=t.dtype)]
        if t.dim() > 1:
            wrong.append(dev(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2])
        for bad in wrong:
            with pytest.raises(ValueError, match=name):
                B.moe_grouped_product(cfg, *{**op, name: bad}.values(), stream=0)
        with pytest.raises(ValueError, match="device"):
            B.moe_grouped_product(cfg, *{**op, name: t.as_subclass(OnAnother)}.values(), stream=0)
        with pytest.raises(ValueError, match="CUDA"):
            B.moe_grouped_product(cfg, *{**op, name: torch.zeros(t.shape, dtype=t.dtype)}.values(),
                                  stream=0)
    assert len(calls) == n
    with pytest.raises(KeyError):
        B.make_product_config(R, E, N, K, "backward")


def test_quantisation_refuses_types_and_sizes(calls):
    cfg = B.make_micro_config(R, K, "nv", groups=E, src_rows=5, copies=2)
    size = B._scale_bytes(R, K, E, cfg.format)
    op = dict(x=dev(5, K), dest=dev(5, 2, dtype=I32), offsets=dev(E + 1, dtype=I32),
              factor=dev(1, dtype=F32), codes=dev(R, K // 2, dtype=U8), scales=dev(size, dtype=U8),
              ws=dev(256, dtype=U8))
    B.moe_micro_quantize(cfg, *op.values(), stream=0)
    B.moe_micro_quantize(cfg, *{**op, "factor": None}.values(), stream=0)
    n = len(calls)
    for name, bad in (("x", dev(6, K)), ("x", dev(5, K, dtype=F32)), ("dest", dev(10, dtype=torch.int64)),
                      ("dest", dev(9, dtype=I32)), ("offsets", dev(E, dtype=I32)),
                      ("factor", dev(2, dtype=F32)), ("factor", dev(1)),
                      ("codes", dev(R, K, dtype=U8)), ("scales", dev(size - 1, dtype=U8))):
        with pytest.raises(ValueError, match=name):
            B.moe_micro_quantize(cfg, *{**op, name: bad}.values(), stream=0)
    mx = B.make_micro_config(R, K, "mx", groups=E, src_rows=5, copies=2)
    with pytest.raises(ValueError, match="factor"):
        B.moe_micro_quantize(mx, *op.values(), stream=0)
    back = dict(codes=op["codes"], scales=op["scales"], offsets=op["offsets"], factor=op["factor"],
                out=dev(R, K), ws=op["ws"])
    B.moe_micro_dequantize(cfg, *back.values(), stream=0)
    with pytest.raises(ValueError, match="out"):
        B.moe_micro_dequantize(cfg, *{**back, "out": dev(R, K, dtype=F32)}.values(), stream=0)
    with pytest.raises(ValueError, match="device"):
        B.moe_micro_dequantize(cfg, *{**back, "out": dev(R, K).as_subclass(OnAnother)}.values(), stream=0)
    assert len(calls) == n + 1
    with pytest.raises(KeyError):
        B.make_micro_config(R, K, "e4m3")


@pytest.mark.parametrize("swiglu", [False, True])
def test_micro_product_refuses_types_and_sizes(calls, swiglu):
    N = 128
    cfg = B.make_micro_product_config(R, E, N, K, "nv", BF16, swiglu)
    per = 2 * N if swiglu else N
    op = dict(offsets=dev(E + 1, dtype=I32), a=dev(R, K // 2, dtype=U8),
              a_scales=dev(B._scale_bytes(R, K, E, 1), dtype=U8), a_factor=dev(1, dtype=F32),
              w=dev(E * per, K // 2, dtype=U8), w_scales=dev(B._scale_bytes(E * per, K, E, 1), dtype=U8),
              w_factor=dev(E, dtype=F32), out=dev(R, N), ws=dev(256, dtype=U8))
    B.moe_micro_product(cfg, *op.values(), stream=0)
    B.moe_micro_product(cfg, *{**op, "a_factor": None, "w_factor": None}.values(), stream=0)
    n = len(calls)
    for name, t in op.items():
        if name == "ws":
            continue
        with pytest.raises(ValueError, match=name):
            B.moe_micro_product(cfg, *{**op, name: dev(t.numel() - 1, dtype=t.dtype)}.values(), stream=0)
        with pytest.raises(ValueError, match=name):
            B.moe_micro_product(cfg, *{**op, name: dev(*t.shape, dtype=torch.float64)}.values(), stream=0)
    mx = B.make_micro_product_config(R, E, N, K, "mx", BF16, swiglu)
    with pytest.raises(ValueError, match="factor"):
        B.moe_micro_product(mx, *op.values(), stream=0)
    assert len(calls) == n


def test_the_quick_check_leaves_what_is_not_plain(moelib):
    """Without a GPU no operand is a plain one: the module calls nothing and says so."""
    m = B._operands_module()
    cfg = B.make_product_config(4, 1, 8, 8)
    specs = B._product_specs(bytes(cfg))
    t = [torch.zeros(2, dtype=I32), torch.zeros(4, 8, dtype=BF16), torch.zeros(1, 8, 8, dtype=BF16),
         torch.zeros(4, 8, dtype=BF16)]
    ws = torch.zeros(256, dtype=U8)
    assert len(specs.packed) == 4 * 56
    assert m.call(B._address("moe_grouped_product"), bytes(cfg), specs.packed, tuple(t), ws, 0, None) is None
    assert m.call(B._address("moe_grouped_product"), bytes(cfg), specs.packed, tuple(t[:3]), ws, 0, None) is None
    assert m.call(B._address("moe_grouped_product"), bytes(cfg), specs.packed, (1, 2, 3, 4), ws, 0, None) is None
    for bad in ((), (0, b"", b"", t, ws, 0, None), (0, b"", b"", tuple(t), None, 0, None),
                ("x", b"", b"", tuple(t), ws, 0, None)):
        with pytest.raises(TypeError):
            m.call(*bad)
    with pytest.raises(TypeError):
        m.type_code(3)
    assert len({m.type_code(d) for d in (F32, BF16, U8, I32)}) == 4
