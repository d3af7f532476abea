"""Refusals of the operators beside the layer (no GPU): the C calls return the
documented status before any launch, the binding rejects tensors the kernels
could not read as told."""
import ctypes

import pytest

NULL, DIMS, UNSUPPORTED, ALIGN, WORKSPACE, LAUNCH = 1, 2, 3, 4, 5, 6
P = 0x7F0000000000          # an aligned address that no launch will see


def _lib():
    import grouped_gemm_layer_amd as g
    return g, g.load_library()


def test_sort_workspace():
    g, lib = _lib()
    n = ctypes.c_size_t(7)
    assert lib.moe_sort_workspace_size(16384, 8, 128, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.moe_sort_workspace_size(2 ** 31 // 8 - 1, 8, 512, ctypes.byref(n)) == 0
    assert n.value <= 1 << 20
    assert lib.moe_sort_workspace_size(0, 8, 128, ctypes.byref(n)) == 0 and n.value == 0
    for T, k, E, st in ((-1, 8, 128, DIMS), (1, 0, 128, DIMS), (1, 1, 0, DIMS), (2 ** 30, 2, 4, DIMS), (1, 1, 513, UNSUPPORTED)):
        assert lib.moe_sort_workspace_size(T, k, E, ctypes.byref(n)) == st
    assert lib.moe_sort_workspace_size(1, 1, 1, None) == NULL


def test_sort_tokens():
    g, lib = _lib()
    big = 1 << 20
    call = lambda idx=P, T=4096, k=8, E=16, c=P, o=P, s=P, f=P, ws=P, n=big: lib.moe_sort_tokens(  # noqa: E731
        idx, T, k, E, c, o, s, f, ws, n, None)
    assert call(idx=None) == NULL and call(c=None) == NULL and call(s=None) == NULL and call(ws=None) == NULL
    assert call(idx=P + 2) == ALIGN and call(ws=P + 128) == ALIGN
    assert call(n=16) == WORKSPACE
    assert call(E=513) == UNSUPPORTED and call(T=-1) == DIMS


def _rows(lib, name, **kw):
    a = dict(tok=P, ldt=64, rows_p=P, ldr=64, rows=10, T=4, H=64, k=2, typ=1, f2s=P, w=P, other=P, ldo=64, dw=P)
    a.update(kw)
    if name == "permute":
        return lib.moe_permute(a["tok"], a["ldt"], a["T"], a["H"], a["k"], a["typ"], a["f2s"], a["w"], a["rows_p"], a["ldr"],
                               a["rows"], None)
    if name == "permute_backward":
        return lib.moe_permute_backward(a["rows_p"], a["ldr"], a["rows"], a["T"], a["H"], a["k"], a["typ"], a["f2s"], a["w"],
                                        a["other"], a["ldo"], a["tok"], a["ldt"], a["dw"], None)
    if name == "unpermute":
        return lib.moe_unpermute(a["rows_p"], a["ldr"], a["rows"], a["T"], a["H"], a["k"], a["typ"], a["f2s"], a["w"], a["tok"],
                                 a["ldt"], None)
    return lib.moe_unpermute_backward(a["tok"], a["ldt"], a["T"], a["H"], a["k"], a["typ"], a["f2s"], a["w"], a["other"],
                                      a["ldo"], a["rows_p"], a["ldr"], a["rows"], a["dw"], None)


@pytest.mark.parametrize("name", ["permute", "permute_backward", "unpermute", "unpermute_backward"])
def test_row_calls(name):
    g, lib = _lib()
    for kw, st in ((dict(tok=None), NULL), (dict(rows_p=None), NULL), (dict(f2s=None), NULL), (dict(ldt=63), DIMS),
                   (dict(ldr=63), DIMS), (dict(k=0), DIMS), (dict(T=-1), DIMS), (dict(H=-1), DIMS), (dict(rows=-1), DIMS),
                   (dict(T=2 ** 30, k=2), DIMS), (dict(k=33), UNSUPPORTED), (dict(typ=2), UNSUPPORTED),
                   (dict(tok=P + 1), ALIGN), (dict(rows_p=P + 2, typ=0), ALIGN), (dict(w=P + 2), ALIGN), (dict(f2s=P + 1), ALIGN)):
        assert _rows(lib, name, **kw) == st, kw
    if name.endswith("backward"):
        assert _rows(lib, name, other=None) == NULL            # dweights needs the forward's rows
        assert _rows(lib, name, ldo=10) == DIMS
    assert _rows(lib, name, T=0, tok=None, f2s=None) == 0      # nothing to do, nothing launched


def test_mxfp4_quantize():
    g, lib = _lib()
    call = lambda src=P, ld=64, batch=1, rows=4, cols=64, typ=1, along=1, swiglu=0, codes=P, scales=P: lib.moe_mxfp4_quantize(  # noqa: E731
        src, ld, batch, rows, cols, typ, along, swiglu, codes, scales, None)
    assert call(src=None) == NULL and call(codes=None) == NULL and call(scales=None) == NULL
    assert call(ld=63) == DIMS and call(rows=-1) == DIMS and call(along=2) == DIMS and call(swiglu=1) == DIMS
    assert call(typ=7) == UNSUPPORTED and call(along=0, swiglu=1) == UNSUPPORTED and call(cols=2 ** 30 + 1, ld=2 ** 32, swiglu=1) == UNSUPPORTED
    assert call(codes=P + 16) == ALIGN and call(scales=P + 16) == ALIGN and call(src=P + 1) == ALIGN
    assert call(rows=0, src=None, codes=None) == 0 and call(cols=0) == 0 and call(batch=0) == 0


def test_mxfp4_dequantize():
    g, lib = _lib()
    call = lambda codes=P, scales=P, rows=4, cols=64, out=P, ld=64, typ=1: lib.moe_mxfp4_dequantize(  # noqa: E731
        codes, scales, rows, cols, out, ld, typ, None)
    assert call(codes=None) == NULL and call(out=None) == NULL and call(ld=10) == DIMS and call(cols=-3) == DIMS
    assert call(typ=3) == UNSUPPORTED and call(codes=P + 8) == ALIGN and call(out=P + 1) == ALIGN
    assert call(rows=0) == 0


def test_mxfp4_product():
    g, lib = _lib()

    def call(**kw):
        a = dict(a=P, sa=P, a_rows=8, fmt=0, b=P, sb=P, E=4, N=64, K=128, off=P, map=P, div=1, c=P, ldc=64, rows=8, typ=1)
        a.update(kw)
        return lib.moe_mxfp4_product(a["a"], a["sa"], a["a_rows"], a["fmt"], a["b"], a["sb"], a["E"], a["N"], a["K"], a["off"],
                                     a["map"], a["div"], a["c"], a["ldc"], a["rows"], a["typ"], None)

    for kw, st in ((dict(a=None), NULL), (dict(sa=None), NULL), (dict(b=None), NULL), (dict(sb=None), NULL), (dict(c=None), NULL),
                   (dict(off=None), NULL), (dict(K=0), DIMS), (dict(E=0), DIMS), (dict(N=-1), DIMS), (dict(div=0), DIMS),
                   (dict(ldc=63), DIMS), (dict(rows=-1), DIMS), (dict(fmt=2), UNSUPPORTED), (dict(typ=2), UNSUPPORTED),
                   (dict(E=513), UNSUPPORTED), (dict(fmt=1, K=100), UNSUPPORTED), (dict(a_rows=1 << 25), UNSUPPORTED),
                   (dict(N=1 << 25, ldc=1 << 25), UNSUPPORTED), (dict(rows=2 ** 31 - 1), UNSUPPORTED),
                   (dict(a=P + 16), ALIGN), (dict(sb=P + 4), ALIGN), (dict(c=P + 1), ALIGN), (dict(off=P + 2), ALIGN),
                   (dict(map=P + 1), ALIGN)):
        assert call(**kw) == st, kw
    assert call(rows=0, c=None) == 0 and call(N=0) == 0


def test_gradients():
    g, lib = _lib()
    n = ctypes.c_size_t(0)
    assert lib.moe_grad_workspace_size(-1, ctypes.byref(n)) == DIMS and lib.moe_grad_workspace_size(1, None) == NULL
    assert lib.moe_grad_workspace_size(500, ctypes.byref(n)) == 0

    def table(*rows):
        t = (g._CTensor * max(len(rows), 1))()
        for c, (data, out, size, typ) in zip(t, rows):
            c.data, c.out, c.n, c.type = data, out, size, typ
        return t

    def norm(rows, sumsq=P, ws=P, size=n.value):
        return lib.moe_grad_norm(ctypes.byref(table(*rows)), len(rows), sumsq, ws, size, None)

    def clip(rows, sumsq=P, max_norm=1.0, out=P):
        return lib.moe_grad_clip(ctypes.byref(table(*rows)), len(rows), sumsq, max_norm, out, None)

    ok = (P, None, 100, 0)
    Q = P + 0x1000000
    for f in (norm, clip):
        assert f([(None, None, 5, 0)]) == NULL and f([ok], sumsq=None) == NULL
        assert f([(P, None, -1, 0)]) == DIMS and f([(P, None, 5, 9)]) == UNSUPPORTED
        assert f([(P + 2, None, 5, 0)]) == ALIGN and f([(P + 1, None, 5, 1)]) == ALIGN and f([ok], sumsq=P + 4) == ALIGN
        assert f([(P, None, 2 ** 40, 0), (P + 2 ** 43, None, 1, 0)]) == DIMS
    assert norm([ok], ws=None) == NULL and norm([ok], ws=P + 8) == ALIGN and norm([ok], size=8) == WORKSPACE
    assert clip([ok, ok]) == UNSUPPORTED and clip([(P + 396, None, 8, 1), ok]) == UNSUPPORTED
    assert clip([ok], max_norm=-1.0) == DIMS and clip([ok], max_norm=float("nan")) == DIMS and clip([ok], out=P + 2) == ALIGN
    assert clip([(P, P + 40, 100, 0)]) == UNSUPPORTED                      # output over its own gradient, shifted
    assert clip([ok, (Q, P, 10, 0)]) == UNSUPPORTED                        # output over another gradient
    assert clip([(P, Q, 100, 0), (P + 400, Q + 396, 10, 0)]) == UNSUPPORTED  # two outputs
    assert lib.moe_grad_norm(None, 3, P, P, 1 << 20, None) == NULL


def test_binding_rejects_what_the_kernels_would_misread():
    import torch
    g, lib = _lib()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)   # noqa: E731
    r = g.RoutingBuffers(i32(4, 2), None, i32(3), i32(4), i32(8), i32(8))
    x, xp = torch.zeros(4, 16), torch.zeros(8, 16)
    bad = [
        lambda: g.sort_tokens(r, u8(0)),                                            # host tensors
        lambda: g.permute(x, r, xp),
        lambda: g.permute(x, r, xp.bfloat16()),                                     # types differ
        lambda: g.permute(x.double(), r, xp.double()),
        lambda: g.permute(x, r, torch.zeros(8, 15)),                                # widths differ
        lambda: g.permute(x.t().contiguous().t(), r, xp),                           # columns are not contiguous
        lambda: g.permute(x[:1].expand(4, 16), r, xp),                              # rows overlap
        lambda: g.permute(torch.zeros(5, 16), r, xp),                               # maps of another batch
        lambda: g.permute(x, r, xp, weights=torch.zeros(4, 2).double()),
        lambda: g.permute(x, r, xp, weights=torch.zeros(4, 3)),
        lambda: g.permute_backward(xp, r, x, dweights=torch.zeros(4, 2)),           # no x for the dots
        lambda: g.unpermute_backward(x, r, xp, rows=torch.zeros(7, 16), dweights=torch.zeros(4, 2)),
        lambda: g.sort_tokens(g.RoutingBuffers(i32(4, 2).long(), None, i32(3), i32(4), i32(8), i32(8)), u8(0)),
        lambda: g.sort_tokens(g.RoutingBuffers(i32(4, 2), None, i32(3), i32(3), i32(8), i32(8)), u8(0)),
        lambda: g.mxfp4_quantize(x, u8(4, 16), u8(4, 2)),                           # scales of another width
        lambda: g.mxfp4_quantize(x, u8(4, 15), u8(4, 1)),
        lambda: g.mxfp4_quantize(x.half(), u8(4, 16), u8(4, 1)),
        lambda: g.mxfp4_quantize(torch.zeros(4, 15), u8(4, 16), u8(4, 1), swiglu=True),
        lambda: g.mxfp4_quantize(torch.zeros(2, 4, 8, 16), u8(64, 16), u8(64, 1)),
        lambda: g.mxfp4_quantize(torch.zeros(2, 8, 16)[:, :4], u8(2, 4, 16), u8(2, 4, 1)),   # a gap between matrices
        lambda: g.mxfp4_dequantize(u8(4, 16), u8(4, 2), x),
        lambda: g.mxfp4_dequantize(u8(4, 16), u8(4, 1), torch.zeros(2, 4, 16)[:, :2]),
        lambda: g.mxfp4_product(u8(8, 16), u8(8, 1), u8(5, 16), u8(5, 1), torch.zeros(8, 5), k=32, a_format="mxfp6"),
        lambda: g.mxfp4_product(u8(7, 16), u8(7, 1), u8(5, 16), u8(5, 1), torch.zeros(8, 5), k=32),
        lambda: g.mxfp4_product(u8(8, 16), u8(8, 1), u8(5, 16), u8(5, 2), torch.zeros(8, 5), k=32),
        lambda: g.mxfp4_product(u8(8, 16), u8(8, 1), u8(5, 16), u8(5, 1), torch.zeros(8, 5), k=32, row_map=i32(7)),
        lambda: g.mxfp4_product(u8(8, 16), u8(8, 1), u8(5, 16), u8(5, 1), torch.zeros(8, 5), k=32, offsets=i32(2).long()),
        lambda: g.GradientList([]),
        lambda: g.GradientList([torch.zeros(4, 4).t()[:, :2]]),
        lambda: g.GradientList([x], out=[x, x]),
        lambda: g.GradientList([x], out=[x.bfloat16()]),
        lambda: g.GradientList([x.half()]),
        lambda: g.grad_norm([x], torch.zeros(1), u8(1 << 16)),
        lambda: g.grad_clip([x], torch.zeros(1, dtype=torch.float64), 1.0),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted", i)
