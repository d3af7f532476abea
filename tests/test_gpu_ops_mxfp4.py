"""MXFP4 quantiser, its inverse and the grouped product, through the binding.

Codes, scales and decoded values are compared bit for bit with the definition
in NumPy float64.  The product's bound: products of codes are exact; the matrix
instruction sums 128 of them in fp32 and n = ceil(K / 128) such sums are added
in fp32, so |err| <= (n + 2) 2^-23 sum|terms| with MXFP4 rows (the sums
themselves came out exact to 2^-24 of the magnitudes; a factor of two covers
their order), and 2e-4 sum|terms| with MXFP8 rows (the instruction aligns
their products to the largest and keeps about 1e-4 of the magnitudes), plus
half a unit of the output type.
"""
import numpy as np
import pytest

import _mxfp4_reference as mx

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _values(rng, rows, cols, typ):
    """Values over many binades as the type holds them: ties, zero blocks,
    negative zeros, subnormals, the largest numbers, blocks that are not finite."""
    import torch
    v = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    v = v.astype(np.float32)
    flat = v.reshape(-1)
    n = flat.size
    flat[: n // 16] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0], n // 16)
    if n > 400:
        flat[100:140] = 0.0
        flat[140:150] = -0.0
        flat[150:190] = np.float32(2.0 ** -140) if typ == "fp32" else np.float32(2.0 ** -132)
        flat[200] = 3.0e38
        flat[240] = np.inf
        flat[300] = np.nan
        flat[380] = -np.inf
    t = torch.from_numpy(v).to(_dt(typ)).cuda()
    return t, t.double().cpu().numpy()


SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 8), (33, 1), (70, 45), (64, 256), (255, 130), (257, 129), (300, 2048),
          (513, 515), (1, 5000), (5000, 1), (31, 96)]


@pytest.mark.parametrize("typ", ["bf16", "fp32"])
@pytest.mark.parametrize("along", [1, 0])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_and_back_bit_exact(shape, along, typ):
    import torch
    import grouped_gemm_layer_amd as g
    rows, cols = shape
    print(f"[mxfp4] {shape} along={along} {typ}", flush=True)
    t, v = _values(np.random.default_rng(rows * 7 + cols), rows, cols, typ)
    w = v if along else v.T
    code, s = mx.encode(w)
    kb = s.shape[1]
    codes = torch.full((w.shape[0], kb * 16), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((w.shape[0], kb), 0xAB, dtype=torch.uint8, device="cuda")
    g.mxfp4_quantize(t, codes, scales, along=along)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), mx.pack(code))
    want = mx.decode(mx.pack(code), s, w.shape[1])
    # 3e38 = 3.53 * 2^126 becomes 4 * 2^126 = 2^128, which is past the largest number of both types: infinite
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    for out_t in ("fp32", "bf16"):
        out = torch.full((w.shape[0], w.shape[1] + 3), 9.0, dtype=_dt(out_t), device="cuda")
        g.mxfp4_dequantize(codes, scales, out[:, 1:1 + w.shape[1]])
        got = out.double().cpu().numpy()
        assert np.array_equal(got[:, 1:-2], want, equal_nan=True)
        assert np.all(got[:, 0] == 9) and np.all(got[:, -2:] == 9)


@pytest.mark.parametrize("typ", ["bf16", "fp32"])
def test_quantize_pitch_and_batch(typ):
    """Rows inside wider rows, and a batch of matrices, transposed each by itself."""
    import torch
    import grouped_gemm_layer_amd as g
    t, v = _values(np.random.default_rng(5), 3 * 65, 90, typ)
    wide = torch.full((3 * 65, 101), float("nan"), dtype=_dt(typ), device="cuda")
    wide[:, 5:95] = t
    src = wide.view(3, 65, 101)[:, :, 5:95]
    for along in (1, 0):
        r, n = (65, 90) if along else (90, 65)
        kb = -(-n // 32)
        codes = torch.empty(3, r, kb * 16, dtype=torch.uint8, device="cuda")
        scales = torch.empty(3, r, kb, dtype=torch.uint8, device="cuda")
        g.mxfp4_quantize(src, codes, scales, along=along)
        for b in range(3):
            m = v.reshape(3, 65, 90)[b]
            code, s = mx.encode(m if along else m.T)
            assert np.array_equal(codes[b].cpu().numpy(), mx.pack(code))
            assert np.array_equal(scales[b].cpu().numpy(), s)


@pytest.mark.parametrize("typ", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 32), (7, 45), (64, 768), (33, 1000)], ids=str)
def test_quantize_swiglu(shape, typ):
    """SiLU(g1) g3 in front: the fp32 value is off the exact one by at most 2^-21
    of it (exp, reciprocal and two products, each within 2 units of 2^-24; the
    exponent's rounding adds |g1| 2^-24 with |g1| < 8 here), so a code may only
    differ where that value lies that close to the middle between two codes,
    and then by one step; a scale likewise next to its border."""
    import torch
    import grouped_gemm_layer_amd as g
    rows, cols = shape
    rng = np.random.default_rng(cols)
    t = torch.from_numpy(np.clip(rng.standard_normal((rows, 2 * cols)) * 2, -8, 8).astype(np.float32)).to(_dt(typ)).cuda()
    v = t.double().cpu().numpy()
    a = v[:, :cols] / (1 + np.exp(-v[:, :cols])) * v[:, cols:]
    kb = -(-cols // 32)
    codes = torch.empty(rows, kb * 16, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, kb, dtype=torch.uint8, device="cuda")
    g.mxfp4_quantize(t, codes, scales, swiglu=True)
    got = mx.decode(codes.cpu().numpy(), scales.cpu().numpy(), cols)
    lo, s_lo = mx.encode(np.abs(a) * (1 - 2.0 ** -21))
    hi, s_hi = mx.encode(np.abs(a) * (1 + 2.0 ** -21))
    s = scales.cpu().numpy()
    assert np.all((s >= s_lo) & (s <= s_hi))
    lo, hi = mx.decode(mx.pack(lo), s_lo, cols), mx.decode(mx.pack(hi), s_hi, cols)
    sure = np.repeat(s_lo == s_hi, 32, axis=1)[:, :cols]
    assert np.all(((np.abs(got) >= lo) & (np.abs(got) <= hi))[sure])
    assert np.mean(lo != hi) < 1e-3                     # the test leaves next to nothing open
    assert np.array_equal(np.signbit(got), np.signbit(a))


def test_dequantize_every_scale():
    """All 16 codes under all 256 scale bytes."""
    import torch
    import grouped_gemm_layer_amd as g
    packed = np.tile(np.array([c | (15 - c) << 4 for c in range(16)], dtype=np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    want = mx.decode(packed, scales, 32)
    for typ in ("fp32", "bf16"):
        out = torch.empty(256, 32, dtype=_dt(typ), device="cuda")
        g.mxfp4_dequantize(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), out)
        got = out.double().cpu().numpy()
        big = np.abs(want) >= 2.0 ** 128
        assert np.array_equal(got[~big], want[~big], equal_nan=True)
        assert np.all(np.isinf(got[big])) and np.array_equal(np.sign(got[big]), np.sign(want[big]))


class Product:
    """Operands of one grouped product and its fp64 result."""

    def __init__(self, counts, N, K, fmt, T=None, k=1, seed=0, gap=0, dense=False):
        import torch
        rng = np.random.default_rng(seed + N * 3 + K)
        self.E, self.N, self.K, self.fmt, self.k = len(counts), N, K, fmt, k
        self.counts = np.asarray(counts)
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        M = int(self.offsets[-1])
        self.rows = M + gap
        self.kb = -(-K // 32)
        self.map = None
        A = self.rows if T is None else T
        if T is not None:                                # gathered: flat slots of T tokens, some negative
            m = rng.integers(0, T * k, self.rows).astype(np.int32)
            if M > 5:
                m[rng.integers(0, M, 2)] = -1
            self.map = m
        av = rng.standard_normal((A, K)) * np.exp2(rng.integers(-3, 4, (A, 1)))
        code, self.sa = mx.encode(av)
        if fmt == "mxfp4":
            self.a = mx.pack(code)
            self.av = mx.decode(self.a, self.sa, K)
        else:
            # random E4M3 codes whose magnitudes spread over a few binades
            self.a = (rng.integers(0x28, 0x60, (A, K)) | (rng.integers(0, 2, (A, K)) << 7)).astype(np.uint8)
            self.av = mx.decode_mxfp8(self.a, self.sa)
        bv = rng.standard_normal((self.E * N, K)) * 0.05
        code, self.sb = mx.encode(bv)
        self.b = mx.pack(code)
        self.bv = mx.decode(self.b, self.sb, K).reshape(self.E, N, K)
        up = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
        self.args = [up(self.a), up(self.sa), up(self.b).view(self.E, N, -1), up(self.sb).view(self.E, N, -1)]
        self.kw = dict(k=K, a_format=fmt, offsets=None if dense else up(self.offsets))
        if self.map is not None:
            self.kw.update(row_map=up(self.map), row_div=k)

    def reference(self):
        src = np.arange(self.rows) if self.map is None else np.where(self.map < 0, -1, self.map // self.k)
        x = np.where((src >= 0)[:, None], self.av[np.maximum(src, 0)], 0.0)
        out, mag = (np.zeros((self.rows, self.N)) for _ in range(2))
        for e in range(self.E):
            r = slice(self.offsets[e], self.offsets[e + 1])
            out[r] = x[r] @ self.bv[e].T
            mag[r] = np.abs(x[r]) @ np.abs(self.bv[e]).T
        return out, mag

    def check(self, c, typ, ref=None):
        want, mag = ref or self.reference()
        M = int(self.offsets[-1])
        got = c.double().cpu().numpy()
        rel = (-(-self.K // 128) + 2) * 2.0 ** -23 if self.fmt == "mxfp4" else 2e-4
        err, lim = np.abs(got[:M] - want[:M]), rel * mag[:M] + 1.01 * U[typ] * np.abs(want[:M])
        assert np.all(err <= lim), f"worst {np.max(err - lim)}, largest value {np.abs(want).max()}"
        return got


CASES = [
    # counts, N, K, T, k
    ([1], 1, 1, None, 1),
    ([3], 5, 31, None, 1),
    ([1, 0, 2], 17, 32, None, 1),
    ([0, 0, 0, 4], 64, 128, None, 1),
    ([16, 17, 1, 0, 33], 48, 160, 9, 3),
    ([2] * 40, 100, 96, 12, 2),
    ([1, 0, 1, 0, 0, 1], 1536, 2048, 4, 8),
    ([130, 0, 5, 64], 130, 256, 50, 4),
    ([257], 257, 288, None, 1),
    ([40, 300, 0, 12, 129], 136, 1120, 100, 6),
    ([300, 256, 700], 520, 544, 400, 2),
    ([5] * 300 + [0] * 212, 33, 64, 64, 4),
    ([1024], 256, 512, None, 1),
    ([5, 0, 17, 1], 50, 1632, 9, 3),
    ([3, 30], 33, 4128, None, 1),
]
# long enough for the tiles through LDS: 128 x 128, then 256 x 256; K of whole and of broken steps, words and stages
TILED = [
    ([3000, 5100], 4200, 40, None, 1),
    ([100] * 400 + [0] * 112, 360, 160, 64, 4),
    ([140, 900, 0, 12, 329], 1336, 1120, 100, 6),
    ([130, 0, 5, 64, 2700], 1500, 512, 50, 4),
    ([1000, 24, 1], 1230, 1664, None, 1),
    ([30] * 10, 2451, 2048, 12, 7),
    ([257, 1], 3601, 2080, None, 1),
    ([1700, 1, 5000], 4100, 1152, 700, 3),
    ([4090], 4090, 2170, None, 1),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("case", TILED, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[1]}-{c[2]}")
def test_product_tiled(case, fmt):
    import torch
    import grouped_gemm_layer_amd as g
    counts, N, K, T, k = case
    if fmt == "mxfp8":
        K = -(-K // 32) * 32
    print(f"[product] {len(counts)} experts, {sum(counts)} rows, N={N} K={K} {fmt}", flush=True)
    p = Product(counts, N, K, fmt, T, k)
    ref = p.reference()
    for typ in ("bf16", "fp32"):
        c = torch.full((p.rows, N + 3), 5.0, dtype=_dt(typ), device="cuda")
        g.mxfp4_product(*p.args, c[:, 2:2 + N], **p.kw)
        p.check(c[:, 2:2 + N], typ, ref)
        assert bool((c[:, :2] == 5).all()) and bool((c[:, -1:] == 5).all())
        c2 = torch.empty(p.rows, N, dtype=_dt(typ), device="cuda")
        g.mxfp4_product(*p.args, c2, **p.kw)
        assert torch.equal(c2, c[:, 2:2 + N])


@pytest.mark.parametrize("typ", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[1]}-{c[2]}")
def test_product(case, fmt, typ):
    import torch
    import grouped_gemm_layer_amd as g
    counts, N, K, T, k = case
    if fmt == "mxfp8":
        K = -(-K // 32) * 32
    print(f"[product] {len(counts)} experts, {sum(counts)} rows, N={N} K={K} {fmt} {typ}", flush=True)
    p = Product(counts, N, K, fmt, T, k)
    c = torch.full((p.rows, N + 3), 5.0, dtype=_dt(typ), device="cuda")
    g.mxfp4_product(*p.args, c[:, 2:2 + N], **p.kw)
    got = p.check(c[:, 2:2 + N], typ)
    assert np.all(c[:, :2].cpu().float().numpy() == 5) and np.all(c[:, -1:].cpu().float().numpy() == 5)
    c2 = torch.empty(p.rows, N, dtype=_dt(typ), device="cuda")
    g.mxfp4_product(*p.args, c2, **p.kw)
    assert torch.equal(c2, c[:, 2:2 + N])                # the pitch changes nothing


@pytest.mark.parametrize("rows,N,K", [(1, 200, 384), (16, 200, 384), (200, 200, 384), (900, 200, 384),
                                      (1500, 3800, 384), (4090, 4090, 1024)])
def test_product_without_experts(rows, N, K):
    import torch
    import grouped_gemm_layer_amd as g
    p = Product([rows], N, K, "mxfp4", dense=True)
    c = torch.empty(rows, N, device="cuda")
    g.mxfp4_product(*p.args, c, **p.kw)
    p.check(c, "fp32")


@pytest.mark.parametrize("counts,N,K", [([3, 0, 5], 72, 256), ([100, 70, 0], 72, 256), ([600, 300], 72, 256),
                                        ([100, 1900, 0], 1100, 1024), ([4000, 2700], 4100, 1024)])
def test_rows_behind_the_last_stay(counts, N, K):
    """c longer than the rows routed: the rest is left as it was; no rows at all; offsets past c are cut."""
    import torch
    import grouped_gemm_layer_amd as g
    p = Product(counts, N, K, "mxfp4", T=20, k=2, gap=37)
    c = torch.full((p.rows, N), 5.0, device="cuda")
    g.mxfp4_product(*p.args, c, **p.kw)
    p.check(c, "fp32")
    M = sum(counts)
    assert torch.equal(c[M:], torch.full_like(c[M:], 5.0))
    c.fill_(5.0)
    g.mxfp4_product(*p.args, c, **dict(p.kw, offsets=torch.zeros(p.E + 1, dtype=torch.int32, device="cuda")))
    assert torch.equal(c, torch.full_like(c, 5.0))
    far = p.kw["offsets"].clone()
    far[-1] += 1000
    buf = torch.full((p.rows + 2000, N), 5.0, device="cuda")
    g.mxfp4_product(*p.args, buf[:p.rows], **dict(p.kw, offsets=far))
    assert torch.equal(buf[p.rows:], torch.full_like(buf[p.rows:], 5.0))


@pytest.mark.parametrize("rows,N,K", [(8, 90, 352), (100, 90, 352), (400, 90, 352), (1600, 1100, 1056), (3300, 4100, 1024)])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_scale_255_makes_what_it_enters_nan(fmt, rows, N, K):
    import torch
    import grouped_gemm_layer_amd as g
    p = Product([rows, rows], N, K, fmt)
    sa, sb = p.args[1], p.args[3]
    sa[3, 2] = 255
    sb[1, 7, 10] = 255
    c = torch.empty(p.rows, N, device="cuda")
    g.mxfp4_product(*p.args, c, **p.kw)
    nan = torch.zeros(p.rows, N, dtype=torch.bool, device="cuda")
    nan[3] = True
    nan[rows:, 7] = True
    assert torch.equal(c.isnan(), nan)


@pytest.mark.parametrize("rows", [6, 90, 600])
def test_inputs_from_the_quantisers(rows):
    """Quantised on the GPU and multiplied, against the same in fp64; MXFP8 rows from the layer's quantiser."""
    import torch
    import grouped_gemm_layer_amd as g
    gen = torch.Generator("cuda").manual_seed(rows)
    x = torch.randn(rows, 256, device="cuda", generator=gen).bfloat16()
    w = (0.02 * torch.randn(2 * 64, 256, device="cuda", generator=gen)).bfloat16()
    cw, sw = torch.empty(128, 128, dtype=torch.uint8, device="cuda"), torch.empty(128, 8, dtype=torch.uint8, device="cuda")
    g.mxfp4_quantize(w, cw, sw)
    bv = mx.decode(cw.cpu().numpy(), sw.cpu().numpy(), 256).reshape(2, 64, 256)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    for fmt in ("mxfp4", "mxfp8"):
        if fmt == "mxfp4":
            ca, sa = torch.empty(rows, 128, dtype=torch.uint8, device="cuda"), torch.empty(rows, 8, dtype=torch.uint8, device="cuda")
            g.mxfp4_quantize(x, ca, sa)
            av = mx.decode(ca.cpu().numpy(), sa.cpu().numpy(), 256)
        else:
            ca, sa = torch.empty(rows, 256, dtype=torch.uint8, device="cuda"), torch.empty(rows, 8, dtype=torch.uint8, device="cuda")
            g.mxfp8_quantize(x, 1, ca, sa)
            av = mx.decode_mxfp8(ca.cpu().numpy(), sa.cpu().numpy())
        c = torch.empty(rows, 64, device="cuda")
        g.mxfp4_product(ca, sa, cw.view(2, 64, -1), sw.view(2, 64, -1), c, k=256, a_format=fmt, offsets=off)
        got = c.double().cpu().numpy()
        for e, r in enumerate((slice(0, rows // 3), slice(rows // 3, rows))):
            want, mag = av[r] @ bv[e].T, np.abs(av[r]) @ np.abs(bv[e]).T
            assert np.all(np.abs(got[r] - want) <= (4 * 2.0 ** -23 if fmt == "mxfp4" else 2e-4) * mag + 2.0 ** -24 * np.abs(want))


def test_large_output_offsets():
    """c past 4 GiB: rows at both ends are right."""
    import torch
    import grouped_gemm_layer_amd as g
    rows, N = 1_060_000, 1024
    p = Product([64], N, 64, "mxfp4", dense=True)
    a_map = (torch.arange(rows, device="cuda") % 64).to(torch.int32)
    c = torch.empty(rows, N, device="cuda", dtype=torch.float32)
    g.mxfp4_product(*p.args, c, k=64, row_map=a_map)
    first = c[:64].clone()
    p.check(first, "fp32")
    for at in (64, 524288, rows // 64 * 64 - 64):
        assert torch.equal(c[at:at + 64], first)
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("counts,N,K", [([3, 0, 5], 136, 512), ([100, 70, 0, 40], 136, 512), ([300, 600], 136, 512),
                                        ([300, 1600], 1136, 1024), ([4000, 2700], 4100, 1024)])
def test_graph_replays_and_streams(counts, N, K):
    import torch
    import grouped_gemm_layer_amd as g
    p = Product(counts, N, K, "mxfp4", T=30, k=4)
    x = torch.randn(30, K, device="cuda").bfloat16()
    c = torch.empty(p.rows, N, dtype=torch.bfloat16, device="cuda")

    def step():
        g.mxfp4_quantize(x, p.args[0], p.args[1])
        g.mxfp4_product(*p.args, c, **p.kw)

    step()
    eager = c.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.zero_()
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        c.zero_()
        torch.randn(1 << 20, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, eager)
