"""The operators beside the layer in a row, as a program calls them: an expert
layer on MXFP4 weights (serving), the experts of a training step with their
gradients and the clipping, and both captured and replayed.

Bounds.  Of the serving layer each stage is held against fp64 of what the stage
before left on the device: products to the roundings of their fp32 sums and of
their output (2^-8 relative for bf16), codes exactly, the weighted sum over k
rows to (k + 1) 2^-24 of its terms' magnitudes and one rounding.  In the
training step the experts are fp64 products rounded to fp32 once, so a value
made of n roundings one after another is off by at most n 2^-24 of its terms'
magnitudes: n = 2 + k for outputs and token gradients (product or weight,
expert, sum over k), n = 2 for weight gradients, H + 2 for the dots.
"""
import numpy as np
import pytest

import _mxfp4_reference as mx
from test_gpu_ops_rows import gpu_sort, make_idx

pytestmark = pytest.mark.gpu

U32, UB = 2.0 ** -24, 2.0 ** -8


def _u8(*shape):
    import torch
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


class Serving:
    """T tokens of H values, E experts of width I: token codes once, each
    expert's rows through two products with SwiGLU between, weighted sum."""

    def __init__(self, T, H, I, E, k, fmt="mxfp4", seed=0):
        import torch
        gen = torch.Generator("cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.T, self.H, self.I, self.E, self.k, self.fmt = T, H, I, E, k, fmt
        self.x = rn(T, H).bfloat16()
        self.w13, self.w2 = (0.1 * rn(E, 2 * I, H)).bfloat16(), (0.1 * rn(E, H, I)).bfloat16()
        self.gate = torch.rand(T, k, device="cuda", generator=gen)
        kh, ki, M = -(-H // 32), -(-I // 32), T * k
        self.c13, self.s13, self.c2, self.s2 = _u8(E, 2 * I, kh * 16), _u8(E, 2 * I, kh), _u8(E, H, ki * 16), _u8(E, H, ki)
        self.cx, self.sx = _u8(T, H if fmt == "mxfp8" else kh * 16), _u8(T, kh)
        self.cp, self.sp = _u8(M, kh * 16), _u8(M, kh)
        self.ca, self.sa = _u8(M, ki * 16), _u8(M, ki)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.g13, self.g13p, self.o = (torch.zeros(M, n, **bf) for n in (2 * I, 2 * I, H))
        self.xp, self.y = torch.zeros(M, H, **bf), torch.zeros(T, H, **bf)

    def weights(self):
        import grouped_gemm_layer_amd as g
        g.mxfp4_quantize(self.w13, self.c13, self.s13)
        g.mxfp4_quantize(self.w2, self.c2, self.s2)

    def route(self, idx, ws):
        import grouped_gemm_layer_amd as g
        import torch
        i32 = dict(dtype=torch.int32, device="cuda")
        if not hasattr(self, "r"):
            self.r = g.RoutingBuffers(idx, None, torch.zeros(self.E, **i32), torch.zeros(self.E + 1, **i32),
                                      torch.zeros(self.T * self.k, **i32), torch.zeros(self.T * self.k, **i32))
        g.sort_tokens(self.r, ws)

    def forward(self):
        import grouped_gemm_layer_amd as g
        r = self.r
        if self.fmt == "mxfp8":
            g.mxfp8_quantize(self.x, 1, self.cx, self.sx)
        else:
            g.mxfp4_quantize(self.x, self.cx, self.sx)
        g.mxfp4_product(self.cx, self.sx, self.c13, self.s13, self.g13, self.H, a_format=self.fmt, offsets=r.offsets,
                        row_map=r.sorted_to_flat, row_div=self.k)
        g.mxfp4_quantize(self.g13, self.ca, self.sa, swiglu=True)
        g.mxfp4_product(self.ca, self.sa, self.c2, self.s2, self.o, self.I, offsets=r.offsets)
        g.unpermute(self.o, r, self.y, weights=self.gate)


SHAPES = [(4, 256, 96, 16, 2, False), (33, 160, 64, 7, 3, True), (200, 1000, 72, 5, 4, True), (1, 64, 32, 3, 1, False),
          (2000, 512, 384, 4, 2, True)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,H,I,E,k,masked", SHAPES)
def test_serving_layer(T, H, I, E, k, masked, fmt):
    import torch
    import grouped_gemm_layer_amd as g
    if fmt == "mxfp8":
        H = -(-H // 32) * 32
    s = Serving(T, H, I, E, k, fmt)
    idx = torch.from_numpy(make_idx(np.random.default_rng(T), T, k, E, masked)).cuda()
    ws = g.alloc_workspace(max(256, g.sort_workspace_size(T, k, E)), "cuda")
    s.weights()
    s.route(idx, ws)
    s.forward()
    off = s.r.offsets.cpu().numpy()
    n, f = off[-1], s.r.sorted_to_flat.cpu().numpy()
    npy = lambda t: t.cpu().numpy()  # noqa: E731
    xv = mx.decode(npy(s.cx), npy(s.sx), H) if fmt == "mxfp4" else mx.decode_mxfp8(npy(s.cx), npy(s.sx))
    code, scale = mx.encode(s.w13.double().cpu().numpy().reshape(-1, H))
    assert np.array_equal(mx.pack(code), npy(s.c13).reshape(-1, s.c13.shape[-1])) and np.array_equal(scale, npy(s.s13).reshape(-1, scale.shape[1]))
    rel = 2e-4 if fmt == "mxfp8" else (-(-H // 128) + 2) * 2 * U32

    def products(a, codes, scales, K, got, rel):
        for e in range(E):
            r = slice(off[e], off[e + 1])
            b = mx.decode(npy(codes[e]), npy(scales[e]), K)
            want, mag = a[r] @ b.T, np.abs(a[r]) @ np.abs(b).T
            assert np.all(np.abs(got[r] - want) <= rel * mag + 1.01 * UB * np.abs(want)), f"expert {e}"

    products(xv[f[:n] // k], s.c13, s.s13, H, s.g13.double().cpu().numpy(), rel)
    assert not bool(s.g13[n:].any())                              # rows behind the last: as they were
    products(mx.decode(npy(s.ca), npy(s.sa), I), s.c2, s.s2, I, s.o.double().cpu().numpy(), (-(-I // 128) + 2) * 2 * U32)
    rows = npy(s.r.flat_to_sorted)
    o = np.where((rows >= 0)[:, None], s.o.double().cpu().numpy()[np.maximum(rows, 0)], 0.0).reshape(T, k, H)
    terms = o * s.gate.double().cpu().numpy()[..., None]
    want = terms.sum(1)
    assert np.all(np.abs(s.y.double().cpu().numpy() - want) <= (k + 1) * U32 * np.abs(terms).sum(1) + 1.01 * UB * np.abs(want))

    # rows moved first and quantised then are the rows gathered by the product: equal bits
    if fmt == "mxfp4":
        g.permute(s.x, s.r, s.xp)
        g.mxfp4_quantize(s.xp, s.cp, s.sp)
        g.mxfp4_product(s.cp, s.sp, s.c13, s.s13, s.g13p, H, offsets=s.r.offsets)
        assert torch.equal(s.g13p[:n], s.g13[:n])


def test_serving_layer_replayed():
    """One graph for all routings: its replays read the indices anew."""
    import torch
    import grouped_gemm_layer_amd as g
    T, H, I, E, k = 40, 256, 128, 12, 3
    s = Serving(T, H, I, E, k)
    ws = g.alloc_workspace(max(256, g.sort_workspace_size(T, k, E)), "cuda")
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    s.weights()
    rng = np.random.default_rng(5)
    draws = [torch.from_numpy(make_idx(rng, T, k, E, m)).cuda() for m in (False, True, True)] + [torch.full((T, k), -1, dtype=torch.int32, device="cuda")]
    want = []
    for d in draws:
        idx.copy_(d)
        s.route(idx, ws)
        s.forward()
        want.append(s.y.clone())
    assert not bool(want[-1].any())                                # no slot has an expert: sums over nothing
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        s.route(idx, ws)
        s.forward()
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(2):
        for d, w in zip(draws, want):
            idx.copy_(d)
            s.y.fill_(3.0)
            torch.randn(1 << 18, device="cuda").sum().item()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(s.y, w)


def test_two_layers_at_once():
    """Two sets of buffers on two streams do not touch each other."""
    import torch
    import grouped_gemm_layer_amd as g
    runs = []
    for seed, (T, H, I, E, k) in enumerate([(900, 256, 128, 6, 2), (5, 512, 64, 30, 4)]):
        s = Serving(T, H, I, E, k, seed=seed)
        ws = g.alloc_workspace(max(256, g.sort_workspace_size(T, k, E)), "cuda")
        idx = torch.from_numpy(make_idx(np.random.default_rng(seed), T, k, E, True)).cuda()
        s.weights()
        s.route(idx, ws)
        s.forward()
        runs.append((s, ws, idx, s.y.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, idx, _, st in runs:
            with torch.cuda.stream(st):
                s.y.zero_()
                s.route(idx, ws)
                s.forward()
    torch.cuda.synchronize()
    for s, _, _, want, _ in runs:
        assert torch.equal(s.y, want)


class Training:
    """y = sum_j w o[row], o = W[e] x: forward, gradients of x, w and W, clipping."""

    def __init__(self, T, H, E, k, idx):
        import torch
        gen = torch.Generator("cuda").manual_seed(T)
        rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.T, self.H, self.E, self.k = T, H, E, k
        self.x, self.W, self.dy = rn(T, H), 0.1 * rn(E, H, H), rn(T, H)
        self.w = torch.rand(T, k, device="cuda", generator=gen)
        self.r = gpu_sort(idx, E)
        self.off = self.r.offsets.tolist()
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.xp, self.o, self.do, self.dxp = (z(T * k, H) for _ in range(4))
        self.y, self.dx, self.dw, self.dW = z(T, H), z(T, H), z(T, k), z(E, H, H)

    def experts(self):
        return [slice(self.off[e], self.off[e + 1]) for e in range(self.E)]

    def step(self, max_norm):
        import grouped_gemm_layer_amd as g
        g.permute(self.x, self.r, self.xp)
        for e, s in enumerate(self.experts()):
            self.o[s] = (self.xp[s].double() @ self.W[e].double().T).float()
        g.unpermute(self.o, self.r, self.y, weights=self.w)
        g.unpermute_backward(self.dy, self.r, self.do, weights=self.w, rows=self.o, dweights=self.dw)
        for e, s in enumerate(self.experts()):
            self.dxp[s] = (self.do[s].double() @ self.W[e].double()).float()
            self.dW[e] = (self.do[s].double().T @ self.xp[s].double()).float()
        g.permute_backward(self.dxp, self.r, self.dx)
        self.raw = [self.dW.clone(), self.dw.clone()]
        return g.GradientList([self.dW, self.dw]).clip(max_norm)

    def loss(self, x, w, W, idx):
        """<y, dy> and its terms' sums of magnitudes, in fp64 on the CPU."""
        y = np.zeros((self.T, self.H))
        for t in range(self.T):
            for j in range(self.k):
                if 0 <= idx[t, j] < self.E:
                    y[t] += w[t, j] * (W[idx[t, j]] @ x[t])
        return y


@pytest.mark.parametrize("T,H,E,k,masked", [(1, 3, 2, 1, False), (40, 33, 5, 3, True), (64, 16, 4, 2, False)])
def test_training_step(T, H, E, k, masked):
    import torch
    idx = make_idx(np.random.default_rng(T + 1), T, k, E, masked)
    s = Training(T, H, E, k, idx)
    x, w, W, dy = (t.double().cpu().numpy() for t in (s.x, s.w, s.W, s.dy))
    norm = s.step(0.75)
    got = {n: getattr(s, n).double().cpu().numpy() for n in ("y", "dx")}
    dW, dw = (t.double().cpu().numpy() for t in s.raw)
    want = {n: np.zeros_like(v) for n, v in (("y", dy), ("dx", x), ("dw", w), ("dW", W))}
    mag = {n: np.zeros_like(v) for n, v in want.items()}
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            for n, v, a in (("y", w[t, j] * (W[e] @ x[t]), w[t, j] * (np.abs(W[e]) @ np.abs(x[t]))),
                            ("dx", w[t, j] * (W[e].T @ dy[t]), w[t, j] * (np.abs(W[e]).T @ np.abs(dy[t])))):
                want[n][t] += v
                mag[n][t] += a
            want["dw"][t, j] = dy[t] @ W[e] @ x[t]
            mag["dw"][t, j] = np.abs(dy[t]) @ np.abs(W[e]) @ np.abs(x[t])
            want["dW"][e] += w[t, j] * np.outer(dy[t], x[t])
            mag["dW"][e] += w[t, j] * np.abs(np.outer(dy[t], x[t]))
    for n, g_, rounds in (("y", got["y"], 2 + k), ("dx", got["dx"], 2 + k), ("dw", dw, H + 2), ("dW", dW, 2)):
        assert np.all(np.abs(g_ - want[n]) <= 1.001 * rounds * U32 * mag[n]), n

    # against differences: along one direction of all three at once, the loss is a cubic in the step h, so that
    # (L(h) - L(-h)) / 2h is off by h^2 times its third coefficient
    rng = np.random.default_rng(0)
    d = [rng.standard_normal(v.shape) for v in (x, w, W)]
    h = 1e-4
    L = [float((s.loss(x + c * d[0], w + c * d[1], W + c * d[2], idx) * dy).sum()) for c in (h, -h)]
    third = abs(float((s.loss(d[0], d[1], d[2], idx) * dy).sum()))
    slope = float((got["dx"] * d[0]).sum() + (dw * d[1]).sum() + (dW * d[2]).sum())
    err = sum(float((r * U32 * mag[n] * np.abs(v)).sum()) for n, v, r in (("dx", d[0], 2 + k), ("dw", d[1], H + 2), ("dW", d[2], 2)))
    scale = sum(abs(v) for v in L)
    assert abs((L[0] - L[1]) / (2 * h) - slope) <= 1.001 * (err + h * h * third) + 1e-12 * (scale + 1) / h

    ref = np.sqrt((dW ** 2).sum() + (dw ** 2).sum())
    assert abs(float(norm) - ref) <= 2 * U32 * ref
    f = min(1.0, 0.75 / ref)
    for t, raw in ((s.dW, dW), (s.dw, dw)):
        assert np.all(np.abs(t.double().cpu().numpy() - f * raw) <= 3 * U32 * f * np.abs(raw))


def test_backward_rows_captured():
    """The row calls of forward and backward in one graph, replayed on new values."""
    import torch
    import grouped_gemm_layer_amd as g
    T, H, E, k = 130, 72, 6, 4
    idx = make_idx(np.random.default_rng(9), T, k, E, True)
    s = Training(T, H, E, k, idx)
    gl = g.GradientList([s.dx, s.dw])

    def run():
        g.permute(s.x, s.r, s.xp, weights=s.w)
        g.unpermute(s.xp, s.r, s.y, weights=s.w)
        g.unpermute_backward(s.dy, s.r, s.do, weights=s.w, rows=s.xp, dweights=s.dw)
        g.permute_backward(s.do, s.r, s.dx)
        gl.clip(1.0)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(3):
        for t in (s.x, s.dy):
            t.normal_()
        run()
        want = [t.clone() for t in (s.y, s.dx, s.dw, gl.norm)]
        for t in (s.y, s.dx, s.dw, gl.norm):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((s.y, s.dx, s.dw, gl.norm), want):
            assert torch.equal(t, w)
