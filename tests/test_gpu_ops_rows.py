"""Rows sorted by expert and back (sort, permute, unpermute and their
gradients) against plain fp64 NumPy, through the binding.

Bounds.  The maps are whole numbers and must be equal.  A copied row must be
equal bit for bit.  A weighted row is one fp32 product rounded once to the
storage type: |err| <= (2^-24 + u)|v| with u = 2^-8 (bf16) or 0 more (fp32),
doubled below for the double rounding.  A sum of n terms in fp32: each term's
product and each addition round once, so |err| <= (n + 1) 2^-24 sum|terms|,
plus the final rounding u|v|; a dot over H values likewise with n = H.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def np_sort(idx, E):
    """counts, offsets, sorted_to_flat, flat_to_sorted by the definition."""
    flat = idx.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    counts = np.array([(key == e).sum() for e in range(E)], dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = offsets[-1]
    s2f = np.where(np.arange(flat.size) < n, order, -1).astype(np.int32)
    f2s = np.full(flat.size, -1, dtype=np.int32)
    f2s[order[:n]] = np.arange(n, dtype=np.int32)
    return counts, offsets, s2f, f2s


def make_idx(rng, T, k, E, masked):
    """[T, k] int32 expert ids; with `masked`, some outside [0, E) (far outside
    too), and whole tokens without an expert."""
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    if masked and T:
        idx[rng.random((T, k)) < 0.3] = -1
        idx[rng.random((T, k)) < 0.1] = E
        idx[rng.random((T, k)) < 0.05] = -2 ** 31
        idx[rng.random((T, k)) < 0.05] = 2 ** 31 - 1
        idx[rng.random(T) < 0.2] = -1
    return idx


def gpu_sort(idx, E):
    import torch
    import grouped_gemm_layer_amd as g
    T, k = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    r = g.RoutingBuffers(torch.from_numpy(idx).cuda(), None, torch.full((E,), -9, **i32),
                         torch.full((E + 1,), -9, **i32), torch.full((T * k,), -9, **i32),
                         torch.full((T * k,), -9, **i32))
    ws = torch.full((g.sort_workspace_size(T, k, E),), 0xAB, dtype=torch.uint8, device="cuda")
    g.sort_tokens(r, ws)
    return r


def _maps(r):
    return [t.cpu().numpy() for t in (r.counts, r.offsets, r.sorted_to_flat, r.flat_to_sorted)]


@pytest.mark.parametrize("T,k,E,masked", [
    (0, 2, 5, False), (1, 1, 1, False), (1, 8, 128, False), (1, 4, 3, True), (7, 3, 512, True), (63, 1, 2, False),
    (512, 8, 128, False), (512, 8, 128, True), (513, 8, 100, True), (4097, 1, 511, False), (5000, 7, 512, True),
    (16384, 8, 128, False), (40000, 8, 33, True),
])
def test_sort_is_exact(T, k, E, masked):
    print(f"[sort] T={T} k={k} E={E} masked={masked}", flush=True)
    rng = np.random.default_rng(T * 31 + k * 7 + E)
    idx = make_idx(rng, T, k, E, masked)
    for got, want in zip(_maps(gpu_sort(idx, E)), np_sort(idx, E)):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("T,fill", [(300, -1), (300, 4), (9000, -1), (9000, 4)])
def test_sort_all_masked_and_one_expert(T, fill):
    idx = np.full((T, 2), fill, dtype=np.int32)
    for got, want in zip(_maps(gpu_sort(idx, 6)), np_sort(idx, 6)):
        assert np.array_equal(got, want)


def test_sort_equals_route_on_the_routers_indices():
    """On the router's own indices the sort gives the router's maps."""
    import torch
    import grouped_gemm_layer_amd as g
    T, E, k = 3000, 96, 8
    d = g.Dims.of(T, 64, 64, E, k, "bf16")
    ref = g.alloc_routing(d)
    logits = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    g.route(d, logits, ref, g.alloc_workspace(g.workspace_size(d)[0]))
    got = g.alloc_routing(d)
    got.topk_idx = ref.topk_idx
    g.sort_tokens(got, g.alloc_workspace(g.sort_workspace_size(T, k, E)))
    for name in ("counts", "offsets", "sorted_to_flat", "flat_to_sorted"):
        assert torch.equal(getattr(got, name), getattr(ref, name)), name


class Rows:
    """Inputs of one shape: token rows and expert rows, as tensors whose rows
    may sit in wider ones (pitch), and their fp64 values."""

    def __init__(self, T, H, k, E, typ, masked, pad, seed, weights):
        import torch
        rng = np.random.default_rng(seed)
        self.typ, self.T, self.H, self.k = typ, T, H, k
        self.idx = make_idx(rng, T, k, E, masked)
        self.r = gpu_sort(self.idx, E)
        self.counts, self.offsets, self.s2f, self.f2s = np_sort(self.idx, E)
        self.n, self.M = int(self.offsets[-1]), T * k
        self.dt = _torch_type(typ)
        self.pad = pad
        self.w = rng.standard_normal((T, k)).astype(np.float32) if weights else None
        self.wt = None if self.w is None else torch.from_numpy(self.w).cuda()
        self.rng = rng

    def matrix(self, rows, fill=None):
        """A [rows, H] tensor inside one with `pad` more columns, and its values."""
        import torch
        v = self.rng.standard_normal((rows, self.H + self.pad)).astype(np.float32)
        t = torch.from_numpy(v).to(self.dt).cuda()
        if fill is not None:
            t.fill_(fill)
        t = t[:, self.pad // 2:self.pad // 2 + self.H]
        return t, t.double().cpu().numpy()

    def weight(self):
        return np.ones((self.T, self.k)) if self.w is None else self.w.astype(np.float64)


def bound_close(got, want, absum, terms, u):
    err = np.abs(got - want)
    lim = (terms + 1) * U32 * absum * 1.01 + u * np.abs(want) * 1.01 + 1e-45
    assert np.all(err <= lim), f"worst {np.max(err - lim)} over the bound at {np.unravel_index(np.argmax(err - lim), err.shape)}"


SHAPES = [
    # T, H, k, E, type, masked, pad, weights
    (1, 8, 1, 1, "bf16", False, 0, False),
    (1, 1, 1, 4, "fp32", False, 0, True),
    (5, 7, 3, 6, "bf16", True, 0, True),
    (33, 64, 8, 16, "bf16", False, 0, True),
    (17, 512, 2, 8, "fp32", True, 0, False),
    (40, 515, 4, 8, "bf16", True, 3, True),
    (21, 1001, 6, 12, "fp32", True, 5, True),
    (9, 1024, 8, 16, "bf16", False, 0, True),
    (64, 2048, 8, 128, "bf16", False, 0, True),
    (12, 4099, 8, 16, "bf16", True, 1, True),
    (6, 9000, 5, 9, "fp32", False, 0, True),
    (11, 300, 9, 32, "bf16", True, 0, True),       # more slots than one batch of rows
    (7, 2500, 32, 64, "fp32", True, 0, True),
    (700, 96, 4, 20, "bf16", True, 0, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_there_and_back(shape):
    import torch
    import grouped_gemm_layer_amd as g
    T, H, k, E, typ, masked, pad, weights = shape
    print(f"[rows] {shape}", flush=True)
    s = Rows(T, H, k, E, typ, masked, pad, 11 + T + H, weights)
    u, w, n, M = U[typ], s.weight(), s.n, s.M
    x, xv = s.matrix(T)
    tok, slot = s.s2f[:n] // k, s.s2f[:n]
    wr = w.reshape(-1)[slot][:, None]

    xp, _ = s.matrix(M, fill=-3.0)                  # rows behind the last stay -3
    g.permute(x, s.r, xp, weights=s.wt)
    got = xp.double().cpu().numpy()
    assert np.all(got[n:] == -3.0)
    if weights:
        bound_close(got[:n], wr * xv[tok], np.abs(wr * xv[tok]), 0, u)
    else:
        assert np.array_equal(got[:n], xv[tok])

    rows, rv = s.matrix(M)
    rows[n:] = float("nan")                         # rows no slot names are not read
    rv[n:] = 0
    live = (s.f2s >= 0).reshape(T, k)
    byslot = np.where(live.reshape(-1)[:, None], rv[np.maximum(s.f2s, 0)], 0.0).reshape(T, k, H)
    terms = w[:, :, None] * byslot
    y, _ = s.matrix(T, fill=float("nan"))
    g.unpermute(rows, s.r, y, weights=s.wt)
    bound_close(y.double().cpu().numpy(), terms.sum(1), np.abs(terms).sum(1), k, u)

    dx, _ = s.matrix(T, fill=float("nan"))
    dw = torch.full((T, k), float("nan"), device="cuda")
    g.permute_backward(rows, s.r, dx, weights=s.wt, x=x, dweights=dw)
    assert torch.equal(dx.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))   # the same sum
    prod = byslot * xv[:, None, :]
    bound_close(dw.double().cpu().numpy(), prod.sum(2), np.abs(prod).sum(2), H, 0)
    assert np.all(dw.cpu().numpy()[~live] == 0)

    drows, _ = s.matrix(M, fill=-3.0)
    dw2 = torch.full((T, k), float("nan"), device="cuda")
    g.unpermute_backward(x, s.r, drows, weights=s.wt, rows=rows, dweights=dw2)
    assert torch.equal(drows.contiguous().view(torch.uint8), xp.contiguous().view(torch.uint8))
    bound_close(dw2.double().cpu().numpy(), prod.sum(2), np.abs(prod).sum(2), H, 0)
    assert np.all(dw2.cpu().numpy()[~live] == 0)


def test_gradients_against_differences():
    """<dy, unpermute(rows, w)> and <dxp, permute(x, w)> are linear in each
    argument: a central difference in a random direction equals the gradient's
    product with it, up to the fp32 rounding of both sides (values of order 1,
    H = 40 sums of k = 3 terms: 1e-4 of the magnitudes is far above it, and far
    below a wrong gradient)."""
    import torch
    import grouped_gemm_layer_amd as g
    s = Rows(50, 40, 3, 7, "fp32", True, 0, 77, True)
    x, _ = s.matrix(50)
    rows, _ = s.matrix(s.M)
    dy, _ = s.matrix(50)
    d = dict(rows=s.matrix(s.M)[0], w=s.matrix(50)[0][:, :3].contiguous(), x=s.matrix(50)[0])

    def y_of(rows, w):
        y = torch.empty(50, 40, device="cuda")
        g.unpermute(rows.contiguous(), s.r, y, weights=w.contiguous())
        return y.double()

    drows = torch.zeros(s.M, 40, device="cuda")
    dw = torch.empty(50, 3, device="cuda")
    g.unpermute_backward(dy, s.r, drows, weights=s.wt, rows=rows, dweights=dw)
    h = 0.5
    for grad, a, b in ((drows, lambda t: (rows + t * d["rows"], s.wt), d["rows"]),
                       (dw, lambda t: (rows, s.wt + t * d["w"]), d["w"])):
        diff = float(((y_of(*a(h)) - y_of(*a(-h))) * dy.double()).sum() / (2 * h))
        want = float((grad.double() * b.double()).sum())
        assert abs(diff - want) <= 1e-4 * float((grad.double() * b.double()).abs().sum())

    def xp_of(x, w):
        xp = torch.zeros(s.M, 40, device="cuda")
        g.permute(x.contiguous(), s.r, xp, weights=w.contiguous())
        return xp.double()

    dx = torch.empty(50, 40, device="cuda")
    g.permute_backward(rows, s.r, dx, weights=s.wt, x=x, dweights=dw)
    live = torch.zeros(s.M, 1, device="cuda", dtype=torch.float64)
    live[:s.n] = 1
    for grad, a, b in ((dx, lambda t: (x + t * d["x"], s.wt), d["x"]), (dw, lambda t: (x, s.wt + t * d["w"]), d["w"])):
        diff = float(((xp_of(*a(h)) - xp_of(*a(-h))) * rows.double() * live).sum() / (2 * h))
        want = float((grad.double() * b.double()).sum())
        assert abs(diff - want) <= 1e-4 * float((grad.double() * b.double()).abs().sum())


def test_masked_slots_and_values_that_are_not_finite():
    """Weights of masked slots are not used, NaN or not; a NaN or infinity in a
    named row reaches exactly its token; copies keep a NaN's bits."""
    import torch
    import grouped_gemm_layer_amd as g
    idx = np.array([[0, 1], [-1, 1], [-1, 7], [2, 2]], dtype=np.int32)
    r = gpu_sort(idx, 3)
    w = torch.tensor([[0.5, 2.0], [float("nan"), 1.0], [float("inf"), float("nan")], [1.0, -1.0]], device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        x = torch.ones(4, 24, dtype=dt, device="cuda")
        x[0, 3] = float("nan")
        x[3, 5] = float("inf")
        xp = torch.zeros(8, 24, dtype=dt, device="cuda")
        g.permute(x, r, xp, weights=w)
        xp2 = torch.zeros_like(xp)
        g.permute(x, r, xp2)
        row = r.flat_to_sorted.view(4, 2).tolist()
        assert torch.equal(xp2[row[0][0]].view(torch.uint8), x[0].view(torch.uint8))
        assert xp[row[0][0]].isnan().sum() == 1 and xp[row[3][1], 5] == float("-inf")
        y = torch.empty(4, 24, dtype=dt, device="cuda")
        g.unpermute(xp, r, y, weights=w)
        assert torch.equal(y[2], torch.zeros_like(y[2]))               # no slot: zero, whatever the weights
        assert y[1].isfinite().all() and y[0].isnan().sum() == 1
        assert y[3, 5].item() == float("inf") and y[3].isfinite().sum() == 23   # inf * 1 + (-inf) * -1
        dw = torch.empty(4, 2, device="cuda")
        g.unpermute_backward(torch.ones_like(x), r, torch.zeros_like(xp), weights=w, rows=xp2, dweights=dw)
        assert dw[2].tolist() == [0.0, 0.0] and dw[1, 0] == 0.0 and dw[1, 1].item() == 24.0


def test_maps_that_point_outside_are_ignored():
    """Rows past the buffer (a capacity smaller than the rows routed) are
    neither written nor read."""
    import torch
    import grouped_gemm_layer_amd as g
    T, k, H, cap = 30, 4, 72, 50
    idx = np.random.default_rng(3).integers(0, 5, (T, k)).astype(np.int32)
    r = gpu_sort(idx, 5)
    x = torch.randn(T, H, device="cuda")
    buf = torch.full((cap + 40, H), 7.0, device="cuda")
    g.permute(x, r, buf[:cap])
    assert torch.equal(buf[cap:], torch.full_like(buf[cap:], 7.0))
    f2s = r.flat_to_sorted.view(T, k).long()
    y = torch.empty(T, H, device="cuda")
    g.unpermute(buf[:cap], r, y)
    n = (f2s < cap).sum(1, keepdim=True)
    assert torch.allclose(y, x * n, rtol=1e-6)
    empty = torch.empty(0, H, device="cuda")
    g.unpermute(empty, r, y)
    assert torch.equal(y, torch.zeros_like(y))
    g.permute(x, r, empty)


def test_offsets_past_32_bits():
    """Expert rows of more than 4 GiB, the last ones read and written."""
    import torch
    import grouped_gemm_layer_amd as g
    T, k, H = 1_100_000, 1, 2048
    idx = torch.zeros(T, 1, dtype=torch.int32)
    idx[::2] = 1
    r = gpu_sort(idx.numpy(), 2)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    xp = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    g.permute(x, r, xp)
    assert torch.equal(xp[:T // 2], x[1::2]) and torch.equal(xp[T // 2:], x[::2])
    y = torch.empty_like(x)
    g.unpermute(xp, r, y)
    assert torch.equal(y, x)
    del x, xp, y
    torch.cuda.empty_cache()


def test_more_tokens_than_a_launch_takes():
    """2^22 tokens a launch: those behind get the same."""
    import torch
    import grouped_gemm_layer_amd as g
    T, k, H, E = 2 ** 22 + 4099, 2, 9, 5
    idx = torch.randint(-1, E, (T, k), dtype=torch.int32)
    r = gpu_sort(idx.numpy(), E)
    x, w = torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")
    n = int(r.offsets[-1])
    xp = torch.full((T * k, H), 7.0, device="cuda")
    g.permute(x, r, xp, weights=w)
    f = r.sorted_to_flat[:n].long()
    assert torch.equal(xp[:n], w.view(-1)[f, None] * x[f // k]) and bool((xp[n:] == 7).all())
    y, dw = torch.empty_like(x), torch.empty(T, k, device="cuda")
    g.permute_backward(xp, r, y, weights=w, x=x, dweights=dw)
    rows = torch.where((r.flat_to_sorted >= 0)[:, None], xp[r.flat_to_sorted.clamp(min=0).long()], 0.0).view(T, k, H).double()
    want = (w[..., None] * rows).sum(1)
    assert bool(((y - want).abs() <= 4 * U32 * (w[..., None] * rows).abs().sum(1)).all())
    want, mag = (x[:, None] * rows).sum(2), (x[:, None] * rows).abs().sum(2)
    assert bool(((dw - want).abs() <= (H + 2) * U32 * mag).all())
    del x, w, xp, y, rows, want, mag
    torch.cuda.empty_cache()


def test_no_tokens():
    import torch
    import grouped_gemm_layer_amd as g
    r = gpu_sort(np.zeros((0, 4), dtype=np.int32), 3)
    assert r.counts.tolist() == [0, 0, 0] and r.offsets.tolist() == [0, 0, 0, 0]
    x, xp = torch.empty(0, 16, device="cuda"), torch.full((5, 16), 2.0, device="cuda")
    g.permute(x, r, xp)
    g.unpermute(xp, r, x)
    assert torch.equal(xp, torch.full_like(xp, 2.0))


def test_graph_and_side_stream():
    """Sort, rows there and back and both gradients, captured on a stream of
    their own: every replay, with other work in between, gives the eager bits."""
    import torch
    import grouped_gemm_layer_amd as g
    T, k, H, E = 900, 8, 256, 24
    rng = np.random.default_rng(8)
    idx = make_idx(rng, T, k, E, True)
    r = gpu_sort(idx, E)
    w = torch.rand(T, k, device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    xp, drows = (torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, dw2 = torch.empty_like(w), torch.empty_like(w)
    ws = g.alloc_workspace(g.sort_workspace_size(T, k, E))
    outs = [xp, drows, y, dx, dw, dw2, r.counts, r.offsets, r.sorted_to_flat, r.flat_to_sorted]

    def step():
        g.sort_tokens(r, ws)
        g.permute(x, r, xp, weights=w)
        g.unpermute(xp, r, y, weights=w)
        g.unpermute_backward(x, r, drows, weights=w, rows=xp, dweights=dw)
        g.permute_backward(drows, r, dx, weights=w, x=x, dweights=dw2)

    step()
    eager = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.randn(1 << 20, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
