"""Gradient norm and clipping against float64, through the binding.

Bounds.  The squares are exact in fp64 (24-bit factors) and their sum of n terms
is off by at most n 2^-53 of itself in any order (n < 2^25 here: below 2^-28);
the norm is rounded once to fp32.  A clipped value: factor (half a unit of fp32,
plus the norm's 2^-28), product, final rounding: (2^-24 + 2^-28 + 2^-24 + u)|v|.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _grads(sizes, types, scale=1.0, seed=0, pad=0):
    """Tensors of the given sizes and types; with `pad`, views at odd places of one buffer."""
    import torch
    rng = np.random.default_rng(seed)
    out = []
    for n, typ in zip(sizes, types):
        v = torch.from_numpy((scale * rng.standard_normal(n)).astype(np.float32)).to(_dt(typ)).cuda()
        if pad:
            buf = torch.full((n + 2 * pad,), 3.0, dtype=v.dtype, device="cuda")
            buf[pad:pad + n] = v
            v = buf[pad:pad + n]
        out.append(v)
    return out


def _norm(grads):
    return math.sqrt(math.fsum(float(np.sum(t.double().cpu().numpy() ** 2)) for t in grads))


def _close(got, old, factor):
    u = 2.0 ** -8 if "bfloat16" in str(got.dtype) else 2.0 ** -24
    want = old.double().cpu().numpy() * factor
    err = np.abs(got.double().cpu().numpy() - want)
    # below the normal numbers a rounding is half a step of the subnormals
    assert np.all(err <= (2.2 * 2.0 ** -24 + u) * 1.01 * np.abs(want) + (2.0 ** -134 if u > 1e-3 else 2.0 ** -149))


CASES = [
    ([1], ["fp32"]), ([1], ["bf16"]), ([0, 7, 0], ["fp32", "bf16", "fp32"]), ([16384], ["fp32"]), ([16385, 3], ["bf16", "fp32"]),
    ([100000, 1, 33, 4097], ["fp32", "bf16", "fp32", "bf16"]),
    ([3, 5, 7] * 50, ["bf16", "fp32", "bf16"] * 50),          # more tensors than one launch takes
    ([1000] * 96, ["fp32"] * 96), ([1000] * 97, ["bf16"] * 97),
    ([40_000_000, 12345], ["fp32", "bf16"]),
]


@pytest.mark.parametrize("pad", [0, 1, 5])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{sum(c[0])}")
def test_clip(case, pad):
    import torch
    import grouped_gemm_layer_amd as g
    sizes, types = case
    print(f"[clip] {len(sizes)} tensors, {sum(sizes)} values, pad {pad}", flush=True)
    grads = _grads(sizes, types, pad=pad)
    old = [t.clone() for t in grads]
    norm = _norm(old)
    for max_norm in (norm * 2, norm * 0.3):
        lst = g.GradientList(grads)
        got = lst.clip(max_norm)
        assert abs(float(lst.sumsq) - norm ** 2) <= 2.0 ** -28 * norm ** 2
        assert abs(float(got) - norm) <= (2.0 ** -24 + 2.0 ** -28) * norm
        for t, o in zip(grads, old):
            if max_norm > norm:
                assert torch.equal(t, o)
            else:
                _close(t, o, max_norm / norm)
    if pad:
        for t in grads:
            base = t._base
            assert torch.equal(base[:pad], torch.full_like(base[:pad], 3.0))
            assert torch.equal(base[-pad:], torch.full_like(base[-pad:], 3.0))


def test_clip_into_other_tensors_and_the_plain_calls():
    import torch
    import grouped_gemm_layer_amd as g
    grads = _grads([5000, 17, 300], ["fp32", "bf16", "fp32"], seed=3)
    old = [t.clone() for t in grads]
    norm = _norm(old)
    for max_norm in (0.4 * norm, 3 * norm):
        out = [torch.full_like(t, 9.0) for t in grads]
        sumsq = torch.empty(1, dtype=torch.float64, device="cuda")
        n = torch.empty(1, device="cuda")
        g.grad_norm(grads, sumsq, g.alloc_workspace(g.grad_workspace_size(3)))
        g.grad_clip(grads, sumsq, max_norm, norm=n, out=out)
        for t, o, v in zip(grads, old, out):
            assert torch.equal(t, o)
            if max_norm > norm:
                assert torch.equal(v, o)
            else:
                _close(v, o, max_norm / norm)
        assert abs(float(n) - norm) <= 2.0 ** -23 * norm


def test_norm_over_ranks():
    """sumsq added up in between, as ranks do: the joint norm clips both lists."""
    import torch
    import grouped_gemm_layer_amd as g
    a, b = _grads([4000], ["fp32"], seed=1), _grads([900, 20], ["bf16", "fp32"], seed=2)
    old = [t.clone() for t in a + b]
    norm = _norm(old)
    la, lb = g.GradientList(a), g.GradientList(b)
    total = la.sum_squares() + lb.sum_squares()
    la.sumsq.copy_(total)
    lb.sumsq.copy_(total)
    la.scale(1.0)
    lb.scale(1.0)
    for t, o in zip(a + b, old):
        _close(t, o, 1.0 / norm)


@pytest.mark.parametrize("scale", [1e20, 1e-30, 3e38])
def test_squares_outside_fp32(scale):
    """Squares that fp32 cannot hold: the norm is right all the same."""
    import torch
    import grouped_gemm_layer_amd as g
    n = 1000
    t = torch.full((n,), scale, device="cuda")
    t[::2] *= -0.5
    old = t.clone()
    norm = _norm([old])
    lst = g.GradientList([t])
    got = lst.clip(norm / 4)
    if norm < 3.4e38:
        assert abs(float(got) - norm) <= 2.0 ** -23 * norm
    else:
        assert float(got) == float("inf")            # the fp32 output; sumsq holds it
    assert abs(float(lst.sumsq) - norm ** 2) <= 2.0 ** -40 * norm ** 2
    _close(t, old, np.float32(norm / 4) / norm) if norm / 4 < 3.4e38 else None


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_clips_nothing(bad):
    import torch
    import grouped_gemm_layer_amd as g
    grads = _grads([70000, 40], ["fp32", "bf16"])
    grads[1][7] = bad
    old = [t.clone() for t in grads]
    out = [torch.zeros_like(t) for t in grads]
    got = g.GradientList(grads, out=out).clip(1.0)
    assert not math.isfinite(float(got))
    for o, v in zip(old, out):
        assert torch.equal(o.view(torch.uint8), v.view(torch.uint8))
    g.GradientList(grads).clip(1.0)
    for o, v in zip(old, grads):
        assert torch.equal(o.view(torch.uint8), v.view(torch.uint8))


def test_zero_gradients_zero_limit_and_no_values():
    import torch
    import grouped_gemm_layer_amd as g
    z = torch.zeros(100, device="cuda")
    assert float(g.GradientList([z]).clip(0.0)) == 0.0 and not z.isnan().any()
    t = torch.ones(100, device="cuda")
    assert float(g.GradientList([t]).clip(0.0)) == 10.0 and torch.equal(t, z)
    e = torch.empty(0, device="cuda")
    assert float(g.GradientList([e]).clip(1.0)) == 0.0
    sumsq = torch.full((1,), 5.0, dtype=torch.float64, device="cuda")
    g.grad_norm([], sumsq, g.alloc_workspace(0))
    assert float(sumsq) == 0.0


def test_overlapping_tensors_are_refused():
    import torch
    import grouped_gemm_layer_amd as g
    t = torch.ones(100, device="cuda")
    for pair in ([t, t], [t[:60], t[59:]], [t[10:20], t]):
        with pytest.raises(g.MoeError) as ei:
            g.GradientList(pair).clip(1.0)
        assert ei.value.status == 3
    with pytest.raises(g.MoeError):
        g.GradientList([t[:50]], out=[t[1:51]]).clip(1.0)
    assert torch.equal(t, torch.ones_like(t))
    g.GradientList([t[:50], t[50:]]).clip(5.0)          # neighbours are fine
    assert abs(float(t.norm()) - 5.0) < 1e-5


def test_results_do_not_change_and_graphs_replay():
    import torch
    import grouped_gemm_layer_amd as g
    grads = _grads([300000, 77, 4096], ["fp32", "bf16", "fp32"], seed=9)
    out = [torch.empty_like(t) for t in grads]
    lst = g.GradientList(grads, out=out)
    lst.clip(2.0)
    first = [t.clone() for t in out] + [lst.norm.clone(), lst.sumsq.clone()]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lst.clip(2.0)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        lst.clip(2.0)
    for _ in range(3):
        for t in (*out, lst.norm, lst.sumsq):
            t.zero_()
        torch.randn(1 << 20, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, lst.norm, lst.sumsq), first):
            assert torch.equal(a, b)
