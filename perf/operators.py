"""The operators around the expert layer, as cases to measure: rows sorted by
expert and back, the 4-bit microscaled format and its grouped product, and the
gradient norm with clipping.

`run` computes one pass in plain torch operations, or, where `own` is true,
through the package's entry points.  `exact` is the same result from the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a few sequences generating one token each: the latency of the sort and the row copies
        dict(name="dispatch decode", op="dispatch", tokens=4, hidden=2048, experts=128, here=128, top_k=8, type="bf16",
             weights=False, backward=False),
        # one training batch of the Qwen3-30B-A3B layer, rows out to the experts and the gradient back
        dict(name="dispatch train", op="dispatch", tokens=16384, hidden=2048, experts=128, here=128, top_k=8,
             type="bf16", weights=False, backward=True),
        # expert parallel, a quarter of the experts on this GPU, gates applied in front of them; odd row length
        dict(name="dispatch local fp32", op="dispatch", tokens=1777, hidden=1001, experts=160, here=40, top_k=6,
             type="fp32", weights=True, backward=True),
        # one token for each of 32 sequences back from the experts, at the Qwen3-235B-A22B width
        dict(name="combine decode", op="combine", tokens=32, hidden=4096, experts=128, here=128, top_k=8, type="bf16",
             weights=True, backward=False),
        # the training batch back from the experts, with the gradients of rows and gates
        dict(name="combine train", op="combine", tokens=16384, hidden=2048, experts=128, here=128, top_k=8,
             type="bf16", weights=True, backward=True),
        # activations of 64 tokens between the two expert products: SwiGLU, then 4 bits
        dict(name="quantize swiglu", op="quantize", batch=1, rows=512, cols=768, along=1, type="bf16", swiglu=True),
        # all W13 of the layer once per optimizer step, transposed for the backward product
        dict(name="quantize weights", op="quantize", batch=128, rows=1536, cols=2048, along=0, type="bf16",
             swiglu=False),
        # the first expert product of four tokens: weight reads only
        dict(name="product decode", op="product", tokens=4, top_k=8, experts=128, n=1536, k=2048, a="mxfp4"),
        # a short prompt on 48 experts with odd sizes and 8-bit activations
        dict(name="product prompt", op="product", tokens=833, top_k=6, experts=48, n=1000, k=1120, a="mxfp8"),
        # the training batch or a long prompt: the first expert product of the Qwen3-30B-A3B layer
        dict(name="product batch", op="product", tokens=16384, top_k=8, experts=128, n=1536, k=2048, a="mxfp4"),
        # many small bf16 tensors of odd lengths (norm weights, biases, adapters)
        dict(name="clip many", op="clip", tensors=211, values=3300001, type="bf16", ratio=0.5),
        # the fp32 main gradients of one Qwen3-30B-A3B layer
        dict(name="clip layer", op="clip", tensors=6, values=604000000, type="fp32", ratio=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "quantize", "product", "clip"])
    if op in ("dispatch", "combine"):
        experts = _log(rng, 4, 256)
        k = rng.randint(1, min(8, experts))
        c = dict(op=op, tokens=_log(rng, 1, 16384), hidden=_log(rng, 33, 4100), experts=experts,
                 here=rng.choice([experts, max(1, experts // 4)]), top_k=k, type=rng.choice(["bf16", "bf16", "fp32"]),
                 weights=rng.random() < 0.6, backward=rng.random() < 0.6)
        if rng.random() < 0.5:
            c["hidden"] = max(64, c["hidden"] // 64 * 64)
        while c["tokens"] * c["top_k"] * c["hidden"] * (2 if c["type"] == "bf16" else 4) > (1 << 29):
            c["tokens"] = max(1, c["tokens"] // 2 - 1)
        return c
    if op == "quantize":
        batch = _log(rng, 1, 32)
        rows, cols = _log(rng, 1, 8192), _log(rng, 17, 8192)
        while batch * rows * cols > 1 << 27:
            rows = max(1, rows // 2 - 1)
        if rng.random() < 0.5:
            cols = max(32, cols // 32 * 32)
        swiglu = rng.random() < 0.4
        return dict(op=op, batch=1 if swiglu else batch, rows=rows, cols=cols, along=1 if swiglu else rng.randint(0, 1),
                    type=rng.choice(["bf16", "fp32"]), swiglu=swiglu)
    if op == "product":
        a = rng.choice(["mxfp4", "mxfp8"])
        experts = _log(rng, 1, 128)
        k = rng.randint(1, min(8, experts))
        kk = _log(rng, 64, 4096)
        kk = max(64, kk // 32 * 32) if a == "mxfp8" or rng.random() < 0.5 else kk
        c = dict(op=op, tokens=_log(rng, 1, 16384), top_k=k, experts=experts, n=_log(rng, 40, 4096), k=kk, a=a)
        while c["tokens"] * c["top_k"] * c["n"] * c["k"] > (1 << 37):
            c["tokens"] = max(1, c["tokens"] // 2 - 1)
        while c["experts"] * c["n"] * c["k"] > (1 << 28):
            c["n"] = c["n"] // 2 + 1
        return c
    tensors = _log(rng, 1, 300)
    return dict(op=op, tensors=tensors, values=_log(rng, 1000, 100000000), type=rng.choice(["bf16", "fp32", "mixed"]),
                ratio=rng.choice([0.1, 0.7, 2.0]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _experts_of(c, gen):
    """[tokens, top_k] distinct experts a token, more to some experts than to others; ids from `here` on live elsewhere."""
    bias = 0.7 * torch.randn(c["experts"], generator=gen, device=DEV)
    z = torch.randn(c["tokens"], c["experts"], generator=gen, device=DEV) + bias
    return z.topk(c["top_k"], dim=1).indices.to(torch.int32).contiguous()


def _maps(idx, here):
    """counts, offsets, sorted_to_flat, flat_to_sorted of the stable sort of the slots by expert."""
    flat = idx.reshape(-1).long()
    live = (flat >= 0) & (flat < here)
    key = torch.where(live, flat, here)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=idx.device)
    counts = (key[:, None] == torch.arange(here, device=idx.device)).sum(0) if key.numel() * here < 1 << 28 else \
        torch.zeros(here + 1, dtype=torch.long, device=idx.device).index_add_(0, key, torch.ones_like(key))[:here]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    s2f = torch.where(torch.arange(order.numel(), device=idx.device) < offsets[-1], order, -1)
    f2s = torch.where(live, place, -1)
    return [v.to(torch.int32) for v in (counts, offsets, s2f, f2s)]


def _blocks(v):
    """[.., n] -> [.., ceil(n / 32), 32], zeros behind the end."""
    n = v.shape[-1]
    return torch.nn.functional.pad(v, (0, -n % 32)).unflatten(-1, (-1, 32))


def _scale_exp(v, top_m, top_e):
    """The smallest X with amax <= m 2^e 2^X over the last dimension (m 2^e the format's largest value, 0.5 <= m < 1)."""
    m, e = torch.frexp(v.abs().amax(-1))
    x = (e - top_e + (m > top_m)).clamp(-127, 127)
    return torch.where(m == 0, -127, x)


def _round_e2m1(y):
    """The nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 with the sign of y; ties to the even code."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(y.dtype)
    return torch.copysign((a / step).round() * step, y)


def _quantized(v):
    """([.., blocks, 32] values on the e2m1 grid, [.., blocks] exponents) of the rows of v."""
    b = _blocks(v)
    x = _scale_exp(b, 0.75, 3)
    half = (-x) // 2  # the power of two in two factors: 2^127 and beyond leave the range of one
    y = b * torch.ldexp(torch.ones_like(b[..., 0]), half)[..., None] * torch.ldexp(torch.ones_like(b[..., 0]), -x - half)[..., None]
    return _round_e2m1(y), x


def _mx4_codes(v):
    """MXFP4 codes [.., 16 a block] (low half first) and scale bytes [.., blocks] of the rows of v."""
    y, x = _quantized(v)
    a = y.abs()
    code = (torch.minimum(2 * a, a + 2) - (a > 4).to(a.dtype)).to(torch.uint8)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    return packed.flatten(-2).contiguous(), (x + 127).to(torch.uint8).contiguous()


def _mx8_codes(v):
    """MXFP8 codes and scale bytes of the rows of v (the row length a multiple of 32)."""
    b = _blocks(v)
    x = _scale_exp(b, 0.875, 9)
    q = (b * torch.ldexp(torch.ones_like(b[..., 0]), -x)[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-2).contiguous(), (x + 127).to(torch.uint8).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    s = dict(case=c)
    if c["op"] in ("dispatch", "combine"):
        dt = TYPES[c["type"]]
        T, H, k = c["tokens"], c["hidden"], c["top_k"]
        M = T * k
        s["idx"] = _experts_of(c, gen)
        s["weights"] = rnd(T, k).softmax(1).contiguous() if c["weights"] else None
        i32 = dict(dtype=torch.int32, device=DEV)
        if c["op"] == "dispatch":
            s["x"] = rnd(T, H).to(dt)
            s["xp"] = torch.zeros(M, H, dtype=dt, device=DEV)
            s["maps"] = [torch.empty(c["here"], **i32), torch.empty(c["here"] + 1, **i32), torch.empty(M, **i32),
                         torch.empty(M, **i32)]
            if c["backward"]:
                s["dxp"] = rnd(M, H).to(dt)
                s["dx"] = torch.empty(T, H, dtype=dt, device=DEV)
        else:
            s["maps"] = _maps(s["idx"], c["here"])
            s["rows"] = rnd(M, H).to(dt)
            s["y"] = torch.empty(T, H, dtype=dt, device=DEV)
            if c["backward"]:
                s["dy"] = rnd(T, H).to(dt)
                s["drows"] = torch.zeros(M, H, dtype=dt, device=DEV)
        if c["backward"] and c["weights"]:
            s["dw"] = torch.empty(T, k, device=DEV)
    elif c["op"] == "quantize":
        wide = c["cols"] * (2 if c["swiglu"] else 1)
        v = rnd(c["batch"], c["rows"], wide)
        if not c["swiglu"]:
            v *= 0.02 * torch.exp(0.5 * rnd(c["batch"], c["rows"], 1))
        s["src"] = v.to(TYPES[c["type"]])
    elif c["op"] == "product":
        idx = _experts_of(dict(c, here=c["experts"]), gen)
        counts, s["offsets"], s["s2f"], _ = _maps(idx, c["experts"])
        s["counts"] = counts.tolist()
        x = rnd(c["tokens"], c["k"]).to(torch.bfloat16).float()
        s["a"] = _mx4_codes(x) if c["a"] == "mxfp4" else _mx8_codes(x)
        w = [_mx4_codes(0.02 * rnd(c["n"], c["k"])) for _ in range(c["experts"])]
        s["b"] = [torch.stack(t) for t in zip(*w)]
        s["out"] = torch.empty(c["tokens"] * c["top_k"], c["n"], dtype=torch.bfloat16, device=DEV)
    else:
        n, total = c["tensors"], c["values"]
        rng = np.random.default_rng([n, total])  # the lengths are the program's, the values the seed's
        cut = rng.dirichlet(np.full(n, 0.6)) * max(total - n, 0)
        whole = 128 if total % 128 == 0 else 1  # whole matrices in one flat buffer, or odd lengths
        sizes = ((1 + cut.astype(np.int64) + whole - 1) // whole * whole).tolist()
        kinds = [torch.bfloat16 if c["type"] == "bf16" or (c["type"] == "mixed" and i % 2) else torch.float32 for i in range(n)]
        s["grads"] = [(0.01 * rnd(m)).to(dt) for m, dt in zip(sizes, kinds)]
        s["flat"] = {dt: torch.empty(sum(m for m, d in zip(sizes, kinds) if d == dt), dtype=dt, device=DEV) for dt in set(kinds)}
        at, s["out"] = {dt: 0 for dt in s["flat"]}, []
        for m, dt in zip(sizes, kinds):
            s["out"].append(s["flat"][dt][at[dt]:at[dt] + m])
            at[dt] += m
        s["max_norm"] = float(c["ratio"] * 0.01 * math.sqrt(sum(sizes)))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return {"dispatch": _dispatch, "combine": _combine, "quantize": _quantize, "product": _product,
            "clip": _clip}[state["case"]["op"]](state)


def _dispatch(s):
    c, w = s["case"], s["weights"]
    if own:
        import grouped_gemm_layer_amd as g
        r = g.RoutingBuffers(s["idx"], w, *s["maps"])
        ws = g.alloc_workspace(g.sort_workspace_size(c["tokens"], c["top_k"], c["here"]))
        g.sort_tokens(r, ws)
        g.permute(s["x"], r, s["xp"], weights=w)
        if c["backward"]:
            g.permute_backward(s["dxp"], r, s["dx"], weights=w, x=s["x"] if c["weights"] else None, dweights=s.get("dw"))
        out = dict(counts=r.counts, offsets=r.offsets, s2f=r.sorted_to_flat, f2s=r.flat_to_sorted, xp=s["xp"])
        if c["backward"]:
            out["dx"] = s["dx"]
            if c["weights"]:
                out["dw"] = s["dw"]
        return out
    counts, offsets, s2f, f2s = _maps(s["idx"], c["here"])
    out = dict(counts=counts, offsets=offsets, s2f=s2f, f2s=f2s)
    flat = s2f.clamp(min=0).long()
    rows = s["x"].float()[flat // c["top_k"]]
    if c["weights"]:
        rows = rows * w.reshape(-1)[flat][:, None]
    out["xp"] = torch.where((s2f >= 0)[:, None], rows, 0).to(s["x"].dtype)
    if c["backward"]:
        back = _rows_of_tokens(s["dxp"], f2s, c["top_k"])
        out["dx"] = (back * w[:, :, None] if c["weights"] else back).sum(1).to(s["x"].dtype)
        if c["weights"]:
            out["dw"] = (back * s["x"].float()[:, None, :]).sum(-1)
    return out


def _rows_of_tokens(rows, f2s, k):
    """[tokens, k, H] rows in 32 bits; zeros for slots without a row."""
    got = torch.where((f2s >= 0)[:, None], rows.float()[f2s.clamp(min=0).long()], 0)
    return got.unflatten(0, (-1, k))


def _combine(s):
    c, w = s["case"], s["weights"]
    if own:
        import grouped_gemm_layer_amd as g
        r = g.RoutingBuffers(s["idx"], w, *s["maps"])
        g.unpermute(s["rows"], r, s["y"], weights=w)
        out = dict(y=s["y"])
        if c["backward"]:
            g.unpermute_backward(s["dy"], r, s["drows"], weights=w, rows=s["rows"] if c["weights"] else None,
                                 dweights=s.get("dw"))
            out["drows"] = s["drows"]
            if c["weights"]:
                out["dw"] = s["dw"]
        return out
    _, _, s2f, f2s = s["maps"]
    rows = _rows_of_tokens(s["rows"], f2s, c["top_k"])
    out = dict(y=(rows * w[:, :, None] if c["weights"] else rows).sum(1).to(s["rows"].dtype))
    if c["backward"]:
        flat = s2f.clamp(min=0).long()
        d = s["dy"].float()[flat // c["top_k"]]
        if c["weights"]:
            d = d * w.reshape(-1)[flat][:, None]
            out["dw"] = (rows * s["dy"].float()[:, None, :]).sum(-1)
        out["drows"] = torch.where((s2f >= 0)[:, None], d, 0).to(s["dy"].dtype)
    return out


def _quantize(s):
    c, src = s["case"], s["src"]
    dt = torch.bfloat16 if c["swiglu"] else src.dtype
    if own:
        import grouped_gemm_layer_amd as g
        r, n = (c["rows"], c["cols"]) if c["along"] else (c["cols"], c["rows"])
        blocks = -(-n // 32)
        codes = torch.empty(c["batch"], r, 16 * blocks, dtype=torch.uint8, device=DEV)
        scales = torch.empty(c["batch"], r, blocks, dtype=torch.uint8, device=DEV)
        g.mxfp4_quantize(src, codes, scales, along=c["along"], swiglu=c["swiglu"])
        out = torch.empty(c["batch"], r, n, dtype=dt, device=DEV)
        g.mxfp4_dequantize(codes, scales, out)
        return out
    if c["swiglu"]:  # in 64 bits: values next to a rounding border
        g1, g3 = src.double().chunk(2, -1)
        v = g1 / (1 + torch.exp(-g1)) * g3
    else:
        v = src.float()
        v = v if c["along"] else v.transpose(-1, -2)
    y, x = _quantized(v)
    return torch.ldexp(y, x[..., None]).flatten(-2)[..., :v.shape[-1]].to(dt).contiguous()


def _values(codes, scales, fmt, k, dt=torch.float32):
    """The values that codes and scales stand for, [.., k]."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).to(dt)
    else:
        low, high = codes & 15, codes >> 4
        c = torch.stack([low, high], -1).flatten(-2).long()
        v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dt, device=codes.device)[c]
    v = v.unflatten(-1, (-1, 32)) * torch.exp2(scales.to(dt) - 127)[..., None]
    return v.flatten(-2)[..., :k]


def _product(s):
    c = s["case"]
    if own:
        import grouped_gemm_layer_amd as g
        g.mxfp4_product(*s["a"], *s["b"], s["out"], k=c["k"], a_format=c["a"], offsets=s["offsets"], row_map=s["s2f"],
                        row_div=c["top_k"])
        return s["out"]
    a = _values(*s["a"], c["a"], c["k"])
    rows = (s["s2f"] // c["top_k"]).split(s["counts"])
    return torch.cat([(a[r] @ _values(q, x, "mxfp4", c["k"]).t()).to(torch.bfloat16) for r, q, x in zip(rows, *s["b"])
                      if len(r)])


def _clip(s):
    if own:
        import grouped_gemm_layer_amd as g
        grads = g.GradientList(s["grads"], out=s["out"])
        norm = grads.clip(s["max_norm"])
        return dict(norm=norm, grads=list(s["flat"].values()))
    norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt()
    f = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    new = [(t.float() * f).to(t.dtype) for t in s["grads"]]
    return dict(norm=norm.float(), grads=[torch.cat([t for t in new if t.dtype == dt]) for dt in s["flat"]])


# ---------------------------------------------------------------------------
# Work of one pass: inputs read once, outputs written once
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("dispatch", "combine"):
        es = 2 if c["type"] == "bf16" else 4
        T, H, M = c["tokens"], c["hidden"], c["tokens"] * c["top_k"]
        L = M * c["here"] / c["experts"]  # rows that live here, on average
        maps = 12 * M if c["op"] == "dispatch" else 4 * M
        n, f = (T + L) * H * es + maps + (4 * M if c["weights"] else 0), L * H
        if c["backward"]:
            n += (T + L) * H * es + 4 * M
            f += L * H
            if c["weights"]:  # the gates' gradient reads the other operand too
                n += (T if c["op"] == "dispatch" else L) * H * es + 8 * M
                f += 2 * L * H
        return dict(bytes=n, flops=f * (2 if c["weights"] else 1))
    if c["op"] == "quantize":
        es = 2 if c["type"] == "bf16" else 4
        n = c["batch"] * c["rows"] * c["cols"]
        return dict(bytes=n * es * (2 if c["swiglu"] else 1) + n * (0.5 + 1 / 32) + n * (2 if c["swiglu"] else es),
                    flops=4 * n)
    if c["op"] == "product":
        M, ka = c["tokens"] * c["top_k"], (0.5 if c["a"] == "mxfp4" else 1.0) + 1 / 32
        hit = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["tokens"])  # experts with a row, on average
        return dict(bytes=c["tokens"] * c["k"] * ka + hit * c["n"] * c["k"] * (0.5 + 1 / 32) + M * c["n"] * 2 + 4 * M,
                    flops=2 * M * c["n"] * c["k"])
    es = {"bf16": 2, "fp32": 4, "mixed": 3}[c["type"]]
    return dict(bytes=2 * es * c["values"], flops=3 * c["values"])


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    f64 = torch.float64
    if c["op"] in ("dispatch", "combine"):
        k, H = c["top_k"], c["hidden"]
        idx = s["idx"].cpu().numpy().reshape(-1)
        live = np.flatnonzero(idx < c["here"])
        order = live[np.lexsort((live, idx[live]))]  # flat slots by expert, then by slot
        slot = torch.from_numpy(order).to(DEV)
        tok = slot // k
        n = slot.numel()
        w = s["weights"].to(f64).reshape(-1)[slot] if c["weights"] else torch.ones(n, dtype=f64, device=DEV)

        def out_rows(v):  # rows of tokens, weighted, in expert order
            r = torch.zeros(c["tokens"] * k, H, dtype=f64, device=DEV)
            r[:n] = v.to(f64)[tok] * w[:, None]
            return r

        def to_tokens(rows):
            return torch.zeros(c["tokens"], H, dtype=f64, device=DEV).index_add_(0, tok, rows[:n].to(f64) * w[:, None])

        def dots(rows, v):
            d = torch.zeros(c["tokens"] * k, dtype=f64, device=DEV)
            d[slot] = torch.linalg.vecdot(rows[:n].to(f64), v.to(f64)[tok])
            return d.reshape(-1, k)

        if c["op"] == "dispatch":
            r = dict(counts=None, offsets=None, s2f=None, f2s=None, xp=out_rows(s["x"]))
            if c["backward"]:
                r["dx"] = to_tokens(s["dxp"])
                if c["weights"]:
                    r["dw"] = dots(s["dxp"], s["x"])
            return r
        r = dict(y=to_tokens(s["rows"]))
        if c["backward"]:
            r["drows"] = out_rows(s["dy"])
            if c["weights"]:
                r["dw"] = dots(s["rows"], s["dy"])
        return r
    if c["op"] == "quantize":
        v = s["src"]
        if c["swiglu"]:
            v = v.to(f64)
            v = v[..., :c["cols"]] * torch.sigmoid(v[..., :c["cols"]]) * v[..., c["cols"]:]
        elif not c["along"]:
            v = v.transpose(-1, -2)
        return torch.stack([_nearest(b.to(f64)) for b in v])
    if c["op"] == "product":
        a = _values(*s["a"], c["a"], c["k"], f64)
        out, at = torch.zeros(len(s["s2f"]), c["n"], dtype=f64, device=DEV), 0
        for e, m in enumerate(s["counts"]):
            rows = torch.div(s["s2f"][at:at + m], c["top_k"], rounding_mode="floor").long()
            b = _values(s["b"][0][e], s["b"][1][e], "mxfp4", c["k"], f64)
            out[at:at + m] = torch.mm(a.index_select(0, rows), b.t().contiguous())
            at += m
        return out
    total = math.sqrt(math.fsum(float(torch.dot(p, p)) for t in s["grads"] for p in t.to(f64).split(1 << 24)))
    f = s["max_norm"] / total if total > s["max_norm"] else 1.0
    return dict(norm=torch.tensor(total, dtype=f64),
                grads=[torch.cat([t.to(f64) * f for t in s["grads"] if t.dtype == dt]) for dt in s["flat"]])


def _nearest(v):
    """The values that the 4-bit format holds for a matrix whose rows are cut into blocks of 32: by search in the list of values."""
    r, n = v.shape
    p = torch.zeros(r, -(-n // 32) * 32, dtype=v.dtype, device=v.device)
    p[:, :n] = v
    p = p.reshape(-1, 32)
    amax = p.abs().max(1).values
    x = torch.ceil(torch.log2(torch.clamp(amax / 6, min=2.0 ** -127)))
    x = x - ((x > -127) & (6 * torch.exp2(x - 1) >= amax)).to(v.dtype)  # log2 rounds: look at both neighbours
    x = x + (6 * torch.exp2(x) < amax).to(v.dtype)
    y = p / torch.exp2(x)[:, None]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=v.dtype, device=v.device)
    at = torch.searchsorted(grid, y.abs().contiguous()).clamp(1, 7)  # grid[at - 1] < |y| <= grid[at]
    low, high = y.abs() - grid[at - 1], grid[at] - y.abs()
    take = torch.where((low < high) | ((low == high) & (at % 2 == 1)), at - 1, at)
    return (torch.sign(y) * grid[take] * torch.exp2(x)[:, None]).reshape(r, -1)[:, :n]
