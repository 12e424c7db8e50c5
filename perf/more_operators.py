"""What is measured of the operators around experts held in 4 bits.

Five kinds of case:
  combine   the gradient of the weighted sum of a token's expert rows: of the rows and of the routing weights
  permute   the gradient of the rows sorted by expert: of the tokens
  rows      token rows quantised to MXFP4 (E2M1 codes, one power-of-two scale per 32 values of a row) and read back
  weights   expert matrices quantised to MXFP4 (a scale per 32 values of a column) and read back
  ffn       the grouped SwiGLU FFN of MXFP4 experts whose input rows and activations are MXFP4 too
The plain forms are elementary torch operations in 32 bits; the experts' products run as one batched product over the
experts' rows, padded to the longest expert."""
import math

import torch

own = False

GROUP = 32  # values that share a scale


def listed():
    return [
        # the gradients of a decode-sized batch: launch latency
        {"name": "combine small", "kind": "combine", "T": 16, "E": 8, "k": 2, "H": 4096, "f32": False},
        # a training micro-batch of a 128-expert layer
        {"name": "combine large", "kind": "combine", "T": 8192, "E": 128, "k": 8, "H": 2048, "f32": False},
        {"name": "permute small", "kind": "permute", "T": 64, "E": 8, "k": 2, "H": 2048, "f32": False, "add": True},
        # the widest rows, with the residual's gradient added
        {"name": "permute large", "kind": "permute", "T": 4096, "E": 256, "k": 8, "H": 7168, "f32": False, "add": True},
        # a short batch of ragged width
        {"name": "rows small", "kind": "rows", "R": 300, "C": 2016, "f32": False},
        # activations of a training micro-batch
        {"name": "rows large", "kind": "rows", "R": 32768, "C": 4096, "f32": False},
        # fp32 master weights of a small ragged layer
        {"name": "weights small", "kind": "weights", "G": 8, "K": 640, "N": 416, "f32": True},
        # one projection of eight very wide experts
        {"name": "weights large", "kind": "weights", "G": 8, "K": 4096, "N": 14336, "f32": False},
        # a small ragged layer (no size a multiple of a tile)
        {"name": "ffn ragged", "kind": "ffn", "T": 300, "H": 640, "F": 416, "E": 8, "k": 2},
        # 128 narrow experts at a prefill batch
        {"name": "ffn 128 experts", "kind": "ffn", "T": 8192, "H": 2048, "F": 768, "E": 128, "k": 8},
        # what one of eight expert-parallel ranks receives: 32 experts of 7168 x 2048, about 128 rows each
        {"name": "ffn 32 wide experts", "kind": "ffn", "T": 4096, "H": 7168, "F": 2048, "E": 32, "k": 1},
        # eight very wide experts
        {"name": "ffn 8 experts", "kind": "ffn", "T": 4096, "H": 4096, "F": 14336, "E": 8, "k": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["combine", "permute", "rows", "weights", "ffn"])
    if kind in ("combine", "permute"):
        while True:
            E = rng.choice([4, 8, 12, 16, 40, 60, 64, 128, 160, 256])
            c = {"kind": kind, "T": _log(rng, 1, 32768), "E": E, "k": rng.randint(1, min(8, E)), "H": 8 * _log(rng, 4, 1024),
                 "f32": rng.random() < 0.3}
            if kind == "permute":
                c["add"] = rng.random() < 0.5
            if c["T"] * c["k"] * c["H"] <= 4096 * 8 * 7168:
                return c
    if kind == "rows":
        return {"kind": kind, "R": _log(rng, 1, 16384), "C": 32 * _log(rng, 1, 224), "f32": rng.random() < 0.3}
    if kind == "weights":
        while True:
            c = {"kind": kind, "G": rng.choice([1, 2, 8, 16, 60, 128]), "K": 32 * _log(rng, 1, 224), "N": 32 * _log(rng, 1, 448),
                 "f32": rng.random() < 0.3}
            if c["G"] * c["K"] * c["N"] <= 8 * 4096 * 14336 // 2:
                return c
    while True:
        c = {"kind": kind, "T": _log(rng, 1, 8192), "H": 32 * _log(rng, 4, 224), "F": 32 * _log(rng, 3, 448),
             "E": rng.choice([2, 4, 8, 16, 24, 32, 64, 128]), "k": 1}
        c["k"] = rng.randint(1, min(8, c["E"]))
        if c["E"] * c["H"] * c["F"] <= 8 * 4096 * 14336 and c["T"] * c["k"] * c["H"] * c["F"] <= 8192 * 4096 * 14336:
            return c


def work(case):
    kind = case["kind"]
    size = 4 if case.get("f32") else 2
    if kind == "combine":
        T, k, H = case["T"], case["k"], case["H"]
        # dY and the rows read, the rows' gradients written; places, weights and their gradients
        return {"bytes": (T + 2 * T * k) * H * size + 12 * T * k, "flops": 3 * T * k * H}
    if kind == "permute":
        T, k, H = case["T"], case["k"], case["H"]
        return {"bytes": (T * k + T + case["add"] * T) * H * size + 4 * T * k, "flops": T * k * H}
    if kind in ("rows", "weights"):
        n = case["R"] * case["C"] if kind == "rows" else case["G"] * case["K"] * case["N"]
        # read, coded (written, and read again by whoever uses it), and the values written
        return {"bytes": n * (size + 2 * (0.5 + 1 / GROUP) + 2), "flops": 4 * n}
    T, H, F, E, k = (case[n] for n in "THFEk")
    M = T * k
    return {"bytes": 3 * min(E, M) * H * F * (0.5 + 1 / GROUP) + 2 * T * H + 2 * M * H, "flops": 6 * M * H * F}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _routing(T, E, k, g):
    """Picks of a router with somewhat uneven experts, their weights, and the sorting: places of the assignments, their
    inverse and the experts' offsets."""
    lean = 0.5 * torch.randn(E, generator=g, device="cuda")
    top, idx = torch.topk(torch.randn(T, E, generator=g, device="cuda") + lean, k, dim=1)
    flat = idx.reshape(-1)
    row_src = torch.sort(flat, stable=True)[1]
    assign_row = torch.empty_like(row_src)
    assign_row[row_src] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return {"w": torch.softmax(top, 1), "row_src": row_src.to(torch.int32), "assign_row": assign_row.to(torch.int32),
            "offsets": offsets.to(torch.int32), "longest": int(counts.max())}


def _activations(R, C, g):
    """Rows of different sizes with a few large columns."""
    x = torch.randn(R, C, generator=g, device="cuda") * torch.exp(torch.randn(R, 1, generator=g, device="cuda"))
    return x * (1 + 20 * (torch.rand(C, generator=g, device="cuda") < 0.01))


def _experts(G, K, N, g):
    """MXFP4 codes [G, K/2, N] and scales [G, K/32, N] of a layer's weights."""
    q = torch.empty(G, K // 2, N, dtype=torch.uint8, device="cuda")
    s = torch.empty(G, K // GROUP, N, dtype=torch.uint8, device="cuda")
    for e in range(G):
        v, sc = _mx4(0.02 * torch.randn(N, K, generator=g, device="cuda"))
        lo, hi = v[:, 0::2].abs(), v[:, 1::2].abs()
        # the code of a magnitude 0, .5, 1, 1.5, 2, 3, 4, 6, and the sign above it
        code = lambda m: torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)  # noqa: E731
        lo = code(lo) | (v[:, 0::2] < 0).to(torch.uint8) << 3
        hi = code(hi) | (v[:, 1::2] < 0).to(torch.uint8) << 3
        q[e], s[e] = (lo | hi << 4).T, sc.T
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    if kind in ("combine", "permute"):
        T, E, k, H = case["T"], case["E"], case["k"], case["H"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        s = {"kind": kind} | _routing(T, E, k, g)
        rows = lambda n: torch.randn(n, H, generator=g, device="cuda").to(dt)  # noqa: E731
        if kind == "combine":
            return s | {"dy": rows(T), "yp": rows(T * k)}
        return s | {"dxp": rows(T * k), "add": rows(T) if case["add"] else None, "k": k}
    if kind == "rows":
        x = _activations(case["R"], case["C"], g)
        return {"kind": kind, "x": x if case["f32"] else x.to(torch.bfloat16)}
    if kind == "weights":
        w = 0.02 * torch.randn(case["G"], case["K"], case["N"], generator=g, device="cuda")
        return {"kind": kind, "w": w if case["f32"] else w.to(torch.bfloat16)}
    T, H, F, E, k = (case[n] for n in "THFEk")
    s = {"kind": kind, "k": k, "x": torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)} | _routing(T, E, k, g)
    s["W1"], s["S1"] = _experts(E, H, F, g)
    s["W3"], s["S3"] = _experts(E, H, F, g)
    s["W2"], s["S2"] = _experts(E, F, H, g)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _mx4(v):
    """What the codes of fp32 rows stand for before their scales, and the E8M0 scale bytes: the scale is 2 to the
    exponent of the group's largest magnitude less 2, the codes 0, .5, 1, 1.5, 2, 3, 4, 6 (nearest, ties to even)."""
    t = v.reshape(v.shape[0], -1, GROUP)
    m, e = torch.frexp(t.abs().amax(2))
    e = torch.where(m == 0, torch.zeros_like(e), torch.clamp(e - 3, -127, 127))
    t = torch.ldexp(t, -e.unsqueeze(2))
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    return torch.where(t < 0, -a, a).reshape(v.shape), (e + 127).to(torch.uint8)


def _rounded(v):
    """fp32 rows rounded to MXFP4 values."""
    c, s = _mx4(v)
    return torch.ldexp(c.reshape(v.shape[0], -1, GROUP), s.int().unsqueeze(2) - 127).reshape(v.shape)


def _held(q, s):
    """The fp32 matrices [G, K, N] that codes and scales stand for."""
    G, K2, N = q.shape
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(mags + [-m for m in mags], device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], 2).reshape(G, -1, GROUP, N)
    return torch.ldexp(v, s.int().unsqueeze(2) - 127).reshape(G, 2 * K2, N)


def _plain_ffn(s):
    k, off = s["k"], s["offsets"].long()
    M, F = s["row_src"].numel(), s["W1"].shape[2]
    at = off[:-1].unsqueeze(1) + torch.arange(s["longest"], device="cuda")
    rows = torch.where(at < off[1:].unsqueeze(1), at, torch.full_like(at, M))
    r = torch.arange(M, device="cuda")
    e = torch.searchsorted(off, r, right=True) - 1
    place = e * s["longest"] + r - off[e]
    x = _rounded(s["x"].float())[s["row_src"].long() // k]
    x = torch.cat([x, torch.zeros_like(x[:1])])[rows]
    g = torch.bmm(x, _held(s["W1"], s["S1"]))
    u = torch.bmm(x, _held(s["W3"], s["S3"]))
    h = _rounded((g * torch.sigmoid(g) * u).reshape(-1, F)).reshape(g.shape)
    y = torch.bmm(h, _held(s["W2"], s["S2"]))
    return {"y": y.reshape(-1, y.shape[2])[place].bfloat16()}


def _plain(s):
    kind = s["kind"]
    if kind == "combine":
        dy, at = s["dy"].float(), s["assign_row"].long()
        T, k = s["w"].shape
        dy = dy.repeat_interleave(k, 0)
        dyp = torch.empty(T * k, dy.shape[1], device="cuda").index_copy_(0, at, s["w"].reshape(-1, 1) * dy)
        return {"dyp": dyp.to(s["yp"].dtype), "dw": (s["yp"].float()[at] * dy).sum(1).reshape(T, k)}
    if kind == "permute":
        dx = s["dxp"].float()[s["assign_row"].long()].reshape(-1, s["k"], s["dxp"].shape[1]).sum(1)
        return {"dx": (dx if s["add"] is None else dx + s["add"].float()).to(s["dxp"].dtype)}
    if kind == "rows":
        return {"x": _rounded(s["x"].float()).bfloat16()}
    if kind == "weights":
        G, K, N = s["w"].shape
        v = _rounded(s["w"].float().transpose(1, 2).reshape(G * N, K))
        return {"w": v.reshape(G, N, K).transpose(1, 2).contiguous().bfloat16()}
    return _plain_ffn(s)


def _own(s):
    import mixture_experts_layer_count_amd as moe
    kind = s["kind"]
    if kind == "combine":
        dyp, dw = moe.combine_backward(s["dy"], s["yp"], s["assign_row"], s["w"])
        return {"dyp": dyp, "dw": dw}
    if kind == "permute":
        return {"dx": moe.permute_backward(s["dxp"], s["assign_row"], s["k"], dX_add=s["add"])}
    if kind == "rows":
        return {"x": moe.dequantize_mxfp4_rows(*moe.quantize_mxfp4_rows(s["x"]))}
    if kind == "weights":
        return {"w": moe.dequantize_mxfp4_weights(*moe.quantize_mxfp4_weights(s["w"]))}
    return {"y": moe.grouped_ffn(s["x"], s["offsets"], s["W1"], s["W3"], s["W2"], s["S1"], s["S3"], s["S2"],
                                 row_src=s["row_src"], k=s["k"], path="tiled_a4")}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
_MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_rounded(v):
    """Each group of 32 rounded to the nearest of the 15 values times its scale: the count of the borders between
    neighbours that a magnitude passes (or reaches, where the tie goes up) is its place among the eight magnitudes."""
    t = v.double().reshape(v.shape[0], -1, GROUP)
    top = t.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    scale = torch.exp2(torch.where(top > 0, torch.clamp(e - 2, -127, 127), torch.zeros_like(e)))
    a = t.abs() / scale
    place = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):
        border = (_MAGS[i] + _MAGS[i + 1]) / 2
        place += (a >= border) if i % 2 else (a > border)
    return (torch.tensor(_MAGS, dtype=torch.float64, device=v.device)[place] * torch.sign(t) * scale).reshape(v.shape)


def _exact_held(q, s):
    """The matrix [K, N] that one expert's codes and scales stand for."""
    c = torch.stack([q & 15, q >> 4], 1).reshape(-1, q.shape[1]).int()
    f, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(f == 0, m / 2, (1 + m / 2) * torch.exp2(f.double() - 1))
    return torch.where(c >= 8, -v, v) * torch.exp2(s.double() - 127).repeat_interleave(GROUP, 0)


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "combine":
        T, k = s["w"].shape
        at = s["assign_row"].long()
        a = torch.argsort(at)  # the assignment that each row holds
        dy = s["dy"].double()[a // k]
        dw = torch.empty(T * k, dtype=torch.float64, device="cuda")
        dw[a] = (s["yp"].double() * dy).sum(1)
        return {"dyp": s["w"].double().reshape(-1)[a].unsqueeze(1) * dy, "dw": dw.reshape(T, k)}
    if kind == "permute":
        dx = torch.zeros(s["w"].shape[0], s["dxp"].shape[1], dtype=torch.float64, device="cuda")
        dx.index_add_(0, s["row_src"].long() // s["k"], s["dxp"].double())
        return {"dx": dx if s["add"] is None else dx + s["add"].double()}
    if kind == "rows":
        return {"x": _exact_rounded(s["x"])}
    if kind == "weights":
        return {"w": torch.stack([_exact_rounded(w.T.contiguous()).T for w in s["w"]])}
    k, off = s["k"], s["offsets"].tolist()
    x = _exact_rounded(s["x"])
    y = torch.empty(s["row_src"].numel(), x.shape[1], dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            xe = x[s["row_src"][lo:hi].long() // k]
            g, u = (xe @ _exact_held(s[w][e], s[c][e]) for w, c in (("W1", "S1"), ("W3", "S3")))
            y[lo:hi] = _exact_rounded(g / (1 + torch.exp(-g)) * u) @ _exact_held(s["W2"][e], s["S2"][e])
    return {"y": y}
