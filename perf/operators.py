"""Cases that measure the per-position operators around triangle attention.

Three operators of a pair block, each beside the attention kernels it feeds:

* ``norm``: layer normalisation of a pair tensor over its channels, the forward pass and the
  backward pass with the reduction of the weight's and bias's gradients;
* ``act8``: the 8-bit activation checkpoint (codes in blocks of 32 channels that share a power-of-two
  scale), packed and restored on its own, or written by the norm's forward pass and used by its
  backward pass in place of the activation;
* ``relpos``: the learned relative position bias by buckets in the layout the attention reads, and
  the gradient of its table.

``own`` false computes the plain form with elementary torch operations; ``own`` true calls the
package.
"""
import math

import torch

own = False

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NB = {"clip": 65, "log": 32, "far": 40}  # buckets of each family of edges (without the one for other chains)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, rows, C, x="bf16", y="bf16", step=True, ckpt="", affine=True):
    return {"name": name, "op": "norm", "rows": rows, "C": C, "x": x, "y": y, "step": step, "ckpt": ckpt,
            "affine": affine}


def _act8(name, rows, C, x="bf16", kind="int8"):
    return {"name": name, "op": "act8", "rows": rows, "C": C, "x": x, "kind": kind}


def _relpos(name, B, H, Nq, Nk, edges="clip", chains=1, base=False, step=False):
    return {"name": name, "op": "relpos", "B": B, "H": H, "Nq": Nq, "Nk": Nk, "edges": edges, "chains": chains,
            "base": base, "step": step}


def listed():
    return [
        # the smallest pair tensor of the tests (N = 32, 128 channels): the launch counts, not the bytes
        _norm("norm fwd tiny", 32 * 32, 128, step=False),
        # one training step of the norm before the attention at crop 384, BF16 throughout
        _norm("norm step crop384", 384 * 384, 128),
        # crop 768 with the residual stream kept in FP32 and the attention fed in BF16
        _norm("norm step crop768 f32", 768 * 768, 128, x="f32", y="bf16"),
        # an odd row length and an odd number of rows, FP32 throughout: nothing is 16-byte aligned
        _norm("norm step odd", 10007, 387, x="f32", y="f32"),
        # crop 768 with the activation kept in 8 bits between the passes: the forward pass writes it, the
        # backward pass restores the norm's output from it and takes the gradients
        _norm("norm step crop768 int8", 768 * 768, 128, ckpt="int8"),
        # any activation of crop 640 packed for the way to the backward pass and restored there
        _act8("act8 crop640 int8", 640 * 640, 128),
        # the 8-bit floating form on an FP32 activation whose last block of channels is cut short
        _act8("act8 odd e4m3", 20011, 209, x="f32", kind="e4m3"),
        # the bias of a tiny crop
        _relpos("relpos fwd tiny", 1, 4, 32, 32),
        # one query row against a long sequence
        _relpos("relpos fwd one row", 1, 16, 1, 4096, edges="log"),
        # a training step at crop 768 with three chains, the bias added to a projected pair bias
        _relpos("relpos step crop768", 1, 4, 768, 768, chains=3, base=True, step=True),
        # a batch of odd length with far-reaching logarithmic buckets
        _relpos("relpos step odd far", 2, 12, 1031, 1031, edges="far", step=True),
        # the largest bias: a long sequence with many heads
        _relpos("relpos step 2048", 1, 16, 2048, 2048, chains=4, step=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "act8", "relpos", "relpos"])
    if op == "relpos":
        H, edges, chains = _log_int(rng, 1, 24), rng.choice(["clip", "log", "far"]), rng.choice([1, 1, 2, 5])
        if rng.random() < 0.2:
            c = _relpos("", rng.choice([1, 2]), H, _log_int(rng, 1, 16), _log_int(rng, 16, 4096), edges, chains,
                        rng.random() < 0.5)
        else:
            N = _log_int(rng, 17, 1100)
            c = _relpos("", rng.choice([1, 1, 2]), H, N, N, edges, chains, rng.random() < 0.5, rng.random() < 0.7)
    else:
        C = rng.choice([32, 64, 128, 128, 256, 384, 512, 1024, rng.randrange(16, 300), rng.randrange(300, 2000)])
        rows = _log_int(rng, 1, max(2, 40_000_000 // C))
        x = rng.choice(["bf16", "bf16", "f32"])
        if op == "act8":
            c = _act8("", rows, C, x, rng.choice(["int8", "e4m3"]))
        else:
            c = _norm("", rows, C, x, rng.choice(["bf16", "f32"]), rng.random() < 0.8,
                      rng.choice(["", "", "int8", "e4m3"]), rng.random() < 0.8)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _edges(kind):
    """Ascending distances: the bucket of a distance is the number of edges that are not above it."""
    if kind == "clip":  # distances clipped at 32 to either side, one bucket each
        return list(range(-31, 33))
    # per side: exact up to a quarter of the buckets, then growing geometrically to the largest distance
    half, far = (16, 128) if kind == "log" else (20, 200000)
    exact = half // 2
    up = list(range(1, exact + 1))
    up += [math.ceil(exact * (far / exact) ** (k / (half - exact)) - 1e-9) for k in range(1, half - exact)]
    return sorted(-u + 1 for u in up) + up + [far]


def _activation(g, rows, C, dtype):
    """Rows of a residual stream: channels of unequal scale and offset, a few of them far out."""
    scale = 0.5 + torch.rand(C, generator=g, device="cuda")
    scale[:: max(1, C // 3)] *= 6.0
    shift = 0.3 * torch.randn(C, generator=g, device="cuda")
    return torch.randn(rows, C, generator=g, device="cuda").mul_(scale).add_(shift).to(DT[dtype])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "relpos":
        B, H, Nq, Nk = case["B"], case["H"], case["Nq"], case["Nk"]
        n = max(Nq, Nk)
        edges = _edges(case["edges"])
        # residue numbers that start anew in each chain, with gaps where residues are missing
        step = 1 + (torch.rand(B, n, generator=g, device="cuda") < 0.03).int() * 7
        chain = (torch.arange(n, device="cuda") * case["chains"] // n).int().expand(B, n).contiguous()
        pos = torch.cumsum(step, 1).int()
        first = torch.searchsorted(chain, chain)
        pos = pos - torch.gather(pos, 1, first)
        s["pos_k"], s["pos_q"] = pos[:, :Nk].contiguous(), pos[:, n - Nq:].contiguous()
        s["grp_k"] = s["grp_q"] = None
        if case["chains"] > 1:
            s["grp_k"], s["grp_q"] = chain[:, :Nk].contiguous(), chain[:, n - Nq:].contiguous()
        nb = len(edges) + 1 + (case["chains"] > 1)
        s["table"] = torch.randn(nb, H, generator=g, device="cuda")
        pad = (Nk + 7) // 8 * 8  # rows of the bias are padded to a multiple of 8, as the attention wants them
        mk = lambda: torch.randn(B, H, Nq, pad, generator=g, device="cuda").to(torch.bfloat16)[..., :Nk]  # noqa: E731
        s["base"] = mk() if case["base"] else None
        s["dbias"] = mk() if case["step"] else None
        s["edges"] = torch.tensor(edges, device="cuda", dtype=torch.int32)
        return s
    rows, C = case["rows"], case["C"]
    s["x"] = _activation(g, rows, C, case["x"])
    if case["op"] == "norm":
        s["w"] = s["b"] = None
        if case["affine"]:
            s["w"] = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
            s["b"] = 0.1 * torch.randn(C, generator=g, device="cuda")
        if case["step"]:
            s["dy"] = torch.randn(rows, C, generator=g, device="cuda").to(DT[case["y"]])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pack(x, kind):
    """(values by block of 32 channels in units of the block's scale, scale): the scale is the least power
    of two under which the block's largest magnitude stays within the code's range."""
    rows, C = x.shape
    nblk = (C + 31) // 32
    v = torch.zeros(rows, nblk * 32, device=x.device)
    v[:, :C] = x
    v = v.view(rows, nblk, 32)
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    e = e - 7 + (m > 127 / 128).int() if kind == "int8" else e - 9 + (m > 448 / 512).int()
    e = e.clamp_min(-126)
    one = torch.ones((), device=x.device)
    u = v * torch.ldexp(one, -e)
    u = u.round() if kind == "int8" else u.to(torch.float8_e4m3fn).float()
    return u, torch.ldexp(one, e)


def _unpack(packed, C):
    u, scale = packed
    return (u * scale).flatten(1)[:, :C]


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    w, b = s["w"], s["b"]
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
    affine = lambda h: h if w is None else h * w + b  # noqa: E731
    out = {"y": affine(xc * rstd).to(DT[case["y"]])}
    if case["ckpt"]:
        packed = _pack(x, case["ckpt"])
    if case["step"]:
        if case["ckpt"]:
            x = _unpack(packed, case["C"])
        h = (x - mean) * rstd
        if case["ckpt"]:
            out["y again"] = affine(h).to(DT[case["y"]])
        dy = s["dy"].float()
        dh = dy if w is None else dy * w
        c1, c2 = dh.mean(1, keepdim=True), (dh * h).mean(1, keepdim=True)
        out["dx"] = (rstd * (dh - c1 - h * c2)).to(DT[case["x"]])
        if w is not None:
            out["dw"], out["db"] = (dy * h).sum(0), dy.sum(0)
    elif case["ckpt"]:
        out["kept"] = _unpack(packed, case["C"]).to(DT[case["x"]])
    return out


def _plain_relpos(s):
    delta = s["pos_k"][:, None, :].long() - s["pos_q"][:, :, None].long()
    bucket = torch.bucketize(delta, s["edges"].long(), right=True)
    if s["grp_k"] is not None:
        bucket = torch.where(s["grp_k"][:, None, :] == s["grp_q"][:, :, None], bucket, s["edges"].numel() + 1)
    bias = s["table"].t()[:, bucket].transpose(0, 1)
    if s["base"] is not None:
        bias = bias + s["base"].float()
    out = {"bias": bias.to(torch.bfloat16)}
    if s["dbias"] is not None:
        nb = s["table"].shape[0]
        # per query row first, then over the rows: the clipped buckets sum millions of terms
        hot = (bucket[:, :, None, :] == torch.arange(nb, device=bucket.device)[:, None]).float()
        out["dtable"] = (hot @ s["dbias"].float().permute(0, 2, 3, 1)).sum((0, 1))
    return out


def run(s):
    case = s["case"]
    if own:
        return _own(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "act8":
        return {"x": _unpack(_pack(s["x"].float(), case["kind"]), case["C"]).to(DT[case["x"]])}
    return _plain_relpos(s)


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _own(s):
    import triangle_attention_biomolecular_b200 as T
    case = s["case"]
    if case["op"] == "act8":
        return {"x": T.act8_unpack(T.act8_pack(s["x"], case["kind"]))}
    if case["op"] == "relpos":
        out = {"bias": T.relpos_forward(s["table"], s["edges"], s["pos_q"], s["pos_k"], s["grp_q"], s["grp_k"],
                                        base=s["base"])}
        if s["dbias"] is not None:
            out["dtable"] = T.relpos_backward(s["dbias"], s["edges"], s["pos_q"], s["pos_k"], s["grp_q"], s["grp_k"])
        return out
    y, stats, kept = T.norm_forward(s["x"], s["w"], s["b"], EPS, out_dtype=DT[case["y"]],
                                    checkpoint=case["ckpt"] or None)
    out = {"y": y}
    if case["step"]:
        if kept is not None:
            out["y again"] = T.norm_restore(kept, stats, s["w"], s["b"], out_dtype=DT[case["y"]])
        dx, dw, db = T.norm_backward(s["x"] if kept is None else kept, stats, s["dy"], s["w"])
        out["dx"] = dx
        if dw is not None:
            out["dw"], out["db"] = dw, db
    elif kept is not None:
        out["kept"] = T.act8_unpack(kept)
    return out


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "relpos":
        n = case["B"] * case["H"] * case["Nq"] * case["Nk"]
        nb = NB[case["edges"]] + (case["chains"] > 1)
        pos = 4 * case["B"] * (case["Nq"] + case["Nk"]) * (2 if case["chains"] > 1 else 1)
        return {"bytes": 2 * n * (1 + case["base"] + case["step"]) + 4 * nb * case["H"] * (1 + case["step"]) + pos,
                "flops": n * (case["base"] + case["step"])}
    n = case["rows"] * case["C"]
    if case["op"] == "act8":
        return {"bytes": 2 * n * size[case["x"]], "flops": 4 * n}
    sides = size[case["x"]] + size[case["y"]]
    if not case["step"]:
        return {"bytes": n * (sides + (size[case["x"]] if case["ckpt"] else 0)), "flops": (8 + 4 * bool(case["ckpt"])) * n}
    again = size[case["y"]] if case["ckpt"] else 0
    return {"bytes": n * (2 * sides + again) + 16 * case["C"] * case["affine"], "flops": (20 + 8 * bool(case["ckpt"])) * n}


def _e4m3_exact(v):
    """Round to 3 mantissa bits (ties to even), smallest exponent -6, in 64 bits."""
    a = v.abs()
    step = torch.full_like(a, 2.0 ** -9)
    for e in range(-5, 9):
        step = torch.where(a >= 2.0 ** e, torch.full_like(a, 2.0 ** (e - 3)), step)
    return torch.round(v / step) * step


def _kept_exact(x, kind):
    rows, C = x.shape
    top = 127.0 if kind == "int8" else 448.0
    v = torch.nn.functional.pad(x, (0, -C % 32)).view(rows, -1, 32)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((amax / top).clamp_min(2.0 ** -126)))
    e = torch.where(amax > top * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= top * torch.exp2(e - 1), e - 1, e).clamp_min(-126)
    u = v / torch.exp2(e)
    u = torch.round(u) if kind == "int8" else _e4m3_exact(u)
    return (u * torch.exp2(e)).view(rows, -1)[:, :C]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "relpos":
        out = {}
        delta = s["pos_k"].double()[:, None, :] - s["pos_q"].double()[:, :, None]
        bucket = torch.zeros_like(delta, dtype=torch.int64)
        for e in s["edges"].tolist():
            bucket += delta >= e
        if s["grp_k"] is not None:
            bucket[s["grp_k"][:, None, :] != s["grp_q"][:, :, None]] = s["edges"].numel() + 1
        table = s["table"].double()
        bias = torch.stack([table[:, h][bucket] for h in range(case["H"])], 1)
        out["bias"] = bias if s["base"] is None else bias + s["base"].double()
        if s["dbias"] is not None:
            flat = bucket.flatten()
            out["dtable"] = torch.stack([
                torch.stack([g[flat == k].sum() for k in range(table.shape[0])])
                for g in s["dbias"].double().transpose(0, 1).flatten(1)], 1)
        return out
    x = s["x"].double()
    if case["op"] == "act8":
        return {"x": _kept_exact(x, case["kind"])}
    mean = x.sum(1, keepdim=True) / case["C"]
    var = (x - mean).square().sum(1, keepdim=True) / case["C"]
    rstd = 1.0 / (var + EPS).sqrt()
    w = torch.ones(case["C"], device="cuda", dtype=torch.float64) if s["w"] is None else s["w"].double()
    b = torch.zeros_like(w) if s["b"] is None else s["b"].double()
    out = {"y": (x - mean) * rstd * w + b}
    kept = _kept_exact(x, case["ckpt"]) if case["ckpt"] else x
    if case["step"]:
        h = (kept - mean) * rstd
        if case["ckpt"]:
            out["y again"] = h * w + b
        dy = s["dy"].double()
        dh = dy * w
        out["dx"] = (dh - (dh.sum(1, keepdim=True) + h * (dh * h).sum(1, keepdim=True)) / case["C"]) * rstd
        if s["w"] is not None:
            out["dw"], out["db"] = (dy * h).sum(0), dy.sum(0)
    elif case["ckpt"]:
        out["kept"] = kept
    return out
