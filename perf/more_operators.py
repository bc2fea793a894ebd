"""Cases of a linear layer's 8-bit training operators: the cast to block-scaled e4m3, the product, and the RMS norm around it.

Four operators, each with its plain form (whole-array torch operations in 32 bits) and, where ``own`` is true, the library's calls:

* ``cast``  -- a matrix, its transpose, or both, to e4m3 codes with one power-of-two scale per 128 elements of a row
  (activations, output grads) or per 128x128 tile (weights);
* ``gemm``  -- out[m][n] (+)= sum over k of a[m][k] b[n][k], both operands so held, scales per block of 128 in k;
* ``norm``  -- h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w, with y in 8 bits;
* ``norm_grad`` -- the norm's backward pass: the grad of h, and the weight's grad summed over the rows.

The 8-bit format: with A the largest magnitude of a block and e the least integer >= -126 with A <= 448 * 2^e, the block's scale is 2^e (held
as e8m0: e + 127 in a byte) and an element's code is the e4m3 number nearest to x * 2^-e, ties to even.  A matrix of R x C is held as R rows of
codes, each padded with zeros to a multiple of 128, and as one row of scales for each 128 columns: R scales, padded to a multiple of 16, where
the blocks are 128 elements of a row, or one for each 128 rows.  Codes are returned as e4m3 values, in units of their block's scale, and scales as e8m0.
"""
import math

import torch

own = False

B = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ---- cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # One token's activation before a projection of hidden size 4096: latency is all there is.
        {"name": "cast one token", "op": "cast", "rows": 1, "cols": 4096, "type": "bf16", "kind": "row", "want": "codes"},
        # The grad of a projection's output: rows for the input's grad, transposed for the weight's; a batch that is not full.
        {"name": "cast output grad", "op": "cast", "rows": 8191, "cols": 4096, "type": "bf16", "kind": "row", "want": "both"},
        # A feed-forward weight after its step, for the forward pass and, transposed, for the input's grad.
        {"name": "cast ffn weight", "op": "cast", "rows": 14336, "cols": 4096, "type": "bf16", "kind": "tile", "want": "both"},
        # One token through a feed-forward projection: the weight is read once.
        {"name": "gemm one token", "op": "gemm", "m": 1, "n": 14336, "k": 4096, "kind": "tile", "out": "bf16", "add": False},
        # A batch of 1024 tokens through a small model's qkv projection.
        {"name": "gemm small qkv", "op": "gemm", "m": 1024, "n": 2304, "k": 768, "kind": "tile", "out": "f16", "add": False},
        # A small model's logits over a vocabulary of 50257 for an odd number of tokens.
        {"name": "gemm logits ragged", "op": "gemm", "m": 777, "n": 50257, "k": 768, "kind": "tile", "out": "f32", "add": False},
        # A weight's grad over 8192 tokens, added to the fp32 main grads.
        {"name": "gemm weight grad", "op": "gemm", "m": 4096, "n": 4096, "k": 8192, "kind": "row", "out": "f32", "add": True},
        # 8192 tokens through a feed-forward projection.
        {"name": "gemm ffn", "op": "gemm", "m": 8192, "n": 14336, "k": 4096, "kind": "tile", "out": "bf16", "add": False},
        # One token's norm between two layers; the norm vectors are fp32.
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "wtype": "f32", "residual": True},
        # A batch of 8192 tokens of hidden size 8192.
        {"name": "norm batch", "op": "norm", "rows": 8192, "cols": 8192, "type": "bf16", "wtype": "f32", "residual": True},
        # A small model's norm backward over an odd number of fp16 tokens, its output's grad in fp32.
        {"name": "norm_grad ragged", "op": "norm_grad", "rows": 1023, "cols": 768, "type": "f16", "dtype": "f32", "wtype": "f16",
         "residual": False, "add": False},
        # 8192 tokens of hidden size 4096, with the residual's grad, the weight's added to the fp32 main grads.
        {"name": "norm_grad batch", "op": "norm_grad", "rows": 8192, "cols": 4096, "type": "bf16", "dtype": "bf16", "wtype": "f32",
         "residual": True, "add": True},
    ]


def draw(rng):
    """Casts and norms of 1 to 16384 rows and columns (norms: 64 to 16384 columns), products of 1 to 16384 rows and depths and up to 65536
    columns, odd sizes among them, none dearer than the largest listed case of its operator."""
    def spread(lo, hi):
        n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
        # about half of a model's sizes are multiples of 64
        return n if n < 128 or rng.random() < 0.5 else n // 64 * 64

    op = rng.choice(["cast", "gemm", "gemm", "norm", "norm_grad"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "cast":
        cols = spread(1, 16384)
        kind = rng.choice(["row", "tile"])
        return {"op": op, "rows": spread(1, min(16384, 14336 * 4096 // cols)), "cols": cols, "type": t, "kind": kind,
                "want": rng.choice(["codes", "transposed", "both"]), "normed": kind == "row" and rng.random() < 0.4}
    if op == "gemm":
        k, n = spread(1, 16384), spread(16, 65536)
        m = spread(1, max(1, min(16384, 8192 * 14336 * 4096 // (n * k), 14336 * 8192 // n)))
        kind = rng.choice(["tile", "row"])
        return {"op": op, "m": m, "n": n, "k": k, "kind": kind, "out": t, "add": kind == "row" and rng.random() < 0.7}
    cols = spread(64, 16384)
    rows = spread(1, min(16384, 8192 * (8192 if op == "norm" else 4096) // cols))
    case = {"op": op, "rows": rows, "cols": cols, "type": t, "wtype": rng.choice(["f32", t]), "residual": rng.random() < 0.7}
    if op == "norm_grad":
        case.update(dtype=rng.choice([t, "f32"]), add=rng.random() < 0.5)
    return case


# ---- the 8-bit format ----------------------------------------------------------------------------------------------

def _padded(x):
    """`x` with zeros up to whole blocks of columns."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % B))


def _encode(x, kind):
    """fp32 matrix to its codes and scales, laid out as the format says."""
    rows = x.shape[0]
    x = _padded(x)
    groups = x.shape[1] // B
    if kind == "row":
        x = x.view(rows, groups, B)
        top = x.abs().amax(2)
    else:
        x = torch.nn.functional.pad(x, (0, 0, 0, -rows % B)).view(-1, B, groups, B)
        top = x.abs().amax((1, 3))
    # 448 is 1.75 * 2^8: the exponent of the magnitude, one more where its mantissa is over 1.75, minus 8
    code = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    inverse = ((254 - code) << 23).view(torch.float32)
    q = x * (inverse[:, :, None] if kind == "row" else inverse[:, None, :, None])
    q = q.to(torch.float8_e4m3fn).view(-1, groups * B)[:rows]
    scales = code.to(torch.uint8).t()
    if kind == "row":
        scales = torch.nn.functional.pad(scales, (0, -rows % 16), value=1)
    return q.contiguous(), scales.contiguous().view(torch.float8_e8m0fnu)


def _decode(codes, scales, rows, cols, kind):
    """The fp32 matrix that codes and scales stand for."""
    e = (scales.view(torch.uint8).to(torch.int32) << 23).view(torch.float32)
    e = e[:, :rows].t() if kind == "row" else e.t().repeat_interleave(B, 0)[:rows]
    return (codes.float().view(rows, -1, B) * e[:, :, None]).view(rows, -1)[:, :cols]


def _held(pair, rows, cols):
    """Codes and scales as outputs, without what pads them."""
    codes, scales = pair
    return {"codes": codes[:, :cols], "scales": scales[:, :rows]}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _inputs(case, seed):
    """Inputs from the seed alone; identical for both forms and for exact()."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def tokens(rows, cols, sigma):
        # activations and their grads: tokens differ by a factor of a few, and so do channels
        return normal(rows, cols).mul_(sigma).mul_(normal(rows, 1).mul_(0.7).exp_()).mul_(normal(1, cols).mul_(0.7).exp_())

    op, s = case["op"], {"case": case}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _encode(tokens(m, k, 1.0), "row")
        s["b"] = _encode(normal(n, k).mul_(0.02) if case["kind"] == "tile" else tokens(n, k, 1e-3), case["kind"])
        # main grads of the micro-batches before
        s["out"] = normal(m, n).mul_(1e-2).to(TYPES[case["out"]]) if case["add"] else \
            torch.empty(m, n, dtype=TYPES[case["out"]], device=dev)
        return s
    rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]
    if op == "cast":
        s["x"] = (normal(rows, cols).mul_(0.02) if case["kind"] == "tile" else tokens(rows, cols, 1.0)).to(t)
        if case.get("normed"):
            s["row"] = s["x"].float().square().mean(1).add_(EPS).rsqrt_()
            s["col"] = normal(cols).mul_(0.1).add_(1.0)
        return s
    s["weight"] = normal(cols).mul_(0.1).add_(1.0).to(TYPES[case["wtype"]])
    x = tokens(rows, cols, 0.5)
    if op == "norm":
        s["x"] = x.to(t)
        if case["residual"]:
            s["residual"] = tokens(rows, cols, 1.0).to(t)
        return s
    s["h"] = x.to(t)
    s["rstd"] = s["h"].float().square().mean(1).add_(EPS).rsqrt_()
    s["dy"] = tokens(rows, cols, 1e-2).to(TYPES[case["dtype"]])
    if case["residual"]:
        s["dh"] = tokens(rows, cols, 1e-2).to(t)
    s["dweight"] = normal(cols).mul_(1e-2) if case["add"] else torch.empty(cols, device=dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import sharded_mixed_precision_amd as D
        from sharded_mixed_precision_amd.arena import fp8_alloc

        def scratch(n):
            return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

        op = case["op"]
        if op == "gemm":
            m, n, k = case["m"], case["n"], case["k"]
            s["a8"] = D.fp8_matrix(*s["a"], m, k, "row")
            s["b8"] = D.fp8_matrix(*s["b"], n, k, case["kind"])
            s["workspace"] = scratch(D.dopt_fp8_gemm_workspace_bytes(m, n, k))
            return s
        rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]
        if op == "cast":
            s["to"] = {"codes": fp8_alloc(rows, cols, case["kind"]) if case["want"] != "transposed" else None,
                       "transposed": fp8_alloc(cols, rows, case["kind"]) if case["want"] != "codes" else None}
        elif op == "norm":
            s["h"] = torch.empty(rows, cols, dtype=t, device="cuda") if case["residual"] else None
            s["rstd"] = torch.empty(rows, device="cuda")
            s["q"] = fp8_alloc(rows, cols, "row")
        else:
            s["dx"] = torch.empty(rows, cols, dtype=t, device="cuda")
            s["workspace"] = scratch(D.dopt_rmsnorm_grad_workspace_bytes(rows, cols))
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _plain_cast(s, case):
    x = s["x"].float()
    if "row" in s:
        x = x * s["row"][:, None] * s["col"]
    got = {}
    if case["want"] != "transposed":
        got["codes"] = _held(_encode(x, case["kind"]), *x.shape)
    if case["want"] != "codes":
        got["transposed"] = _held(_encode(x.t().contiguous(), case["kind"]), x.shape[1], x.shape[0])
    return got


def _plain_gemm(s, case):
    m, n, k = case["m"], case["n"], case["k"]
    out = _decode(*s["a"], m, k, "row") @ _decode(*s["b"], n, k, case["kind"]).t()
    if case["add"]:
        out = out + s["out"].float()
    s["out"] = out.to(TYPES[case["out"]])
    return {"out": s["out"]}


def _plain_norm(s, case):
    got = {}
    h = s["x"]
    if case["residual"]:
        got["h"] = h = (h.float() + s["residual"].float()).to(h.dtype)
    h = h.float()
    rstd = (h.square().mean(1) + EPS).rsqrt()
    got["rstd"] = rstd
    got["y"] = _held(_encode(h * rstd[:, None] * s["weight"].float(), "row"), *h.shape)
    return got


def _plain_norm_grad(s, case):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
    if case["residual"]:
        dx = dx + s["dh"].float()
    dw = (dy * (h * rstd)).sum(0)
    s["dweight"] = s["dweight"] + dw if case["add"] else dw
    return {"dx": dx.to(s["h"].dtype), "dweight": s["dweight"]}


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"cast": _plain_cast, "gemm": _plain_gemm, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[op](s, case)
    import sharded_mixed_precision_amd as D

    stream = torch.cuda.current_stream()
    if op == "cast":
        to = s["to"]
        D.dopt_fp8_cast(s["x"], to["codes"], to["transposed"], s.get("row"), s.get("col"), stream)
        return {k: _held((q.codes, q.scales), q.rows, q.cols) for k, q in to.items() if q is not None}
    if op == "gemm":
        D.dopt_fp8_gemm(s["a8"], s["b8"], s["out"], case["add"], s["workspace"], stream)
        return {"out": s["out"]}
    if op == "norm":
        D.dopt_rmsnorm(s["x"], s["weight"], EPS, residual=s.get("residual"), h=s["h"], q=s["q"], rstd=s["rstd"], stream=stream)
        got = {"rstd": s["rstd"], "y": _held((s["q"].codes, s["q"].scales), s["q"].rows, s["q"].cols)}
        if s["h"] is not None:
            got["h"] = s["h"]
        return got
    D.dopt_rmsnorm_grad(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], dh=s.get("dh"), accumulate=case["add"],
                        workspace=s["workspace"], stream=stream)
    return {"dx": s["dx"], "dweight": s["dweight"]}


def work(case):
    """Each input read once, each output written once."""
    op = case["op"]

    def held(rows, cols, kind):
        return rows * cols + (rows if kind == "row" else -(-rows // B)) * -(-cols // B)

    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": held(m, k, "row") + held(n, k, case["kind"]) + m * n * BYTES[case["out"]] * (2 if case["add"] else 1),
                "flops": 2 * m * n * k}
    rows, cols, t = case["rows"], case["cols"], BYTES[case["type"]]
    n = rows * cols
    if op == "cast":
        out = (held(rows, cols, case["kind"]) if case["want"] != "transposed" else 0) + \
            (held(cols, rows, case["kind"]) if case["want"] != "codes" else 0)
        return {"bytes": n * t + out + (4 * (rows + cols) if case.get("normed") else 0), "flops": 3 * n}
    w = cols * BYTES[case["wtype"]]
    if op == "norm":
        return {"bytes": n * t * (3 if case["residual"] else 1) + w + 4 * rows + held(rows, cols, "row"), "flops": 8 * n}
    return {"bytes": n * (t * (3 if case["residual"] else 2) + BYTES[case["dtype"]]) + w + 4 * rows + 4 * cols * (2 if case["add"] else 1),
            "flops": 11 * n}


# ---- the definition in 64 bits -------------------------------------------------------------------------------------

def exact(case, seed):
    """The outputs from the formulas in 64 bits."""
    x = _inputs(case, seed)
    op = case["op"]

    def wide(key):
        return x[key].to(torch.float64)

    def to_codes(v, kind):
        high = B if kind == "tile" else 1
        r, c = v.shape
        nr, nc = -(-r // high), -(-c // B)
        blocks = v.new_zeros(nr * high, nc * B)
        blocks[:r, :c] = v
        blocks = blocks.reshape(nr, high, nc, B)
        top = torch.maximum(blocks.amax(dim=(1, 3)), -blocks.amin(dim=(1, 3)))
        # top / 448 = f * 2^p with f in [1/2, 1): the least power of two that is not below it
        f, p = torch.frexp(top / 448.0)
        p = torch.where(f == 0.5, p - 1, p)
        p = torch.where(top > 0, p, -126).clamp(min=-126).to(torch.float64)
        z = blocks / torch.exp2(p)[:, None, :, None]
        # spacing of e4m3 at z: 2^-3 of its power of two, 2^-9 below 2^-6
        step = torch.exp2((torch.frexp(z)[1] - 1).clamp(min=-6).to(torch.float64) - 3)
        z = torch.round(z / step) * step
        return {"codes": z.reshape(nr * high, nc * B)[:r, :c], "scales": torch.exp2(p).transpose(0, 1)}

    def value(pair, rows, cols, kind):
        at = torch.arange(rows, device=pair[1].device) // (B if kind == "tile" else 1)
        unit = pair[1].to(torch.float64)[:, at].transpose(0, 1).repeat_interleave(B, dim=1)
        return (pair[0].to(torch.float64) * unit)[:, :cols]

    if op == "cast":
        v = wide("x")
        if "row" in x:
            v = v * wide("row").unsqueeze(1) * wide("col").unsqueeze(0)
        return {k: to_codes(u, case["kind"]) for k, u in (("codes", v), ("transposed", v.transpose(0, 1)))
                if case["want"] in (k, "both")}
    if op == "gemm":
        a = value(x["a"], case["m"], case["k"], "row")
        b = value(x["b"], case["n"], case["k"], case["kind"])
        out = torch.matmul(a, b.transpose(0, 1))
        return {"out": out + wide("out") if case["add"] else out}
    if op == "norm":
        h = wide("x")
        got = {}
        if case["residual"]:
            got["h"] = h + wide("residual")
            h = got["h"].to(TYPES[case["type"]]).to(torch.float64)  # what is kept is what is normed
        rstd = 1.0 / ((h ** 2).sum(1) / h.shape[1] + EPS).sqrt()
        got.update(rstd=rstd, y=to_codes(h * rstd.unsqueeze(1) * wide("weight"), "row"))
        return got
    h, dy, w, rstd = wide("h"), wide("dy"), wide("weight"), wide("rstd")
    normed = h * rstd.unsqueeze(1)
    along = (dy * w * normed).sum(1, keepdim=True) / h.shape[1]
    dx = (dy * w - normed * along) * rstd.unsqueeze(1)
    if case["residual"]:
        dx = dx + wide("dh")
    dw = (dy * normed).sum(0)
    return {"dx": dx, "dweight": dw + wide("dweight") if case["add"] else dw}
