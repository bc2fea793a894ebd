"""Cases of the AdamW step over a list of tensors, with 32-bit and with 8-bit moments.

Four operators, each with its plain form (whole-array torch operations) and,
where ``own`` is true, the library's calls:

* ``step8``  -- unscale, global norm, clip and AdamW over a list of tensors whose moments are held in 8 bits;
* ``step32`` -- the same step with fp32 moments;
* ``stats``  -- the sum of squares and the zero count of a list's grads (the pass before a cross-rank norm);
* ``export`` / ``import`` -- the 8-bit moments to fp32 checkpoint arrays in list order, and back.

A list's params and grads are views of one flat array each, every tensor
starting on a multiple of 128 elements, as a flat param buffer holds them.
The optimizer state is in the same index space.  8-bit moments: per tensor,
blocks of 128 elements; m as e4m3 codes times a block scale, v as e4m3 codes
of its square root times a block scale; a scale is the block's largest
magnitude / 448.
"""
import math
import random

import torch

own = False

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
TINY = 2.0 ** -100        # a block whose largest magnitude is below this is held as zeros
CAP_M = 2.0 ** 127        # block magnitudes are cut here, so that a decoded value stays finite
CAP_R = 18446742974197923840.0  # the largest fp32 number below 2^64: its square is finite
LEAST = 2.0 ** -9         # the smallest e4m3 magnitude
LR, BETA1, BETA2, EPS, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 1.0
DECAYS = (0.01, 0.0)      # weight decay of matrices and of vectors (two hyper-groups)


# ---- cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # Smallest call: four tensors of a toy model, 2,608 elements.  Latency is all there is.
        {"name": "step8 tiny", "op": "step8", "pd": "bf16", "gd": "bf16", "list": "tiny"},
        # Every parameter of GPT-2 small as its own tensor: 148 tensors, 124 M elements, vectors among matrices.
        {"name": "step8 gpt2-small", "op": "step8", "pd": "bf16", "gd": "bf16", "list": "gpt2-small"},
        # Adapters and heads of all sizes: 500 tensors of odd sizes from 1 to 150 k, fp16 with a loss scale.
        {"name": "step8 ragged f16", "op": "step8", "pd": "f16", "gd": "f16", "list": "random", "n": 500, "lo": 1,
         "hi": 150001, "sizes": 7},
        # One rank's 1/8 shard of Llama-3-8B's matrices, bf16 params with fp32 main grads: 226 tensors, 1.0e9 elements.
        {"name": "step8 llama3-8b rank", "op": "step8", "pd": "bf16", "gd": "f32", "list": "llama3-8b/8"},
        # The same calls with fp32 moments: the smallest, a whole small model held in fp32 throughout ...
        {"name": "step32 tiny", "op": "step32", "pd": "bf16", "gd": "bf16", "list": "tiny"},
        {"name": "step32 gpt2-small f32", "op": "step32", "pd": "f32", "gd": "f32", "list": "gpt2-small"},
        # ... and one rank's 1/64 shard of Llama-3-70B: 723 tensors, 1.1e9 elements.
        {"name": "step32 llama3-70b rank", "op": "step32", "pd": "bf16", "gd": "bf16", "list": "llama3-70b/64"},
        # The norm of a list's grads before a cross-rank sum: many small tensors, and a large shard.
        {"name": "stats ragged f32", "op": "stats", "pd": "f32", "gd": "f32", "list": "random", "n": 1500, "lo": 1,
         "hi": 40001, "sizes": 11},
        {"name": "stats llama3-70b rank", "op": "stats", "pd": "bf16", "gd": "bf16", "list": "llama3-70b/64"},
        # Saving and loading a run with 8-bit moments: a small model, and a rank's shard.
        {"name": "export gpt2-small", "op": "export", "pd": "bf16", "gd": "bf16", "list": "gpt2-small"},
        {"name": "import gpt2-small", "op": "import", "pd": "bf16", "gd": "bf16", "list": "gpt2-small"},
        {"name": "export llama3-8b rank", "op": "export", "pd": "bf16", "gd": "f32", "list": "llama3-8b/8"},
    ]


def draw(rng):
    """A list of 1 to 1500 tensors, each of 0 to 2^26 elements, at most 6e8 in all, of the usual types."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["step8", "step8", "step32", "stats", "export", "import"])
    pd, gd = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
    n = spread(1, 1500)
    hi = spread(1, min(1 << 26, 600_000_000 // n))
    return {"op": op, "pd": pd, "gd": gd, "list": "random", "n": n, "lo": rng.choice([0, 1, hi // 16, hi // 2]),
            "hi": hi, "sizes": rng.randrange(1 << 30)}


def _llama(layers, h, kv, ffn, vocab, parts):
    """A rank's 1/parts of each tensor: embedding, per layer q, k, v, o, gate, up, down and two norms, head, norm."""
    per = [h, h * h, h * kv, h * kv, h * h, h, h * ffn, h * ffn, h * ffn]
    return [x // parts for x in [vocab * h] + per * layers + [h, vocab * h]]


def _sizes(case):
    """The tensors' sizes, and which of them decay (matrices)."""
    kind = case["list"]
    if kind == "tiny":
        return [2048, 32, 512, 16], [0, 1, 0, 1]
    if kind == "gpt2-small":
        h = 768
        layer = [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h]
        sizes = [50257 * h, 1024 * h] + layer * 12 + [h, h]
        return sizes, [0 if x >= h * h else 1 for x in sizes]
    if kind == "llama3-8b/8":
        sizes = [x for x in _llama(32, 4096, 1024, 14336, 128256, 8) if x != 512]  # the norm vectors are fp32: not here
        return sizes, [0] * len(sizes)
    if kind == "llama3-70b/64":
        sizes = _llama(80, 8192, 1024, 28672, 128256, 64)
        return sizes, [0 if x > 128 else 1 for x in sizes]
    rng = random.Random(case["sizes"])
    lo, hi = case["lo"], case["hi"]
    # a third of the tensors spread evenly over the range, the others over its logarithm
    sizes = [rng.randint(lo, hi) if rng.random() < 1 / 3 else
             min(hi, max(lo, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))) for _ in range(case["n"])]
    sizes[0] = max(sizes[0], 1)
    return sizes, [rng.randint(0, 1) for _ in sizes]


def _starts(sizes):
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return starts, at


def _scale(case):
    return 65536.0 if case["gd"] == "f16" else 1.0


# ---- inputs ------------------------------------------------------------------------------------------------------

def _inputs(case, seed):
    """Inputs from the seed alone; identical for both forms and for exact()."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    sizes, groups = _sizes(case)
    starts, total = _starts(sizes)
    n_el = sum(sizes)
    blocks = total // BLOCK
    counts = torch.tensor([-(-n // BLOCK) for n in sizes], device=dev)
    owner = torch.repeat_interleave(torch.arange(len(sizes), device=dev), counts, output_size=blocks)
    begin, size = torch.tensor(starts, device=dev), torch.tensor(sizes, device=dev)
    lane = torch.arange(BLOCK, device=dev)
    # which slots of the index space hold an element, one row per block
    inside = (torch.arange(blocks, device=dev) * BLOCK - begin[owner])[:, None] + lane < size[owner][:, None] \
        if blocks else torch.zeros(0, BLOCK, dtype=torch.bool, device=dev)

    def normal(sigma):
        return torch.randn(blocks, BLOCK, generator=gen, device=dev).mul_(sigma).mul_(inside)

    s = {"case": case, "sizes": sizes, "starts": starts, "total": total, "n_el": n_el, "groups": groups,
         "inside": inside, "scale": _scale(case), "t": 100}
    op = case["op"]
    sigma = 1e-3 if total > 1e6 else 0.05
    if op != "export":
        # grads of one step, times the loss scale, some exactly zero
        g = normal(sigma * s["scale"])
        g.mul_(torch.rand(blocks, 1, generator=gen, device=dev) < 0.98)
        s["grad"] = g.to(TYPES[case["gd"]]).view(-1)
        del g
    if op == "stats":
        return s
    w = normal(0.02)
    s["param"] = w.to(TYPES[case["pd"]]).view(-1)
    if op == "import":
        # fp32 arrays of a checkpoint, in list order without gaps
        at = inside.view(-1).nonzero().view(-1)
        s["at"] = at
        s["x_master"] = w.view(-1)[at]
        s["x_m"] = torch.randn(n_el, generator=gen, device=dev).mul_(sigma / 3)
        s["x_v"] = torch.randn(n_el, generator=gen, device=dev).mul_(sigma).square_()
    if case["pd"] != "f32":
        s["master"] = w.view(-1)
    m = normal(sigma / 3)
    # v over several octaves: a few steps' mean square times a spread per element
    v = normal(sigma).square_().add_(torch.rand(blocks, BLOCK, generator=gen, device=dev).mul_(sigma * sigma).mul_(inside))
    if op == "step32":
        s["exp_avg"], s["exp_avg_sq"] = m.view(-1), v.view(-1)
    else:
        s["exp_avg"], s["exp_avg_scale"] = _encode(m, CAP_M)
        s["exp_avg_sq"], s["exp_avg_sq_scale"] = _encode(v.sqrt_(), CAP_R, True)
    if op == "export":
        s["at"] = inside.view(-1).nonzero().view(-1)
    # weight decay of each block's hyper-group, as the factor 1 - lr * decay
    factor = torch.tensor([1.0 - LR * d for d in DECAYS], dtype=torch.float64, device=dev)
    group = torch.tensor(groups, dtype=torch.int64, device=dev)
    s["keep"] = factor[group[owner]].float()[:, None] if blocks else factor[:0].float()[:, None]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import sharded_mixed_precision_amd as D
        from sharded_mixed_precision_amd.arena import ListArrays

        eight = case["op"] in ("step8", "export", "import")
        specs = [D.TensorSpec(n, case["pd"], case["gd"], h) for n, h in zip(s["sizes"], s["groups"])]
        plan = D.dopt_list_build(specs, "e4m3" if eight else "f32")
        dev = "cuda"
        views = {k: [s[k][a:a + n] for a, n in zip(s["starts"], s["sizes"])] for k in ("param", "grad") if k in s}
        if "param" not in views:  # the statistics read grads only
            views["param"] = [torch.zeros(n, dtype=TYPES[case["pd"]], device=dev) for n in s["sizes"]]
        arrays = ListArrays(plan)
        tensors = D.list_tensors(plan, views["param"], views.get("grad"), arrays.state)
        stream = torch.cuda.current_stream()
        D.dopt_list_init(plan, tensors, D.scaler_cfg(initial_scale=s["scale"]), arrays.workspace, stream)
        for k in ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            if k in s:
                arrays.state[k].copy_(s[k])
                s[k] = arrays.state[k]
        D.dopt_list_scalars_set(plan, arrays.workspace, {"step_count": s["t"], "loss_scale": s["scale"],
                                                        "growth_tracker": 0, "hysteresis_tracker": 1}, stream)
        at = plan.stats_record_offset
        s.update(plan=plan, tensors=tensors, workspace=arrays.workspace, arrays=arrays, views=views,
                 record=arrays.workspace[at:at + 16].view(torch.float64),
                 hparams=D.hparams_array([(LR, BETA1, BETA2, EPS, d) for d in DECAYS]))
        if case["op"] == "export":
            s.update({k: torch.empty(s["n_el"], device=dev) for k in ("x_master", "x_m", "x_v")})
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _encode(x, cap, root=False):
    """Blocks (rows) of fp32 values as e4m3 codes and one fp32 scale each."""
    top = x.abs().amax(1, keepdim=True)
    live = top >= TINY
    scale = torch.where(live, top.clamp(max=cap) * (1.0 / 448.0), 0.0)
    q = torch.where(live, x * torch.reciprocal(scale), 0.0).clamp(-448.0, 448.0)
    if root:  # a second moment that is not zero keeps a code that is not zero
        q = torch.where(x > 0, q.clamp(min=LEAST), q)
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _decode(codes, scale):
    return codes.view(-1, BLOCK).float() * scale[:, None]


def _unscaled(s):
    return s["grad"].view(-1, BLOCK).float() * (1.0 / s["scale"])


def _plain_step(s, eight):
    # the grads are finite here, so the step is never skipped
    s["t"] += 1
    t = s["t"]
    g = _unscaled(s)
    norm = g.double().square().sum().sqrt()
    g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    low = s["case"]["pd"] != "f32"
    p = (s["master"] if low else s["param"]).view(-1, BLOCK) * s["keep"]
    if eight:
        m = _decode(s["exp_avg"], s["exp_avg_scale"])
        r = _decode(s["exp_avg_sq"], s["exp_avg_sq_scale"])
        v = r * r
    else:
        m, v = s["exp_avg"].view(-1, BLOCK), s["exp_avg_sq"].view(-1, BLOCK)
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    r = v.sqrt()
    # a divisor held in a tensor: a division, where a number would be turned into a product with its reciprocal
    root2 = torch.full((), math.sqrt(1.0 - BETA2 ** t), device=r.device)
    p = p - (LR / (1.0 - BETA1 ** t)) * (m / (r / root2 + EPS))
    if low:
        s["master"] = p.view(-1)
    s["param"] = p.to(s["param"].dtype).view(-1)
    if eight:
        s["exp_avg"], s["exp_avg_scale"] = _encode(m, CAP_M)
        s["exp_avg_sq"], s["exp_avg_sq_scale"] = _encode(r, CAP_R, True)
    else:
        s["exp_avg"], s["exp_avg_sq"] = m.view(-1), v.view(-1)


def _plain_stats(s):
    g = _unscaled(s)
    zeros = (g == 0).sum() - (s["total"] - s["n_el"])
    s["record"] = torch.stack([g.double().square().sum(), zeros.double()])


def _plain_export(s):
    r = _decode(s["exp_avg_sq"], s["exp_avg_sq_scale"])
    s["x_master"] = (s["master"] if "master" in s else s["param"])[s["at"]]
    s["x_m"] = _decode(s["exp_avg"], s["exp_avg_scale"]).view(-1)[s["at"]]
    s["x_v"] = (r * r).view(-1)[s["at"]]


def _plain_import(s):
    def spread(x):
        return torch.zeros(s["total"], device=x.device).index_copy_(0, s["at"], x)

    p = spread(s["x_master"])
    if "master" in s:
        s["master"] = p
    s["param"] = p.to(s["param"].dtype)
    s["exp_avg"], s["exp_avg_scale"] = _encode(spread(s["x_m"]).view(-1, BLOCK), CAP_M)
    s["exp_avg_sq"], s["exp_avg_sq_scale"] = _encode(spread(s["x_v"]).view(-1, BLOCK).sqrt(), CAP_R, True)


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import sharded_mixed_precision_amd as D

        stream = torch.cuda.current_stream()
        if op in ("step8", "step32"):
            D.dopt_list_step(s["plan"], s["tensors"], s["hparams"], MAX_NORM, s["workspace"], stream, want_stats=False)
        elif op == "stats":
            D.dopt_list_stats(s["plan"], s["tensors"], s["workspace"], stream)
        elif op == "export":
            D.dopt_list_export(s["plan"], s["tensors"], s["x_master"], s["x_m"], s["x_v"], s["workspace"], stream)
        else:
            D.dopt_list_import(s["plan"], s["tensors"], s["x_master"], s["x_m"], s["x_v"], s["workspace"], stream)
    elif op in ("step8", "step32"):
        _plain_step(s, op == "step8")
    elif op == "stats":
        _plain_stats(s)
    elif op == "export":
        _plain_export(s)
    else:
        _plain_import(s)
    return {k: s[k] for k in _outputs(s["case"])}


def _outputs(case):
    """What a pass writes.  8-bit moments are e4m3 values in units of their block's scale."""
    op = case["op"]
    if op == "stats":
        return ["record"]
    if op == "export":
        return ["x_master", "x_m", "x_v"]
    moments = ["exp_avg", "exp_avg_sq"] + ([] if op == "step32" else ["exp_avg_scale", "exp_avg_sq_scale"])
    return ["param"] + (["master"] if case["pd"] != "f32" else []) + moments


def work(case):
    """Each input read once, each output written once."""
    sizes, _ = _sizes(case)
    n, blocks = sum(sizes), sum(-(-x // BLOCK) for x in sizes)
    pb, gb = BYTES[case["pd"]], BYTES[case["gd"]]
    low = case["pd"] != "f32"
    op = case["op"]
    state8 = 2 * n + 8 * blocks  # both moments' codes and scales, one way
    if op == "stats":
        return {"bytes": gb * n + 16, "flops": 3 * n}
    if op == "export":
        return {"bytes": 4 * n + state8 + 12 * n, "flops": 3 * n}
    if op == "import":
        return {"bytes": 12 * n + (4 + pb if low else 4) * n + state8, "flops": 8 * n}
    weights = 8 + pb if low else 8
    return {"bytes": gb * n + weights * n + (2 * state8 if op == "step8" else 16 * n), "flops": (32 if op == "step8" else 20) * n}


# ---- the definition in 64 bits -------------------------------------------------------------------------------------

def exact(case, seed):
    """The outputs from the formulas in 64 bits.  Codes are the e4m3 numbers nearest to value / scale."""
    x = _inputs(case, seed)
    op = case["op"]
    rows = (-1, BLOCK)

    def wide(key):
        return x[key].to(torch.float64).view(rows)

    def held(key):
        return wide(key) * x[key + "_scale"].to(torch.float64).unsqueeze(1)

    def to_codes(y, second):
        peak = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values) if len(y) else y.new_zeros(0)
        unit = torch.where(peak < TINY, 0.0, peak / 448.0)
        z = (y / torch.where(unit > 0, unit, 1.0).unsqueeze(1)) * (unit > 0).unsqueeze(1)
        # spacing of e4m3 at z: 2^-3 of its power of two, 2^-9 below 2^-6
        _, e = torch.frexp(z)
        step = torch.exp2((e - 1).clamp(min=-6).to(torch.float64) - 3)
        c = torch.round(z / step) * step
        if second:
            c = torch.where((y > 0) & (c == 0), LEAST, c)
        return c.view(-1), unit

    if op == "stats":
        g = wide("grad") / x["scale"]
        z = ((g == 0) & x["inside"]).sum()
        return {"record": torch.stack([(g * g).sum(), z.to(torch.float64)])}
    if op == "export":
        where = x["inside"]
        weights = x["master"] if "master" in x else x["param"]
        return {"x_master": weights.to(torch.float64).view(rows)[where], "x_m": held("exp_avg")[where],
                "x_v": held("exp_avg_sq")[where] ** 2}
    if op == "import":
        def laid(key):
            y = torch.zeros_like(x["inside"], dtype=torch.float64)
            y[x["inside"]] = x[key].to(torch.float64)
            return y

        weights, m, root = laid("x_master"), laid("x_m"), laid("x_v").sqrt()
    else:
        t = x["t"] + 1
        g = wide("grad") / x["scale"]
        g = g * min(1.0, MAX_NORM / (math.sqrt(float((g * g).sum())) + 1e-6))
        m = held("exp_avg") if op == "step8" else wide("exp_avg")
        v = held("exp_avg_sq") ** 2 if op == "step8" else wide("exp_avg_sq")
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g * g - v)
        root = v.sqrt()
        weights = wide("master") if "master" in x else wide("param")
        weights = weights * x["keep"].to(torch.float64) \
            - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    got = {"param": weights.reshape(-1), "master": weights.reshape(-1)}
    if op == "step32":
        got.update(exp_avg=m.reshape(-1), exp_avg_sq=v.reshape(-1))
    else:
        got["exp_avg"], got["exp_avg_scale"] = to_codes(m, False)
        got["exp_avg_sq"], got["exp_avg_sq_scale"] = to_codes(root, True)
    return {k: got[k] for k in _outputs(case)}
