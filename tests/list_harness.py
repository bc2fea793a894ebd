"""The list step in plain numpy: the formulas in 64 bits with the error bounds
of their fp32 evaluation, and the same operations in fp32 (numpy's are IEEE,
one rounding each) for bit equality."""
import math

import numpy as np
import torch

BLOCK = 128
U = 2.0 ** -24  # half a step of fp32
TINY = 2.0 ** -100
CAP = {"m": np.float32(2.0 ** 127), "r": np.float32(2.0 ** 64 - 2.0 ** 40)}
LEAST = 2.0 ** -9
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# half a step of the 16-bit types, relative to the value; below their normal range half the smallest number
HALF = {"bf16": (2.0 ** -9 * 2, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (0.0, 0.0)}
_CODES = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float32).numpy()


def e4m3_value(codes: np.ndarray) -> np.ndarray:
    return _CODES[codes]


def e4m3_round(q: np.ndarray) -> np.ndarray:
    """Nearest e4m3 number, ties to even, of |q| <= 448 in double (exact)."""
    q = q.astype(np.float64)
    _, e = np.frexp(q)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(q / step) * step


def e4m3_code(v: np.ndarray) -> np.ndarray:
    return torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _blocks(x: np.ndarray) -> np.ndarray:
    n = -(-x.size // BLOCK) * BLOCK
    out = np.zeros(n, x.dtype)
    out[:x.size] = x
    return out.reshape(-1, BLOCK)


def encode(x: np.ndarray, kind: str):
    """(codes uint8 of x.size, scales fp32 per block) in the stated fp32 operations."""
    b = _blocks(x.astype(np.float32))
    with np.errstate(all="ignore"):
        a = np.abs(b).max(1)  # a NaN wins
        live = ~(a < np.float32(TINY))
        s = np.where(live, np.where(a > CAP[kind], CAP[kind], a) * np.float32(1.0 / 448.0), np.float32(0)).astype(np.float32)
        inv = (np.float32(1) / s).astype(np.float32)
        q = (b * inv[:, None]).astype(np.float32)
        q = np.where(live[:, None], np.clip(q, np.float32(-448), np.float32(448)), np.float32(0))
        if kind == "r":
            q = np.where((b > 0) & live[:, None], np.maximum(q, np.float32(LEAST)), q)
        v = e4m3_round(np.nan_to_num(q, nan=0.0))
        v = np.where(np.signbit(q) & (v == 0), -0.0, v)
    return e4m3_code(v.reshape(-1))[:x.size], s


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    s = np.repeat(scales, BLOCK)[:codes.size]
    with np.errstate(all="ignore"):
        return (e4m3_value(codes) * s).astype(np.float32)


def step_f32(raw, p, m, v, hp, t, inv, clip):
    """(p, m, v, sqrt v) after one update, every operation rounded to fp32."""
    f = np.float32
    lr, b1, b2, eps, wd = hp
    with np.errstate(all="ignore"):
        g = raw.astype(f) * f(inv)
        if clip is not None:
            g = g * f(clip)
        p = p * f(1.0 - lr * wd)
        m = f(b1) * m + f(1.0 - b1) * g
        v = f(b2) * v + f(1.0 - b2) * (g * g)
        r = np.sqrt(v)
        d = r / f(math.sqrt(1.0 - b2 ** t)) + f(eps)
        p = p - f(lr / (1.0 - b1 ** t)) * (m / d)
    return p, m, v, r


def step_f64(raw, p, m, v, hp, t, inv, clip):
    """The formulas in 64 bits, and how far an fp32 evaluation of each result
    may be off: per operation half a step (U) of its result, per fp32 constant
    half a step of it.  g: inverse scale, clip and their products, 4U of g.
    m: two products of a constant, 2U + 2U + 4U, and the sum, within 7U of
    M = |b1 m| + |(1-b1) g|.  v: 2U of its first term, 2*4U + U + 2U of its second, U for
    the sum: 12U.  sqrt: half of that and U: 7U.  d: sqrt, a constant, a
    division, eps, a sum: 11U of d.  m/d * step: m's own, 11U + U (division)
    + 2U (step and product).  p: 2U of p for the decay, U of the result."""
    x = [a.astype(np.float64) for a in (raw, p, m, v)]
    lr, b1, b2, eps, wd = hp
    g = x[0] * inv * (1.0 if clip is None else clip)
    p1 = x[1] * (1.0 - lr * wd)
    m1 = b1 * x[2] + (1.0 - b1) * g
    v1 = b2 * x[3] + (1.0 - b2) * g * g
    r1 = np.sqrt(v1)
    d = r1 / math.sqrt(1.0 - b2 ** t) + eps
    k = lr / (1.0 - b1 ** t)
    p2 = p1 - k * (m1 / d)
    big = np.abs(b1 * x[2]) + np.abs((1.0 - b1) * g)
    tiny = 2.0 ** -147  # a few steps of the subnormal range, where half a step is not relative
    tm, tv, tr = 8 * U * big + tiny, 13 * U * v1 + tiny, 8 * U * r1 + math.sqrt(2.0 ** -147)
    tp = U * (3 * np.abs(p1) + 1.01 * np.abs(p2)) + k / d * (8 * U * big + 15 * U * np.abs(m1)) \
        + k * np.abs(m1) / d * (math.sqrt(2.0 ** -147) / d) + tiny
    return (p2, m1, v1, r1), (tp, tm, tv, tr)


def near_e4m3(name, codes, scales, exact, tol, root):
    """codes * scales against the 64-bit values they hold: half a step of
    e4m3 (2^-4 of the value, 2^-10 of the scale below 2^-6; a nonzero square
    root may be raised to 2^-9 of it), the fp32 error of the value itself, and
    4U for the scale, its reciprocal and the two products."""
    s = np.repeat(scales.astype(np.float64), BLOCK)[:codes.size]
    got = e4m3_value(codes).astype(np.float64) * s
    bound = np.maximum((2.0 ** -4 + 8 * U) * (np.abs(exact) + tol), (2.0 ** -9 if root else 2.0 ** -10) * s) \
        + tol + 8 * U * np.abs(exact) + TINY
    bad = ~(np.abs(got - exact) <= bound)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4], exact[bad][:4])
    peak = np.abs(_blocks(exact)).max(1)
    ptol = _blocks(np.broadcast_to(tol, exact.shape)).max(1)
    ok = np.abs(scales * 448.0 - peak) <= ptol + 4 * U * peak + TINY
    assert ok.all(), (name, "scale", scales[~ok][:4], peak[~ok][:4])


def within(name, got, exact, tol):
    bad = ~(np.abs(got.astype(np.float64) - exact) <= tol)
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4], exact[bad][:4], np.broadcast_to(tol, exact.shape)[bad][:4])


class ListCase:
    """Tensors of a list at chosen alignments, with guards around each."""

    def __init__(self, sizes, types, state, seed=0, hgroups=None, shift=1, sigma=1e-2, scale=1.0, dynamic=False,
                 zero_frac=0.05, device="cuda"):
        import sharded_mixed_precision_amd as D
        from sharded_mixed_precision_amd.arena import ListArrays
        self.D, self.device, self.scale = D, device, scale
        self.rng = np.random.default_rng(seed)
        n = len(sizes)
        types = [types[i % len(types)] for i in range(n)]
        hg = [hgroups[i % len(hgroups)] if hgroups else 0 for i in range(n)]
        self.specs = [D.TensorSpec(s, pd, gd, h) for s, (pd, gd), h in zip(sizes, types, hg)]
        self.L = D.dopt_list_build(self.specs, state)
        self.A = ListArrays(self.L, device)
        self.hps = [(1e-3, 0.9, 0.999, 1e-8, 0.01), (3e-4, 0.8, 0.99, 1e-6, 0.0), (1e-2, 0.95, 0.9, 1e-4, 0.1)]
        self.params, self.grads, self.store = [], [], []
        for i, s in enumerate(self.specs):
            p, ps = self._place(s.numel, s.param_dtype, shift * i)
            g, gs = self._place(s.numel, s.grad_dtype, shift * (i + 3))
            w = torch.from_numpy(self.rng.standard_normal(s.numel).astype(np.float32) * 0.05)
            p.copy_(w.to(TORCH[s.param_dtype]))
            self.params.append(p)
            self.grads.append(g)
            self.store += [(ps, p, 7.0), (gs, g, 7.0)]
        self.new_grads(sigma, zero_frac)
        self.t = D.list_tensors(self.L, self.params, self.grads, self.A.state)
        self.scaler = D.scaler_cfg(dynamic, scale)
        self.stream = torch.cuda.current_stream() if device == "cuda" else None

    def _place(self, n, dt, shift):
        """A view of n elements, shift % 9 elements past a 512-byte boundary, in a store filled with 7."""
        off = 64 + shift % 9
        store = torch.full((off + n + 64,), 7.0, dtype=TORCH[dt], device=self.device)
        return store[off:off + n], store

    def new_grads(self, sigma=1e-2, zero_frac=0.05):
        for g in self.grads:
            x = self.rng.standard_normal(g.numel()) * sigma * self.scale
            x[self.rng.random(g.numel()) < zero_frac] = 0.0
            g.copy_(torch.from_numpy(x.astype(np.float32)).to(g.dtype))

    def init(self):
        self.D.dopt_list_init(self.L, self.t, self.scaler, self.A.workspace, self.stream)

    def host(self, x):
        x = x.detach().cpu()
        return x.view(torch.uint8).numpy().copy() if x.dtype == torch.float8_e4m3fn else x.float().numpy().copy()

    def part(self, name, i, blocks=False):
        """Tensor i's part of a state array on the host."""
        info = self.L.tensor(i)
        a, n = info["arena_offset"], info["numel"]
        if blocks:
            a, n = a // BLOCK, -(-n // BLOCK)
        return self.host(self.A.state[name][a:a + n])

    def snapshot(self):
        """Per tensor what the next step starts from."""
        out = []
        for i, s in enumerate(self.specs):
            d = {"raw": self.host(self.grads[i]), "param": self.host(self.params[i])}
            d["p"] = self.part("master", i) if s.param_dtype != "f32" else d["param"]
            if self.L.state_kind == "e4m3":
                d["cm"], d["sm"] = self.part("exp_avg", i), self.part("exp_avg_scale", i, True)
                d["cr"], d["sr"] = self.part("exp_avg_sq", i), self.part("exp_avg_sq_scale", i, True)
                d["m"] = decode(d["cm"], d["sm"])
                r = decode(d["cr"], d["sr"])
                d["v"] = (r * r).astype(np.float32)
            else:
                d["m"], d["v"] = self.part("exp_avg", i), self.part("exp_avg_sq", i)
            out.append(d)
        return out

    def gaps(self):
        """Bytes that no call may write: around the tensors, and between the arena's tensors."""
        out = []
        for store, view, _ in self.store:
            a = (view.data_ptr() - store.data_ptr()) // store.element_size()
            out += [self.host(store[:a]), self.host(store[a + view.numel():])]
        infos = self.L.tensors()
        for name in ("master", "exp_avg", "exp_avg_sq"):
            if name in self.A.state:
                arr = self.host(self.A.state[name])
                keep = np.ones(arr.size, bool)
                for i in infos:
                    keep[i["arena_offset"]:i["arena_offset"] + i["numel"]] = False
                out.append(arr[keep])
        return out

    def check_step(self, before, st, exact=True):
        """The state and params after one step that started from `before`
        (stats st), against the 64-bit formulas within their bounds and the
        fp32 operations bit for bit."""
        inv = float(np.float32(1.0 / self.scale))
        sumsq = sum(float(np.sum((b["raw"].astype(np.float64) * inv) ** 2)) for b in before)
        zeros = sum(int(np.sum(b["raw"] == 0)) for b in before)
        # sums of squares in double: n additions, each within 2^-53 of the sum
        assert math.isclose(st["sumsq"], sumsq, rel_tol=1e-9), (st["sumsq"], sumsq)
        assert st["num_zeros"] == zeros
        clip = st["clip_coef"] if st["clip_applied"] else None
        after = self.snapshot()
        for i, (s, b, a) in enumerate(zip(self.specs, before, after)):
            hp, args = self.hps[s.hgroup], (b["raw"], b["p"], b["m"], b["v"])
            (p, m, v, r), (tp, tm, tv, tr) = step_f64(*args, hp, st["step_count"], inv, clip)
            name = f"tensor {i} {s}"
            within(name + " p", a["p"], p, tp)
            rel, low = HALF[s.param_dtype]
            within(name + " param", a["param"], p, tp + np.maximum(rel * (np.abs(p) + tp), low))
            if self.L.state_kind == "e4m3":
                near_e4m3(name + " m", a["cm"], a["sm"], m, tm, False)
                near_e4m3(name + " r", a["cr"], a["sr"], r, tr, True)
            else:
                within(name + " m", a["m"], m, tm)
                within(name + " v", a["v"], v, tv)
            if exact:
                self.same(name, a, *step_f32(*args, hp, st["step_count"], inv, clip))

    def same(self, name, a, p, m, v, r):
        def eq(what, x, y):
            x, y = np.ascontiguousarray(x), np.ascontiguousarray(y)
            bad = x.view(np.uint8 if x.dtype == np.uint8 else np.uint32) != y.view(np.uint8 if y.dtype == np.uint8 else np.uint32)
            if x.dtype != np.uint8:
                bad &= ~(np.isnan(x) & np.isnan(y))
            assert not bad.any(), (name, what, int(bad.sum()), x[bad][:4], y[bad][:4])

        eq("p", a["p"], p)
        if self.L.state_kind == "e4m3":
            for key, x in (("m", m), ("r", r)):
                c, s = encode(x, key)
                eq("scale of " + key, a["s" + key], s)
                ok = ~np.isnan(np.repeat(s, BLOCK)[:c.size])
                eq("codes of " + key, a["c" + key][ok], c[ok])
        else:
            eq("m", a["m"], m)
            eq("v", a["v"], v)
