"""GPU tests of the list step whose 8-bit moments are rounded by chance
('e4m3_sr'): every code against the stated fp32 operations and random words
bit for bit, whole runs against fp32 moments, capture, parts and checkpoints."""
import numpy as np
import pytest
import torch

from tests import gpu_harness as G
from tests import list_dither as S
from tests import list_harness as H

pytestmark = pytest.mark.gpu

PAIRS = [(p, g) for p in ("bf16", "f16", "f32") for g in ("bf16", "f16", "f32")]


@pytest.fixture(autouse=True)
def _announce(request):
    G.log(f"[gpu-test] start {request.node.name}")
    yield
    torch.cuda.synchronize()


class Case(H.ListCase):
    """A ListCase of kind e4m3_sr."""

    def __init__(self, sizes, types, **kw):
        super().__init__(sizes, types, "e4m3_sr", **kw)

    def snapshot(self):
        out = []
        for i, s in enumerate(self.specs):
            d = {"raw": self.host(self.grads[i]), "param": self.host(self.params[i])}
            d["p"] = self.part("master", i) if s.param_dtype != "f32" else d["param"]
            d["cm"], d["sm"] = self.part("exp_avg", i), self.part("exp_avg_scale", i, True)
            d["cr"], d["sr"] = self.part("exp_avg_sq", i), self.part("exp_avg_sq_scale", i, True)
            d["m"], r = H.decode(d["cm"], d["sm"]), H.decode(d["cr"], d["sr"])
            d["v"] = (r * r).astype(np.float32)
            out.append(d)
        return out

    def check(self, before, st, seed):
        """One step from `before`: params, masters, codes and scales bit for bit, and the
        codes within a step of e4m3 of the 64-bit formulas."""
        clip, t, inv = (st["clip_coef"] if st["clip_applied"] else None), st["step_count"], float(np.float32(1.0 / self.scale))
        for i, (s, b, a) in enumerate(zip(self.specs, before, self.snapshot())):
            hp, args, name = self.hps[s.hgroup], (b["raw"], b["p"], b["m"], b["v"]), f"tensor {i} {s}"
            p, m, _, r = H.step_f32(*args, hp, t, inv, clip)
            assert np.array_equal(a["p"], p), name
            want = torch.from_numpy(p).to(H.TORCH[s.param_dtype]).float().numpy()
            assert np.array_equal(a["param"], want), name
            w = S.words(self.L.tensor(i)["arena_offset"], s.numel, t, seed)
            for key, x in (("m", m), ("r", r)):
                c, sc = S.encode(x, key, w)
                assert np.array_equal(a["s" + key], sc), (name, key)
                bad = a["c" + key] != c
                assert not bad.any(), (name, key, int(bad.sum()), a["c" + key][bad][:4], c[bad][:4])
            (p64, m64, _, r64), (tp, tm, _, tr) = H.step_f64(*args, hp, t, inv, clip)
            H.within(name, a["p"], p64, tp)
            for key, x, tol in (("m", m64, tm), ("r", r64, tr)):
                sc = np.repeat(a["s" + key].astype(np.float64), 128)[:s.numel]
                got = H.e4m3_value(a["c" + key]).astype(np.float64) * sc
                # a whole step: 2^-3 of the value's power of two, 2^-9 of the scale below 2^-6; then 4 fp32 roundings
                bound = np.maximum(2.0 ** -3 * (np.abs(x) + tol), 2.0 ** -9 * sc) * (1 + 8 * H.U) + tol + 8 * H.U * np.abs(x) + H.TINY
                H.within(f"{name} {key}", got, x, bound)


def run(c, steps=2, seed=0, max_norm=1.0):
    D = c.D
    c.init()
    if seed:
        D.dopt_list_set_seed(c.L, seed, c.A.workspace, c.stream)
    gaps = c.gaps()
    for k in range(steps):
        if k:
            c.new_grads()
        before = c.snapshot()
        st = D.dopt_list_step(c.L, c.t, c.hps, max_norm, c.A.workspace, c.stream)
        assert st["step_count"] == k + 1 and not st["skipped"]
        c.check(before, st, seed)
    for x, y in zip(gaps, c.gaps()):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(p))
def test_types(pair):
    run(Case([1, 300, 4097], [pair], seed=1))
    run(Case([1, 300, 20_000], [pair], seed=1), seed=(1 << 64) - 3)


@pytest.mark.parametrize("sizes", [[1], [127], [129], [2047], [2049], [0, 5, 0], [8192], [8193], [70_001], [16384, 16385, 3]], ids=str)
def test_sizes(sizes):
    run(Case(sizes, [("bf16", "bf16")], seed=2, hgroups=[1, 0, 2]), steps=3, seed=77)


@pytest.mark.parametrize("shift", [1, 4])
def test_many_tensors_of_mixed_types(shift):
    rng = np.random.default_rng(shift)
    run(Case([int(x) for x in rng.integers(0, 700, 600)], PAIRS, seed=4, hgroups=[0, 2, 1], shift=shift), seed=1 << 40)


def test_late_steps_and_seeds():
    """The number of the step and the seed beyond 32 bits, and a seed changed between two steps."""
    c = Case([3000, 70], [("bf16", "f32")], seed=3)
    c.init()
    D = c.D
    for t, seed in ((7, 5), ((1 << 33) + 9, 5), ((1 << 33) + 9, 5 + (1 << 50))):
        D.dopt_list_scalars_set(c.L, c.A.workspace, {"step_count": t, "loss_scale": 1.0, "growth_tracker": 0,
                                                     "hysteresis_tracker": 1}, c.stream)
        D.dopt_list_set_seed(c.L, seed, c.A.workspace, c.stream)
        before = c.snapshot()
        st = D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream)
        assert st["step_count"] == t + 1
        c.check(before, st, seed)


def test_zero_subnormal_and_huge_grads():
    for scale in (0.0, 1e-40, 1e-25, 1e20):
        c = Case([700, 128], [("f32", "f32")], seed=8)
        c.init()
        for _ in range(2):
            c.new_grads(sigma=scale)
            before = c.snapshot()
            st = c.D.dopt_list_step(c.L, c.t, c.hps, 0.0, c.A.workspace, c.stream)
            assert not st["skipped"]
            for s, b, a in zip(c.specs, before, c.snapshot()):
                p, m, _, r = H.step_f32(b["raw"], b["p"], b["m"], b["v"], c.hps[0], st["step_count"], 1.0, None)
                assert np.array_equal(a["p"], p) and np.isfinite(a["m"]).all() and np.isfinite(a["v"]).all()
                assert ((a["cr"] > 0) | (r < 2.0 ** -100) == (r > 0) | (r < 2.0 ** -100)).all()


def test_steps_in_parts_and_from_two_sizes_of_list_are_the_step():
    cs = [Case([3000, 70, 1], [("bf16", "bf16"), ("f32", "f32")], seed=11) for _ in range(3)]
    for c in cs:
        c.init()
        c.D.dopt_list_set_seed(c.L, 3, c.A.workspace, c.stream)
    (a, b, d), D = cs, cs[0].D
    for _ in range(3):
        D.dopt_list_step(a.L, a.t, a.hps, 1.0, a.A.workspace, a.stream, want_stats=False)  # one launch
        D.dopt_list_prepare(b.L, b.t, b.hps, 1.0, b.A.workspace, b.stream)
        D.dopt_list_apply(b.L, b.t, b.A.workspace, b.stream)
        D.dopt_list_stats(d.L, d.t, d.A.workspace, d.stream)
        D.dopt_list_finalize(d.L, d.hps, 1.0, d.A.workspace, d.stream)
        D.dopt_list_apply(d.L, d.t, d.A.workspace, d.stream)
    for x, y, z in zip(*(c.snapshot() for c in cs)):
        assert all(np.array_equal(x[k], y[k]) and np.array_equal(x[k], z[k]) for k in x)


@pytest.mark.parametrize("sizes", [[40_000, 70, 300], [900, 70]], ids=str)
def test_captured_step(sizes):
    """Replays of a captured step take the random words of their own step."""
    a, b, other = (Case(sizes, [("bf16", "bf16"), ("f32", "f32")], seed=12) for _ in range(3))
    D, s = a.D, torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for c in (a, b, other):
            c.stream = s
            c.init()
            D.dopt_list_set_seed(c.L, 9, c.A.workspace, s)
            D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            D.dopt_list_step(a.L, a.t, a.hps, 1.0, a.A.workspace, torch.cuda.current_stream(), want_stats=False)
    for k in range(4):
        with torch.cuda.stream(s):
            b.new_grads()
            for x, y in zip(a.grads, b.grads):
                x.copy_(y)
            graph.replay()
            D.dopt_list_step(other.L, other.t, other.hps, 1.0, other.A.workspace, s)
            before = b.snapshot()
            st = D.dopt_list_step(b.L, b.t, b.hps, 1.0, b.A.workspace, s)
        torch.cuda.synchronize()
        b.check(before, st, 9)
        assert D.dopt_list_read_stats(a.L, a.A.workspace, s) == st
        for x, y in zip(a.snapshot(), b.snapshot()):
            assert all(np.array_equal(x[i], y[i]) for i in x), k


def test_checkpoint():
    """Import rounds to nearest; export gives what is held; init resets the seed."""
    c = Case([5, 2049, 0, 128, 30_001], [("bf16", "f32"), ("f32", "f32"), ("f16", "f16")], seed=9)
    run(c, 2, seed=21)
    D, n = c.D, c.L.numel
    out = [torch.empty(n, device="cuda") for _ in range(3)]
    D.dopt_list_export(c.L, c.t, *out, c.A.workspace, c.stream)
    snap = c.snapshot()
    for key, o in zip(("p", "m", "v"), out):
        assert np.array_equal(o.cpu().numpy(), np.concatenate([b[key] for b in snap]))
    x = [torch.randn(n, device="cuda"), torch.randn(n, device="cuda"), torch.randn(n, device="cuda").square()]
    D.dopt_list_import(c.L, c.t, *x, c.A.workspace, c.stream)
    for info, a in zip(c.L.tensors(), c.snapshot()):
        sl = slice(info["export_offset"], info["export_offset"] + info["numel"])
        for key, y in (("m", x[1]), ("r", x[2].sqrt())):
            codes, sc = H.encode(y[sl].cpu().numpy(), key)
            assert np.array_equal(a["c" + key], codes) and np.array_equal(a["s" + key], sc)
    c.init()
    before = c.snapshot()
    c.check(before, D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream), 0)


@pytest.mark.parametrize("n", [8000, 40_000])  # one launch a step, and two
def test_second_moments_follow_their_grads_over_a_run(n):
    """Half of the elements' grads grow by 3 and the others' fall to a tenth
    after 1000 of 9000 steps: sqrt(v) against that of a list with fp32 moments
    that takes the same grads.  Bounds as derived in test_list_dither_cpu.py."""
    c, d = Case([n], [("f32", "f32")], seed=1), H.ListCase([n], [("f32", "f32")], "f32", seed=1)
    D = c.D
    for x in (c, d):
        x.init()
        x.hps = [(1e-4, 0.9, 0.999, 1e-8, 0.0)]
    even = torch.arange(n, device="cuda") % 2 == 0
    gen = torch.Generator("cuda").manual_seed(5)
    late = torch.where(even, 3e-2, 1e-3)
    for t in range(1, 9001):
        g = torch.randn(n, device="cuda", generator=gen) * (late if t > 1000 else 1e-2)
        for x in (c, d):
            x.grads[0].copy_(g)
            D.dopt_list_step(x.L, x.t, x.hps, 0.0, x.A.workspace, x.stream, want_stats=False)
        if t % 1500 == 0:
            torch.cuda.synchronize()
            G.log(f"[gpu-test] step {t}")
    ratio = np.sqrt(c.snapshot()[0]["v"]) / np.sqrt(d.snapshot()[0]["v"])
    for part in (ratio[::2], ratio[1::2]):
        beyond = ((part > 2) | (part < 0.5)).mean()
        assert abs(part.mean() - 1) < 0.12 and beyond < 0.03, (part.mean(), beyond)
    assert np.isfinite(c.params[0].cpu().numpy()).all()
