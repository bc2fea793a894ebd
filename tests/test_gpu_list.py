"""GPU tests of the tensor-list step: every element of params and state against
the 64-bit formulas within the bounds of their fp32 evaluation, and against
the same fp32 operations in numpy bit for bit."""
import math

import numpy as np
import pytest
import torch

import synth
from synth.models import ParamSpec
from tests import gpu_harness as G
from tests import list_harness as H

pytestmark = pytest.mark.gpu

PAIRS = [(p, g) for p in ("bf16", "f16", "f32") for g in ("bf16", "f16", "f32")]
STATES = ("f32", "e4m3")


@pytest.fixture(autouse=True)
def _announce(request):
    G.log(f"[gpu-test] start {request.node.name}")
    yield
    torch.cuda.synchronize()


def run(c, steps=2, max_norm=1.0, exact=True):
    D = c.D
    c.init()
    gaps = c.gaps()
    for k in range(steps):
        if k:
            c.new_grads()
        before = c.snapshot()
        st = D.dopt_list_step(c.L, c.t, c.hps, max_norm, c.A.workspace, c.stream)
        assert st["step_count"] == k + 1 and not st["skipped"]
        c.check_step(before, st, exact)
    for x, y in zip(gaps, c.gaps()):
        assert np.array_equal(x, y)
    return st


def test_e4m3_hardware_conversion_is_the_plain_one():
    """Every code decoded, and values at, beside and between all of them
    encoded, through import and export."""
    import sharded_mixed_precision_amd as D
    codes = [x for x in range(256) if x & 0x7f != 0x7f]
    vals = H._CODES[codes].astype(np.float64)
    pos = np.sort(np.unique(np.abs(vals)))
    mids = (pos[1:] + pos[:-1]) / 2
    some = np.concatenate([vals, mids, -mids, np.nextafter(mids.astype(np.float32), np.float32(1e9)),
                           np.nextafter(mids.astype(np.float32), np.float32(0))]).astype(np.float32)
    rows = -(-some.size // 127)
    x = np.zeros((rows, 128), np.float32)
    x[:, 0] = 448.0
    x.reshape(-1)[np.flatnonzero(np.arange(rows * 128) % 128)[:some.size]] = some
    n = x.size
    c = H.ListCase([n], [("f32", "f32")], "e4m3")
    c.init()
    dev = [torch.from_numpy(a.reshape(-1).copy()).cuda() for a in (x, x, np.abs(x) ** 2)]
    D.dopt_list_import(c.L, c.t, *dev, c.A.workspace, c.stream)
    got = c.snapshot()[0]
    root = np.sqrt((np.abs(x) ** 2).reshape(-1))
    for key, want in (("m", x.reshape(-1)), ("r", root)):
        wc, ws = H.encode(want, key)
        assert np.array_equal(got["s" + key], ws) and np.array_equal(got["c" + key], wc), key
    out = [torch.empty(n, device="cuda") for _ in range(3)]
    D.dopt_list_export(c.L, c.t, *out, c.A.workspace, c.stream)
    r = H.decode(got["cr"], got["sr"])
    for o, want in zip(out, (x.reshape(-1), H.decode(got["cm"], got["sm"]), r * r)):
        assert np.array_equal(o.cpu().numpy(), want)


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(p))
def test_types(pair, state):
    run(H.ListCase([1, 300, 4097], [pair], state, seed=1))


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("sizes", [[1], [2], [7], [8], [127], [128], [129], [2047], [2048], [2049], [0, 5, 0],
                                   [70001], [16384, 16385, 3]], ids=str)
def test_sizes(sizes, state):
    run(H.ListCase(sizes, [("bf16", "bf16")], state, seed=2))


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("shift", range(9))
def test_alignments(shift, state):
    """Params and grads at every offset of 0 to 8 elements from an aligned address."""
    run(H.ListCase([5000, 2048, 333], [("f16", "bf16"), ("bf16", "f32"), ("f32", "f32")], state, seed=3, shift=shift))


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("n", [239, 240, 241, 480, 481, 1000])
def test_many_tensors(n, state):
    """More tensors than one launch takes, of mixed types and hyper-groups."""
    rng = np.random.default_rng(n)
    sizes = [int(x) for x in rng.integers(0, 700, n)]
    run(H.ListCase(sizes, [("bf16", "bf16")] if n % 2 else PAIRS, state, seed=4, hgroups=[0, 2, 1]))


@pytest.mark.parametrize("state", STATES)
def test_larger_than_one_grid(state):
    """More tiles than workgroups in both passes (grid-stride)."""
    run(H.ListCase([34_000_001, 3, 2_000_000], [("bf16", "bf16")], state, seed=5), steps=1)


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("sizes", [[2048] * 4, [2048] * 5, [8192], [8193], [2048 * 256], [2048 * 256 + 1],
                                   [3, 2048 * 128, 7, 2048 * 124]], ids=str)
def test_launch_rules(sizes, state):
    """On either side of a whole step in one launch (4 tiles), and of pass 1
    finished by its last workgroup (64 partials of 4 tiles)."""
    run(H.ListCase(sizes, [("bf16", "bf16")], state, seed=15, hgroups=[1, 0, 2]))


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("pairs", [PAIRS[i:i + 4] for i in (0, 3, 5)], ids=lambda p: " ".join("-".join(x) for x in p))
def test_one_launch_of_mixed_types(pairs, state):
    run(H.ListCase([1000, 17, 2048, 5], pairs, state, seed=16, hgroups=[2, 0, 1], shift=3), steps=3)


@pytest.mark.parametrize("state", STATES)
def test_no_tensors(state):
    c = H.ListCase([], [("bf16", "bf16")], state)
    c.init()
    st = c.D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream)
    assert st["sumsq"] == 0 and st["num_zeros"] == 0 and st["step_count"] == 1 and not st["skipped"]
    z = H.ListCase([0, 0], [("bf16", "bf16")], state)
    z.init()
    assert z.D.dopt_list_step(z.L, z.t, z.hps, 1.0, z.A.workspace, z.stream)["step_count"] == 1


@pytest.mark.parametrize("state", STATES)
def test_clip_and_no_clip(state):
    st = run(H.ListCase([3000, 55], [("bf16", "bf16")], state, seed=6, sigma=1.0), max_norm=1e-2)
    assert st["clip_applied"] == 1
    st = run(H.ListCase([3000, 55], [("bf16", "bf16")], state, seed=6, sigma=1.0), max_norm=0.0)
    assert st["clip_applied"] == 0 and st["clip_coef"] == 1.0


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_overflow_skips(state, bad):
    c = H.ListCase([2048, 1, 777], [("f16", "f16")], state, seed=7, scale=1024.0, dynamic=True)
    c.init()
    D = c.D
    st = D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream)
    before = c.snapshot()
    keep = c.grads[1].clone()
    c.grads[1][0] = bad
    st = D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream)
    assert st["skipped"] and st["found_inf"] and st["step_count"] == 1 and st["loss_scale_next"] == 512.0
    for b, a in zip(before, c.snapshot()):
        assert all(np.array_equal(b[k], a[k]) for k in b if k != "raw")
    c.grads[1].copy_(keep)
    assert D.dopt_list_read_stats(c.L, c.A.workspace, c.stream)["skipped"] == 1
    c.scale = 512.0
    before = c.snapshot()
    st = D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream)
    assert st["step_count"] == 2 and st["loss_scale_used"] == 512.0
    c.check_step(before, st)


@pytest.mark.parametrize("kind", ["zeros", "tiny", "huge", "one-spike", "subnormal"])
@pytest.mark.parametrize("state", STATES)
def test_extreme_grads(kind, state):
    """Zero blocks, magnitudes whose squares underflow or overflow fp32, and a
    spike that leaves the rest of its block near the smallest code."""
    c = H.ListCase([700, 128], [("f32", "f32")], state, seed=8)
    c.init()
    for k in range(3):
        for g in c.grads:
            x = torch.randn(g.numel(), generator=torch.Generator().manual_seed(k)).cuda()
            g.copy_({"zeros": x * 0, "tiny": x * 1e-25, "huge": x * 1e20, "subnormal": x * 1e-40,
                     "one-spike": torch.where(torch.arange(g.numel(), device="cuda") % 128 == 5,
                                              x * (1e9 if k == 0 else 0.0), x)}[kind])
        before = c.snapshot()
        # no clip: squares reach beyond the fp32 range on purpose
        st = c.D.dopt_list_step(c.L, c.t, c.hps, 0.0, c.A.workspace, c.stream)
        assert not st["skipped"]
        clip, after = None, c.snapshot()
        for s, b, a in zip(c.specs, before, after):
            c.same(kind, a, *H.step_f32(b["raw"], b["p"], b["m"], b["v"], c.hps[s.hgroup], st["step_count"], 1.0, clip))
            assert np.isfinite(a["param"]).all() and np.isfinite(a["m"]).all()
            if state == "e4m3":  # finite second moments too: they are cut, not overflowed
                assert np.isfinite(a["v"]).all()
                _, m, v, r = H.step_f32(b["raw"], b["p"], b["m"], b["v"], c.hps[0], st["step_count"], 1.0, clip)
                assert ((a["v"] > 0) | (a["cr"] > 0) == (r > 0)).all()  # none that was seen is dropped


@pytest.mark.parametrize("state", STATES)
def test_export_import_between_kinds(state):
    """Export of one kind, import into the other, export again: fp32 arrays
    unchanged by the fp32 kind, and the stated encoding by the 8-bit one."""
    sizes, types = [5, 2049, 0, 128, 30_001], [("bf16", "f32"), ("f32", "f32"), ("f16", "f16")]
    c = H.ListCase(sizes, types, state, seed=9)
    run(c, 2)
    D, n = c.D, c.L.numel
    out = [torch.full((n + 3,), 5.0, device="cuda")[1:n + 1] for _ in range(3)]
    D.dopt_list_export(c.L, c.t, *out, c.A.workspace, c.stream)
    snap = c.snapshot()
    for key, o in zip(("p", "m", "v"), out):
        assert np.array_equal(o.cpu().numpy(), np.concatenate([b[key] for b in snap]))
        assert o._base[0] == 5.0 and (o._base[n + 1:] == 5.0).all()
    for other in STATES:
        d = H.ListCase(sizes, types, other, seed=10)
        d.init()
        gaps = d.gaps()
        D.dopt_list_import(d.L, d.t, *out, d.A.workspace, d.stream)
        D.dopt_list_scalars_set(d.L, d.A.workspace, D.dopt_list_scalars_get(c.L, c.A.workspace, c.stream), d.stream)
        for i, (b, a) in enumerate(zip(snap, d.snapshot())):
            assert np.array_equal(a["p"], b["p"])
            assert torch.equal(d.params[i], torch.from_numpy(b["p"]).cuda().to(d.params[i].dtype))
            d.same("imported", a, b["p"], b["m"], b["v"], np.sqrt(b["v"]))
        for x, y in zip(gaps, d.gaps()):
            assert np.array_equal(x, y)
        before = d.snapshot()
        st = D.dopt_list_step(d.L, d.t, d.hps, 1.0, d.A.workspace, d.stream)
        assert st["step_count"] == 3
        d.check_step(before, st)


def test_import_of_nan_and_infinity():
    """A NaN makes its own block NaN and no other; infinite moments are cut."""
    c = H.ListCase([128 * 5], [("f32", "f32")], "e4m3")
    c.init()
    x = torch.ones(3, 640, device="cuda")
    x[1, 3], x[1, 130], x[1, 260] = math.nan, math.inf, -math.inf
    x[2, 400], x[2, 520] = math.nan, math.inf
    x[2, 600] = -1.0  # no square root
    c.D.dopt_list_import(c.L, c.t, *x, c.A.workspace, c.stream)
    out = [torch.empty(640, device="cuda") for _ in range(3)]
    c.D.dopt_list_export(c.L, c.t, *out, c.A.workspace, c.stream)
    m, v = out[1].cpu().numpy(), out[2].cpu().numpy()
    assert np.isnan(m[:128]).all() and np.isfinite(m[128:]).all() and m[130] > 1e38 and m[260] < -1e38
    assert np.isnan(v[384:]).all() and (v[:384] == v[0]).all() and math.isclose(v[0], 1.0, rel_tol=1e-6)


@pytest.mark.parametrize("state", STATES)
def test_step_in_parts_is_the_step(state):
    cs = [H.ListCase([3000, 70, 1], [("bf16", "bf16"), ("f32", "f32")], state, seed=11) for _ in range(3)]
    for c in cs:
        c.init()
    D = cs[0].D
    a, b, d = cs
    for _ in range(2):
        D.dopt_list_step(a.L, a.t, a.hps, 1.0, a.A.workspace, a.stream, want_stats=False)
        D.dopt_list_prepare(b.L, b.t, b.hps, 1.0, b.A.workspace, b.stream)
        D.dopt_list_apply(b.L, b.t, b.A.workspace, b.stream)
        D.dopt_list_stats(d.L, d.t, d.A.workspace, d.stream)
        D.dopt_list_finalize(d.L, d.hps, 1.0, d.A.workspace, d.stream)
        D.dopt_list_apply(d.L, d.t, d.A.workspace, d.stream)
    stats = [D.dopt_list_read_stats(c.L, c.A.workspace, c.stream) for c in cs]
    assert stats[0] == stats[1] == stats[2]
    for x, y, z in zip(*(c.snapshot() for c in cs)):
        assert all(np.array_equal(x[k], y[k]) and np.array_equal(x[k], z[k]) for k in x)


@pytest.mark.parametrize("sizes", [[40_000, 70, 1, 300], [900, 70, 1], [600_000, 70]], ids=str)
@pytest.mark.parametrize("state", STATES)
def test_captured_step(state, sizes):
    """A captured step replayed, with eager work of two lists between the replays, against eager steps."""
    a, b, other = (H.ListCase(sizes, [("bf16", "bf16"), ("f32", "f32")], state, seed=12) for _ in range(3))
    D = a.D
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for c in (a, b, other):
            c.stream = s
            c.init()
        D.dopt_list_step(a.L, a.t, a.hps, 1.0, a.A.workspace, s)
        D.dopt_list_step(b.L, b.t, b.hps, 1.0, b.A.workspace, s)
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
            D.dopt_list_step(b.L, b.t, b.hps, 1.0, b.A.workspace, s)
        torch.cuda.synchronize()
        assert D.dopt_list_read_stats(a.L, a.A.workspace, s) == D.dopt_list_read_stats(b.L, b.A.workspace, s)
        for x, y in zip(a.snapshot(), b.snapshot()):
            assert all(np.array_equal(x[i], y[i]) for i in x), k


def test_two_lists_on_two_streams():
    """Two lists with workspaces of their own, stepped at once on two streams."""
    pairs = [[H.ListCase([200_000, 70], [("bf16", "bf16")], s, seed=13) for s in STATES] for _ in range(2)]
    for p in pairs:
        for c in p:
            c.init()
    D = pairs[0][0].D
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in STATES]
    for _ in range(5):
        for c, s in zip(pairs[0], streams):
            D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, s, want_stats=False)
    torch.cuda.synchronize()
    for _ in range(5):
        for c in pairs[1]:
            D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream, want_stats=False)
    torch.cuda.synchronize()
    for c, d in zip(*pairs):
        for x, y in zip(c.snapshot(), d.snapshot()):
            assert all(np.array_equal(x[i], y[i]) for i in x)


@pytest.mark.parametrize("state", STATES)
def test_a_modules_params(state):
    """The params of a module as the allocator placed them, with the grads of
    its backward pass, stepped through the default stream; init again begins
    anew."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import ListArrays
    torch.manual_seed(0)
    net = torch.nn.Sequential(torch.nn.Linear(96, 130), torch.nn.GELU(), torch.nn.Linear(130, 33)).cuda()
    params = list(net.parameters())
    net(torch.randn(8, 96, device="cuda")).square().sum().backward()
    L = D.dopt_list_build([D.TensorSpec(p.numel(), "f32", "f32") for p in params], state)
    A, hp = ListArrays(L), (1e-2, 0.9, 0.999, 1e-8, 0.01)
    t = D.list_tensors(L, params, [p.grad for p in params], A.state)
    begin = [p.detach().clone() for p in params]
    for _ in range(2):
        for p, b in zip(params, begin):
            p.data.copy_(b)
        D.dopt_list_init(L, t, D.scaler_cfg(), A.workspace)
        st = D.dopt_list_step(L, t, [hp], 1.0, A.workspace)
        assert st["step_count"] == 1
        clip = st["clip_coef"] if st["clip_applied"] else None
        for p, b in zip(params, begin):
            z = np.zeros(p.numel(), np.float32)
            want = H.step_f32(p.grad.cpu().numpy().reshape(-1), b.cpu().numpy().reshape(-1), z, z, hp, 1, 1.0, clip)[0]
            assert np.array_equal(p.detach().cpu().numpy().reshape(-1), want)


@pytest.mark.parametrize("state", STATES)
@pytest.mark.parametrize("count", [16, 40])
def test_all_hyper_groups(state, count):
    """A list over all 16 hyper-groups, in one launch's and in two launches' form."""
    c = H.ListCase([100 + 37 * i for i in range(count)], [("bf16", "f32")], state, seed=17, hgroups=list(range(16)))
    c.hps = [(1e-3 * (i + 1), 0.9 - 0.01 * i, 0.99 - 0.005 * i, 1e-8 * 4 ** i, 0.01 * i) for i in range(16)]
    run(c)
    s = H.ListCase([100, 2000, 5], [("bf16", "f32")], state, seed=17, hgroups=[15, 3, 8])
    s.hps = c.hps
    run(s)


def test_shared_grads_and_empty_copies():
    import sharded_mixed_precision_amd as D
    c = H.ListCase([3000, 3000], [("bf16", "bf16")], "e4m3", seed=18)
    c.grads[1] = c.grads[0]
    c.t = D.list_tensors(c.L, c.params, c.grads, c.A.state)
    c.init()
    before = c.snapshot()
    c.check_step(before, D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream))
    for sizes in ([], [0, 0]):
        e = H.ListCase(sizes, [("bf16", "bf16")], "e4m3")
        e.init()
        x = [torch.empty(0, device="cuda")] * 3
        D.dopt_list_export(e.L, e.t, *x, e.A.workspace, e.stream)
        D.dopt_list_import(e.L, e.t, *x, e.A.workspace, e.stream)
        D.dopt_list_stats(e.L, e.t, e.A.workspace, e.stream)
        D.dopt_list_apply(e.L, e.t, e.A.workspace, e.stream)


SHARDED = [ParamSpec("emb", 100_003, "bf16", "f32", 1, 0), ParamSpec("w1", 70_001, "bf16", "bf16", 0, 0),
           ParamSpec("n1", 4096, "f32", "f32", 0, 1), ParamSpec("h1", 33_333, "f16", "f16", 0, 0),
           ParamSpec("w2", 123_456, "bf16", "bf16", 0, 1), ParamSpec("n2", 100, "f32", "f32", 0, 0)]
SHARD_HPS = [(1e-3, 0.9, 0.999, 1e-8, 0.01), (3e-4, 0.8, 0.99, 1e-6, 0.0)]


def _bits(x):
    return x.detach().cpu().contiguous().view(torch.uint8).numpy()


@pytest.mark.parametrize("rank", [0, 2])
def test_shards_stepped_as_a_list_are_the_sharded_step(rank):
    """The shards of a layout as a list with fp32 moments: the same params,
    masters and moments as dopt_step, bit for bit, and the same checkpoint."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import DeviceArenas, ListArrays
    lay = D.dopt_build_ranges(SHARDED, 3, rank, 50_000)
    arenas = [DeviceArenas(lay) for _ in range(2)]
    stream = torch.cuda.current_stream()
    for k, inf in enumerate(lay.infos()):
        w = synth.fill_normal(inf["pd"], inf["arena_numel"], 3, synth.weight_stream(k), 0, 0.02)
        for A in arenas:
            A.bufs[k]["param"].copy_(w)
    A, B = arenas
    D.dopt_init_state(lay, A.bufs, D.scaler_cfg(), A.workspace, stream)
    lst = D.dopt_list_from_layout(lay)
    S = ListArrays(lst)
    t = D.list_tensors(lst, *D.shard_views(lay, lst, B.bufs), S.state)
    D.dopt_list_init(lst, t, D.scaler_cfg(), S.workspace, stream)
    n = lst.numel
    for step in (1, 2, 3):
        for k, inf in enumerate(lay.infos()):
            g = synth.fill_normal(inf["gd"], inf["arena_numel"], 3, synth.grad_stream(k), step, 1e-2)
            for X in arenas:
                X.bufs[k]["grad"].copy_(g)
        a = D.dopt_step(lay, A.bufs, SHARD_HPS, 1.0, A.workspace, stream)
        b = D.dopt_list_step(lst, t, SHARD_HPS, 1.0, S.workspace, stream)
        # the two add their squares in different orders: doubles within 1e-12, one fp32 clip
        assert a["clip_applied"] == b["clip_applied"] == 1 and a["num_zeros"] == b["num_zeros"]
        assert math.isclose(a["sumsq"], b["sumsq"], rel_tol=1e-12)
        assert np.float32(a["clip_coef"]) == np.float32(b["clip_coef"])
        x, y = ([torch.empty(n, device="cuda") for _ in range(3)] for _ in range(2))
        D.dopt_state_export(lay, A.bufs, *x, A.workspace, stream)
        D.dopt_list_export(lst, t, *y, S.workspace, stream)
        for u, v in zip(x, y):
            assert np.array_equal(_bits(u), _bits(v)), step
        for u, v in zip(A.bufs, B.bufs):
            assert np.array_equal(_bits(u["param"]), _bits(v["param"])), step


def test_ranks_with_8_bit_moments_exchange_their_record():
    """Three ranks' shards with 8-bit moments, the record summed over the ranks
    before the finalize: every rank clips by the norm of the whole, and
    the checkpoint of one kind continues in the other."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import DeviceArenas, ListArrays
    ranks = []
    stream = torch.cuda.current_stream()
    rng = np.random.default_rng(5)
    total = 0.0
    for r in range(3):
        lay = D.dopt_build_ranges(SHARDED, 3, r, 50_000)
        A = DeviceArenas(lay)
        for b, inf in zip(A.bufs, lay.infos()):
            for key in ("param", "grad"):
                b[key].copy_(torch.from_numpy(rng.standard_normal(inf["arena_numel"]).astype(np.float32) * 0.02))
        lst = D.dopt_list_from_layout(lay, "e4m3")
        S = ListArrays(lst)
        ps, gs = D.shard_views(lay, lst, A.bufs)
        t = D.list_tensors(lst, ps, gs, S.state)
        D.dopt_list_init(lst, t, D.scaler_cfg(), S.workspace, stream)
        total += sum(float(g.double().square().sum()) for g in gs)
        ranks.append((lay, A, lst, S, t))
    for _, _, lst, S, t in ranks:
        D.dopt_list_stats(lst, t, S.workspace, stream)
    at = ranks[0][2].stats_record_offset
    records = [S.workspace[at:at + 16].view(torch.float64) for _, _, _, S, _ in ranks]
    whole = torch.stack(records).sum(0)
    assert math.isclose(float(whole[0]), total, rel_tol=1e-12)
    for rec in records:
        rec.copy_(whole)
    for lay, A, lst, S, t in ranks:
        D.dopt_list_finalize(lst, SHARD_HPS, 1.0, S.workspace, stream)
        st = D.dopt_list_read_stats(lst, S.workspace, stream)
        assert st["clip_applied"] and math.isclose(st["clip_coef"], 1.0 / (math.sqrt(total) + 1e-6), rel_tol=1e-12)
        D.dopt_list_apply(lst, t, S.workspace, stream)
        # the 8-bit checkpoint loads into the flat step's fp32 state
        x = [torch.empty(lst.numel, device="cuda") for _ in range(3)]
        D.dopt_list_export(lst, t, *x, S.workspace, stream)
        D.dopt_init_state(lay, A.bufs, D.scaler_cfg(), A.workspace, stream)
        D.dopt_state_import(lay, A.bufs, *x, A.workspace, stream)
        D.dopt_state_scalars_set(lay, A.workspace, D.dopt_list_scalars_get(lst, S.workspace, stream), stream)
        y = [torch.empty(lst.numel, device="cuda") for _ in range(3)]
        D.dopt_state_export(lay, A.bufs, *y, A.workspace, stream)
        assert all(torch.equal(u, v) for u, v in zip(x, y))
        assert D.dopt_step(lay, A.bufs, SHARD_HPS, 1.0, A.workspace, stream)["step_count"] == 2


@pytest.mark.parametrize("unit", [2, 512])
@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("state", STATES)
def test_tensors_far_apart(state, n, unit):
    """Params and grads in turn at either end of 10 GiB, so that no 32-bit
    number of elements reaches from one to the next, at odd offsets and at
    offsets of a common 512 bytes: the results, norm and checkpoint of the
    same tensors side by side, bit for bit."""
    rng = np.random.default_rng(n)
    sizes = [9000] + [int(x) for x in rng.integers(1, 3000, n - 1)]
    near, far = (H.ListCase(sizes, [("bf16", "bf16")], state, seed=14) for _ in range(2))
    span, D = 10 << 30, near.D
    field = torch.zeros(span, dtype=torch.uint8, device="cuda")
    at = [0, span]
    moved = {"params": [], "grads": []}
    for i, x in enumerate(sizes):
        for name, side in (("params", i % 2), ("grads", 1 - i % 2)):
            if side:  # from the top down
                at[1] -= -(-(2 * x + 2) // unit) * unit
                a = at[1]
            else:
                a = at[0]
                at[0] += -(-(2 * x + 2) // unit) * unit
            v = field[a:a + 2 * x].view(torch.bfloat16)
            v.copy_(getattr(far, name)[i])
            moved[name].append(v)
    far.params, far.grads, far.store = moved["params"], moved["grads"], []
    far.t = D.list_tensors(far.L, far.params, far.grads, far.A.state)
    for c in (near, far):
        c.init()
    for _ in range(2):
        a, b = (D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream) for c in (near, far))
        assert a == b
    for x, y in zip(near.snapshot(), far.snapshot()):
        assert all(np.array_equal(x[k], y[k]) for k in x)
    xs = [[torch.empty(c.L.numel, device="cuda") for _ in range(3)] for c in (near, far)]
    for c, x in zip((near, far), xs):
        D.dopt_list_export(c.L, c.t, *x, c.A.workspace, c.stream)
        D.dopt_list_import(c.L, c.t, *x, c.A.workspace, c.stream)
    assert all(torch.equal(u, v) for u, v in zip(*xs))
    for x, y in zip(near.snapshot(), far.snapshot()):
        assert all(np.array_equal(x[k], y[k]) for k in x)


def test_offsets_beyond_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements, and one after it: the
    first and last elements of both, and a stretch across the 2^31st."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import ListArrays
    n, tail = (1 << 31) + 5001, 777
    L = D.dopt_list_build([D.TensorSpec(n, "bf16", "bf16"), D.TensorSpec(tail, "bf16", "bf16")], "e4m3")
    A = ListArrays(L)
    params = [torch.full((k,), 0.5, dtype=torch.bfloat16, device="cuda") for k in (n, tail)]
    grads = [torch.zeros(k, dtype=torch.bfloat16, device="cuda") for k in (n, tail)]
    places = [(0, slice(0, 3000)), (0, slice((1 << 31) - 1024, (1 << 31) + 1024)), (0, slice(n - 128 * 9 - n % 128, n)),
              (1, slice(0, tail))]
    for i, sl in places:
        g = grads[i][sl]
        g.copy_(torch.randn(g.numel(), device="cuda", generator=torch.Generator("cuda").manual_seed(sl.start % 97)))
    t = D.list_tensors(L, params, grads, A.state)
    stream = torch.cuda.current_stream()
    D.dopt_list_init(L, t, D.scaler_cfg(), A.workspace, stream)
    hp = (1e-3, 0.9, 0.999, 1e-8, 0.01)
    st = D.dopt_list_step(L, t, [hp], 1.0, A.workspace, stream)
    want = sum(float(grads[i][sl].double().square().sum()) for i, sl in places)
    assert math.isclose(st["sumsq"], want, rel_tol=1e-9)
    assert st["num_zeros"] == n + tail - sum(int((grads[i][sl] != 0).sum()) for i, sl in places)
    for i, sl in places:
        raw = grads[i][sl].float().cpu().numpy()
        a = L.tensor(i)["arena_offset"] + sl.start
        z = np.zeros(raw.size, np.float32)
        p, m, v, r = H.step_f32(raw, z + np.float32(0.5), z, z, hp, 1, 1.0, st["clip_coef"])
        assert np.array_equal(A.state["master"][a:a + raw.size].cpu().numpy(), p)
        for key, x in (("exp_avg", m), ("exp_avg_sq", r)):
            assert a % 128 == 0
            c, s = H.encode(x, "m" if key == "exp_avg" else "r")
            assert np.array_equal(_bits(A.state[key][a:a + raw.size]), c)
            whole = raw.size // 128
            assert np.array_equal(A.state[key + "_scale"][a // 128:a // 128 + whole].cpu().numpy(), s[:whole])
    # a place that had no grad only decayed
    assert float(A.state["master"][1 << 30]) == float(np.float32(0.5) * np.float32(1 - 1e-5))
