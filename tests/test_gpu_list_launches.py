"""GPU tests of the list calls where a pass takes several launches: more
tensors of one type pair than a launch's arguments hold (480 in pass 2 and the
copies, 800 in pass 1), near and far apart, more tiles than a launch takes
(2^15 with fp32 moments, 2^16 with 8-bit ones), and pass 1 of more than 512 MiB
of grads in each type."""
import math

import numpy as np
import pytest
import torch

from tests import gpu_harness as G
from tests import list_dither as S
from tests import list_harness as H
from tests.test_gpu_list import run
from tests.test_gpu_list_dither import Case
from tests.test_gpu_list_dither import run as run_by_chance

pytestmark = pytest.mark.gpu

STATES = ("f32", "e4m3", "e4m3_sr")


@pytest.fixture(autouse=True)
def _announce(request):
    G.log(f"[gpu-test] start {request.node.name}")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _sizes(n):
    return [int(x) for x in np.random.default_rng(n).integers(1, 500, n)]


@pytest.mark.parametrize("n", [800, 801, 1700])
@pytest.mark.parametrize("state", STATES)
def test_more_tensors_than_a_launch_of_either_pass(n, state):
    """Tensors of one type pair, none empty: 2 to 4 launches of pass 2 and 1 to 3 of pass 1."""
    pair, hg = [("bf16", "f32")], [0, 2, 1]
    if state == "e4m3_sr":
        run_by_chance(Case(_sizes(n), pair, seed=21, hgroups=hg), seed=4)
    else:
        run(H.ListCase(_sizes(n), pair, state, seed=21, hgroups=hg))


@pytest.mark.parametrize("state", STATES)
def test_many_tensors_far_apart(state):
    """1700 tensors of one type pair, params and grads in turn at either end of
    10 GiB at odd offsets, so that every launch takes its addresses from the
    table: the step, export and import of the same tensors side by side."""
    sizes = _sizes(1700)
    near, far = (H.ListCase(sizes, [("bf16", "bf16")], state, seed=22, hgroups=[0, 2, 1]) for _ in range(2))
    D, span = near.D, 10 << 30
    field, lo, hi = torch.zeros(span, dtype=torch.uint8, device="cuda"), 0, span
    moved = {"params": [], "grads": []}
    for i, x in enumerate(sizes):
        for name, side in (("params", i % 2), ("grads", 1 - i % 2)):
            if side:
                hi -= 2 * x + 2
            v = field[hi if side else lo:][:2 * x].view(torch.bfloat16)
            lo += 0 if side else 2 * x + 2
            v.copy_(getattr(far, name)[i])
            moved[name].append(v)
    far.params, far.grads, far.store = moved["params"], moved["grads"], []
    far.t = D.list_tensors(far.L, far.params, far.grads, far.A.state)
    assert max(p.data_ptr() for p in far.params) - min(p.data_ptr() for p in far.params) > 2 << 32  # beyond 32 bits of 2 bytes
    for c in (near, far):
        c.init()
    for _ in range(2):
        a, b = (D.dopt_list_step(c.L, c.t, c.hps, 1.0, c.A.workspace, c.stream) for c in (near, far))
        assert a == b
    out = [[torch.empty(c.L.numel, device="cuda") for _ in range(3)] for c in (near, far)]
    for c, x in zip((near, far), out):
        D.dopt_list_export(c.L, c.t, *x, c.A.workspace, c.stream)
    assert all(torch.equal(u, v) for u, v in zip(*out))
    assert all(float(x.abs().max()) > 0 for x in out[0])
    for c, x in zip((near, far), out):
        for y in x:
            y.mul_(0.5)
        D.dopt_list_import(c.L, c.t, *x, c.A.workspace, c.stream)
    for u, v in zip(near.params + list(near.A.state.values()), far.params + list(far.A.state.values())):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("pair", [("bf16", "f32"), ("f32", "bf16")], ids=lambda p: "-".join(p))
@pytest.mark.parametrize("state", STATES)
def test_more_tiles_than_a_launch(state, pair):
    """One tensor of more tiles than a launch of pass 2 and the copies takes,
    and the same elements as a list of tensors of 2^20: no launch of theirs
    begins inside a tensor.  Step, export and import give the same bits, and at the
    pieces' borders those of the fp32 operations."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import ListArrays
    tiles = 1 << (15 if state == "f32" else 16)
    n, part = (2 * tiles + 3) * 2048 + 777, 1 << 20
    gen = torch.Generator("cuda").manual_seed(3)
    pd, gd = H.TORCH[pair[0]], H.TORCH[pair[1]]
    w = torch.randn(n, device="cuda", generator=gen).mul_(0.05).to(pd)
    g = torch.randn(n, device="cuda", generator=gen).mul_(1e-2).to(gd)
    cuts = [(a, min(part, n - a)) for a in range(0, n, part)]
    runs = []
    hp, stream = (1e-3, 0.9, 0.999, 1e-8, 0.01), torch.cuda.current_stream()
    for pieces in ([(0, n)], cuts):
        p = w.clone()
        L = D.dopt_list_build([D.TensorSpec(k, *pair) for _, k in pieces], state)
        A = ListArrays(L)
        t = D.list_tensors(L, [p[a:a + k] for a, k in pieces], [g[a:a + k] for a, k in pieces], A.state)
        D.dopt_list_init(L, t, D.scaler_cfg(), A.workspace, stream)
        for _ in range(2):
            st = D.dopt_list_step(L, t, [hp], 0.0, A.workspace, stream)
        runs.append((L, t, A, p, st))
    a, b = runs

    def same():
        assert torch.equal(a[3].view(torch.uint8), b[3].view(torch.uint8))
        for key in a[2].state:
            assert torch.equal(a[2].state[key].view(torch.uint8), b[2].state[key].view(torch.uint8)), key

    same()
    assert a[4]["num_zeros"] == b[4]["num_zeros"] and math.isclose(a[4]["sumsq"], b[4]["sumsq"], rel_tol=1e-9)
    border = tiles * 2048
    for lo, hi in ((0, 512), (border - 512, border + 512), (2 * border - 512, 2 * border + 512), (n - 777 - 256, n)):
        raw, p = g[lo:hi].float().cpu().numpy(), w[lo:hi].float().cpu().numpy()
        m = v = np.zeros(hi - lo, np.float32)
        for k in (1, 2):
            p, m, v, r = H.step_f32(raw, p, m, v, hp, k, 1.0, None)
            if state != "f32" and k == 1:
                if state == "e4m3_sr":
                    word = S.words(lo, hi - lo, 1, 0)
                    m, r = (H.decode(*S.encode(x, key, word)) for key, x in (("m", m), ("r", r)))
                else:
                    m, r = (H.decode(*H.encode(x, key)) for key, x in (("m", m), ("r", r)))
                v = (r * r).astype(np.float32)
        assert np.array_equal((a[2].state["master"] if "master" in a[2].state else a[3])[lo:hi].cpu().numpy(), p), (lo, hi)
    out = [[torch.empty(n, device="cuda") for _ in range(3)] for _ in runs]
    for (L, t, A, _, _), x in zip(runs, out):
        D.dopt_list_export(L, t, *x, A.workspace, stream)
    assert all(torch.equal(u, v) for u, v in zip(*out))
    if state == "f32":
        assert torch.equal(out[0][1], a[2].state["exp_avg"][:n]) and torch.equal(out[0][2], a[2].state["exp_avg_sq"][:n])
    for (L, t, A, _, _), x in zip(runs, out):
        D.dopt_list_import(L, t, *[y.mul_(0.75) for y in x], A.workspace, stream)
    same()
    if state == "f32":
        assert torch.equal(a[2].state["exp_avg"][:n], out[0][1]) and torch.equal(a[2].state["exp_avg_sq"][:n], out[0][2])
    assert torch.equal(a[3], out[0][0].to(pd))


@pytest.mark.parametrize("gd", ["f32", "f16", "bf16"])
def test_statistics_of_more_grads_than_the_last_level_cache_keeps(gd):
    """More than 512 MiB of grads, at an odd offset and with a ragged end, where
    pass 1 reads them in its other way: the sum of squares in 64 bits and the
    count of zeros, and the same list's grads with an infinity among them."""
    import sharded_mixed_precision_amd as D
    from sharded_mixed_precision_amd.arena import ListArrays
    dt = H.TORCH[gd]
    n = (512 << 20) // (4 if gd == "f32" else 2) + 12_345
    store = torch.zeros(n + 9, dtype=dt, device="cuda")
    store[:] = float("nan")  # what is not of the tensors is not read
    g = store[3:3 + n]
    gen = torch.Generator("cuda").manual_seed(7)
    for a in range(0, n, 1 << 26):
        x = torch.randn(min(1 << 26, n - a), device="cuda", generator=gen)
        g[a:a + x.numel()] = x.mul_(x.abs() > 0.05)
    sizes = [n - 5001, 0, 5001]
    L = D.dopt_list_build([D.TensorSpec(k, gd, gd) for k in sizes], "f32")
    A = ListArrays(L)
    params = [torch.zeros(k, dtype=dt, device="cuda") for k in sizes]
    t = D.list_tensors(L, params, [g[:sizes[0]], None, g[sizes[0]:]], A.state)
    stream = torch.cuda.current_stream()
    D.dopt_list_init(L, t, D.scaler_cfg(), A.workspace, stream)
    D.dopt_list_stats(L, t, A.workspace, stream)
    at = L.stats_record_offset
    rec = A.workspace[at:at + 16].view(torch.float64).tolist()
    sumsq = sum(float(g[a:a + (1 << 26)].double().square().sum()) for a in range(0, n, 1 << 26))
    # each of n additions in double within 2^-53 of the sum, on both sides
    assert math.isclose(rec[0], sumsq, rel_tol=2 * n * 2.0 ** -53)
    assert rec[1] == sum(int((g[a:a + (1 << 26)] == 0).sum()) for a in range(0, n, 1 << 26))
    g[n // 2] = math.inf
    st = D.dopt_list_step(L, t, [(1e-3, 0.9, 0.999, 1e-8, 0.01)], 1.0, A.workspace, stream)
    assert st["skipped"] and st["step_count"] == 0 and not float(params[0].abs().max())
