"""The rounding of a list's 8-bit moments by chance, in plain numpy: the random
words, the rounding itself, and runs of moments against fp32 ones."""
import numpy as np

from tests import list_harness as H

F = np.float32
M32 = np.uint64(0xFFFFFFFF)


def philox(counter, key, rounds):
    """Philox4x32 (Salmon, Moraes, Dror, Shaw 2011): counter (..., 4) and key of two words -> (..., 4)."""
    c = [np.asarray(x, np.uint64) for x in np.moveaxis(np.asarray(counter, np.uint64), -1, 0)]
    k = [int(x) for x in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & M32,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1).astype(np.uint32)


def words(first, n, step, seed):
    """The random words of elements first .. first + n - 1 of an arena (first a multiple of 4)."""
    quads = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    t = np.full_like(quads, step)
    c = np.stack([quads & M32, quads >> np.uint64(32), t & M32, t >> np.uint64(32)], -1)
    return philox(c, (seed & 0xFFFFFFFF, seed >> 32), 7).reshape(-1)[:n]


def chance(q, u):
    """|q| <= 448 to one of the two e4m3 numbers around it; u: 16 random bits each."""
    a = np.abs(q).astype(F)
    low = a < F(2.0 ** -6)
    b = np.where(low, a + F(2.0 ** -6), a).astype(F).view(np.uint32)
    y = ((b + (u.astype(np.uint32) << np.uint32(4)) + np.uint32(8)) & np.uint32(0xFFF00000)).view(F)
    return np.copysign(np.where(low, y - F(2.0 ** -6), y), q).astype(F)


def encode(x, kind, w):
    """(codes, scales) as list_harness.encode, rounded by chance with the random words w."""
    b = H._blocks(x.astype(F))
    u = np.zeros(b.size, np.uint32)
    u[:x.size] = w >> np.uint32(16) if kind == "r" else w & np.uint32(0xFFFF)
    with np.errstate(all="ignore"):
        a = np.abs(b).max(1)
        live = ~(a < F(H.TINY))
        s = np.where(live, np.where(a > H.CAP[kind], H.CAP[kind], a) * F(1.0 / 448.0), F(0)).astype(F)
        q = np.clip((b * (F(1) / s).astype(F)[:, None]).astype(F), F(-448), F(448))
        q = np.where(live[:, None], np.nan_to_num(q, nan=0.0), F(0)).astype(F)
        v = chance(q.reshape(-1), u).reshape(q.shape)
        if kind == "r":
            v = np.where((b > 0) & live[:, None], np.maximum(v, F(H.LEAST)), v)
        v = np.where(live[:, None], v, F(0))
    return H.e4m3_code(v.reshape(-1))[:x.size], s


def run(sigma, steps, blocks, by_chance, seed=1, at=()):
    """Decoded sqrt(v) over sqrt(v) of fp32 moments, per element, after each of
    the steps `at`; sigma(t) is the standard deviation of the step's grads."""
    rng = np.random.default_rng(seed)
    n = 128 * blocks
    v32, r = np.zeros(n, F), np.zeros(n, F)
    b2, o = F(0.999), F(1.0 - 0.999)
    out = []
    for t in range(1, steps + 1):
        g = (rng.standard_normal(n) * sigma(t)).astype(F)
        v32 = b2 * v32 + o * (g * g)
        x = np.sqrt(b2 * (r * r) + o * (g * g))
        r = H.decode(*(encode(x, "r", rng.integers(0, 1 << 32, n, dtype=np.uint32)) if by_chance else H.encode(x, "r")))
        if t in at:
            out.append(r / np.sqrt(v32))
    return out
