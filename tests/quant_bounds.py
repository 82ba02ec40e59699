"""How far the 4-bit attention may be from its float64 definition, for one unit's rows and dims.

With p_t the softmax weights (float64) of the tokens a row sees, x_t what the store gives for V, o the result, 15 s_t the
range of a token's group and M_t = m + 15 s its maximum, the kernels' roundings are:
  * a weight: to f16, 2^-11, and its logit in float32: sums of |q| (|n s| + |m|) in some twenty steps of 2^-24, taken
    as 2^-18 of that sum.  It moves the result by p_t (x_t - o), numerator and denominator together.
  * its product with s: 2^-11 of it, times a code of at most 15.
  * M_t: 2^-11 of it (in every second tile; counted in all).
These are independent from token to token, so their squares add up: V_d.  A rounding is uniform at best, a third of
its largest square, so six roots of V_d is more than ten standard deviations, and more than the sum of all for a dozen
tokens; for the norm over the 128 dims, which share a weight's rounding and in groups of 32 a product's, three roots
of the sum of V_d.
  * weights and products among f16's subnormals: 2^(e - 35) of the largest weight each, e the exponent of the largest s.
  * float32 sums over at most 1 / 32 of the tokens' number of steps: 2^-24 a step of half the codes' part.
  * the result to bf16: 2^-8 of it."""
import numpy as np

from oracle import quant_oracle as Q


def _v_scales(blocks):
    """s and m of V, float64 [64 n, 128] each, of blocks uint8 [n, 10240]."""
    t = blocks.reshape(-1, 4, Q.TILE_BYTES)
    i, g = np.arange(16)[:, None], np.arange(4)[None]
    out = []
    for which in (0, 1):
        at = np.broadcast_to(Q.scale_place("v", which, i, g), (16, 4))
        b = np.ascontiguousarray(np.stack((t[:, :, at], t[:, :, at + 1]), -1)).view(np.float16)[..., 0]
        out.append(np.repeat(b.astype(np.float64), 32, -1).reshape(-1, 128))
    return out


def expect(q, blocks, at, length, nq, scale):
    """q [R, 128] float64 (row r is query token r % nq), blocks uint8 [n, 10240] and their tokens' positions at [n, 64]:
    the result [R, 128], the bound of each value [R, 128] and the bound of each row's norm [R]."""
    k, v, size_k, _ = (x.reshape(-1, 128) for x in Q.unpack(blocks))
    s, m = _v_scales(blocks)
    at = np.asarray(at).reshape(-1)
    late = nq - 1 - np.arange(q.shape[0]) % nq
    see = (at[None] >= 0) & (at[None] < (length - late)[:, None])
    some = see.any(1)
    z = np.where(see, q @ k.T * scale, -np.inf)
    p = np.exp(z - np.where(some, z.max(1, initial=-np.inf), 0)[:, None])
    p /= np.where(some, p.sum(1), 1)[:, None]
    step, top = 15 * s, np.abs(m + 15 * s)
    o = p @ v
    weight = (p * (2.0 ** -11 + 2.0 ** -18 * (np.abs(q) @ size_k.T) * scale)) ** 2
    # sum of weight (v - o)^2
    var = np.maximum(weight @ v ** 2 - 2 * o * (weight @ v) + o ** 2 * weight.sum(1, keepdims=True), 0)
    var += p ** 2 @ (2.0 ** -22 * (step ** 2 + top ** 2))
    largest = np.where(see, s.max(1)[None], 0).max(1)
    e = np.maximum(np.floor(np.log2(np.maximum(largest, 1))), 0)[:, None]
    far = see @ np.abs(v) + see.sum(1, keepdims=True) * (np.abs(o) + 15)  # at least the sum of |v - o| + 15
    rest = 2.0 ** (e - 35) * p.max(1, keepdims=True) * far + 2.0 ** -24 * see.sum(1, keepdims=True) / 32 * (p @ step) / 2
    tol = 2.0 ** -8 * np.abs(o) + 1.01 * (6 * np.sqrt(var) + rest)
    norm = 2.0 ** -8 * np.linalg.norm(o, axis=1) + 1.01 * (3 * np.sqrt(var.sum(1)) + np.linalg.norm(rest, axis=1))
    return o, tol, np.where(some, norm, 0)


def within(got, ref, tol, norm):
    """Whether got [R, 128] is within both bounds."""
    err = np.abs(got - ref)
    return bool((err <= tol).all() and (np.linalg.norm(err, axis=1) <= norm).all())


# units, blocks a unit: a cluster per unit (few, and so many that they fill the device), equal pieces of all units, one CTA
# per unit
PLANS = {"cluster": (6, 24), "full-wave": (64, 40), "pieces": (12, 130), "unit-a-cta": (600, 9)}
FORMS = [(8, 1), (8, 2), (8, 4)]  # q heads and query tokens of a unit: 8, 16 and 32 rows


def lengths(units, nb):
    """Ragged lengths: all of it, none, one token, and odd ones between a tenth and all."""
    n = np.linspace(0.1, 1.0, units) * 64 * nb
    n = n.astype(np.int64) | 1
    n[0], n[1], n[2] = 64 * nb, 0, 1
    return np.minimum(n, 64 * nb)
