"""The bounds that the GPU tests of the 4-bit attention use (tests/quant_bounds.py) can fail: at every shape they are used
at, they let a result with the kernels' own roundings through and stop zeros, a lost or doubled block and a lost half block."""
import math

import numpy as np
import pytest

from oracle import quant_oracle as Q
from tests import quant_bounds as QB


def _bf16(x):
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1) >> 16 << 16).astype(np.uint32)).view(np.float32).astype(np.float64)


def _unit(nb, rows, seed):
    rng = np.random.default_rng(seed)
    k, v = _bf16(rng.standard_normal((2, nb, 64, 128)))
    q = rng.standard_normal((rows, 128))
    q = _bf16(q * math.sqrt(128) / np.linalg.norm(q, axis=1, keepdims=True))
    return Q.pack(k, v), q


def _rounded(q, blocks, length, nq, scale):
    """The result with the kernels' 16-bit roundings: weights up to 2^14, products with s, maxima in every second tile."""
    k, v, _, _ = (x.reshape(-1, 128) for x in Q.unpack(blocks))
    s, m = QB._v_scales(blocks)
    n = np.where(s > 0, (v - m) / np.where(s > 0, s, 1), 0)
    odd = (np.arange(len(k)) // 16 % 2 == 1)[:, None]
    f16 = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    out = np.zeros(q.shape)
    for r in range(q.shape[0]):
        see = np.arange(len(k)) < length - (nq - 1 - r % nq)
        if see.any():
            z = k[see] @ q[r] * scale
            w = f16(np.exp(z - z.max()) * 2.0 ** 12)[:, None]
            low = f16(w * s[see]) * n[see] + w * m[see]
            high = w * f16(m[see] + 15 * s[see]) - f16(w * s[see]) * (15 - n[see])
            out[r] = np.where(odd[see], high, low).sum(0) / w.sum()
    return _bf16(out)


@pytest.mark.parametrize("group,nq", QB.FORMS)
@pytest.mark.parametrize("plan", QB.PLANS)
def test_bounds_let_roundings_through_and_stop_lost_blocks(plan, group, nq):
    units, nb = QB.PLANS[plan]
    scale = 1 / math.sqrt(128)
    lens = QB.lengths(units, nb)
    for length in sorted({int(lens[0]), int(lens[2]), int(lens[3])}):
        blocks, q = _unit(nb, group * nq, length)
        at = np.arange(64 * nb).reshape(nb, 64)
        ref, tol, norm = QB.expect(q, blocks, at, length, nq, scale)
        assert QB.within(_rounded(q, blocks, length, nq, scale), ref, tol, norm)
        seen = np.abs(ref).sum(1) > 0
        assert not QB.within(0 * ref, ref, tol, norm)
        held = -(-length // 64)
        if held < 2:
            continue

        def other(keep):
            """Every row's result over the listed blocks, as far as it sees them."""
            return _bf16(QB.expect(q, blocks[keep], at[keep], length, nq, scale)[0])

        everything = np.arange(held)
        for lost in (0, held // 2):
            for wrong in (other(np.delete(everything, lost)), other(np.append(everything, lost))):
                err = np.abs(wrong - ref)
                # in every row that sees anything
                assert ((np.linalg.norm(err, axis=1) > norm) | (err > tol).any(1))[seen].all(), (length, lost)
        half = at.copy()
        half[held // 2, 32:] = -1
        if held > 2:
            wrong = _bf16(QB.expect(q, blocks, half, length, nq, scale)[0])
            assert not QB.within(wrong, ref, tol, norm)
