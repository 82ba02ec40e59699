"""The attention over the 4-bit store in each form of its kernels (8, 16 and 32 query rows a unit) and each way to share
the work (clusters, pieces, a CTA a unit), within bounds that a lost or doubled block does not pass
(tests/quant_bounds.py, tests/test_quant_bounds_cpu.py)."""
import math

import numpy as np
import pytest

from oracle import quant_oracle as Q
from tests import quant_bounds as QB

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402

BB = N.NOSA_QUANT_BLOCK_BYTES
SCALE = 1 / math.sqrt(128)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _store(k, v):
    """The store of k, v [units, n, 128] (bf16 on the device; n a whole number of blocks)."""
    units, n = k.shape[:2]
    store = torch.zeros((units, n // 64, BB), dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(k, v, store, units, n, n // 64, stream=_stream())
    return store


def _normal(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


def _queries(seed, units, group, nq):
    q = _normal(seed, units, group, nq, 128)
    return (q / q.norm(dim=-1, keepdim=True) * math.sqrt(128)).to(torch.bfloat16)


def _attend(q, store, lens, sel=None, slot=None, scale=0.0):
    units, group, nq = q.shape[:3]
    nb = store.shape[1]
    blocks = nb if sel is None else sel.shape[1]
    size = N.nosa_quant_scratch_bytes(units, group * nq, blocks)
    scratch = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    if sel is None:
        N.nosa_quant_dense_attend(q, store, units, group, nq, nb, lens, 64 * nb, out, scratch, size, softmax_scale=scale,
                                  stream=_stream())
    else:
        N.nosa_quant_attend(q, store, sel, slot, units, group, nq, nb, blocks, lens, out, scratch, size,
                            softmax_scale=scale, stream=_stream())
    torch.cuda.synchronize()
    assert int(scratch[:4].view(torch.int32).item()) == 0
    return out.double().cpu().numpy()


def _check(got, q, blocks, at, length, scale=SCALE):
    """One unit: got, q [group, nq, 128], blocks uint8 [n, 10240] at the positions at [n, 64]."""
    nq = q.shape[1]
    ref, tol, norm = QB.expect(q.double().cpu().numpy().reshape(-1, 128), blocks, at, int(length), nq, scale)
    got = got.reshape(-1, 128)
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    assert (np.linalg.norm(err, axis=1) <= norm).all(), (np.linalg.norm(err, axis=1) / np.maximum(norm, 1e-300)).max()
    assert not got[norm == 0].any()  # a row that sees nothing


def _some(units):
    return sorted({0, 1, 2, 3, units // 2, units - 2, units - 1})


@pytest.mark.parametrize("group,nq", QB.FORMS)
@pytest.mark.parametrize("plan", QB.PLANS)
def test_ragged_batches(plan, group, nq):
    units, nb = QB.PLANS[plan]
    k, v = (_normal(s, units, 64 * nb, 128).to(torch.bfloat16) for s in (1, 2))
    store = _store(k, v)
    q, lens = _queries(3, units, group, nq), QB.lengths(units, nb)
    rng = np.random.default_rng(4)
    order = np.stack([rng.permutation(nb) for _ in range(units)])
    # the blocks of each unit put at other rows of the store, listed in any order with gaps between
    moved = torch.empty_like(store)
    rows = torch.from_numpy(order).cuda()
    moved.scatter_(1, rows[:, :, None].expand(-1, -1, BB), store)  # block b is in row order[b]
    sel = np.full((units, nb + 4), -1)
    slot = np.zeros((units, nb + 4), np.int64)
    for u in range(units):
        place = np.sort(rng.permutation(nb + 4)[:nb])
        sel[u, place] = rng.permutation(nb)
        slot[u, place] = order[u][sel[u, place]]
    dense = _attend(q, store, _i32(lens))
    listed = _attend(q, store, _i32(lens), _i32(sel))
    cached = _attend(q, moved, _i32(lens), _i32(sel), _i32(slot))
    assert np.array_equal(listed, cached)
    at = np.arange(64 * nb).reshape(nb, 64)
    for u in _some(units):
        blocks = store[u].cpu().numpy()
        for got in (dense, listed):
            _check(got[u], q[u], blocks, at, lens[u])
    # the units that were not looked at: the two calls differ by their roundings (2^-8 and less than 2^-6.9 each)
    for a, b in zip(dense, listed):
        assert np.linalg.norm(a - b) <= 2.0 ** -5 * np.linalg.norm(a)


@pytest.mark.parametrize("group,nq", QB.FORMS)
@pytest.mark.parametrize("plan", ["cluster", "pieces"])
def test_selections_count_what_they_list(plan, group, nq):
    """Some blocks left out, one listed twice, one behind the context."""
    units, nb = QB.PLANS[plan]
    k, v = (_normal(s, units, 64 * nb, 128).to(torch.bfloat16) for s in (5, 6))
    store, q = _store(k, v), _queries(7, units, group, nq)
    rng = np.random.default_rng(8)
    lens = np.full(units, 64 * (nb - 2) + 37)
    most = nb - 3
    sel = np.stack([rng.permutation(nb)[:most] for _ in range(units)])
    sel[:, 1] = sel[:, 0] = nb - 2  # the last, partial block twice
    got = _attend(q, store, _i32(lens), _i32(sel))
    for u in _some(units):
        at = sel[u][:, None] * 64 + np.arange(64)
        _check(got[u], q[u], store[u].cpu().numpy()[sel[u]], at, lens[u])


def _values(what, k, v, q):
    """k, v [units, n, 128] and q [units, group, nq, 128] float32 on the device, made into the case."""
    n = k.shape[1]
    if what == "large-v":
        v[:, n // 3:] *= 60.0
    if what == "huge-v":  # a few tokens, scales of thousands
        v[:, ::67] *= 9000.0
    if what == "small-v":
        v *= 1e-4
    if what == "mixed-groups":  # each group of dims another size
        v *= torch.tensor([0.01, 1.0, 12.0, 200.0], device="cuda").repeat_interleave(32)
    if what == "offset-v":  # minima far from zero
        v += 30.0
    if what == "growing":  # keys along the first row's query, ever longer: references rise all the time
        k += torch.linspace(0, 25, n, device="cuda")[None, :, None] * q[:, 0, 0][:, None] / 4
    if what == "growing-large-v":
        k += torch.linspace(0, 25, n, device="cuda")[None, :, None] * q[:, 0, 0][:, None] / 4
        v *= torch.linspace(0.1, 100, n, device="cuda")[None, :, None]
    if what == "peaked":
        q *= 8
    return k, v, q


@pytest.mark.parametrize("group,nq", QB.FORMS)
@pytest.mark.parametrize("plan", ["cluster", "pieces"])
@pytest.mark.parametrize("what", ["large-v", "huge-v", "small-v", "mixed-groups", "offset-v", "growing", "growing-large-v",
                                  "peaked"])
def test_value_ranges(what, plan, group, nq):
    units, nb = QB.PLANS[plan]
    q = _queries(9, units, group, nq).float()
    k, v, q = _values(what, *(_normal(s, units, 64 * nb, 128) for s in (10, 11)), q)
    q = q.to(torch.bfloat16)
    store = _store(k.to(torch.bfloat16), v.to(torch.bfloat16))
    lens = np.full(units, 64 * nb - 11)
    got = _attend(q, store, _i32(lens))
    at = np.arange(64 * nb).reshape(nb, 64)
    for u in (0, units // 2, units - 1):
        _check(got[u], q[u], store[u].cpu().numpy(), at, lens[u])


@pytest.mark.parametrize("group,nq", QB.FORMS)
@pytest.mark.parametrize("plan", QB.PLANS)
def test_nan_groups(plan, group, nq):
    """A NaN in V reaches its group's dims of the rows that see the token, one in K the whole row, and both nothing else:
    seen by all, by the last query token alone, by none; in a stage's first and second tile."""
    units, nb = QB.PLANS[plan]
    k, v = (_normal(s, units, 64 * nb, 128).to(torch.bfloat16) for s in (12, 13))
    q = _queries(14, units, group, nq)
    clean = _store(k, v)
    lens = np.full(units, 64 * nb - 20)
    lens[1], lens[4] = 64 * nb - 36, 64 * nb - 10  # the last token in a stage's second tile, in the first and second half
    end = lens - 1
    bad = np.zeros((units, group, nq, 128), bool)
    v[0, end[0], 40] = float("nan")
    bad[0, :, nq - 1, 32:64] = True
    k[1, end[1], 3] = float("inf")
    bad[1, :, nq - 1] = True
    v[2, 10, 127] = float("inf")
    bad[2, :, :, 96:] = True
    v[3, 63, 0], k[3, end[3] + 1, 5], v[3, end[3] + 2, 64] = -float("inf"), float("nan"), float("nan")
    bad[3, :, :, :32] = True
    if nq > 1:
        v[4, end[4] - nq + 2, 70] = float("nan")  # seen by all query tokens but the first
        bad[4, :, 1:, 64:96] = True
    store = _store(k, v)
    at = np.arange(64 * nb).reshape(nb, 64)
    for sel in (None, _i32(np.tile(np.arange(nb), (units, 1)))):
        got = _attend(q, store, _i32(lens), sel)
        assert np.array_equal(np.isnan(got), bad)
        for u in range(5):
            # the other values: those of a store without the NaN, but for the token that had it (K: nowhere else)
            host = clean[u].cpu().numpy()
            ref, tol, _ = QB.expect(q[u].double().cpu().numpy().reshape(-1, 128), host, at, int(lens[u]), nq, SCALE)
            ok = ~bad[u].reshape(-1, 128)
            assert (np.abs(got[u].reshape(-1, 128) - ref)[ok] <= tol[ok]).all()


@pytest.mark.parametrize("group,nq", QB.FORMS)
def test_long_means(group, nq):
    """65,536 tokens that nearly cancel, 320 units of them: a warp's sums run over 270 (8 rows) to 2,156 tiles (32 rows).

    The error's norm over the result's.  Rounding to bf16 is uniform in +-2^-8 of the value's power of two: 2^-8 / sqrt(3)
    of the value in the mean square, 2^-8.8.  A token's weight and its product with s are rounded by 2^-11 at most,
    independently, so that their errors add up as the tokens' values do: sqrt(2 / 3) 2^-11 times the size of a code's part
    against its value's, 8.7 against 3.7 in units of s: 2^-10.1.  Together 2^-8.68; a tenth more for the finite number of
    values."""
    units, nb = 320, 1024
    k, v = (_normal(s, 1, 64 * nb, 128).to(torch.bfloat16) for s in (15, 16))
    one = _store(k, v)
    store = one.expand(units, -1, -1).contiguous()
    q = _queries(17, units, group, nq)
    got = torch.from_numpy(_attend(q, store, _i32([64 * nb] * units))).cuda()
    kk, vv, _, _ = Q.unpack(one[0].cpu().numpy())
    k, v = torch.from_numpy(kk).cuda().view(-1, 128), torch.from_numpy(vv).cuda().view(-1, 128)
    at = torch.arange(64 * nb, device="cuda")
    for u in (0, 3, units // 2, units - 1):
        for i in range(nq):
            z = (q[u, :, i].double() @ k.T * SCALE).masked_fill(at >= 64 * nb - (nq - 1 - i), -math.inf)
            ref = torch.softmax(z, -1) @ v
            assert ((got[u, :, i] - ref).norm() / ref.norm()).item() <= 1.1 * 2.0 ** -8.68
