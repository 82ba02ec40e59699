"""The 8-bit KV block store on the GPU against its float64 oracle (oracle/byte_oracle.py): the bytes that
nosa_byte_append writes and the blocks that nosa_byte_read gives are compared for equality, the attention and its
masses within bounds counted from their roundings (see _expect)."""
import math

import numpy as np
import pytest

from oracle import byte_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402

BB = N.NOSA_BYTE_BLOCK_BYTES


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _i32(values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


# ------------------------------------------------------------------------------------------ append
def _filled(rng, units, nb):
    """A store whose blocks hold values of different sizes."""
    k, v = (rng.standard_normal((units * nb, 64, 128)) * np.exp2(rng.integers(-3, 4, (units * nb, 1, 1))) for _ in range(2))
    return O.pack(k, v).reshape(units, nb, BB)


def _append_check(k, v, before, pos, count, slot_blk=None, use_err=True):
    """Appends into a copy of `before` and compares every byte; returns the error word."""
    units, nb = before.shape[:2]
    store = torch.from_numpy(before).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N.nosa_byte_append(k, v, store, units, k.shape[1], nb, pos=None if pos is None else _i32(pos),
                       count=None if count is None else _i32(count), slot_blk=None if slot_blk is None else _i32(slot_blk),
                       err_out=err if use_err else None, stream=_stream())
    torch.cuda.synchronize()
    ref = before.copy()
    flag = O.append(ref, _f64(k), _f64(v), [0] * units if pos is None else pos,
                    [k.shape[1]] * units if count is None else count, slot_blk)
    got = store.cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    if use_err:
        assert int(err.item()) == int(flag)
    return int(err.item())


@pytest.mark.parametrize("size", [1.0, 8.0, 2.0 ** -9], ids=["same", "larger", "smaller"])
@pytest.mark.parametrize("n,pos,count", [
    (1, [0, 63, 64, 190], None),              # single tokens, two of which begin a block
    (1, [15, 16, 17, 100], [1, 0, 1, 1]),     # one unit writes nothing
    (2, [15, 31, 62, 63], None),              # two tokens over a tile's, a block's edge
    (37, [0, 5, 16, 150], [37, 36, 1, 0]),    # ragged starts and counts
    (64, None, None), (65, None, [65, 64, 17, 2]), (191, [1, 0, 1, 1], None), (192, None, None),
], ids=["one", "one-masked", "edges", "ragged", "block", "block+1", "odd", "full"])
def test_append_writes_the_oracles_bytes(n, pos, count, size):
    """With tokens that need larger scales than the blocks have, the same, or smaller ones."""
    rng = np.random.default_rng(n)
    k, v = (_bf16(rng, 4, n, 128) * size for _ in range(2))
    _append_check(k, v, _filled(rng, 4, 3), pos, count)


def test_append_out_of_range_is_flagged_and_left_out():
    rng = np.random.default_rng(5)
    k, v = _bf16(rng, 6, 20, 128), _bf16(rng, 6, 20, 128)
    before = _filled(rng, 6, 2)
    assert _append_check(k, v, before, [-7, 120, 128, 1 << 30, -(1 << 31), 3], [20, 20, 1, 20, 20, 20]) == 1
    assert _append_check(k, v, before, [0] * 6, [21, -1, 5, 0, 20, 1 << 30]) == 1
    assert _append_check(k, v, before, [0] * 6, [20] * 6) == 0
    _append_check(k, v, before, [-7] * 6, [21] * 6, use_err=False)


def test_append_through_a_slot_table():
    rng = np.random.default_rng(6)
    k, v = _bf16(rng, 5, 70, 128), _bf16(rng, 5, 70, 128)
    slots = np.full((5, 300), -1, np.int32)
    slots[0, [299, 3]] = [8, 9]                   # blocks in no order
    slots[1, [260, 7]] = 8                        # one block in two rows: the lowest counts
    slots[2, 0] = 9                               # a block that no row holds
    slots[3, [1, 0, 5]] = [33554431, 33554430, 0]  # the end of int32's positions
    slots[4, :] = np.arange(300)
    pos, count = [8 * 64 + 60, 8 * 64 + 1, 8 * 64 + 60, 2 ** 31 - 70, 18000], [68, 63, 20, 70, 70]
    before = np.zeros((5, 300, BB), np.uint8)
    before[:, :10] = _filled(rng, 5, 10)
    assert _append_check(k, v, before, pos, count, slots) == 1
    count[2] = 0
    assert _append_check(k, v, before, pos, count, slots) == 0
    assert _append_check(k[4:], v[4:], before[4:], [64 * 300 - 10], [20], slots[4:]) == 1  # the block behind the last row


def _odd_tokens():
    """Tokens whose values are where quantising can go wrong, one kind per block of 64."""
    rng = np.random.default_rng(9)
    g = rng.standard_normal((9, 64, 128))
    g[0] = np.repeat(O.E4M3[np.arange(0, 127)], 65)[: 64 * 128].reshape(64, 128)  # all codes, up to 448
    g[1] = 0.0
    g[1, 5, 7] = -0.0
    g[2] = rng.integers(-500, 500, (64, 128)) * 0.5                    # many exact ties
    g[3] *= 1e-38                                                      # below the least scale's normal range
    g[4] *= 1e38                                                       # near bf16's largest
    g[5] *= np.exp2(rng.integers(-40, 40, (64, 1)))                     # tokens of all sizes
    g[6, 3, 1], g[6, 9, 127], g[6, 40, 64] = np.nan, np.inf, -np.inf
    g[7] = np.nan
    g[8, 63, 127] = 448.0 * 8
    return torch.from_numpy(g.reshape(1, 576, 128)).float().to(torch.bfloat16).cuda()


def test_append_odd_values():
    x = _odd_tokens()
    y = x.flip(1).contiguous()
    _append_check(x, y, np.zeros((1, 9, BB), np.uint8), None, None)
    rng = np.random.default_rng(1)
    _append_check(x, y, _filled(rng, 1, 10), [37], None)
    # one by one into what was there, each checked against the oracle's own step
    store = _filled(rng, 1, 10)
    for i in range(300, 450, 7):
        ref = store.copy()
        t = torch.from_numpy(store).cuda()
        N.nosa_byte_append(x[:, i].contiguous(), y[:, i].contiguous(), t, 1, 1, 10, pos=_i32([i + 5]), stream=_stream())
        O.append(ref, _f64(x[:, i:i + 1]), _f64(y[:, i:i + 1]), [i + 5], [1])
        store = t.cpu().numpy()
        assert np.array_equal(store, ref), i


def test_append_into_what_was_never_written():
    """Scales that no append has written count as none: the codes there stay as they are."""
    rng = np.random.default_rng(12)
    before = rng.integers(0, 256, (6, 1, BB), dtype=np.uint8)
    for u, s in enumerate([np.nan, np.inf, -4.0, 3.0, 2.0 ** -120, 2.0 ** 121]):
        before[u, 0, O.SCALES:O.SCALES + 8] = np.array([s, s], np.float32).view(np.uint8)
    _append_check(_bf16(rng, 6, 9, 128), _bf16(rng, 6, 9, 128), before, [3, 20, 30, 40, 50, 55], None)


def test_append_batch_of_many_units_and_long_prompt():
    rng = np.random.default_rng(11)
    _append_check(_bf16(rng, 300, 1, 128), _bf16(rng, 300, 1, 128), _filled(rng, 300, 2), rng.integers(0, 128, 300).tolist(), None)
    k, v = _bf16(rng, 1, 4100, 128), _bf16(rng, 1, 4100, 128)
    _append_check(k, v, np.full((1, 65, BB), 0xA5, np.uint8), None, None)


def test_append_twice_is_the_same():
    rng = np.random.default_rng(13)
    k, v = _bf16(rng, 3, 50, 128) * 30, _bf16(rng, 3, 50, 128) * 30
    store = torch.from_numpy(_filled(rng, 3, 3)).cuda()
    got = []
    for _ in range(2):
        N.nosa_byte_append(k, v, store, 3, 50, 3, pos=_i32([10, 63, 64]), stream=_stream())
        got.append(store.cpu())
    assert torch.equal(*got)


def test_append_and_read_past_32_bit_offsets():
    nb = 2 ** 32 // BB + 3  # the last blocks of the first unit start beyond 4 GiB
    store = torch.zeros((2, nb, BB), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    k, v = _bf16(rng, 2, 70, 128), _bf16(rng, 2, 70, 128)
    pos = [64 * nb - 70, 64 * nb - 75]
    N.nosa_byte_append(k, v, store, 2, 70, nb, pos=_i32(pos), stream=_stream())
    kv = torch.empty((2, 2, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    blocks = torch.tensor([[nb - 2, nb - 1]] * 2, dtype=torch.int32, device="cuda")
    N.nosa_byte_read(store, 2, nb, blocks, 2, kv, stream=_stream())
    torch.cuda.synchronize()
    ref = np.zeros((2, 2, BB), np.uint8)
    O.append(ref, _f64(k), _f64(v), [p - 64 * (nb - 2) for p in pos], [70, 70])
    assert np.array_equal(store[:, nb - 2:].cpu().numpy(), ref)
    want = np.stack(O.unpack(ref.reshape(-1, BB)), 1).reshape(2, 2, 2, 64, 128)
    assert torch.equal(kv.cpu(), torch.from_numpy(want).float().to(torch.bfloat16))


# ------------------------------------------------------------------------------------------ read
def test_read_lists_lengths_and_slots():
    rng = np.random.default_rng(21)
    units, nb = 3, 5
    store = _filled(rng, units, nb)
    store[1, 2, :64] = 0x7F  # some NaN
    st = torch.from_numpy(store).cuda()
    values = np.stack(O.unpack(store.reshape(-1, BB)), 1).reshape(units, nb, 2, 64, 128)
    blocks = np.array([[0, 4, 4, -1], [2, 1, -5, 0], [3, 2, 1, 0]], np.int32)
    for lens in (None, [0, 130, 256 + 17]):
        for slots in (None, np.array([[1, 0, 3, 99], [4, 4, -3, 2], [0, 0, 1, 2]], np.int32)):
            kv = torch.full((units, 4, 2, 64, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            N.nosa_byte_read(st, units, nb, _i32(blocks), 4, kv, slots=None if slots is None else _i32(slots),
                             lens=None if lens is None else _i32(lens), err_out=err, stream=_stream())
            want = np.zeros(kv.shape)
            for u in range(units):
                for j, b in enumerate(blocks[u]):
                    if b >= 0:
                        left = 64 if lens is None else min(max(lens[u] - 64 * b, 0), 64)
                        want[u, j, :, :left] = values[u, b if slots is None else slots[u, j]][:, :left]
            want = torch.from_numpy(want).float().to(torch.bfloat16)
            assert torch.equal(torch.nan_to_num(kv.cpu(), 99.0), torch.nan_to_num(want, 99.0))
            assert err.item() == 0
    kv = torch.empty((units, 5, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    N.nosa_byte_read(st, units, nb, None, 5, kv, stream=_stream())
    assert torch.equal(torch.nan_to_num(kv.cpu(), 99.0), torch.nan_to_num(torch.from_numpy(values).float().to(torch.bfloat16), 99.0))


@pytest.mark.parametrize("blocks,slots", [([[0, 5]], None), ([[1, 0]], [[0, -1]]), ([[9, 1]], [[0, 5]])])
def test_read_rows_outside_are_flagged(blocks, slots):
    rng = np.random.default_rng(22)
    st = torch.from_numpy(_filled(rng, 1, 5)).cuda()
    kv = torch.full((1, 2, 2, 64, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N.nosa_byte_read(st, 1, 5, _i32(blocks), 2, kv, slots=None if slots is None else _i32(slots), err_out=err, stream=_stream())
    assert err.item() == 1 and (kv[0, 1] == 0).all() and (kv[0, 0] != 0).any()


# ------------------------------------------------------------------------------------------ attention
def _expect(q, k, v, at, length, nq, scale):
    """The oracle's result and masses of one unit, and how far the kernels' may be from them.

    With p_t a row's weights, o its result and S_t = scale sum |q| |k_t|: a logit is a float32 sum and a few products, in
    some twenty steps of 2^-24 at most of S_t, taken as 2^-18 S_t, and with more than 8 rows small values of q are off
    by 2^-21 of the row's largest, Q (two e4m3 codes a value): 2^-21 Q scale sum |k_t|; it moves a weight by as much, relative.  A weight that
    multiplies V is rounded to f16, 2^-11, or is off by 2^-35 of the row's largest where it is small.  These are
    independent from token to token: with e_t the sum of both, V = sum (p_t e_t v_t)^2 + (p_t 2^-18 S_t o)^2 is at
    least three times the error's variance, so six roots of V is more than ten standard deviations, and more than the
    sum of all for three dozen tokens.  Float32 sums over a warp's 32 tokens at a time: 2^-24 of sum p |v| per step,
    at most one per half block and twenty more.  The result to bf16: 2^-8.
    A mass has float32 weights (2^-21: exponential, reference, sum) and their logits, numerator and denominator."""
    out, mass = O.attend(q, k, v, at, length, nq, scale)
    token = np.asarray(at)[:, None] * 64 + np.arange(64)
    tol, off = np.zeros(out.shape), np.zeros(mass.shape)
    kk, vv, seen = k.reshape(-1, 128), v.reshape(-1, 128), (np.asarray(at)[:, None] >= 0) & (token >= 0)
    for r in range(q.shape[0]):
        see = (seen & (token < length - (nq - 1 - r % nq))).reshape(-1)
        if not see.any():
            continue
        z = kk[see] @ q[r] * scale
        p = np.exp(z - z.max())
        p /= p.sum()
        d = 2.0 ** -18 * (np.abs(kk[see]) @ np.abs(q[r])) * scale
        if q.shape[0] > 8:
            d += 2.0 ** -21 * np.abs(q[r]).max() * np.abs(kk[see]).sum(1) * scale
        x, o = vv[see], out[r]
        var = ((p * (2.0 ** -11 + d))[:, None] * x) ** 2 + ((p * d)[:, None] * o) ** 2
        steps = see.sum() / 32 + 20
        tol[r] = (2.0 ** -8 * np.abs(o) + 1.01 * 6 * np.sqrt(var.sum(0)) + 2.0 ** -35 * p.max() * np.abs(x).sum(0)
                  + 2.0 ** -24 * steps * (p @ np.abs(x)))
        each = np.zeros(see.shape)
        each[see] = p * (2.0 ** -21 + 1.01 * (d + p @ d))
        off += each.reshape(-1, 64).sum(1)
    return out, mass, tol, off


def _attend(q, store, lens, group, nq, nb, *, sel=None, slots=None, max_len=None, scale=0.0, mass=True, scratch=None):
    """q [units, rows, 128] bf16; the result, the masses and the error word."""
    units, rows = q.shape[:2]
    blocks = sel.shape[1] if sel is not None else -(-max_len // 64)
    if scratch is None:
        scratch = torch.zeros(N.nosa_byte_scratch_bytes(units, rows, blocks, mass), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    m = torch.full((units, blocks), 7.0, dtype=torch.float32, device="cuda") if mass else None
    kw = dict(mass=m, softmax_scale=scale, stream=_stream())
    if sel is None:
        N.nosa_byte_dense_attend(q, store, units, group, nq, nb, lens, max_len, out, scratch, scratch.numel(), **kw)
    else:
        N.nosa_byte_attend(q, store, sel, slots, units, group, nq, nb, sel.shape[1], lens, out, scratch, scratch.numel(), **kw)
    torch.cuda.synchronize()
    return out, m, int(scratch[:4].view(torch.int32).item())


def _check(q, store, lens, group, nq, nb, *, units=None, sel=None, slots=None, max_len=None, scale=0.0, err=0):
    """Compares the units listed (all by default) with the oracle; returns the result and the masses."""
    st, ln = torch.from_numpy(store).cuda(), _i32(lens)
    s, sl = (None if x is None else _i32(x) for x in (sel, slots))
    out, mass, word = _attend(q, st, ln, group, nq, nb, sel=s, slots=sl, max_len=max_len, scale=scale)
    again, none, _ = _attend(q, st, ln, group, nq, nb, sel=s, slots=sl, max_len=max_len, scale=scale, mass=False)
    assert none is None and torch.equal(out.view(torch.int16), again.view(torch.int16))  # the masses change nothing
    assert word == err
    got, gm, qq = _f64(out), _f64(mass), _f64(q)
    for u in range(q.shape[0]) if units is None else units:
        at = np.arange(-(-max_len // 64)) if sel is None else np.asarray(sel[u])
        rows = at if slots is None else np.asarray(slots[u])
        at = np.where((at >= 0) & (rows >= 0) & (rows < nb), at, -1)
        k, v = O.unpack(store[u, np.where(at >= 0, rows, 0)])
        ref, m, tol, off = _expect(qq[u], k, v, at, max(lens[u], 0), nq, scale or 1 / math.sqrt(128))
        assert np.array_equal(np.isnan(got[u]), np.isnan(ref)), u
        assert (np.abs(got[u] - ref) <= tol)[~np.isnan(ref)].all(), (u, np.nanmax(np.abs(got[u] - ref) / (tol + 1e-30)))
        assert np.array_equal(np.isnan(gm[u]), np.isnan(m)), u
        assert (np.abs(gm[u] - m) <= off)[~np.isnan(m)].all(), (u, np.nanmax(np.abs(gm[u] - m) / (off + 1e-30)))
    return out, mass


def _queries(rng, units, rows):
    q = rng.standard_normal((units, rows, 128))
    return torch.from_numpy(q / np.linalg.norm(q, axis=-1, keepdims=True) * math.sqrt(128)).to(torch.bfloat16).cuda()


# units, blocks a unit: how CTAs share them (few units with a cluster each, a wave of them, pieces, a unit a CTA, more than one)
PLANS = {"cluster": (6, 24), "wave": (100, 12), "pieces": (12, 130), "units-in-pieces": (200, 40), "unit-a-cta": (152, 9),
         "rounds": (310, 5), "many": (2100, 2)}
FORMS = [(1, 1), (8, 1), (3, 2), (1, 9), (8, 2), (1, 17), (7, 3), (8, 4), (1, 32)]  # q heads and query tokens of a unit: 1 to 32 rows


@pytest.fixture(scope="module")
def many_blocks():
    """Blocks to build stores from (packing them anew for every test would take minutes)."""
    return _filled(np.random.default_rng(31), 1, 400)[0]


def _store(rng, many_blocks, units, nb):
    return many_blocks[rng.integers(0, len(many_blocks), (units, nb))]


def _some(units):
    return sorted({0, 1, 2, 3, units // 2, units - 1})


def _lengths(units, nb, nq):
    """Ragged lengths: all of it, none, one token, fewer than the query tokens, and odd ones."""
    n = (np.linspace(0.1, 1.0, units) * 64 * nb).astype(np.int64) | 1
    n[:4] = [64 * nb, 0, 1, max(nq - 1, 1)]
    return np.minimum(n, 64 * nb)


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("plan", PLANS)
def test_dense_in_every_form(plan, group, nq, many_blocks):
    units, nb = PLANS[plan]
    rng = np.random.default_rng(units + group + nq)
    store = _store(rng, many_blocks, units, nb)
    lens = _lengths(units, nb, nq)
    for u in _some(units):  # behind the context there may be anything
        tail = store[u, max(lens[u], 0) // 64:]
        i = lens[u] % 64
        if len(tail):
            tail[0, np.concatenate([O.AT["k"][i:].ravel(), O.AT["v"][i:].ravel()])] = 0x7F
            tail[1:] = 0xFF
            if i == 0:
                tail[0] = 0xFF
    _check(_queries(rng, units, group * nq), store, lens, group, nq, nb, units=_some(units), max_len=64 * nb)


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("plan", PLANS)
def test_listed_in_every_form(plan, group, nq, many_blocks):
    units, n = PLANS[plan]
    nb = 2 * n
    rng = np.random.default_rng(7 * units + group + nq)
    store = _store(rng, many_blocks, units, nb)
    lens = _lengths(units, nb, nq)
    sel = np.argsort(rng.random((units, nb)), 1)[:, :n].astype(np.int32)  # in no order, some behind the context
    sel[:, 0] = np.maximum(lens - 1, 0) // 64                             # the last block in any case
    sel[rng.random((units, n)) < 0.1] = -1
    sel[units // 2] = -1                                                  # a unit without a block
    sel[units - 1, -1] = sel[units - 1, 0]                                # a block twice
    _check(_queries(rng, units, group * nq), store, lens, group, nq, nb, units=_some(units), sel=sel)


def test_listed_through_slots(many_blocks):
    rng = np.random.default_rng(41)
    units, nb, n = 5, 20, 300  # more than one batch of the list
    store = _store(rng, many_blocks, units, nb)
    sel = rng.integers(-1, 2000, (units, n)).astype(np.int32)
    slots = rng.integers(0, nb, (units, n)).astype(np.int32)
    lens = [64 * 2000, 64 * 1500 + 3, 5, 0, 2 ** 31 - 1]
    sel[4, 0], slots[4, 0] = 33554431, 3  # the block of the last of int32's positions
    _check(_queries(rng, units, 8), store, lens, 8, 1, nb, sel=sel, slots=slots)
    slots[0, 5], slots[1, 7], sel[0, 5], sel[1, 7] = nb, -1, 3, 4  # rows outside are left out and flagged
    _check(_queries(rng, units, 8), store, lens, 8, 1, nb, sel=sel, slots=slots, err=1)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129])
@pytest.mark.parametrize("group,nq", [(4, 1), (2, 3), (8, 4)])
def test_short_lengths(n, group, nq, many_blocks):
    rng = np.random.default_rng(n)
    store = _store(rng, many_blocks, 4, 3)
    _check(_queries(rng, 4, group * nq), store, [n, n + 1, n - 1, 0], group, nq, 3, max_len=n + 1)


def test_lengths_out_of_range_are_clamped_and_flagged(many_blocks):
    rng = np.random.default_rng(3)
    store, q = _store(rng, many_blocks, 3, 4), _queries(rng, 3, 4)
    st = torch.from_numpy(store).cuda()
    out, mass, err = _attend(q, st, _i32([300, -5, 100]), 4, 1, 4, max_len=200)
    want, wm, _ = _attend(q, st, _i32([200, 0, 100]), 4, 1, 4, max_len=200)
    assert err == 1 and torch.equal(out, want) and torch.equal(mass, wm) and not out[1].any() and not mass[1].any()
    sel = _i32(np.tile(np.arange(4), (3, 1)))
    out, mass, err = _attend(q, st, _i32([200, -5, 100]), 4, 1, 4, sel=sel)
    assert err == 1 and torch.allclose(out.float(), want.float(), rtol=2 ** -7, atol=1e-3) and not mass[1].any()


def test_nan_in_drafted_tokens_reaches_only_the_rows_that_see_them(many_blocks):
    rng = np.random.default_rng(5)
    units, nb, group, nq = 3, 4, 4, 8
    store = _store(rng, many_blocks, units, nb)
    lens = [200, 192 + 3, 130]
    for u, n in enumerate(lens):
        for j, d in ((1, 5), (3, 127), (6, 0)):  # the j-th last tokens' V; the fifth last's K
            t = n - j
            store[u, t // 64, O.AT["v"][t % 64, d]] = 0xFF if j == 3 else 0x7F
        t = n - 5
        store[u, t // 64, O.AT["k"][t % 64, 64]] = 0x7F
    _check(_queries(rng, units, group * nq), store, lens, group, nq, nb, max_len=64 * nb)


def test_blocks_of_very_different_scales(many_blocks):
    """V scales from 2^-100 to 2^100 in one sequence, each in true units; K scales that set logits far apart."""
    rng = np.random.default_rng(8)
    units, nb = 4, 12
    store = _store(rng, many_blocks, units, nb)
    for b in range(nb):
        for u, (ks, vs) in enumerate([(2.0 ** -8, 2.0 ** rng.integers(-100, 100)), (2.0 ** (b % 5 - 8), 2.0 ** -6),
                                      (2.0 ** rng.integers(-20, -8), 2.0 ** rng.integers(-12, 12)), (0.0, 0.0)]):
            store[u, b, O.SCALES:O.SCALES + 8] = np.array([ks, vs], np.float32).view(np.uint8)
    _check(_queries(rng, units, 8), store, [64 * nb - 5] * units, 8, 1, nb, max_len=64 * nb)


@pytest.mark.parametrize("ks", [2.0 ** -118, 2.0 ** -30, 2.0 ** 6, 2.0 ** 20, 2.0 ** 60, 2.0 ** 119])
@pytest.mark.parametrize("scale", [1e-30, 1.0, 2.0 ** 21, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27, 2.0 ** 28, 2.0 ** 29, 2.0 ** 33, 1e30, 3e38])
def test_logits_of_any_size(ks, scale, many_blocks):
    """A token that stands out by far has all the weight; logits that cannot be told apart share it."""
    rng = np.random.default_rng(9)
    store = _store(rng, many_blocks, 2, 6)
    store[..., O.SCALES:O.SCALES + 4] = np.array([ks], np.float32).view(np.uint8)
    q = _queries(rng, 2, 8)
    out, mass, err = _attend(q, torch.from_numpy(store).cuda(), _i32([384, 377]), 8, 1, 6, max_len=384, scale=scale)
    got, gm, qq = _f64(out), _f64(mass), _f64(q)
    assert err == 0 and np.isfinite(got).all() and np.isfinite(gm).all()
    for u, n in enumerate([384, 377]):
        k, v = (x.reshape(-1, 128)[:n] for x in O.unpack(store[u]))
        for r in range(8):
            z = (k @ qq[u, r]) * scale
            spread = np.abs(k) @ np.abs(qq[u, r]) * scale
            if spread.max() < 2.0 ** -12:  # equal weights
                o = v.mean(0)
            else:
                order = np.argsort(z)
                if z[order[-1]] - z[order[-2]] < 2.0 ** -17 * spread.max() + 40:
                    continue
                o = v[order[-1]]
            assert (np.abs(got[u, r] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(v).max()).all()


def test_rows_of_q_that_are_not_finite_or_tiny_or_zero(many_blocks):
    rng = np.random.default_rng(10)
    store = _store(rng, many_blocks, 2, 3)
    q = _queries(rng, 2, 8)
    q[0, 1] = 0
    q[0, 2] *= 2.0 ** -120
    q[0, 3] *= 2.0 ** 100
    q[0, 4, 100] = math.inf
    q[0, 5, 3] = math.nan
    q[0, 6, 17] = 1e4  # one value far above the others
    st = torch.from_numpy(store).cuda()
    out, mass, err = _attend(q, st, _i32([150, 150]), 8, 1, 3, max_len=192)
    assert torch.isnan(out[0, 4:6]).all() and not torch.isnan(out[0, [0, 1, 2, 3, 6, 7]]).any() and torch.isnan(mass[0]).all()
    assert err == 0 and not torch.isnan(out[1]).any() and not torch.isnan(mass[1]).any()
    k, v = (x.reshape(-1, 128)[:150] for x in O.unpack(store[0]))
    for r in (1, 2):
        assert (np.abs(_f64(out)[0, r] - v.mean(0)) <= 2.0 ** -8 * np.abs(v.mean(0)) + 2.0 ** -10 * np.abs(v).max()).all()
    q[0, 3:6] = 1.0
    _check(q, store, [150, 0], 8, 1, 3, max_len=192)
    q[1, 2, 5] = math.nan  # a row that sees nothing is zeros whatever it holds
    out, mass, _ = _attend(q, st, _i32([150, 0]), 8, 1, 3, max_len=192)
    assert not out[1].any() and not mass[1].any()


def test_long_context_and_64_bit_offsets():
    """One unit of 300,000 tokens in a store whose rows go past 4 GiB, values repeated so that the oracle stays small."""
    rng = np.random.default_rng(15)
    nb = 2 ** 32 // BB + 40
    blocks = _filled(rng, 1, 7)[0]
    store = torch.from_numpy(blocks).cuda().repeat(nb // 7 + 1, 1)[:nb].contiguous()
    q = _queries(rng, 1, 8)
    n = 4688
    sel = torch.arange(nb - n, nb, dtype=torch.int32, device="cuda")[None].contiguous()
    out, mass, err = _attend(q, store, _i32([64 * nb]), 8, 1, nb, sel=sel)
    k, v = (np.concatenate([x] * (n // 7 + 2))[:n + 7] for x in O.unpack(blocks))
    first = (nb - n) % 7
    k, v = k[first:first + n], v[first:first + n]
    ref, m, tol, off = _expect(_f64(q)[0], k, v, np.arange(n), 64 * n, 1, 1 / math.sqrt(128))
    assert err == 0 and (np.abs(_f64(out)[0] - ref) <= tol).all() and (np.abs(_f64(mass)[0] - m) <= off).all()
    assert abs(_f64(mass).sum() - 8) < 1e-4


# ------------------------------------------------------------------------------------------ how it is called
def test_scratch_is_monotone_bounded_and_enough(many_blocks):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for mass in (False, True):
        last = 0
        for units, rows, blocks in [(1, 1, 1), (1, 1, 100), (2, 3, 100), (100, 8, 100), (200, 8, 100), (200, 32, 500), (3000, 32, 500)]:
            n = N.nosa_byte_scratch_bytes(units, rows, blocks, mass)
            assert last <= n <= 512 + 536 * rows * (units + 16 * sms) + (16 * (rows + 1) * units * blocks if mass else 0)
            last = n
    assert N.nosa_byte_scratch_bytes(4, 8, 10, True) > N.nosa_byte_scratch_bytes(4, 8, 10)
    for bad in [(0, 8, 10), (4, 0, 10), (4, 33, 10), (4, 8, 0), (4, 8, 16385), (1 << 18, 8, 1 << 13)]:
        assert N.nosa_byte_scratch_bytes(*bad) == 0
    rng = np.random.default_rng(1)
    store, q = torch.from_numpy(_store(rng, many_blocks, 4, 9)).cuda(), _queries(rng, 4, 8)
    need = N.nosa_byte_scratch_bytes(4, 8, 9, True)
    out, mass = torch.empty_like(q), torch.empty(4, 9, device="cuda")
    scratch = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    lens = _i32([500] * 4)
    with pytest.raises(N.NosaError) as e:
        N.nosa_byte_dense_attend(q, store, 4, 8, 1, 9, lens, 576, out, scratch, need - 1, mass=mass, stream=_stream())
    assert e.value.status == N.NOSA_ERR_CAPACITY
    N.nosa_byte_dense_attend(q, store, 4, 8, 1, 9, lens, 576, out, scratch, need, mass=mass, stream=_stream())
    torch.cuda.synchronize()
    assert (scratch[need:] == 0xA5).all()


def test_scratch_of_the_largest_call_serves_smaller_ones_and_its_bytes_do_not_matter(many_blocks):
    rng = np.random.default_rng(2)
    scratch = torch.randint(0, 256, (N.nosa_byte_scratch_bytes(160, 32, 130, True),), dtype=torch.uint8, device="cuda")
    for units, nb, group, nq in [(160, 20, 8, 4), (12, 130, 8, 1), (3, 5, 1, 1), (12, 130, 8, 4)]:
        store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group * nq)
        lens = _i32(_lengths(units, nb, nq)) if units > 4 else _i32([300] * units)
        scratch[:4] = 0
        a = _attend(q, store, lens, group, nq, nb, max_len=64 * nb, scratch=scratch)
        b = _attend(q, store, lens, group, nq, nb, max_len=64 * nb)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] == b[2] == 0


def test_neighbours_and_inputs_are_left_alone(many_blocks):
    rng = np.random.default_rng(4)
    units, nb, rows = 5, 6, 3
    store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, rows)
    before, qb = store.clone(), q.clone()
    out = torch.full((units + 2, rows, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mass = torch.full((units + 2, nb), 7.0, device="cuda")
    scratch = torch.zeros(N.nosa_byte_scratch_bytes(units, rows, nb, True), dtype=torch.uint8, device="cuda")
    N.nosa_byte_dense_attend(q, store, units, rows, 1, nb, _i32([384, 1, 0, 65, 383]), 64 * nb, out[1:], scratch, scratch.numel(),
                             mass=mass[1:], stream=_stream())
    torch.cuda.synchronize()
    assert torch.equal(store, before) and torch.equal(q, qb)
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (mass[0] == 7).all() and (mass[-1] == 7).all()
    assert (out[1:-1] != 7).all() and (mass[1:-1] != 7).all()


def test_replayed_graph_takes_new_lengths_and_runs_beside_another_stream(many_blocks):
    rng = np.random.default_rng(6)
    units, nb, group = 16, 40, 8
    n = 64 * nb
    store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group)
    k, v = _bf16(rng, units, 1, 128), _bf16(rng, units, 1, 128)
    lens, pos = _i32([100] * units), _i32([99] * units)
    need = N.nosa_byte_scratch_bytes(units, group, nb, True)
    scratch = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out, mass = torch.empty_like(q), torch.empty(units, nb, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream().cuda_stream
        N.nosa_byte_append(k, v, store, units, 1, nb, pos=pos, stream=s)
        N.nosa_byte_dense_attend(q, store, units, group, 1, nb, lens, n, out, scratch[0], need, mass=mass, stream=s)
    for length in (100, 1, 777, n):
        lens.fill_(length)
        pos.fill_(length - 1)
        torch.cuda.synchronize()
        graph.replay()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):  # a call of its own, with its own scratch, at the same time
            o2, m2 = torch.empty_like(q), torch.empty(units, nb, device="cuda")
            N.nosa_byte_dense_attend(q, store, units, group, 1, nb, _i32([50] * units), n, o2, scratch[1], need, mass=m2,
                                     stream=other.cuda_stream)
        torch.cuda.synchronize()
        ref, rm, err = _attend(q, store, lens, group, 1, nb, max_len=n)
        assert err == 0 and torch.equal(out, ref) and torch.equal(mass, rm)
        ref, rm, _ = _attend(q, store, _i32([50] * units), group, 1, nb, max_len=n)
        if length - 1 >= 50:  # (the append did not touch what that call attended)
            assert torch.equal(o2, ref) and torch.equal(m2, rm)


def test_the_same_call_gives_the_same_bits(many_blocks):
    rng = np.random.default_rng(16)
    for units, nb, group, nq in [(12, 130, 8, 1), (6, 24, 8, 4), (310, 5, 4, 1)]:
        store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group * nq)
        lens = _i32(_lengths(units, nb, nq))
        runs = [_attend(q, store, lens, group, nq, nb, max_len=64 * nb) for _ in range(5)]
        for out, mass, _ in runs[1:]:
            assert torch.equal(out, runs[0][0]) and torch.equal(mass, runs[0][1])


@pytest.mark.parametrize("group,nq", [(8, 1), (8, 2), (8, 4)])
@pytest.mark.parametrize("plan", ["cluster", "pieces", "rounds"])
@pytest.mark.parametrize("listed", [False, True])
def test_a_wait_that_gives_up_is_reported(plan, group, nq, listed, many_blocks):
    units, nb = PLANS[plan]
    rng = np.random.default_rng(17)
    store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group * nq)
    lens = np.full(units, 64 * nb)
    sel = _i32(np.tile(np.arange(nb), (units, 1))) if listed else None
    call = lambda: _attend(q, store, _i32(lens), group, nq, nb, sel=sel, max_len=64 * nb)  # noqa: E731
    N.nosa_debug_quant_wait(-1)
    try:
        out, mass, err = call()
    finally:
        N.nosa_debug_quant_wait(0)
    assert err == 2
    assert torch.isnan(out).all() and torch.isnan(mass).all()
    out, mass, err = call()
    assert err == 0 and torch.isfinite(out).all() and torch.isfinite(mass).all()


@pytest.mark.parametrize("nq", range(1, 33))
def test_any_number_of_rows(nq, many_blocks):
    rng = np.random.default_rng(nq)
    store = _store(rng, many_blocks, 2, 3)
    _check(_queries(rng, 2, nq), store, [150, nq - 1], 1, nq, 3, max_len=160)


def test_calls_from_two_threads_on_their_own_streams(many_blocks):
    import threading
    rng = np.random.default_rng(18)
    cases, errors = [], []
    for units, nb, group, nq in [(12, 130, 8, 1), (16, 40, 8, 4)]:
        store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group * nq)
        lens = _i32(_lengths(units, nb, nq))
        cases.append((q, store, lens, group, nq, nb, _attend(q, store, lens, group, nq, nb, max_len=64 * nb)))
    torch.cuda.synchronize()

    def work(case):
        try:
            q, store, lens, group, nq, nb, want = case
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out, mass, err = _attend(q, store, lens, group, nq, nb, max_len=64 * nb)
                    assert err == 0 and torch.equal(out, want[0]) and torch.equal(mass, want[1])
        except BaseException as e:  # noqa: BLE001 - handed to the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_first_calls_may_be_made_under_capture():
    """A process whose first use of the store, of eviction and of rotary positions is inside a graph capture."""
    code = """
import torch
from offloadable_block_sparse_gb300 import nosa as N
k = torch.randn(3, 70, 128, device="cuda").to(torch.bfloat16)
q, w = (torch.randn(3, r, 128, device="cuda").to(torch.bfloat16) for r in (8, 32))
store = torch.zeros(3, 2, 16512, dtype=torch.uint8, device="cuda"); lens = torch.full((3,), 70, dtype=torch.int32, device="cuda")
kv = torch.empty(3, 2, 2, 64, 128, dtype=torch.bfloat16, device="cuda"); sel = torch.tensor([[0, 1]] * 3, dtype=torch.int32, device="cuda")
a, b, c = torch.empty_like(q), torch.empty_like(q), torch.empty_like(w)
m, acc, sc = torch.empty(3, 2, device="cuda"), torch.zeros(3, 2, device="cuda"), torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
turned, back = torch.empty_like(k), torch.empty_like(k)
t = N.nosa_rope_make()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s = torch.cuda.current_stream().cuda_stream
    N.nosa_rope(t, [(k[:, None], turned[:, None])], stream=s)
    N.nosa_rope(t, [(turned[:, None], back[:, None])], inverse=True, stream=s)
    N.nosa_byte_append(k, k, store, 3, 70, 2, stream=s)
    N.nosa_byte_read(store, 3, 2, None, 2, kv, lens=lens, stream=s)
    N.nosa_byte_dense_attend(q, store, 3, 8, 1, 2, lens, 70, a, sc, sc.numel(), stream=s)
    N.nosa_byte_attend(q, store, sel, None, 3, 8, 1, 2, 2, lens, b, sc, sc.numel(), mass=m, stream=s)
    N.nosa_byte_attend(w, store, sel, None, 3, 8, 4, 2, 2, lens, c, sc, sc.numel(), stream=s)
    N.nosa_evict(acc, sel, m, 3, 2, lens, 1, 0, 0, 1.0, acc, sel, stream=s)
g.replay()
torch.cuda.synchronize()
x = kv[:, :, 0].reshape(3, 128, 128)
assert (x[:, :70].float() - k.float()).abs().max() < 0.3 and not x[:, 70:].any()
assert torch.isfinite(a).all() and a.any() and (a.float() - b.float()).abs().max() < 0.1 and torch.isfinite(c).all() and c.any()
assert (m.sum(1) - 8).abs().max() < 1e-3 and (sel == -1).sum() == 3 and (acc > 0).sum() == 3
assert (back.float() - k.float()).abs().max() < 0.1 and not torch.equal(turned, k)
print("ok")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
