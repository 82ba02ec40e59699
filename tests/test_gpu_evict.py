"""Eviction and rotary positions on the GPU against their float64 oracle (oracle/byte_oracle.py), and a run of them with
the 8-bit store as a decode loop would use them."""
import math

import numpy as np
import pytest

from oracle import byte_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _i32(values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


def _table(rng, units, slots, blocks, fill=1.0):
    """A slot table of distinct blocks below `blocks`, about a share `fill` of the rows held."""
    blk = np.full((units, slots), -1, np.int32)
    for u in range(units):
        n = min(int(round(fill * slots)), blocks)
        blk[u, rng.permutation(slots)[:n]] = rng.permutation(blocks)[:n]
    return blk


# ------------------------------------------------------------------------------------------ eviction
def _evict_check(acc, blk, mass, lens, budget, sink, window, decay, nxt=None, inplace=False):
    units, slots = blk.shape
    a, b = torch.from_numpy(acc).cuda(), torch.from_numpy(blk).cuda()
    ao, bo = (a, b) if inplace else (torch.full_like(a, 7.0), torch.full_like(b, 7))
    row = torch.full((units,), 7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N.nosa_evict(a, b, None if mass is None else torch.from_numpy(mass).cuda(), units, slots,
                 None if lens is None else _i32(lens), budget, sink, window, decay, ao, bo,
                 next_block=None if nxt is None else _i32(nxt), next_slot=row, err_out=err, stream=_stream())
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", over="ignore"):
        ra, rb, rr, flag = O.evict(acc, blk, mass, lens, budget, sink, window, decay, nxt)
    assert np.array_equal(bo.cpu().numpy(), rb), np.argwhere(bo.cpu().numpy() != rb)[:4]
    assert np.array_equal(ao.cpu().numpy(), ra)  # the same two float32 roundings
    assert np.array_equal(row.cpu().numpy(), rr) and err.item() == 4 * flag
    if not inplace:
        assert np.array_equal(a.cpu().numpy(), acc, equal_nan=True) and np.array_equal(b.cpu().numpy(), blk)


@pytest.mark.parametrize("slots", [1, 2, 31, 128, 129, 256, 257, 1025, 2048, 2049, 16384])
@pytest.mark.parametrize("goal", ["step", "quarter", "none", "all"])
def test_evict_takes_the_oracles_rows(slots, goal):
    rng = np.random.default_rng(slots)
    units = 7
    blk = _table(rng, units, slots, 2 * slots + 40, 0.9 if goal == "none" else 1.0)
    acc, mass = (np.exp(2 * rng.standard_normal((units, slots))).astype(np.float32) for _ in range(2))
    budget = {"step": slots, "quarter": (slots + 3) // 4, "none": slots, "all": 0}[goal]
    top = blk.max(1) + 1
    nxt = np.where(np.arange(units) % 3 == 0, -1, np.where(np.arange(units) % 3 == 1, top, blk[:, 0]))
    lens = 64 * top + np.arange(units) * 9
    for inplace in (False, True):
        _evict_check(acc, blk, mass, lens, budget, 1, min(16, slots // 2), 0.97, nxt, inplace)


def test_evict_equal_weights_fall_by_block():
    rng = np.random.default_rng(2)
    blk = _table(rng, 6, 300, 1000)
    acc = rng.integers(0, 3, (6, 300)).astype(np.float32)
    acc[2:4] = 0.0
    acc[3, ::2] = -0.0  # equal to 0
    for budget in (299, 298, 150, 7, 0):
        _evict_check(acc, blk, None, None, budget, 0, 0, 1.0)


def test_evict_odd_weights():
    rng = np.random.default_rng(3)
    blk = _table(rng, 5, 64, 100)
    acc = rng.standard_normal((5, 64)).astype(np.float32)
    acc[0, ::3], acc[1, ::4], acc[2, ::5] = np.nan, np.inf, 1e-45
    mass = rng.random((5, 64)).astype(np.float32)
    mass[3, ::3], mass[4, ::3] = np.nan, 3e38
    acc[4, ::3] = 3e38
    for decay in (0.0, 0.5, 1.0, 3.0):
        for budget in (64, 63, 40, 3):
            _evict_check(acc, blk, mass, [6400] * 5, budget, 2, 5, decay, [100] * 5)


def test_evict_protected_blocks_stay():
    blk = np.array([[0, 1, 5, 6, 7, -1], [0, 1, 2, 9, 8, 7]], np.int32)
    acc = np.zeros((2, 6), np.float32)
    _evict_check(acc, blk, None, [512, 640], 1, 2, 3, 1.0, [8, 10])      # only what may go goes
    _evict_check(acc, blk, None, [512, 640], 0, 100, 0, 1.0, [8, 10])    # nothing may: no row for the second unit
    _evict_check(acc, blk, None, [512, 640], 0, 0, 100, 1.0, [8, 9])
    _evict_check(acc, blk, None, [0, -5], 0, 0, 0, 1.0, [8, 10])         # blocks behind the context are the window's
    _evict_check(acc, blk, None, None, 0, 0, 0, 1.0, [8, 9])
    _evict_check(acc, np.full((2, 6), -3, np.int32), None, [512, 640], 0, 0, 0, 1.0, [8, -9])
    _evict_check(acc, blk, None, [2 ** 31 - 1] * 2, 3, 0, 1, 1.0, [33554431, 33554431])


def test_evict_rows_with_the_same_block():
    rng = np.random.default_rng(7)
    blk = rng.integers(-1, 40, (6, 200)).astype(np.int32)
    acc = rng.permutation(1200).reshape(6, 200).astype(np.float32)
    nxt = [int(blk[0].max()), 41, -1, 3, 44, int(blk[5, 5])]
    for budget in (200, 199, 198, 90, 1):
        _evict_check(acc, blk, None, [2560] * 6, budget, 1, 2, 0.5, nxt)
    for budget in (3, 2):  # one or two rows have to go: of equal weights all three of block 9 do
        b = torch.tensor([[4, 9, 9, 9]], dtype=torch.int32, device="cuda")
        a = torch.ones(1, 4, device="cuda")
        N.nosa_evict(a, b, None, 1, 4, None, budget, 0, 0, 1.0, a, b, stream=_stream())
        assert b.tolist() == [[4, -1, -1, -1]] and a.tolist() == [[1, 0, 0, 0]]


def test_evict_without_optional_outputs_and_many_units():
    rng = np.random.default_rng(5)
    units, slots = 3000, 40
    blk = _table(rng, units, slots, 90)
    acc = rng.random((units, slots)).astype(np.float32)
    a, b = torch.from_numpy(acc).cuda(), torch.from_numpy(blk).cuda()
    N.nosa_evict(a, b, None, units, slots, None, 11, 0, 0, 1.0, a, b, stream=_stream())
    ra, rb, _, _ = O.evict(acc, blk, None, None, 11, 0, 0, 1.0)
    assert np.array_equal(b.cpu().numpy(), rb) and np.array_equal(a.cpu().numpy(), ra)


# ------------------------------------------------------------------------------------------ rotary positions
def _rope_check(x, y, kw, pos, count=None, inverse=False, rows=None):
    """One tensor against the oracle; what lies behind a sequence's tokens must be left as it was.

    Angles are off by 2^-25 of a turn's half at most (an integer's rounding to float32) and by the sine's and cosine's own
    errors, 2 units of 2^-24; two products and a sum in float32 add 2^-23 of |x| + |x'|; the result to bf16 2^-8."""
    t = N.nosa_rope_make(**kw)
    n = x.shape[2]
    before, xin = y.clone(), x.double().cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N.nosa_rope(t, [(x, y)], pos=None if pos is None else _i32(pos), count=None if count is None else _i32(count),
                inverse=inverse, err_out=err, stream=_stream())
    torch.cuda.synchronize()
    f = O.frequencies(t.rot_dims, **{k: v for k, v in kw.items() if k not in ("rot_dims", "interleaved", "attention_factor")})
    factor = float(np.float32(kw.get("attention_factor", 1.0)))
    p = np.zeros(x.shape[0]) if pos is None else np.asarray(pos)
    want = O.rope(xin, p, f, kw.get("interleaved", False), factor, inverse)
    got, old = y.double().cpu().numpy(), before.double().cpu().numpy()
    c = np.full(x.shape[0], n) if count is None else np.clip(count, 0, n)
    # the largest |x| of a row bounds |x| + |x'| by half; float64's own angle: |p f| 2^-52, the table's 2^-54 |p|
    big = np.abs(xin).max(-1, keepdims=True)
    far = (np.abs(p).reshape(-1, 1, 1, 1) + n) * 2.0 ** -50
    tol = 2.0 ** -8 * np.abs(want) + 2 * big * factor * (math.pi * 2.0 ** -25 + 2.0 ** -22 + far)
    for b in range(x.shape[0]):
        assert (np.abs(got[b, :, :c[b]] - want[b, :, :c[b]]) <= tol[b, :, :c[b]]).all(), b
        assert np.array_equal(got[b, :, c[b]:], old[b, :, c[b]:])
    r = t.rot_dims
    assert all(np.array_equal(got[b, :, :c[b], r:], xin[b, :, :c[b], r:]) for b in range(x.shape[0]))
    assert err.item() == int(count is not None and (np.asarray(count) != c).any())
    return y


def _values(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [2, 6, 16, 48, 64, 96, 112, 126, 128])
def test_rope_parts_of_the_head(rot, interleaved):
    rng = np.random.default_rng(rot)
    for batch, heads, n in [(1, 1, 1), (3, 5, 70), (2, 33, 9), (1, 64, 3)]:
        x = _values(rng, batch, heads, n, 128)
        kw = dict(rot_dims=rot, interleaved=interleaved)
        pos = rng.integers(0, 100000, batch)
        out = _rope_check(x, torch.full_like(x, 7.0), kw, pos)
        same = _rope_check(x, x.clone(), kw, pos)
        assert torch.equal(out, same)
        N.nosa_rope(N.nosa_rope_make(**kw), [(x, x)], pos=_i32(pos), stream=_stream())  # in place
        assert torch.equal(x, out)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling=N.NOSA_ROPE_LINEAR, factor=4.0), dict(scaling=N.NOSA_ROPE_BASE, factor=8.0),
                                     dict(scaling=N.NOSA_ROPE_PARTS, factor=8.0, original=8192.0, attention_factor=1.21),
                                     dict(base=5e6, attention_factor=0.5)])
def test_rope_scalings_at_far_positions(scaling):
    rng = np.random.default_rng(1)
    x = _values(rng, 6, 2, 5, 128)
    _rope_check(x, torch.empty_like(x).fill_(7.0), scaling, [0, 1, 131071, 1048573, 2 ** 31 - 6, -3])
    _rope_check(x, torch.empty_like(x).fill_(7.0), scaling, None)


@pytest.mark.parametrize("rot", [64, 62, 128])
def test_rope_strides_counts_and_alignment(rot):
    rng = np.random.default_rng(rot)
    kw = dict(rot_dims=rot, base=500000.0)
    flat = _values(rng, 3, 40, 7, 128)                       # [sequence][token][head][dim]
    x = flat.transpose(1, 2)
    y = torch.full((3, 7, 40, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    pos, count = [5, 90000, 33], [40, 0, 17]
    a = _rope_check(x, y, kw, pos, count)
    b = _rope_check(x, torch.full_like(flat, 7.0).transpose(1, 2), kw, pos, count)
    assert torch.equal(a, b)
    _rope_check(x, torch.full_like(flat, 7.0).transpose(1, 2), kw, pos, [41, -1, 40])
    wide = torch.full((3 * 7 * 40 * 131 + 1,), 7.0, dtype=torch.bfloat16, device="cuda")[1:]  # rows at odd values
    z = wide.as_strided((3, 7, 40, 128), (7 * 40 * 131, 40 * 131, 131, 1))
    c = _rope_check(x, z, kw, pos, count)
    assert torch.equal(c, a) and (wide.as_strided((3, 7, 40, 3), (7 * 40 * 131, 40 * 131, 131, 1), wide.storage_offset() + 128) == 7).all()
    d = _rope_check(c, y.clone(), kw, pos)                   # and read from there
    assert torch.equal(d, _rope_check(c.contiguous(), y.clone(), kw, pos))
    one = x[:1, :1].expand(3, 7, 40, 128)                    # a broadcast input
    _rope_check(one, torch.full_like(y, 7.0), kw, pos)


def test_rope_of_odd_values():
    rng = np.random.default_rng(8)
    x = _values(rng, 1, 2, 64, 128)
    x[0, 0, 3, 5], x[0, 0, 4, 6], x[0, 1, 60, 0] = math.nan, math.inf, 3e38
    x[0, 1, 7] = 1e-40
    x[0, 1, 8] = 0.0
    y = torch.empty_like(x)
    N.nosa_rope(N.nosa_rope_make(), [(x, y)], stream=_stream())
    bad = ~torch.isfinite(y)
    assert bad[0, 0, 3, [5, 69]].all() and bad[0, 0, 4, [6, 70]].all() and bad.sum() <= 6 and not y[0, 1, 8].any()


def test_rope_two_tensors_at_once_and_past_32_bit_offsets():
    rng = np.random.default_rng(9)
    t = N.nosa_rope_make(rot_dims=128, base=500000.0)
    q, k = _values(rng, 2, 40, 33, 128), _values(rng, 2, 3, 33, 128)
    pos, count = _i32([1000, 7]), _i32([33, 20])
    one = [torch.zeros_like(q), torch.zeros_like(k)]
    two = [torch.zeros_like(q), torch.zeros_like(k)]
    N.nosa_rope(t, [(q, one[0]), (k, one[1])], pos=pos, count=count, stream=_stream())
    for x, y in zip((q, k), two):
        N.nosa_rope(t, [(x, y)], pos=pos, count=count, stream=_stream())
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1]) and one[0][1, :, 19].any() and not one[0][1, :, 20:].any()
    big = torch.empty(3 * 2 ** 30 + 4 * 128, dtype=torch.bfloat16, device="cuda")  # rows 2^31 values apart and more
    x = big.as_strided((2, 1, 2, 128), (3 * 2 ** 30, 128, 128, 1))
    x.copy_(q[:, :1, :2])
    y = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    N.nosa_rope(t, [(x, y)], pos=pos, stream=_stream())
    want = torch.zeros_like(y)
    N.nosa_rope(t, [(q[:, :1, :2].contiguous(), want)], pos=pos, stream=_stream())
    assert torch.equal(y, want)


def test_rope_inverse_is_the_gradient():
    """d/dx of sum(g rope(x)) is rope's inverse applied to g: against the formula, and against differences of the forward
    rotation, which is linear: (rope(x + h e_j) - rope(x)) . g / h with h of x's size."""
    rng = np.random.default_rng(10)
    for kw in (dict(rot_dims=64, interleaved=True, attention_factor=1.3), dict()):
        g = _values(rng, 1, 1, 4, 128)
        dx = _rope_check(g, torch.empty_like(g), kw, [777], inverse=True)
        t = N.nosa_rope_make(**kw)
        basis = torch.eye(128, dtype=torch.bfloat16, device="cuda").view(1, 128, 1, 128).expand(1, 128, 4, 128).contiguous()
        turned = torch.empty_like(basis)
        N.nosa_rope(t, [(basis, turned)], pos=_i32([777]), stream=_stream())
        slope = torch.einsum("jtd,td->tj", turned[0].double(), g[0, 0].double())
        # a basis vector has two values, each off by 2^-8 of itself; the gradient by 2^-8 of itself
        tol = 2.0 ** -8 * (dx[0, 0].double().abs() + torch.einsum("jtd,td->tj", turned[0].double().abs(), g[0, 0].double().abs())) + 1e-5
        assert ((dx[0, 0].double() - slope).abs() <= tol).all()


# ------------------------------------------------------------------------------------------ together
def _decode(steps, slots, budget, graph, seed=0):
    """A prompt, then `steps` tokens of 2 sequences (2 kv heads, 4 query heads each): rotate, place, append, attend with
    masses.  Returns what the oracle needs: every step's inputs and outputs."""
    rng = np.random.default_rng(seed)
    B, Hk, G, U = 2, 2, 4, 4
    prompt = [700, 451]
    t = N.nosa_rope_make(base=500000.0)
    store = torch.zeros((U, slots, N.NOSA_BYTE_BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    acc, blk = torch.zeros((U, slots), device="cuda"), torch.full((U, slots), -1, dtype=torch.int32, device="cuda")
    for u in range(U):
        nb = -(-prompt[u // Hk] // 64)
        blk[u, torch.from_numpy(rng.permutation(slots)[:nb]).cuda()] = torch.arange(nb, dtype=torch.int32, device="cuda")
    iota = torch.arange(slots, dtype=torch.int32, device="cuda").repeat(U, 1)
    mass = torch.zeros((U, slots), device="cuda")
    row = torch.zeros(U, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = N.nosa_byte_scratch_bytes(U, G, slots, True)
    scratch = torch.zeros(need, dtype=torch.uint8, device="cuda")
    n = max(prompt)
    x = _values(rng, B, n, Hk + 1, 128)  # k heads of the prompt's projection (and one that is not used)
    kp, vp = torch.zeros((B, Hk, n, 128), dtype=torch.bfloat16, device="cuda"), _values(rng, B, Hk, n, 128)
    counts = _i32(prompt)
    N.nosa_rope(t, [(x[:, :, :Hk].transpose(1, 2), kp)], count=counts, stream=_stream())
    N.nosa_byte_append(kp, vp, store, U, n, slots, count=counts.repeat_interleave(Hk), slot_blk=blk, err_out=err, stream=_stream())
    first = dict(kp=kp.double().cpu().numpy(), vp=vp.double().cpu().numpy(), blk=blk.cpu().numpy(), prompt=prompt)
    xs = _values(rng, steps, B, 1, (G + 1) * Hk, 128)
    vs = _values(rng, steps, B, Hk, 1, 128)
    x, v = xs[0].clone(), vs[0].clone()
    q, k = torch.zeros((B, G * Hk, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, Hk, 1, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((U, G, 128), dtype=torch.bfloat16, device="cuda")
    pos, lens, nxt = counts.clone(), counts.repeat_interleave(Hk), torch.zeros(U, dtype=torch.int32, device="cuda")

    def step():
        s = torch.cuda.current_stream().cuda_stream
        torch.div(lens, 64, rounding_mode="floor", out=nxt)  # the block of the token at position `lens`
        lens.add_(1)
        N.nosa_rope(t, [(x[:, :, :G * Hk].transpose(1, 2), q), (x[:, :, G * Hk:].transpose(1, 2), k)], pos=pos, stream=s)
        N.nosa_evict(acc, blk, mass, U, slots, lens, budget, 1, 2, 0.9, acc, blk, next_block=nxt, next_slot=row, err_out=err, stream=s)
        N.nosa_byte_append(k, v, store, U, 1, slots, pos=pos.repeat_interleave(Hk), slot_blk=blk, err_out=err, stream=s)
        N.nosa_byte_attend(q, store, blk, iota, U, G, 1, slots, slots, lens, out, scratch, need, mass=mass, stream=s)
        pos.add_(1)

    run = step
    if graph:
        saved = [z.clone() for z in (acc, blk, mass, pos, lens, store)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        for z, s in zip((acc, blk, mass, pos, lens, store), saved):
            z.copy_(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    log = []
    for i in range(steps):
        x.copy_(xs[i])
        v.copy_(vs[i])
        run()
        torch.cuda.synchronize()
        log.append([z.clone() for z in (q, k, v, out, mass, acc, blk, row)])
    assert err.item() == 0 and int(scratch[:4].view(torch.int32).item()) == 0
    return first, log


def test_a_decode_loop_with_everything():
    slots, budget, steps = 13, 12, 150
    first, log = _decode(steps, slots, budget, graph=False)
    U, G, Hk = 4, 4, 2
    store = np.zeros((U, slots, O.BLOCK_BYTES), np.uint8)
    blk, acc, mass = first["blk"], np.zeros((U, slots), np.float32), np.zeros((U, slots), np.float32)
    n = first["kp"].shape[2]
    pos = np.repeat(first["prompt"], Hk)
    O.append(store, first["kp"].reshape(U, n, 128), first["vp"].reshape(U, n, 128), [0] * U, pos, blk)
    gone = 0
    for q, k, v, out, m, a, b, row in log:
        before = (blk >= 0).sum()
        acc, blk, want_row, flag = O.evict(acc, blk, mass, pos + 1, budget, 1, 2, 0.9, pos // 64)
        assert not flag and np.array_equal(b.cpu().numpy(), blk) and np.array_equal(a.cpu().numpy(), acc)
        assert np.array_equal(row.cpu().numpy(), want_row) and (blk >= 0).sum(1).max() <= budget
        assert not O.append(store, *(z.double().cpu().numpy().reshape(U, 1, 128) for z in (k, v)), pos, [1] * U, blk)
        pos = pos + 1
        mass = m.cpu().numpy()  # the next step's weights are the kernel's own, so that ranks agree to the last bit
        gone += before - (blk >= 0).sum() + int((row.cpu().numpy() >= 0).sum() and (pos % 64 == 1).sum())
        for u in range(U):
            kk, vv = O.unpack(store[u])
            ref, rm = O.attend(q.double().cpu().numpy().reshape(U, G, 128)[u], kk, vv, blk[u], pos[u], 1, 1 / math.sqrt(128))
            # the bounds that test_gpu_byte.py counts, at their largest here: weights 2^-11 + 2^-12, the result 2^-8
            assert (np.abs(out[u].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * np.abs(vv).max()).all()
            assert np.abs(mass[u] - rm).max() <= 2.0 ** -12
    assert gone > 0


def test_a_captured_decode_loop_is_the_eager_one():
    eager, graph = (_decode(70, 13, 12, graph=g)[1] for g in (False, True))
    for a, b in zip(eager, graph):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
