"""The 4-bit KV block store on the GPU against its float64 oracle (oracle/quant_oracle.py): the bytes
that nosa_quant_append writes and the bf16 blocks that nosa_quant_read gives are compared for equality,
the attention within bounds counted from its roundings (see _tolerance)."""
import math

import numpy as np
import pytest

from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402

BB = N.NOSA_QUANT_BLOCK_BYTES


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ append
def _append_check(k, v, nb, pos, count, seed=0, use_err=True):
    """Appends into a store of random bytes and compares every byte; returns the error word."""
    units = k.shape[0]
    rng = np.random.default_rng(seed)
    before = rng.integers(0, 256, (units, nb, BB), dtype=np.uint8)
    store = torch.from_numpy(before).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    N.nosa_quant_append(k, v, store, units, k.shape[1], nb, pos=None if pos is None else _i32(pos),
                        count=None if count is None else _i32(count), err_out=err if use_err else None, stream=_stream())
    torch.cuda.synchronize()
    ref = before.copy()
    flag = Q.append(ref, _f64(k), _f64(v), [0] * units if pos is None else pos,
                    [k.shape[1]] * units if count is None else count)
    got = store.cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    if use_err:
        assert int(err.item()) == int(flag)
    return int(err.item())


@pytest.mark.parametrize("n,pos,count", [
    (1, [0, 63, 64, 190], None),              # single tokens
    (1, [15, 16, 17, 100], [1, 0, 1, 1]),     # one unit writes nothing
    (2, [15, 31, 62, 63], None),              # two tokens over a tile's, a block's edge
    (37, [0, 5, 16, 150], [37, 36, 1, 0]),    # ragged starts and counts
    (64, None, None), (65, None, [65, 64, 17, 2]), (191, [1, 0, 1, 1], None), (192, None, None),
], ids=["one", "one-masked", "edges", "ragged", "block", "block+1", "odd", "full"])
def test_append_writes_the_oracles_bytes(n, pos, count):
    rng = np.random.default_rng(n)
    _append_check(_bf16(rng, 4, n, 128), _bf16(rng, 4, n, 128), 3, pos, count, seed=n)


def test_append_out_of_range_is_flagged_and_left_out():
    rng = np.random.default_rng(5)
    k, v = _bf16(rng, 6, 20, 128), _bf16(rng, 6, 20, 128)
    assert _append_check(k, v, 2, [-7, 120, 128, 1 << 30, -(1 << 31), 3], [20, 20, 1, 20, 20, 20]) == 1
    assert _append_check(k, v, 2, [0] * 6, [21, -1, 5, 0, 20, 1 << 30]) == 1
    assert _append_check(k, v, 2, [0] * 6, [20] * 6) == 0
    _append_check(k, v, 2, [-7] * 6, [21] * 6, use_err=False)


def _odd_groups():
    """Rows of 128 values whose groups are where quantising can go wrong."""
    g = np.zeros((12, 4, 32))
    rng = np.random.default_rng(9)
    g[0] = rng.integers(-40, 40, (4, 32)) * 0.5                    # many exact ties
    g[1, 0], g[1, 1], g[1, 2], g[1, 3] = 3.0, -2.5, 0.0, -0.0        # constant
    g[2] = np.where(np.arange(32) % 2, 15.0, np.arange(32) * 0.5)    # s = 1, ties
    g[3] = rng.standard_normal((4, 32)) * 1e-6                       # s below f16's normal range
    g[4] = rng.standard_normal((4, 32)) * 1e-9                       # s rounds to zero
    g[5] = rng.standard_normal((4, 32)) * 2e4                        # near f16's range
    g[6] = rng.standard_normal((4, 32)) * 1e6                        # minimum beyond it
    g[7] = np.abs(rng.standard_normal((4, 32))) * 4e5                # range beyond it, minimum within
    g[8] = rng.standard_normal((4, 32))
    g[8, 0, 3], g[8, 1, 31], g[8, 2, 0] = np.nan, np.inf, -np.inf
    g[9, :, 7] = 1.0                                                # one spike
    g[10] = 100 + rng.standard_normal((4, 32)) * 0.5                 # small range on a large offset
    g[11] = rng.standard_normal((4, 32)) * 3e38                      # range overflows float32
    return torch.from_numpy(g.reshape(12, 128)).float().to(torch.bfloat16).cuda()


def test_append_odd_groups():
    x = _odd_groups()
    k = x.repeat(2, 1).view(1, 24, 128).contiguous()
    v = x.flip(0).repeat(2, 1).view(1, 24, 128).contiguous()
    _append_check(k, v, 1, [7], None)


def test_append_batch_of_many_units_and_long_prompt():
    rng = np.random.default_rng(11)
    _append_check(_bf16(rng, 300, 1, 128), _bf16(rng, 300, 1, 128), 2, rng.integers(0, 128, 300).tolist(), None)
    k, v = _bf16(rng, 1, 4100, 128), _bf16(rng, 1, 4100, 128)
    store = torch.full((1, 65, BB), 0xA5, dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(k, v, store, 1, 4100, 65, stream=_stream())
    torch.cuda.synchronize()
    got = store.cpu().numpy()
    whole = Q.pack(_f64(k)[0, :4096].reshape(64, 64, 128), _f64(v)[0, :4096].reshape(64, 64, 128))
    assert np.array_equal(got[0, :64], whole)
    tail = np.full((1, 1, BB), 0xA5, np.uint8)
    Q.append(tail, _f64(k)[:, 4096:], _f64(v)[:, 4096:], [0], [4])
    assert np.array_equal(got[0, 64], tail[0, 0])


def test_append_and_read_past_32_bit_offsets():
    nb = 2 ** 32 // BB + 3  # the last blocks of the first unit start beyond 4 GiB
    store = torch.zeros((2, nb, BB), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    k, v = _bf16(rng, 2, 70, 128), _bf16(rng, 2, 70, 128)
    pos = [64 * nb - 70, 64 * nb - 75]
    N.nosa_quant_append(k, v, store, 2, 70, nb, pos=_i32(pos), stream=_stream())
    kv = torch.empty((2, 2, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    blocks = torch.tensor([[nb - 2, nb - 1]] * 2, dtype=torch.int32, device="cuda")
    N.nosa_quant_read(store, 2, nb, blocks, 2, kv, stream=_stream())
    torch.cuda.synchronize()
    ref = np.zeros((2, 2, BB), np.uint8)
    Q.append(ref, _f64(k), _f64(v), [p - 64 * (nb - 2) for p in pos], [70, 70])
    assert np.array_equal(store[:, nb - 2:].cpu().numpy(), ref)
    kk, vv, _, _ = Q.unpack(ref.reshape(-1, BB))
    want = torch.from_numpy(np.stack((kk, vv), 1).reshape(2, 2, 2, 64, 128)).float().to(torch.bfloat16)
    assert torch.equal(kv.cpu(), want)


# -------------------------------------------------------------------------------------------- read
def _random_store(units, nb, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((2, units * nb, 64, 128)) * scale
    to = lambda x: torch.from_numpy(x).float().to(torch.bfloat16).double().numpy()  # noqa: E731
    return Q.pack(to(k), to(v)).reshape(units, nb, BB)


@pytest.mark.parametrize("units,nb,n_blocks", [(1, 1, 1), (3, 5, 5), (7, 9, 4), (2, 3, 11)])
def test_read_gives_the_oracles_blocks(units, nb, n_blocks):
    store = _random_store(units, nb, units)
    rng = np.random.default_rng(nb)
    lens = rng.integers(0, 64 * nb + 1, units)
    lens[0] = 64 * nb
    blocks = rng.integers(-1, nb, (units, n_blocks)).astype(np.int32)  # repeats and padding
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.from_numpy(store).cuda()
    for use_blocks in (True, False):
        if not use_blocks and n_blocks > nb:
            continue
        for use_lens in (True, False):
            ids = blocks if use_blocks else np.broadcast_to(np.arange(n_blocks), blocks.shape)
            kv = torch.full((units, n_blocks, 2, 64, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
            N.nosa_quant_read(d, units, nb, torch.from_numpy(blocks).cuda() if use_blocks else None, n_blocks, kv,
                              lens=_i32(lens) if use_lens else None, err_out=err, stream=_stream())
            torch.cuda.synchronize()
            ref = np.zeros((units, n_blocks, 2, 64, 128))
            for u in range(units):
                for j, b in enumerate(ids[u]):
                    if b >= 0:
                        k, v, _, _ = Q.unpack(store[u, b][None])
                        at = 64 * b + np.arange(64)
                        keep = (at < lens[u]) if use_lens else np.ones(64, bool)
                        ref[u, j, 0], ref[u, j, 1] = k[0] * keep[:, None], v[0] * keep[:, None]
            # n s + m fits 32 bits before its one rounding to bf16 unless the terms are 2^8 apart
            want = torch.from_numpy(ref).float().to(torch.bfloat16)
            assert torch.equal(kv.cpu(), want)
    assert int(err.item()) == 0


def test_read_ignores_what_lies_behind_the_length_and_flags_bad_blocks():
    store = torch.full((2, 2, BB), 0xFF, dtype=torch.uint8, device="cuda")  # every scale is a NaN
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = torch.full((2, 3, 2, 64, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    blocks = torch.tensor([[0, 1, -5], [1, 2, 1 << 30]], dtype=torch.int32, device="cuda")
    N.nosa_quant_read(store, 2, 2, blocks, 3, kv, lens=_i32([3, -4]), err_out=err, stream=_stream())
    torch.cuda.synchronize()
    got = kv.cpu()
    assert int(err.item()) == 1
    assert got[0, 0, :, :3].isnan().all()  # the tokens there are
    got[0, 0, :, :3] = 0
    assert (got == 0).all()


def test_odd_groups_read_back():
    x = _odd_groups()
    store = torch.zeros((1, 1, BB), dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(x.view(1, 12, 128), x.flip(0).contiguous().view(1, 12, 128), store, 1, 12, 1, stream=_stream())
    kv = torch.empty((1, 1, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
    N.nosa_quant_read(store, 1, 1, None, 1, kv, lens=_i32([12]), stream=_stream())
    torch.cuda.synchronize()
    for got, src in ((kv[0, 0, 0, :12], x), (kv[0, 0, 1, :12], x.flip(0))):
        want = torch.from_numpy(Q.values(*Q.quantise(_f64(src)))).float().to(torch.bfloat16)
        got = got.cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), want.nan_to_num())


# --------------------------------------------------------------------------------------- attention
def _tolerance(ref, q, k, size_k, size_v, seen, scale):
    """Bound of |out - ref| for one unit's row r over the tokens it sees.

    Each weight is rounded to f16 (2^-11) and so is its product with s (2^-11); the softmax sum is that of
    the rounded weights: together 2^-9 of the largest |n s| + |m| covers numerator and denominator.
    Logits: sums of 128 products in float32 (each addition 2^-24 at most 2^-23 of what it adds up, over
    8 steps of 16 and 4 groups): delta = 2^-18 sum |q| (|n s| + |m|) scale, which moves a weight by 2 delta.
    Weights are at least 2^10 at the maximum, and f16 has an absolute error of 2^-25 below 2^-14:
    (15 + 1) 2^-35 (1 + s) a token, taken as 2^-30 (1 + |v|).  Rounding to bf16: 2^-8 of the result."""
    out = np.zeros_like(ref)
    for r in range(q.shape[0]):
        i = seen[r]
        if i.any():
            top = size_v[i].max()
            delta = 2.0 ** -18 * (size_k[i] @ np.abs(q[r])).max() * scale
            out[r] = 2.0 ** -8 * np.abs(ref[r]) + top * (2.0 ** -9 + 4 * delta) + i.sum() * 2.0 ** -30 * (1 + top)
    return out


def _queries(rng, units, group, nq):
    q = rng.standard_normal((units, group, nq, 128))
    q *= math.sqrt(128) / np.linalg.norm(q, axis=-1, keepdims=True)
    return torch.from_numpy(q).float().to(torch.bfloat16).cuda()


def _scratch(units, rows, blocks):
    n = N.nosa_quant_scratch_bytes(units, rows, blocks)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert 256 <= n <= 256 + 520 * rows * (units + 16 * sms)
    return torch.zeros(n, dtype=torch.uint8, device="cuda"), n


def _dense(q, store, lens, max_len, scale=0.0, scratch=None, out=None):
    units, group, nq = q.shape[:3]
    sc, n = scratch or _scratch(units, group * nq, -(-max_len // 64))
    out = torch.full_like(q, float("nan")) if out is None else out
    N.nosa_quant_dense_attend(q, store, units, group, nq, store.shape[1], lens, max_len, out, sc, n,
                              softmax_scale=scale, stream=_stream())
    return out, sc


def _sparse(q, store, sel, slot, lens, scale=0.0):
    units, group, nq = q.shape[:3]
    sc, n = _scratch(units, group * nq, sel.shape[1])
    out = torch.full_like(q, float("nan"))
    N.nosa_quant_attend(q, store, sel, slot, units, group, nq, store.shape[1], sel.shape[1], lens, out, sc, n,
                        softmax_scale=scale, stream=_stream())
    return out, sc


def _check_unit(got, q, blocks, at, length, nq, scale):
    """One unit: got, q [group, nq, 128]; blocks uint8 [n, 10240] and their tokens' positions at [n, 64]."""
    k, v, sk, sv = (x.reshape(-1, 128) for x in Q.unpack(blocks))
    at = at.reshape(-1)
    rows = q.reshape(-1, 128)
    late = nq - 1 - np.arange(rows.shape[0]) % nq
    seen = (at[None] < (length - late)[:, None]) & (at[None] >= 0)
    ref = Q.attend(rows, k, v, seen, scale)
    tol = _tolerance(ref, rows, k, sk, sv, seen, scale)
    err = np.abs(got.reshape(-1, 128) - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err.max(), tol.max())
    assert not got.reshape(-1, 128)[~seen.any(1)].any()  # a row that sees nothing is zero


@pytest.mark.parametrize("units,group,nq,nb,lens", [
    (1, 1, 1, 1, [1]), (2, 8, 1, 1, [0, 64]), (3, 8, 1, 5, [300, 1, 17]), (2, 3, 1, 3, [16, 15]),
    (4, 4, 1, 40, [2560, 2559, 33, 0]), (2, 8, 2, 6, [384, 129]), (3, 8, 4, 9, [576, 3, 2]),
    (2, 5, 3, 4, [1, 255]), (2, 1, 32, 3, [20, 190]), (2, 7, 4, 4, [0, 4]), (1, 8, 1, 130, [8303]),
    (40, 2, 1, 7, [11 * i for i in range(40)]), (2, 4, 8, 33, [2100, 2101]),
], ids=lambda x: str(x) if not isinstance(x, list) else str(len(x)))
def test_dense_attention(units, group, nq, nb, lens):
    host = _random_store(units, nb, units + 7 * nb)
    store = torch.from_numpy(host).cuda()
    # behind each length the store holds what a NaN scale and any code look like
    for u, n in enumerate(lens):
        for b in range(n // 64, nb):
            for i in range(max(n - 64 * b, 0), 64):
                tile, r = 2560 * (i // 16), i % 16
                store[u, b, tile + 2048 + 16 * r:tile + 2064 + 16 * r] = 0xFF
                for which in (0, 1):
                    for gr in range(4):
                        p = tile + Q.scale_place("v", which, r, gr)
                        store[u, b, p:p + 2] = 0xFF
    q = _queries(np.random.default_rng(nb), units, group, nq)
    for scale in (0.0, 0.5):
        out, sc = _dense(q, store, _i32(lens), max(max(lens), 1), scale=scale)
        torch.cuda.synchronize()
        assert int(sc[:4].view(torch.int32).item()) == 0
        for u in range(units):
            at = np.arange(64 * nb).reshape(nb, 64)
            _check_unit(_f64(out[u]), _f64(q[u]), host[u], at, lens[u], nq, scale or 1 / math.sqrt(128))


def test_dense_attention_long_contexts_in_many_chunks():
    units, nb = 2, 1100
    host = _random_store(units, nb, 4)
    store = torch.from_numpy(host).cuda()
    q = _queries(np.random.default_rng(1), units, 8, 1)
    lens = [70000, 35003]
    out, _ = _dense(q, store, _i32(lens), 64 * nb)
    again, _ = _dense(q, store, _i32(lens), 70000)
    torch.cuda.synchronize()
    for u in range(units):
        for got in (out, again):
            _check_unit(_f64(got[u]), _f64(q[u]), host[u], np.arange(64 * nb).reshape(nb, 64), lens[u], 1, 1 / math.sqrt(128))


@pytest.mark.parametrize("group,nq", [(8, 1), (4, 1), (8, 4), (5, 2)])
def test_sparse_attention(group, nq):
    units, nb, most = 5, 23, 9
    host = _random_store(units, nb, 31)
    store = torch.from_numpy(host).cuda()
    rng = np.random.default_rng(8)
    q = _queries(rng, units, group, nq)
    lens = [64 * nb, 64 * nb - 5, 700, 2, 0]
    sel = np.full((units, most), -1, np.int32)
    for u in range(units):
        n = [most, 7, 4, most, 3][u]
        sel[u, rng.permutation(most)[:n]] = rng.permutation(nb)[:n]  # any order, padding anywhere
    sel[1, 0] = sel[1, 1] = (lens[1] - 1) // 64  # the last, partial block twice
    sel[3, 2] = 0                                # two tokens among blocks behind the context
    slot = np.array([rng.permutation(nb)[:most] for _ in range(units)], np.int32)
    for slots in (None, slot):
        out, sc = _sparse(q, store, torch.from_numpy(sel).cuda(), None if slots is None else torch.from_numpy(slots).cuda(),
                          _i32(lens))
        torch.cuda.synchronize()
        assert int(sc[:4].view(torch.int32).item()) == 0
        for u in range(units):
            keep = sel[u] >= 0
            rows = sel[u][keep] if slots is None else slots[u][keep]
            at = sel[u][keep][:, None] * 64 + np.arange(64)
            _check_unit(_f64(out[u]), _f64(q[u]), host[u, rows], at, lens[u], nq, 1 / math.sqrt(128))


def test_attention_out_of_range_is_flagged():
    host = _random_store(2, 3, 1)
    store = torch.from_numpy(host).cuda()
    q = _queries(np.random.default_rng(1), 2, 8, 1)
    out, sc = _dense(q, store, _i32([150, -3]), 100)  # taken as 100 and 0
    torch.cuda.synchronize()
    assert int(sc[:4].view(torch.int32).item()) == 1
    at = np.arange(192).reshape(3, 64)
    for u, n in ((0, 100), (1, 0)):
        _check_unit(_f64(out[u]), _f64(q[u]), host[u], at, n, 1, 1 / math.sqrt(128))
    sel = torch.tensor([[0, 3, 1], [2, 1 << 30, -1]], dtype=torch.int32, device="cuda")  # 3: no such row
    out, sc = _sparse(q, store, sel, None, _i32([192, 192]))
    torch.cuda.synchronize()
    assert int(sc[:4].view(torch.int32).item()) == 1
    for u, keep in ((0, [0, 1]), (1, [2])):
        _check_unit(_f64(out[u]), _f64(q[u]), host[u, keep], at[keep], 192, 1, 1 / math.sqrt(128))


def test_attention_scratch_too_small_is_refused():
    store = torch.from_numpy(_random_store(2, 3, 1)).cuda()
    q = _queries(np.random.default_rng(1), 2, 8, 1)
    n = N.nosa_quant_scratch_bytes(2, 8, 3)
    sc = torch.zeros(n, dtype=torch.uint8, device="cuda")
    with pytest.raises(N.NosaError) as e:
        _dense(q, store, _i32([10, 10]), 192, scratch=(sc, n - 1))
    assert e.value.status == N.NOSA_ERR_CAPACITY
    assert N.nosa_quant_scratch_bytes(0, 8, 3) == 0 and N.nosa_quant_scratch_bytes(2, 33, 3) == 0
    assert N.nosa_quant_scratch_bytes(2, 8, 16385) == 0


@pytest.mark.parametrize("what", ["large-v", "huge-v", "growing", "small-v", "large-q", "tiny-q", "peaked"])
def test_attention_value_ranges(what):
    """Scales beyond 2 (weights x s must stay in f16), maxima that keep growing, tiny and huge queries."""
    rng = np.random.default_rng(17)
    n = 64 * 6
    k, v = rng.standard_normal((2, 1, n, 128))
    q = _f64(_queries(rng, 1, 8, 1))
    if what == "large-v":
        v[:, 150:] *= 60.0
    if what == "huge-v":
        v[:, rng.permutation(n)[:40]] *= 9000.0
    if what == "small-v":
        v *= 1e-4
    if what == "growing":  # keys along the query, ever longer: the logits climb by far more than 2^14 in weight
        k += np.linspace(0, 25, n)[None, :, None] * q[:, 0, 0][:, None] / 4
    if what == "large-q":
        q[:] = 0
        q[..., 0] = 1e30  # logits of 1e29: the tokens with the largest first dim take all
    if what == "tiny-q":
        q *= 1e-30
    if what == "peaked":
        q *= 8
    kd, vd, qd = (torch.from_numpy(x).float().to(torch.bfloat16).cuda() for x in (k, v, q))
    store = torch.zeros((1, 6, BB), dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(kd, vd, store, 1, n, 6, stream=_stream())
    out, _ = _dense(qd, store, _i32([n]), n)
    torch.cuda.synchronize()
    host, got = store.cpu().numpy(), _f64(out[0])
    if what != "large-q":
        _check_unit(got, _f64(qd[0]), host[0], np.arange(n).reshape(6, 64), n, 1, 1 / math.sqrt(128))
        return
    kk, vv, _, _ = Q.unpack(host[0])
    kk, vv = kk.reshape(-1, 128), vv.reshape(-1, 128)
    best = np.nonzero(kk[:, 0] == kk[:, 0].max())[0]  # those that tie share the weight
    ref = vv[best].mean(0)
    assert np.abs(got.reshape(8, 128) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -9 * np.abs(vv[best]).max() * 2


def test_nan_groups_reach_only_the_rows_and_dims_they_should():
    """A NaN in a V group gives NaN in that group's dims for the rows that see the token; a NaN in K gives
    NaN in the whole row; rows that see neither are untouched."""
    rng = np.random.default_rng(23)
    n, nq, group = 100, 4, 2
    k, v = _bf16(rng, 3, n, 128), _bf16(rng, 3, n, 128)
    v[0, 98, 40] = float("nan")   # seen by the last two query tokens; group 1
    k[1, 99, 3] = float("inf")    # seen by the last query token
    v[2, 10, 127] = float("inf")  # seen by all; group 3
    store = torch.zeros((3, 2, BB), dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(k, v, store, 3, n, 2, stream=_stream())
    q = _queries(rng, 3, group, nq)
    out, _ = _dense(q, store, _i32([n] * 3), n)
    torch.cuda.synchronize()
    got = out.cpu()
    bad = torch.zeros((3, group, nq, 128), dtype=torch.bool)
    bad[0, :, 2:, 32:64] = True
    bad[1, :, 3:] = True
    bad[2, :, :, 96:] = True
    assert torch.equal(got.isnan(), bad)
    host = store.cpu().numpy()
    kk, vv, sk, sv = (x.reshape(3, 128, 128) for x in Q.unpack(host.reshape(-1, BB)))
    for u in range(3):
        for i in range(nq):
            seen = np.arange(128)[None] < n - (nq - 1 - i)
            rows = _f64(q[u, :, i])
            ref = Q.attend(rows, np.nan_to_num(kk[u]), np.nan_to_num(vv[u]), np.repeat(seen, group, 0), 1 / math.sqrt(128))
            tol = _tolerance(ref, rows, None, np.nan_to_num(sk[u]), np.nan_to_num(sv[u]), np.repeat(seen, group, 0), 1 / math.sqrt(128))
            err = np.abs(got[u, :, i].double().numpy() - ref)
            ok = ~bad[u, :, i].numpy()
            assert (err[ok] <= tol[ok]).all()


def test_repeated_calls_give_the_same_bits_and_streams_and_graphs_work():
    units, nb = 6, 50
    host = _random_store(units, nb, 12)
    store = torch.from_numpy(host).cuda()
    rng = np.random.default_rng(2)
    q = _queries(rng, units, 8, 1)
    lens = _i32([3200, 3000, 1, 0, 777, 64])
    scratch = _scratch(units, 8, nb)
    first = _dense(q, store, lens, 3200, scratch=scratch)[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = _dense(q, store, lens, 3200, scratch=scratch)[0]
    side.synchronize()
    assert torch.equal(first, second)
    # a decode step captured once: append the token, then attend; lengths and tokens are read on replay
    pos, ln = _i32([3199, 2999, 0, 5, 776, 63]), lens
    k, v = _bf16(rng, units, 1, 128), _bf16(rng, units, 1, 128)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        N.nosa_quant_append(k, v, store, units, 1, nb, pos=pos, stream=_stream())
        _dense(q, store, ln, 3200, scratch=scratch, out=out)
    for step in range(3):
        new = _bf16(rng, 3, units, 1, 128)
        k.copy_(new[0])
        v.copy_(new[1])
        q.copy_(_queries(rng, units, 8, 1))
        pos.copy_(_i32([3197 + step, 2000, 9 + step, step, 100, 0]))
        ln.copy_(pos + 1)
        Q.append(host, _f64(k), _f64(v), pos.tolist(), [1] * units)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(store.cpu().numpy(), host)
        for u in range(units):
            _check_unit(_f64(out[u]), _f64(q[u]), host[u], np.arange(64 * nb).reshape(nb, 64), int(ln[u]), 1, 1 / math.sqrt(128))


def test_a_context_selects_and_the_store_is_attended():
    """The operators as they are used together: a context keeps K/V on the host and selects blocks; the
    prompt and every new token are also written to a 4-bit store on the device, which is attended over
    the selection (nosa_select's own list), in full, and read back into a bf16 cache."""
    torch.cuda.set_device(0)
    B, Hq, Hkv, T0, steps = 2, 16, 2, 1500, 3
    U, G = B * Hkv, Hq // Hkv
    cfg = N.make_config(num_layers=1, batch=B, num_q_heads=Hq, num_kv_heads=Hkv, k_q=4, k_e=6, window_tokens=128,
                        max_context=T0 + steps)
    sizes = N.nosa_query_sizes(cfg)
    cap, nb = sizes.select_slots, sizes.max_blocks
    ctx = N.nosa_create(cfg, _stream())
    try:
        rng = np.random.default_rng(6)
        K, V = _bf16(rng, B, Hkv, T0 + steps, 128), _bf16(rng, B, Hkv, T0 + steps, 128)
        W1 = (rng.standard_normal((Hkv, 128, 128)) / math.sqrt(128)).astype(np.float32)
        W2 = (rng.standard_normal((Hkv, 128)) / math.sqrt(128)).astype(np.float32)
        N.nosa_set_eviction_head(ctx, 0, W1, W2)
        store = torch.zeros((U, nb, BB), dtype=torch.uint8, device="cuda")
        k0, v0 = K[:, :, :T0].contiguous(), V[:, :, :T0].contiguous()
        N.nosa_append_kv(ctx, 0, k0, v0, T0)
        N.nosa_quant_append(k0, v0, store, U, T0, nb, stream=_stream())
        sel = torch.empty((U, cap), dtype=torch.int32, device="cuda")
        host = np.zeros((U, nb, BB), np.uint8)
        Q.append(host, _f64(K).reshape(U, -1, 128), _f64(V).reshape(U, -1, 128), [0] * U, [T0] * U)
        for t in range(steps):
            T = T0 + t + 1
            k, v = K[:, :, T - 1].contiguous(), V[:, :, T - 1].contiguous()
            q = _queries(rng, U, G, 1)
            N.nosa_append_kv(ctx, 0, k, v, 1)
            N.nosa_quant_append(k, v, store, U, 1, nb, pos=_i32([T - 1] * U), stream=_stream())
            N.nosa_select(ctx, 0, q, sel_out=sel)
            lens = _i32([T] * U)
            sparse, sc = _sparse(q, store, sel, None, lens)
            dense, _ = _dense(q, store, lens, 64 * nb)
            kv = torch.empty((U, cap, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
            N.nosa_quant_read(store, U, nb, sel, cap, kv, lens=lens, stream=_stream())
            # the bf16 blocks read back, attended by the bf16 kernel: row i of the cache holds the i-th block
            slots = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(U, 1)
            n_sel = (sel >= 0).sum(1).to(torch.int32)
            plain = torch.empty((U, G, 1, 128), dtype=torch.bfloat16, device="cuda")
            N.nosa_attend_noalloc(q, kv, sel, slots, n_sel, U, G, cap, T, plain, stream=_stream())
            assert N.nosa_sync(ctx) == N.NOSA_OK
            torch.cuda.synchronize()
            new = lambda x: _f64(x).reshape(U, 1, 128)  # noqa: E731
            Q.append(host, new(k), new(v), [T - 1] * U, [1] * U)
            assert np.array_equal(store.cpu().numpy(), host)
            s = sel.cpu().numpy()
            for u in range(U):
                keep = s[u][s[u] >= 0]
                at = keep[:, None] * 64 + np.arange(64)
                _check_unit(_f64(sparse[u]), _f64(q[u]), host[u, keep], at, T, 1, 1 / math.sqrt(128))
                _check_unit(_f64(dense[u]), _f64(q[u]), host[u], np.arange(64 * nb).reshape(nb, 64), T, 1, 1 / math.sqrt(128))
            # the two differ by the rounding of x^ to bf16 (2^-9 of K and V each) and of P to bf16
            assert (sparse.float() - plain.float()).abs().max().item() <= 2e-2
    finally:
        N.nosa_destroy(ctx)


@pytest.mark.parametrize("units,nb,group,nq", [(700, 20, 2, 1), (330, 40, 8, 1), (2100, 3, 1, 1), (400, 12, 4, 5), (310, 30, 8, 2)],
                         ids=["whole", "pieces", "thousands", "32-rows", "16-rows"])
def test_many_units_with_ragged_lengths(units, nb, group, nq):
    """More units than one wave of CTAs, with empty ones among them; pieces that span several units."""
    few = _random_store(8, nb, 77)
    host = np.tile(few, (-(-units // 8), 1, 1))[:units]
    rng = np.random.default_rng(units)
    lens = rng.integers(0, 64 * nb + 1, units)
    lens[::7] = 0
    lens[5] = 64 * nb
    store = torch.from_numpy(host).cuda()
    q = _queries(rng, units, group, nq)
    sel = np.full((units, nb + 3), -1, np.int32)
    for u in range(units):
        sel[u, :nb] = rng.permutation(nb)
    dense, sc = _dense(q, store, _i32(lens), 64 * nb)
    sparse, sc2 = _sparse(q, store, torch.from_numpy(sel).cuda(), None, _i32(lens))  # every block, in any order
    torch.cuda.synchronize()
    assert int(sc[:4].view(torch.int32).item()) == 0 and int(sc2[:4].view(torch.int32).item()) == 0
    at = np.arange(64 * nb).reshape(nb, 64)
    for u in list(range(0, 40)) + list(range(40, units, 37)) + [units - 1]:
        for got in (dense, sparse):
            _check_unit(_f64(got[u]), _f64(q[u]), host[u], at, int(lens[u]), nq, 1 / math.sqrt(128))
    # every unit of both is finite, and the two agree within their roundings to bf16 and f16
    assert torch.isfinite(dense).all() and torch.isfinite(sparse).all()
    assert (dense.float() - sparse.float()).abs().max().item() <= 2 * (2.0 ** -8 + 2.0 ** -9) * 8


@pytest.mark.parametrize("scale,size", [(1e-30, 1e-30), (1e-38, 1.0), (1e30, 1.0), (3e38, 1e30), (0.0, 3e38)])
def test_extreme_scales_give_a_mean_or_the_largest(scale, size):
    """Logits of (almost) zero weigh all tokens alike; logits of any size leave the token with the largest."""
    n = 200
    host = _random_store(1, 4, 3)
    store = torch.from_numpy(host).cuda()
    q = torch.zeros((1, 8, 1, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = size
    out, _ = _dense(q, store, _i32([n]), n, scale=scale)
    torch.cuda.synchronize()
    kk, vv, _, sv = (x.reshape(-1, 128)[:n] for x in Q.unpack(host[0]))
    if scale and scale * size < 1e-3:
        best = np.arange(n)
    else:
        best = np.nonzero(kk[:, 5] == kk[:, 5].max())[0]
        assert best.size == 1
    err = np.abs(_f64(out[0]).reshape(8, 128) - vv[best].mean(0))
    # weights alike: rounding of the products with s (2^-11 of the largest |n s| + |m|) and of the result
    assert (err <= 2.0 ** -8 * np.abs(vv[best].mean(0)) + 2.0 ** -9 * sv.max()).all()


def test_a_selection_of_nothing_gives_zeros():
    store = torch.from_numpy(_random_store(2, 3, 1)).cuda()
    q = _queries(np.random.default_rng(1), 2, 8, 2)
    sel = torch.full((2, 5), -1, dtype=torch.int32, device="cuda")
    sel[1, 3] = 2  # behind the context
    out, sc = _sparse(q, store, sel, None, _i32([192, 100]))
    torch.cuda.synchronize()
    assert not out.any() and int(sc[:4].view(torch.int32).item()) == 0


def test_first_calls_may_be_made_under_capture():
    """A process whose first use of the store is inside a graph capture (nothing is set up before)."""
    code = """
import torch
from offloadable_block_sparse_gb300 import nosa as N
k = torch.randn(3, 70, 128, device="cuda").to(torch.bfloat16); q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
store = torch.zeros(3, 2, 10240, dtype=torch.uint8, device="cuda"); lens = torch.full((3,), 70, dtype=torch.int32, device="cuda")
kv = torch.empty(3, 2, 2, 64, 128, dtype=torch.bfloat16, device="cuda"); sel = torch.tensor([[0, 1]] * 3, dtype=torch.int32, device="cuda")
a, b = torch.empty_like(q), torch.empty_like(q); sc = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s = torch.cuda.current_stream().cuda_stream
    N.nosa_quant_append(k, k, store, 3, 70, 2, stream=s)
    N.nosa_quant_read(store, 3, 2, None, 2, kv, lens=lens, stream=s)
    N.nosa_quant_dense_attend(q, store, 3, 8, 1, 2, lens, 70, a, sc, sc.numel(), stream=s)
    N.nosa_quant_attend(q, store, sel, None, 3, 8, 1, 2, 2, lens, b, sc, sc.numel(), stream=s)
g.replay()
torch.cuda.synchronize()
x = kv[:, :, 0].reshape(3, 128, 128)
assert (x[:, :70].float() - k.float()).abs().max() < 0.6 and not x[:, 70:].any()
assert torch.isfinite(a).all() and a.any() and (a.float() - b.float()).abs().max() < 0.1
print("ok")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("units,group,nq", [(320, 8, 1), (16, 8, 2), (16, 8, 4)], ids=["8-rows", "16-rows", "32-rows"])
def test_long_means_lose_no_more_than_roundings(units, group, nq):
    """65,536 tokens that nearly cancel (a result of 0.006 from values of 1), a unit's tokens in few long sums.

    The error's norm over the result's: rounding to bf16 is at most 2^-8 of each value (2^-9.8 in the mean square);
    a token's weight and its product with s are rounded by 2^-11 at most, independently, so that their errors add up as
    the tokens' values themselves do: sqrt(2 / 3) 2^-11 times the size of a code's part against its value's, 8.7 against
    3.7 in units of s, 2^-10.1.  Together 2^-9; a sum that drifts by 2^-24 of its codes' part a step, 500 steps long, would
    be off by 2^-6."""
    nb = 1024
    one = torch.from_numpy(_random_store(1, nb, 99)).cuda()
    store = one.expand(units, -1, -1).contiguous()
    q = _queries(np.random.default_rng(4), units, group, nq)
    out, _ = _dense(q, store, _i32([64 * nb] * units), 64 * nb)
    torch.cuda.synchronize()
    kk, vv, _, _ = Q.unpack(one[0].cpu().numpy())
    k, v = torch.from_numpy(kk).cuda().view(-1, 128), torch.from_numpy(vv).cuda().view(-1, 128)
    at = torch.arange(64 * nb, device="cuda")
    for u in (0, 3, units - 1):
        for i in range(nq):
            z = (q[u, :, i].double() @ k.T / math.sqrt(128)).masked_fill(at >= 64 * nb - (nq - 1 - i), -math.inf)
            ref = torch.softmax(z, -1) @ v
            assert ((out[u, :, i].double() - ref).norm() / ref.norm()).item() <= 2.0 ** -8


@pytest.mark.parametrize("group,nq", [(8, 1), (8, 2), (8, 4)])
def test_rows_of_q_do_not_touch_each_other(group, nq):
    """A NaN or an infinity in one row of q, and a row of zeros (the mean), leave the other rows as they are."""
    n = 300
    store = torch.from_numpy(_random_store(1, 5, 8)).cuda()
    q = _queries(np.random.default_rng(3), 1, group, nq)
    clean, _ = _dense(q, store, _i32([n]), n)
    clean = clean.clone()
    odd = q.clone()
    odd[0, 1, 0, 7], odd[0, 3, nq - 1, 100], odd[0, 5, 0] = float("nan"), float("inf"), 0
    out, _ = _dense(odd, store, _i32([n]), n)
    torch.cuda.synchronize()
    same = torch.ones((group, nq), dtype=torch.bool)
    same[1, 0] = same[3, nq - 1] = same[5, 0] = False
    assert torch.equal(out[0].cpu()[same], clean[0].cpu()[same])
    assert out[0, 1, 0].isnan().all() and out[0, 3, nq - 1].isnan().all()
    _, vv, _, sv = (x.reshape(-1, 128)[:n - (nq - 1)] for x in Q.unpack(store[0].cpu().numpy()))
    err = np.abs(_f64(out[0, 5, 0]) - vv.mean(0))
    assert (err <= 2.0 ** -8 * np.abs(vv.mean(0)) + 2.0 ** -9 * sv.max()).all()


def test_calls_on_two_streams_with_a_scratch_each():
    """Calls that overlap share nothing but the store: every result is that of the call alone."""
    host = _random_store(12, 60, 5)
    store = torch.from_numpy(host).cuda()
    rng = np.random.default_rng(9)
    work = []
    for nq in (1, 4):
        q = _queries(rng, 12, 8, nq)
        lens = _i32(rng.integers(1, 64 * 60 + 1, 12))
        work.append((q, lens, _scratch(12, 8 * nq, 60), torch.empty_like(q), _dense(q, store, lens, 64 * 60)[0].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(30):
        for s, (q, lens, scratch, out, _) in zip(streams, work):
            with torch.cuda.stream(s):
                out.zero_()
                _dense(q, store, lens, 64 * 60, scratch=scratch, out=out)
        torch.cuda.synchronize()
        for _, _, _, out, alone in work:
            assert torch.equal(out, alone)


def test_attention_past_32_bit_offsets_and_at_the_longest_context():
    nb = 2 ** 32 // BB + 3  # the last blocks of the first unit start beyond 4 GiB
    store = torch.zeros((2, nb, BB), dtype=torch.uint8, device="cuda")
    few = _random_store(2, 2, 6)
    store[:, nb - 2:] = torch.from_numpy(few).cuda()
    q = _queries(np.random.default_rng(1), 2, 8, 1)
    sel = torch.tensor([[nb - 1, nb - 2]] * 2, dtype=torch.int32, device="cuda")
    lens = [64 * nb - 3, 64 * nb - 70]
    out, sc = _sparse(q, store, sel, None, _i32(lens))
    torch.cuda.synchronize()
    assert int(sc[:4].view(torch.int32).item()) == 0
    at = np.arange(64 * (nb - 2), 64 * nb).reshape(2, 64)
    for u in range(2):
        _check_unit(_f64(out[u]), _f64(q[u]), few[u], at, lens[u], 1, 1 / math.sqrt(128))
    del store
    # 1,048,576 tokens: sixteen copies of 65,536, which give what one copy gives
    one = torch.from_numpy(_random_store(1, 1024, 21)).cuda()
    long = one.repeat(1, 16, 1)
    q = _queries(np.random.default_rng(2), 1, 4, 1)
    a, _ = _dense(q, one, _i32([65536]), 65536)
    b, sc = _dense(q, long, _i32([1 << 20]), 1 << 20)
    with pytest.raises(N.NosaError):
        _dense(q, long, _i32([1 << 20]), (1 << 20) + 1, scratch=(sc, sc.numel()))
    torch.cuda.synchronize()
    assert ((a.double() - b.double()).norm() / a.double().norm()).item() <= 2 * 2.0 ** -8  # each as in the test of means
