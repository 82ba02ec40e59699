"""The attention over the 8-bit store at the ends of what the store, the queries and the lists may hold, with 8, 16 and 32
query rows a unit: the kernel of up to 8 rows and both forms of the one for more."""
import math

import numpy as np
import pytest

from oracle import byte_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402
from tests.test_gpu_byte import (_attend, _expect, _f64, _i32, _lengths, _queries, _some, _store,  # noqa: E402
                                 many_blocks)  # noqa: F401 (a fixture)

FORMS = [(8, 1), (8, 2), (8, 4)]  # q heads and query tokens of a unit
WAVE = 2 * torch.cuda.get_device_properties(0).multi_processor_count  # CTAs that are resident at once
# units, blocks a unit: a cluster a unit, equal pieces of few and of many units, a CTA a unit
PLANS = {"cluster": (6, 24), "pieces": (12, 130), "pieces-of-units": (WAVE + 16, 40), "unit-a-cta": (2 * WAVE, 5)}


def _set_scales(store, ks=None, vs=None):
    """Replaces blocks' scales: ks, vs broadcast over [units][blocks]."""
    for x, at in ((ks, O.SCALES), (vs, O.SCALES + 4)):
        if x is not None:
            s = np.ascontiguousarray(np.broadcast_to(np.asarray(x, np.float32), store.shape[:2]))
            store[..., at:at + 4] = s[..., None].view(np.uint8)


def _check(q, store, lens, group, nq, *, units=None, sel=None, slots=None, max_len=None, scale=0.0):
    """Compares the units listed (all by default) with the oracle within _expect's bounds; returns the result and the masses.

    One term more for a mass: it is a float32 sum of 2 rows terms (a half block's sum times two factors, a row at a time)
    by multiply-add.  All are positive, so no partial sum is above the mass, and each step rounds by at most 2^-24 of it:
    2 rows 2^-24 of the mass.  _expect's 2^-21 has room for that with random roundings, not with rows whose terms are all
    equal and round the same way."""
    nb, rows = store.shape[1], group * nq
    st, ln = torch.from_numpy(store).cuda(), _i32(lens)
    s, sl = (None if x is None else _i32(x) for x in (sel, slots))
    out, mass, err = _attend(q, st, ln, group, nq, nb, sel=s, slots=sl, max_len=max_len, scale=scale)
    again, _, _ = _attend(q, st, ln, group, nq, nb, sel=s, slots=sl, max_len=max_len, scale=scale, mass=False)
    assert err == 0 and torch.equal(out.view(torch.int16), again.view(torch.int16))
    got, gm, qq = _f64(out), _f64(mass), _f64(q)
    for u in range(q.shape[0]) if units is None else units:
        at = np.arange(-(-max_len // 64)) if sel is None else np.asarray(sel[u])
        row = at if slots is None else np.asarray(slots[u])
        k, v = O.unpack(store[u, np.where(at >= 0, row, 0)])
        ref, m, tol, off = _expect(qq[u], k, v, at, lens[u], nq, scale or 1 / math.sqrt(128))
        assert np.isfinite(got[u]).all() and np.isfinite(gm[u]).all()
        assert (np.abs(got[u] - ref) <= tol).all(), (u, np.max(np.abs(got[u] - ref) / (tol + 1e-300)))
        off = off + 2 * rows * 2.0 ** -24 * m
        assert (np.abs(gm[u] - m) <= off).all(), (u, np.max(np.abs(gm[u] - m) / (off + 1e-300)))
    return out, mass


# ------------------------------------------------------------------------------------------ V
@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("kind", ["mixed", "equal"])
def test_values_to_the_end_of_the_range(kind, plan, group, nq, many_blocks):
    """V up to 448 2^119, of both signs beside smaller blocks, and of one sign with equal weights: finite as the sum is."""
    units, nb = PLANS[plan]
    rng = np.random.default_rng(50 + units)
    store, q = _store(rng, many_blocks, units, nb), _queries(rng, units, group * nq)
    if kind == "mixed":
        _set_scales(store, vs=np.exp2(rng.choice([119, 118, 100, 81, 80, 60, -6], (units, nb))))
    else:
        store[..., O.AT["v"].ravel()] &= 0x7F
        _set_scales(store, vs=2.0 ** 119)
        q.zero_()
    out, _ = _check(q, store, _lengths(units, nb, nq), group, nq, units=_some(units), max_len=64 * nb)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("plan", PLANS)
def test_large_values_without_weight_leave_the_others_exact(plan, group, nq, many_blocks):
    """Blocks of 448 2^119 whose logits are thousands below: their weight is 0 in 64 bits too, so the result and its bound
    are those of the other blocks alone."""
    units, nb = PLANS[plan]
    rng = np.random.default_rng(60 + units)
    store, q = _store(rng, many_blocks, units, nb), _queries(rng, units, group * nq)
    q[..., 0] = 8.0
    store[..., O.AT["k"][:, 0]] = 0                       # ordinary blocks do not look at that dim
    big = rng.random((units, nb)) < 0.2
    big[:, 0] = False
    big[0], big[1, -1], big[2, 1:] = False, True, True
    x = np.zeros((64, 128))
    x[:, 0] = -448
    where = np.argwhere(big)
    for u, b in where:
        store[u, b, O.AT["k"].ravel()] = O.encode(x).ravel()
        store[u, b, O.SCALES:O.SCALES + 8] = np.array([8.0, 2.0 ** 119], np.float32).view(np.uint8)
    lens = np.full(units, 64 * nb - 5)
    out, mass, err = _attend(q, torch.from_numpy(store).cuda(), _i32(lens), group, nq, nb, max_len=64 * nb)
    got, gm = _f64(out), _f64(mass)
    assert err == 0 and np.isfinite(got).all()
    for u in _some(units):
        k, v = O.unpack(store[u])
        ref, m, tol, off = _expect(_f64(q)[u], k, v, np.where(big[u], -1, np.arange(nb)), lens[u], nq, 1 / math.sqrt(128))
        assert (np.abs(got[u] - ref) <= tol).all(), (u, (np.abs(got[u] - ref) / tol).max())
        assert (np.abs(gm[u] - m) <= off).all()


# ------------------------------------------------------------------------------------------ K
def _codes_of(rng, units, nb, k, v=1.0):
    """A store with the codes of N(0, 1) times k and v, and scales of 1."""
    store = np.zeros((units, nb, O.BLOCK_BYTES), np.uint8)
    for kind, size in (("k", k), ("v", v)):
        x = rng.standard_normal((units, nb, 64, 128)) * size
        store[..., O.AT[kind].ravel()] = O.encode(x).reshape(units, nb, -1)
    _set_scales(store, ks=1.0, vs=1.0)
    return store


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -60, 1.0, 2.0 ** 33, 3e38])
def test_the_largest_of_logits_beyond_float32_takes_all(scale, group, nq):
    """Blocks with different K scales, the larger ones with the smaller codes, so that codes alone mislead.  A logit is off
    by 2^-17 of S = scale sum |q| |k| at most (the sums, the roundings and what 2^90 and beyond keep), so a token that leads
    by that of both and by 40 has a weight of 1 in f16 and float32, the others 0, and the result is its V, which bf16
    holds exactly."""
    rng = np.random.default_rng(70)
    units, blocks = 6, 12
    ks = np.array([119, 118, 114, 112, 107, 98, 90, 80, 60, 20, -20, -118])
    size = np.exp2(rng.uniform(0, 1, (units, blocks)) * np.minimum(119 - ks, 13) - 6)
    store = _codes_of(rng, units, blocks, size[..., None, None])
    order = np.argsort(rng.random((units, blocks)), 1)
    _set_scales(store, ks=np.exp2(ks))
    store = np.take_along_axis(store, order[..., None], 1)
    lens = np.array([64 * blocks] * 3 + [64 * blocks - 37] * 3)
    q = _queries(rng, units, group * nq)
    out, mass, err = _attend(q, torch.from_numpy(store).cuda(), _i32(lens), group, nq, blocks, max_len=64 * blocks, scale=scale)
    got, gm, qq, held = _f64(out), _f64(mass), _f64(q), 0
    assert err == 0 and np.isfinite(got).all() and np.isfinite(gm).all()
    assert (np.abs(gm.sum(1) - group * nq) <= 1e-4).all()
    scale = scale or 1 / math.sqrt(128)
    for u in range(units):
        k, v = (x.reshape(-1, 128) for x in O.unpack(store[u]))
        for r in range(group * nq):
            n = lens[u] - (nq - 1 - r % nq)
            z, s = k[:n] @ qq[u, r] * scale, np.abs(k[:n]) @ np.abs(qq[u, r]) * scale
            top = z.argmax()
            lead = z[top] - z - 2.0 ** -17 * (s[top] + s)
            lead[top] = np.inf
            if lead.min() > 40:
                held += 1
                assert np.array_equal(got[u, r], v[top]), (u, r)
    assert held >= units * group * nq // 2


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("scale,size,ks,codes", [
    (3e38, -9, -118, 0.25),            # the scale in base 2 is beyond float32, the logits are ordinary
    (2.0 ** 100, 0, -110, 2.0 ** 6),    # ... and with larger codes
    (2.0 ** -40, -80, 116, 4.0),       # its product with the row's power of two is below float32's normal range
    (2.0 ** -16, -110, 119, 64.0),
    (2.0 ** -140, 20, 119, 4.0),       # the scale itself is
    (0.0, 120, -118, 2.0),             # rows of q near bf16's largest
    (0.0, -120, 119, 4.0),             # and smallest
], ids=["scale-inf", "scale-large", "alpha-tiny", "alpha-tiniest", "scale-tiny", "q-large", "q-small"])
def test_factors_of_any_size(scale, size, ks, codes, group, nq):
    rng = np.random.default_rng(71)
    store = _codes_of(rng, 3, 5, codes)
    _set_scales(store, ks=2.0 ** ks)
    q = (_queries(rng, 3, group * nq).double() * 2.0 ** size).to(torch.bfloat16)
    _check(q, store, np.array([320, 200, 33]), group, nq, max_len=320, scale=scale)


@pytest.mark.parametrize("group,nq", FORMS)
def test_blocks_of_ordinary_logits_beside_a_huge_scale(group, nq, many_blocks):
    """A block with the largest s_K and codes of zero has logits of zero, also where its factor is beyond float32."""
    rng = np.random.default_rng(72)
    store = _store(rng, many_blocks, 3, 6)
    for b in (0, 3):
        store[:, b, O.AT["k"].ravel()] = 0
    _set_scales(store, ks=np.array([2.0 ** 119, 2.0 ** -8, 2.0 ** -9, 2.0 ** 119, 2.0 ** -7, 2.0 ** -8]))
    _check(_queries(rng, 3, group * nq), store, np.array([384, 300, 250]), group, nq, max_len=384)


# ------------------------------------------------------------------------------------------ scratch
@pytest.mark.parametrize("mass", [False, True])
def test_many_units_want_no_scratch_for_pieces(mass):
    """Beyond 2,048 units a CTA takes a unit: no parts to keep, but the scratch still never shrinks with more units."""
    last, most = 0, 536 * 32 * (2048 + 8 * WAVE)
    for units in (2047, 2048, 2049, 5000, 1 << 20):
        n = N.nosa_byte_scratch_bytes(units, 32, 1, mass)
        assert last <= n <= 512 + most + 16 * 32 * units + (16 * 33 * units if mass else 0)
        last = n


@pytest.mark.parametrize("group,nq", FORMS)
def test_many_units_stay_within_their_scratch(group, nq, many_blocks):
    rng = np.random.default_rng(80)
    units, nb, rows = 2500, 3, group * nq
    store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, rows)
    need = N.nosa_byte_scratch_bytes(units, rows, nb, True)
    scratch = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    scratch[:4] = 0
    lens = _i32(_lengths(units, nb, nq))
    want = _attend(q, store, lens, group, nq, nb, max_len=64 * nb,
                   scratch=torch.zeros(4 * need + (1 << 26), dtype=torch.uint8, device="cuda"))
    out, mass = torch.empty_like(q), torch.empty_like(want[1])
    N.nosa_byte_dense_attend(q, store, units, group, nq, nb, lens, 64 * nb, out, scratch, need, mass=mass,
                             stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert (scratch[need:] == 0xA5).all() and scratch[:4].sum() == 0
    assert torch.equal(out, want[0]) and torch.equal(mass, want[1])


# ------------------------------------------------------------------------------------------ waits
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("plan", PLANS)
def test_a_wait_for_products_that_gives_up_is_reported(plan, group, nq, listed, many_blocks):
    """The copies come in time, the products do not (they are waited for all the same): NaN and bit 1, and the next call is
    whole.  Up to 8 rows there is no such wait."""
    units, nb = PLANS[plan]
    rng = np.random.default_rng(81)
    store, q = torch.from_numpy(_store(rng, many_blocks, units, nb)).cuda(), _queries(rng, units, group * nq)
    lens = _i32(np.full(units, 64 * nb))
    sel = _i32(np.tile(np.arange(nb), (units, 1))) if listed else None
    call = lambda: _attend(q, store, lens, group, nq, nb, sel=sel, max_len=64 * nb)  # noqa: E731
    want = call()
    assert want[2] == 0
    N.nosa_debug_quant_wait(-2)
    try:
        out, mass, err = call()
    finally:
        N.nosa_debug_quant_wait(0)
    if group * nq > 8:
        assert err == 2 and torch.isnan(out).all() and torch.isnan(mass).all()
    else:
        assert err == 0 and torch.equal(out, want[0]) and torch.equal(mass, want[1])
    out, mass, err = call()
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(mass, want[1])


# ------------------------------------------------------------------------------------------ lists
# units, listed blocks: more than the 256 entries that a CTA looks up at a time, in a CTA a unit and in a piece
LISTS = {"unit-a-cta": (2049, 300), "pieces": (17 * WAVE // 20, 512)}


@pytest.mark.parametrize("group,nq", FORMS + [(5, 1), (3, 3)])
@pytest.mark.parametrize("plan", LISTS)
def test_lists_longer_than_a_lookup(plan, group, nq, many_blocks):
    """Lists of which the first 256 entries hold nothing, the others nothing, one block, odd numbers of blocks; through
    slots of a small store."""
    units, n = LISTS[plan]
    rng = np.random.default_rng(90)
    store = _store(rng, many_blocks, units, 5)
    sel = rng.integers(0, 2000, (units, n)).astype(np.int32)
    slots = rng.integers(0, 5, (units, n)).astype(np.int32)
    sel[rng.random((units, n)) < 0.1] = -1
    lens = np.full(units, 64 * 2000)
    sel[0, :256], sel[1, 256:] = -1, -1
    sel[2, 257:] = -1
    sel[2, 256] = 1999
    sel[3] = -1
    sel[3, [7, 255, 256]] = [4, 1000, 9]
    lens[4:8] = [0, 1, 64 * 900 + 33, 64 * 1500]  # entries behind the context are left out
    sel[5, 299] = 0
    sel[8] = np.arange(n)
    _check(_queries(rng, units, group * nq), store, lens, group, nq, units=[0, 1, 2, 3, 4, 5, 6, 7, 8, units // 2, units - 1],
           sel=sel, slots=slots)


@pytest.mark.parametrize("group,nq", FORMS[1:])
def test_listed_rows_past_4_gib(group, nq):
    """4,688 blocks of one unit at the end of a store of more than 4 GiB, values repeated so that the oracle stays small."""
    rng = np.random.default_rng(91)
    nb = 2 ** 32 // O.BLOCK_BYTES + 40
    blocks = _codes_of(rng, 1, 7, 60.0, 60.0)[0]
    blocks[:, O.SCALES:O.SCALES + 8] = np.array([2.0 ** -6, 2.0 ** -6], np.float32).view(np.uint8)
    store = torch.from_numpy(blocks).cuda().repeat(nb // 7 + 1, 1)[:nb].contiguous()
    q, n = _queries(rng, 1, group * nq), 4688
    sel = torch.arange(nb - n, nb, dtype=torch.int32, device="cuda")[None].contiguous()
    out, mass, err = _attend(q, store, _i32([64 * nb]), group, nq, nb, sel=sel)
    k, v = (x[(np.arange(n) + nb - n) % 7] for x in O.unpack(blocks))
    ref, m, tol, off = _expect(_f64(q)[0], k, v, np.arange(nb - n, nb), 64 * nb, nq, 1 / math.sqrt(128))
    assert err == 0 and (np.abs(_f64(out)[0] - ref) <= tol).all() and (np.abs(_f64(mass)[0] - m) <= off).all()


@pytest.mark.parametrize("group", [2, 8])
def test_a_context_selects_and_the_8_bit_store_is_attended(group):
    """nosa_select's own list, -1 entries and all, over a store that got the same tokens."""
    torch.cuda.set_device(0)
    B, Hkv, T0, steps = 2, 2, 1500, 3
    U = B * Hkv
    cfg = N.make_config(num_layers=1, batch=B, num_q_heads=group * Hkv, num_kv_heads=Hkv, k_q=4, k_e=6, window_tokens=128,
                        max_context=T0 + steps)
    sizes = N.nosa_query_sizes(cfg)
    cap, nb = sizes.select_slots, sizes.max_blocks
    stream = torch.cuda.current_stream().cuda_stream
    ctx = N.nosa_create(cfg, stream)
    try:
        rng = np.random.default_rng(92)
        K, V = (torch.from_numpy(rng.standard_normal((B, Hkv, T0 + steps, 128))).to(torch.bfloat16).cuda() for _ in range(2))
        W1 = (rng.standard_normal((Hkv, 128, 128)) / math.sqrt(128)).astype(np.float32)
        W2 = (rng.standard_normal((Hkv, 128)) / math.sqrt(128)).astype(np.float32)
        N.nosa_set_eviction_head(ctx, 0, W1, W2)
        store = torch.zeros((U, nb, O.BLOCK_BYTES), dtype=torch.uint8, device="cuda")
        k0, v0 = K[:, :, :T0].contiguous(), V[:, :, :T0].contiguous()
        N.nosa_append_kv(ctx, 0, k0, v0, T0)
        N.nosa_byte_append(k0, v0, store, U, T0, nb, stream=stream)
        sel = torch.empty((U, cap), dtype=torch.int32, device="cuda")
        for t in range(steps):
            T = T0 + t + 1
            k, v = K[:, :, T - 1].contiguous(), V[:, :, T - 1].contiguous()
            q = _queries(rng, U, group)
            N.nosa_append_kv(ctx, 0, k, v, 1)
            N.nosa_byte_append(k, v, store, U, 1, nb, pos=_i32([T - 1] * U), stream=stream)
            N.nosa_select(ctx, 0, q, sel_out=sel)
            out, mass, err = _attend(q, store, _i32([T] * U), group, 1, nb, sel=sel)
            assert N.nosa_sync(ctx) == N.NOSA_OK and err == 0
            host, s = store.cpu().numpy(), sel.cpu().numpy()
            assert (s >= 0).any(1).all()
            for u in range(U):
                kk, vv = O.unpack(host[u, np.maximum(s[u], 0)])
                ref, m, tol, off = _expect(_f64(q)[u], kk, vv, s[u], T, 1, 1 / math.sqrt(128))
                assert (np.abs(_f64(out)[u] - ref) <= tol).all() and (np.abs(_f64(mass)[u] - m) <= off).all()
    finally:
        N.nosa_destroy(ctx)


# ------------------------------------------------------------------------------------------ q, and the other ranges
@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("above", [6, 12, 13, 16, 20])
def test_small_values_of_q_beside_a_large_one_decide(above, group, nq):
    """One value of each row is 2^above times the others' size, in a dim where K is zero: the logits are the small values'.
    _expect counts what is off by 2^-21 of the row's largest with more than 8 rows."""
    rng = np.random.default_rng(93)
    store = _codes_of(rng, 4, 6, 2.0)
    q = _queries(rng, 4, group * nq)
    dims = rng.integers(0, 128, (4, group * nq))
    store[..., O.AT["k"][:, np.unique(dims)].ravel()] = 0
    for u in range(4):
        q[u, torch.arange(group * nq), torch.from_numpy(dims[u])] = 2.0 ** above * (1 if u % 2 else -1.375)
    _check(q, store, np.array([384, 383, 200, 65]), group, nq, max_len=384)


@pytest.mark.parametrize("group,nq", FORMS[1:])
def test_v_and_k_scales_far_apart_with_many_rows(group, nq, many_blocks):
    """As test_blocks_of_very_different_scales, for the kernel of more than 8 rows."""
    rng = np.random.default_rng(94)
    units, nb = 4, 12
    store = _store(rng, many_blocks, units, nb)
    for b in range(nb):
        for u, (ks, vs) in enumerate([(2.0 ** -8, 2.0 ** rng.integers(-100, 100)), (2.0 ** (b % 5 - 8), 2.0 ** -6),
                                      (2.0 ** rng.integers(-20, -8), 2.0 ** rng.integers(-12, 12)), (0.0, 0.0)]):
            store[u, b, O.SCALES:O.SCALES + 8] = np.array([ks, vs], np.float32).view(np.uint8)
    _check(_queries(rng, units, group * nq), store, np.full(units, 64 * nb - 5), group, nq, max_len=64 * nb)


@pytest.mark.parametrize("group,nq", FORMS[1:])
@pytest.mark.parametrize("ks", [2.0 ** -118, 2.0 ** -30, 2.0 ** 6, 2.0 ** 20, 2.0 ** 60, 2.0 ** 119])
@pytest.mark.parametrize("scale", [1e-30, 1.0, 2.0 ** 21, 2.0 ** 25, 2.0 ** 27, 2.0 ** 29, 2.0 ** 33, 1e30, 3e38])
def test_logits_of_any_size_with_many_rows(ks, scale, group, nq, many_blocks):
    """A token that leads by more than its logit and the others may be off (2^-17 of S, as above) and by 40 has all the weight;
    logits below 2^-12 weigh the same within 2^-11 (twice 2^-12 / ln 2, half a step of f16's 2^-11 besides: 2^-10 of the
    largest |v| covers both)."""
    rng = np.random.default_rng(95)
    store = _store(rng, many_blocks, 2, 6)
    _set_scales(store, ks=ks)
    q = _queries(rng, 2, group * nq)
    lens = [384, 377]
    out, mass, err = _attend(q, torch.from_numpy(store).cuda(), _i32(lens), group, nq, 6, max_len=384, scale=scale)
    got, gm, qq = _f64(out), _f64(mass), _f64(q)
    assert err == 0 and np.isfinite(got).all() and np.isfinite(gm).all()
    for u in range(2):
        k, v = (x.reshape(-1, 128) for x in O.unpack(store[u]))
        for r in range(group * nq):
            n = lens[u] - (nq - 1 - r % nq)
            z, s = k[:n] @ qq[u, r] * scale, np.abs(k[:n]) @ np.abs(qq[u, r]) * scale
            if s.max() < 2.0 ** -12:
                o = v[:n].mean(0)
                assert (np.abs(got[u, r] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(v).max()).all()
                continue
            top = z.argmax()
            lead = z[top] - z - 2.0 ** -17 * (s[top] + s)
            lead[top] = np.inf
            if lead.min() > 40:
                assert np.array_equal(got[u, r], v[top])


@pytest.mark.parametrize("group,nq", FORMS[1:])
def test_rows_of_q_that_are_not_finite_or_tiny_or_zero_with_many_rows(group, nq, many_blocks):
    rng = np.random.default_rng(96)
    store = _store(rng, many_blocks, 2, 3)
    q = _queries(rng, 2, group * nq)
    q[0, 1] = 0
    q[0, 2] *= 2.0 ** -120
    q[0, 3] *= 2.0 ** 100
    q[0, 4, 100] = math.inf
    q[0, 5, 3] = math.nan
    q[0, 6, 17] = 1e4  # one value far above the others
    q[0, 9] = 1e-40    # below bf16's normal range
    st = torch.from_numpy(store).cuda()
    out, mass, err = _attend(q, st, _i32([150, 150]), group, nq, 3, max_len=192)
    rows = [r for r in range(group * nq) if r not in (4, 5)]
    assert torch.isnan(out[0, 4:6]).all() and torch.isfinite(out[0, rows]).all() and torch.isnan(mass[0]).all()
    assert err == 0 and torch.isfinite(out[1]).all() and torch.isfinite(mass[1]).all()
    v = O.unpack(store[0])[1].reshape(-1, 128)
    for r in (1, 2, 9):
        o = v[:150 - (nq - 1 - r % nq)].mean(0)
        assert (np.abs(_f64(out)[0, r] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * np.abs(v).max()).all()
    q[0, 3:6] = 1.0  # the rows beside those, against the oracle
    _check(q, store, np.array([150, 0]), group, nq, max_len=192)
    want = out[0, rows[7:]]
    out, _, _ = _attend(q, st, _i32([150, 150]), group, nq, 3, max_len=192)
    assert torch.equal(out[0, rows[7:]], want)  # what other rows hold changes nothing
    q[1, 2, 5] = math.nan  # a row that sees nothing is zeros whatever it holds
    out, mass, _ = _attend(q, st, _i32([150, 0]), group, nq, 3, max_len=192)
    assert not out[1].any() and not mass[1].any()
