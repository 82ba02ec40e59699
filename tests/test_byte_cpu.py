"""The 8-bit KV block store, eviction and rotary positions without a GPU: the oracle's own pins, the table that
nosa_rope_make fills, and the refusals of the entry points, which come before any CUDA call."""
import ctypes
import math
import os

import numpy as np
import pytest

from offloadable_block_sparse_gb300 import build as B
from offloadable_block_sparse_gb300 import nosa as N
from oracle import byte_oracle as O


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(N.LIB_PATH):
        B.build()


# ------------------------------------------------------------------------------------------ the oracle
def test_oracle_codes():
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F])
    assert np.array_equal(O.encode(O.E4M3[finite]), finite)  # every value is its own code
    assert O.E4M3[0x7E] == 448 and O.E4M3[1] == 2.0 ** -9 and O.E4M3[0x38] == 1
    # ties to even codes, saturation, NaN
    assert list(O.encode([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 464, 1e30, -1e30])) == [0x38, 0x3A, 0, 2, 0x7E, 0x7E, 0xFE]
    assert list(O.encode([np.nan, np.inf, -np.inf])) == [0x7F] * 3
    x = np.random.default_rng(0).uniform(-448, 448, 5000)
    assert (np.abs(O.E4M3[O.encode(x)] - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10)).all()


def test_oracle_scales():
    for x, s in ((448.0, 1.0), (449.0, 2.0), (1.75, 2.0 ** -8), (1.8, 2.0 ** -7), (0.0, 0.0), (1e-45, 2.0 ** -118),
                 (3e38, 2.0 ** 119), (7.0, 2.0 ** -6)):
        assert O.need(np.array([x, -x / 2, np.nan, np.inf])) == s


def test_oracle_layout_is_a_bijection():
    seen = {int(O.place(kind, i, d)) for kind in "kv" for i in range(16) for d in range(128)}
    assert seen == set(range(O.TILE_BYTES))


def test_oracle_tokens_one_by_one():
    """One token at a time ends with the scales of a whole block, and with its codes wherever no step rounded again."""
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((1, 128, 128)) * np.exp(rng.standard_normal((1, 128, 1))) for _ in range(2))
    one, whole = np.zeros((1, 2, O.BLOCK_BYTES), np.uint8), O.pack(k.reshape(2, 64, 128), v.reshape(2, 64, 128))
    for i in range(128):
        assert not O.append(one, k[:, i:i + 1], v[:, i:i + 1], [i], [1])
    assert np.array_equal(O.scales(one[0]), O.scales(whole))
    for a, b, s in zip(O.unpack(one[0]), O.unpack(whole), O.scales(whole).T):
        off, step = np.abs(a - b), s[:, None, None] * 2.0 ** -9
        assert (off[np.abs(b) >= 2.0 ** -6 * s[:, None, None]] == 0).all() or (off <= step).all()
        assert (off <= step).all()
    bulk = np.zeros((1, 2, O.BLOCK_BYTES), np.uint8)
    O.append(bulk, k, v, [0], [128])
    assert np.array_equal(bulk[0], whole)


def test_oracle_evict_by_hand():
    blk = np.array([[0, 7, 3, -1, 9, 5]], np.int32)
    acc = np.array([[0.0, 2.0, 1.0, 9.0, 0.0, 1.0]], np.float32)
    # 5 blocks held, block 10 wanted, budget 4: two go of 3, 5 and 7 (0 is the sink, 9 the window); of 3 and 5, equal at
    # 1, both are below 7's 2
    a, b, row, flag = O.evict(acc, blk, None, [640], 4, 1, 1, 1.0, [10])
    assert list(b[0]) == [0, 7, 10, -1, 9, -1] and list(a[0]) == [0, 2, 0, 0, 0, 0] and row[0] == 2 and not flag
    a, b, row, flag = O.evict(acc, blk, None, [640], 5, 1, 1, 1.0, [10])
    assert list(b[0]) == [0, 7, 3, 10, 9, -1] and row[0] == 3  # the higher of the equal ones
    a, b, row, flag = O.evict(acc[:, :1], blk[:, :1], None, [640], 0, 1, 1, 1.0, [10])
    assert list(b[0]) == [0] and row[0] == -1 and flag


# ------------------------------------------------------------------------------------------ the rotary table
@pytest.mark.parametrize("kw", [dict(), dict(rot_dims=64, base=500000.0), dict(rot_dims=2), dict(rot_dims=98, interleaved=True),
                                dict(scaling=N.NOSA_ROPE_LINEAR, factor=4.0), dict(scaling=N.NOSA_ROPE_BASE, factor=8.0),
                                dict(scaling=N.NOSA_ROPE_BASE, factor=8.0, rot_dims=2),
                                dict(scaling=N.NOSA_ROPE_PARTS, factor=8.0, original=8192.0, low=1.0, high=4.0,
                                     attention_factor=1.2)])
def test_rope_table(kw):
    t = N.nosa_rope_make(**kw)
    rot = kw.get("rot_dims", 128)
    f = O.frequencies(rot, **{k: v for k, v in kw.items() if k not in ("rot_dims", "interleaved", "attention_factor")})
    assert t.rot_dims == rot and t.interleaved == int(kw.get("interleaved", False))
    assert t.attention_factor == np.float32(kw.get("attention_factor", 1.0))
    got = np.array([t.turn[i] / 2.0 ** 64 for i in range(64)])
    # a power, a division and a scaling in float64, each within 2^-51 of its result
    assert (np.abs(got[:rot // 2] - f / (2 * math.pi)) <= 2.0 ** -49 * f / (2 * math.pi) + 2.0 ** -63).all()
    assert not got[rot // 2:].any()


GOOD = dict(rot_dims=128, interleaved=0, scaling=0, base=10000.0, factor=2.0, low=1.0, high=32.0, original=4096.0,
            attention_factor=1.0)


@pytest.mark.parametrize("bad", [dict(rot_dims=0), dict(rot_dims=63), dict(rot_dims=130), dict(rot_dims=-2), dict(interleaved=2),
                                 dict(scaling=4), dict(scaling=-1), dict(base=0.5), dict(base=math.nan), dict(base=math.inf),
                                 dict(scaling=1, factor=0.5), dict(scaling=2, factor=math.inf), dict(scaling=2, factor=1e300),
                                 dict(scaling=3, low=32.0), dict(scaling=3, low=-1.0), dict(scaling=3, original=0.0),
                                 dict(scaling=3, high=math.nan), dict(attention_factor=-1.0), dict(attention_factor=math.nan),
                                 dict(attention_factor=1e39)])
def test_rope_make_refusals(bad):
    with pytest.raises(N.NosaError) as e:
        N.nosa_rope_make(**(GOOD | bad))
    assert e.value.status == N.NOSA_ERR_INVALID_ARG
    N.nosa_rope_make(**GOOD)


def test_rope_make_null_and_size():
    out = N.nosa_rope_table()
    cfg = N.nosa_rope_config(8, *GOOD.values())
    assert N.lib().nosa_rope_make(ctypes.byref(cfg), ctypes.byref(out)) == N.NOSA_ERR_INVALID_ARG
    assert N.lib().nosa_rope_make(None, ctypes.byref(out)) == N.NOSA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------ refusals
P = 1 << 20  # a non-null address that is never read


def _append(**kw):
    a = dict(k=P, v=P, store=P, units=2, n_tokens=5, max_blocks=3, pos=P, count=P, slot_blk=P, err_out=P, stream=None)
    return N.lib().nosa_byte_append(*(a | kw).values())


def _read(**kw):
    a = dict(store=P, units=2, max_blocks=3, blocks=P, slots=P, n_blocks=5, lens=P, kv=P, err_out=P, stream=None)
    return N.lib().nosa_byte_read(*(a | kw).values())


def _dense(**kw):
    a = dict(q=P, store=P, units=2, group=8, n_queries=2, max_blocks=3, lens=P, max_len=190, softmax_scale=0.0,
             out=P, mass=P, scratch=P, scratch_bytes=1 << 30, stream=None)
    return N.lib().nosa_byte_dense_attend(*(a | kw).values())


def _sparse(**kw):
    a = dict(q=P, store=P, sel=P, sel_slot=P, units=2, group=8, n_queries=2, max_blocks=3, max_sel=4, lens=P,
             softmax_scale=0.0, out=P, mass=P, scratch=P, scratch_bytes=1 << 30, stream=None)
    return N.lib().nosa_byte_attend(*(a | kw).values())


def _evict(**kw):
    a = dict(acc=P, slot_blk=P, mass=P, units=2, slots=8, lens=P, budget=4, sink_blocks=1, window_blocks=2, decay=1.0,
             acc_out=P, slot_blk_out=P, next_block=P, next_slot=P, err_out=P, stream=None)
    return N.lib().nosa_evict(*(a | kw).values())


def _view(**kw):
    w = N.nosa_rope_view()
    a = dict(x=P, y=2 * P, heads=4, x_stride=(4096, 1024, 128), y_stride=(4096, 1024, 128)) | kw
    w.x, w.y, w.heads = a["x"], a["y"], a["heads"]
    w.x_stride[:], w.y_stride[:] = a["x_stride"], a["y_stride"]
    return w


def _rope(views=None, table=None, **kw):
    views = [_view()] if views is None else views
    v = (N.nosa_rope_view * max(len(views), 1))(*views)
    a = dict(views=v, n_views=len(views), batch=2, n_tokens=8, pos=P, count=P, inverse=0, err_out=P, stream=None) | kw
    return N.lib().nosa_rope(ctypes.byref(table or N.nosa_rope_make()), *a.values())


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(store=None), dict(units=0), dict(n_tokens=0), dict(max_blocks=0),
                                 dict(k=P + 8), dict(v=P + 2), dict(store=P + 4), dict(pos=P + 2), dict(count=P + 1),
                                 dict(slot_blk=P + 2), dict(err_out=P + 2), dict(units=1 << 20, max_blocks=1 << 12),
                                 dict(units=2 ** 31 - 1, n_tokens=2 ** 30, max_blocks=1), dict(n_tokens=2 ** 30 + 1)])
def test_append_refusals(bad):
    assert _append(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(store=None), dict(kv=None), dict(units=0), dict(max_blocks=0), dict(n_blocks=0),
                                 dict(store=P + 8), dict(kv=P + 8), dict(blocks=P + 2), dict(slots=P + 2), dict(lens=P + 2),
                                 dict(err_out=P + 1), dict(blocks=None, slots=None, n_blocks=4), dict(blocks=None, n_blocks=2),
                                 dict(units=1 << 20, n_blocks=1 << 12), dict(units=1 << 20, max_blocks=1 << 12)])
def test_read_refusals(bad):
    assert _read(**bad) == N.NOSA_ERR_INVALID_ARG


SHARED = [dict(q=None), dict(store=None), dict(lens=None), dict(out=None), dict(scratch=None), dict(units=0),
          dict(units=(1 << 20) + 1), dict(group=0), dict(group=9), dict(n_queries=0), dict(group=8, n_queries=5),
          dict(group=1, n_queries=33), dict(max_blocks=0), dict(softmax_scale=-1.0), dict(softmax_scale=math.nan),
          dict(softmax_scale=math.inf), dict(q=P + 8), dict(store=P + 8), dict(out=P + 8), dict(lens=P + 2), dict(mass=P + 2),
          dict(scratch=P + 128), dict(units=1 << 20, max_blocks=1 << 12), dict(group=2 ** 30, n_queries=2 ** 30)]


@pytest.mark.parametrize("bad", SHARED + [dict(max_len=0), dict(max_len=193), dict(max_len=(1 << 20) + 1, max_blocks=1 << 20)])
def test_dense_refusals(bad):
    assert _dense(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", SHARED + [dict(sel=None), dict(max_sel=0), dict(max_sel=16385), dict(sel=P + 2),
                                          dict(sel_slot=P + 1), dict(units=1 << 18, max_sel=1 << 13)])
def test_sparse_refusals(bad):
    assert _sparse(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(acc=None), dict(slot_blk=None), dict(acc_out=None), dict(slot_blk_out=None), dict(units=0),
                                 dict(slots=0), dict(slots=16385), dict(budget=-1), dict(budget=9), dict(sink_blocks=-1),
                                 dict(window_blocks=-1), dict(decay=-0.5), dict(decay=math.nan), dict(decay=math.inf),
                                 dict(lens=None), dict(acc=P + 2), dict(mass=P + 1), dict(lens=P + 2), dict(next_block=P + 2),
                                 dict(next_slot=P + 2), dict(err_out=P + 2), dict(acc_out=P + 2), dict(slot_blk_out=P + 2)])
def test_evict_refusals(bad):
    assert _evict(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(views=[]), dict(views=[_view()] * 3, n_views=3), dict(batch=0), dict(n_tokens=0),
                                 dict(pos=P + 2), dict(count=P + 2), dict(err_out=P + 2), dict(views=[_view(x=0)]),
                                 dict(views=[_view(y=0)]), dict(views=[_view(heads=0)]), dict(views=[_view(), _view(x=P + 1)]),
                                 dict(views=[_view(x_stride=(-1, 128, 128))]), dict(views=[_view(y_stride=(4096, 127, 128))]),
                                 dict(views=[_view(y_stride=(0, 1024, 128))]), dict(views=[_view(x_stride=(1 << 40, 1024, 128))]),
                                 dict(views=[_view(y=P, x_stride=(8192, 1024, 128))]),
                                 dict(batch=2 ** 30, n_tokens=2 ** 30), dict(batch=1, n_tokens=2 ** 30 + 1),
                                 dict(batch=1, n_tokens=2 ** 31 - 1), dict(views=[_view(heads=2 ** 20 + 1)]),
                                 dict(views=[_view(), _view(heads=2 ** 31 - 1)])])
def test_rope_refusals(bad):
    assert _rope(**bad) == N.NOSA_ERR_INVALID_ARG


def test_rope_refuses_a_foreign_table():
    for field, value in (("struct_size", 4), ("rot_dims", 129), ("rot_dims", 3), ("rot_dims", 0)):
        t = N.nosa_rope_make()
        setattr(t, field, value)
        assert _rope(table=t) == N.NOSA_ERR_INVALID_ARG


def test_binding_checks_views():
    import torch
    x = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)
    for pair in ((x, x[:, :2]), (x, x.transpose(2, 3)), (x[..., :64], x[..., :64])):
        with pytest.raises(ValueError):
            N.nosa_rope(N.nosa_rope_make(), [pair])


def test_without_a_gpu_calls_report_a_status():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_append, _read, _dense, _sparse, _evict, _rope):
        assert call() == N.NOSA_ERR_CUDA
    assert N.nosa_byte_scratch_bytes(4, 8, 100, True) == 0


def test_binding_raises_the_status():
    with pytest.raises(N.NosaError) as e:
        N.nosa_byte_append(None, P, P, 1, 1, 1)
    assert e.value.status == N.NOSA_ERR_INVALID_ARG
    assert N.NOSA_BYTE_BLOCK_BYTES == O.BLOCK_BYTES
