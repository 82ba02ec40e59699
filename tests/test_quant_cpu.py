"""The 4-bit KV block store without a GPU: the oracle's own pins (hand-worked groups, the layout as a
bijection, one token at a time against whole blocks) and the refusals of the entry points, which come
before any CUDA call."""
import ctypes
import os

import numpy as np
import pytest

from offloadable_block_sparse_gb300 import build as B
from offloadable_block_sparse_gb300 import nosa as N
from oracle import quant_oracle as Q


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(N.LIB_PATH):
        B.build()


def test_oracle_hand_worked_groups():
    x = np.zeros(128)
    x[0:32] = np.arange(32) / 2          # 0 .. 15.5: s = f16(31/30), codes rint(x / s)
    x[32:64] = -3.0                       # constant: s = 0, codes 0
    x[64:96] = np.tile([0, 15, 0.5, 1.5], 8)  # s = 1: ties to even codes 0 and 2
    x[96] = np.nan
    codes, s, m = Q.quantise(x)
    assert s[0] == np.float16(15.5 / 15) and m[0] == 0 and codes[31] == 15 and codes[1] == 0 and codes[2] == 1
    assert s[1] == 0 and m[1] == -3 and not codes[32:64].any()
    assert s[2] == 1 and list(codes[64:68]) == [0, 15, 0, 2]
    assert np.isnan(s[3]) and np.isnan(m[3]) and not codes[96:].any()
    back = Q.values(codes, s, m)
    assert (back[32:64] == -3).all() and np.isnan(back[96:]).all()
    # away from clamping a value is at most half a step away
    assert np.abs(back[:32] - x[:32]).max() <= float(s[0]) / 2 + 15 * float(s[0]) * 2.0 ** -11


def test_oracle_layout_is_a_bijection():
    seen = set()
    for kind in "kv":
        for i in range(16):
            for d in range(128):
                byte, shift = Q.code_place(kind, i, d)
                seen.add((byte, shift))
            for gr in range(4):
                for which in (0, 1):
                    at = Q.scale_place(kind, which, i, gr)
                    assert at % 2 == 0
                    seen |= {(at + b, sh) for b in (0, 1) for sh in (0, 4)}
    assert seen == {(b, sh) for b in range(Q.TILE_BYTES) for sh in (0, 4)}


def test_oracle_whole_blocks_equal_tokens_one_by_one():
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((1, 128, 128)) for _ in range(2))
    store = np.zeros((1, 2, Q.BLOCK_BYTES), np.uint8)
    assert not Q.append(store, k, v, [0], [128])
    assert (store[0] == Q.pack(k.reshape(2, 64, 128), v.reshape(2, 64, 128))).all()
    kk, vv, _, _ = Q.unpack(store[0])
    assert np.array_equal(kk.reshape(128, 128), Q.values(*Q.quantise(k[0])))
    assert np.array_equal(vv.reshape(128, 128), Q.values(*Q.quantise(v[0])))


P = 1 << 20  # a non-null address that is never read


def _append(**kw):
    a = dict(k=P, v=P, store=P, units=2, n_tokens=5, max_blocks=3, pos=P, count=P, err_out=P, stream=None)
    return N.lib().nosa_quant_append(*(a | kw).values())


def _read(**kw):
    a = dict(store=P, units=2, max_blocks=3, blocks=P, n_blocks=5, lens=P, kv=P, err_out=P, stream=None)
    return N.lib().nosa_quant_read(*(a | kw).values())


def _dense(**kw):
    a = dict(q=P, store=P, units=2, group=8, n_queries=2, max_blocks=3, lens=P, max_len=190, softmax_scale=0.0,
             out=P, scratch=P, scratch_bytes=1 << 30, stream=None)
    return N.lib().nosa_quant_dense_attend(*(a | kw).values())


def _sparse(**kw):
    a = dict(q=P, store=P, sel=P, sel_slot=P, units=2, group=8, n_queries=2, max_blocks=3, max_sel=4, lens=P,
             softmax_scale=0.0, out=P, scratch=P, scratch_bytes=1 << 30, stream=None)
    return N.lib().nosa_quant_attend(*(a | kw).values())


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(store=None), dict(units=0), dict(n_tokens=0),
                                 dict(max_blocks=0), dict(k=P + 8), dict(v=P + 2), dict(store=P + 4),
                                 dict(pos=P + 2), dict(count=P + 1), dict(err_out=P + 2),
                                 dict(units=1 << 20, max_blocks=1 << 12), dict(units=2 ** 31 - 1, n_tokens=2 ** 31 - 1,
                                                                               max_blocks=1)])
def test_append_refusals(bad):
    assert _append(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(store=None), dict(kv=None), dict(units=0), dict(max_blocks=0), dict(n_blocks=0),
                                 dict(store=P + 8), dict(kv=P + 8), dict(blocks=P + 2), dict(lens=P + 2),
                                 dict(err_out=P + 1), dict(blocks=None, n_blocks=4), dict(units=1 << 20, n_blocks=1 << 12),
                                 dict(units=1 << 20, max_blocks=1 << 12)])
def test_read_refusals(bad):
    assert _read(**bad) == N.NOSA_ERR_INVALID_ARG


SHARED = [dict(q=None), dict(store=None), dict(lens=None), dict(out=None), dict(scratch=None), dict(units=0),
          dict(units=(1 << 20) + 1), dict(group=0), dict(group=9), dict(n_queries=0), dict(group=8, n_queries=5),
          dict(group=1, n_queries=33), dict(max_blocks=0), dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
          dict(softmax_scale=float("inf")), dict(q=P + 8), dict(store=P + 8), dict(out=P + 8), dict(lens=P + 2),
          dict(scratch=P + 128), dict(units=1 << 20, max_blocks=1 << 12), dict(group=2 ** 30, n_queries=2 ** 30)]


@pytest.mark.parametrize("bad", SHARED + [dict(max_len=0), dict(max_len=193), dict(max_len=(1 << 20) + 1, max_blocks=1 << 20)])
def test_dense_refusals(bad):
    assert _dense(**bad) == N.NOSA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", SHARED + [dict(sel=None), dict(max_sel=0), dict(max_sel=16385), dict(sel=P + 2),
                                          dict(sel_slot=P + 1)])
def test_sparse_refusals(bad):
    assert _sparse(**bad) == N.NOSA_ERR_INVALID_ARG


def test_without_a_gpu_calls_report_a_status():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_append, _read, _dense, _sparse):
        assert call() == N.NOSA_ERR_CUDA
    assert N.nosa_quant_scratch_bytes(4, 8, 100) == 0


def test_binding_raises_the_status():
    with pytest.raises(N.NosaError) as e:
        N.nosa_quant_append(None, P, P, 1, 1, 1)
    assert e.value.status == N.NOSA_ERR_INVALID_ARG
    assert N.NOSA_QUANT_BLOCK_BYTES == Q.BLOCK_BYTES
    assert ctypes.sizeof(ctypes.c_size_t) == 8
