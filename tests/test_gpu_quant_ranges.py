"""The attention over the 4-bit store at the ends of its types' ranges, in each of its forms (8, 16 and 32 query
rows a unit), against the float64 oracle's reading of the same store."""
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
FORMS = [(8, 1), (8, 2), (8, 4)]  # q heads and query tokens a unit: 8, 16 and 32 rows


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _store(k, v):
    """k, v float [units, n, 128]: their store on the device, and what it stands for (K, V, |n s| + |m| of V)."""
    units, n = k.shape[:2]
    nb = -(-n // 64)
    kd, vd = (torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda() for x in (k, v))
    store = torch.zeros((units, nb, BB), dtype=torch.uint8, device="cuda")
    N.nosa_quant_append(kd, vd, store, units, n, nb, stream=_stream())
    torch.cuda.synchronize()
    got = Q.unpack(store.cpu().numpy().reshape(-1, BB))
    kk, vv, _, sv = (x.reshape(units, nb * 64, 128)[:, :n] for x in got)
    return store, kk, vv, sv


def _dense(q, store, lens, scale=0.0):
    units, group, nq = q.shape[:3]
    nb = store.shape[1]
    bytes_ = N.nosa_quant_scratch_bytes(units, group * nq, nb)
    scratch = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    N.nosa_quant_dense_attend(q, store, units, group, nq, nb, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              64 * nb, out, scratch, bytes_, softmax_scale=scale, stream=_stream())
    torch.cuda.synchronize()
    assert int(scratch[:4].view(torch.int32).item()) == 0
    return out.double().cpu().numpy()


def _one_token(out, u, n, kk, vv, sv, dim):
    """Every row of unit u has the values of the token it sees with the largest K in `dim`: one token's weight and
    its product with s are rounded to f16 (2^-11 each, of the codes' part), m + 15 s too, and the result to bf16."""
    nq = out.shape[2]
    for i in range(nq):
        see = n - (nq - 1 - i)
        best = np.nonzero(kk[u, :see, dim] == kk[u, :see, dim].max())[0]
        assert best.size == 1
        ref = vv[u, best[0]]
        err = np.abs(out[u, :, i] - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * 16 * sv[u, best[0]]).all(), (i, np.nanmax(err))


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("v_size", [1.0, 60.0, 9000.0])
@pytest.mark.parametrize("q_size", [1e6, 1e9, 1e20])
def test_huge_logits_leave_one_token_whatever_its_scale(group, nq, v_size, q_size):
    rng = np.random.default_rng(41)
    n = 300
    k, v = rng.standard_normal((2, 2, n, 128))
    v *= v_size
    k[0, 251, 5], k[1, 40, 5] = 9.0, 9.0  # far above the others
    store, kk, vv, sv = _store(k, v)
    q = torch.zeros((2, group, nq, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = q_size
    out = _dense(q, store, [n, n])
    for u in range(2):
        _one_token(out, u, n, kk, vv, sv, 5)


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("k_size", [1.0, 3000.0])
@pytest.mark.parametrize("scale,q_size", [(1e30, 1.0), (3e38, 1e30), (0.0, 3e38), (3e38, 3e38)])
def test_extreme_scales_leave_one_token_in_every_form(group, nq, k_size, scale, q_size):
    """Logits up to 2^250 and beyond float32: the token with the largest takes all."""
    rng = np.random.default_rng(43)
    n = 300
    k, v = rng.standard_normal((2, 2, n, 128))
    k[0, 251, 5], k[1, 40, 5] = 9.0, 9.0
    store, kk, vv, sv = _store(k * k_size, v)
    q = torch.zeros((2, group, nq, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = q_size
    out = _dense(q, store, [n, n], scale=scale)
    for u in range(2):
        _one_token(out, u, n, kk, vv, sv, 5)


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("scale_of", ["every-token", "one-token"])
def test_small_groups_keep_their_values_beside_large_ones(group, nq, scale_of):
    """Groups of one value (s = 0) next to a group with scales of 2 and more: weights and the softmax sum meet the same
    minima, so that nothing but float32 sums and the result's rounding to bf16 stands between the value and the output."""
    rng = np.random.default_rng(47)
    n = 200
    k, v = rng.standard_normal((2, 1, n, 128))
    v[..., 0:32] *= 40.0 if scale_of == "every-token" else 1.0
    v[:, 70, 0:32] *= 40.0
    v[..., 32:64], v[..., 64:96], v[..., 96:128] = 1e-4, 1e-5, -3e-6
    store, kk, vv, sv = _store(k, v)
    q = torch.from_numpy(rng.standard_normal((1, group, nq, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = _dense(q, store, [n])
    ref = vv[0, 0, 32:]
    assert (vv[0, :, 32:] == ref).all()
    err = np.abs(out[0, :, :, 32:] - ref)
    # float32 sums over 13 tiles, in units of the sum: less than 2^-16
    assert (err <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref)).all(), (err / np.abs(ref)).max()


@pytest.mark.parametrize("rows,blocks", [(8, 64), (8, 20), (16, 64), (32, 64), (32, 8), (1, 1)])
def test_scratch_for_more_is_enough_for_less(rows, blocks):
    """A program sizes its scratch for its largest batch: fewer units, rows or blocks never want more."""
    size = N.nosa_quant_scratch_bytes
    units = [1, 2, 16, 64, 151, 152, 153, 303, 304, 305, 442, 443, 600, 608, 609, 2048, 2049, 5000, 1 << 20]
    got = [size(u, rows, blocks) for u in units]
    assert got == sorted(got), list(zip(units, got))
    for u in units:
        got = [size(u, r, blocks) for r in range(1, rows + 1)]
        assert got == sorted(got), (u, got)
        got = [size(u, rows, b) for b in (1, 2, 3, 7, 20, 26, 27, 64, 65, 100, 101, 1000, 16384)]
        assert got == sorted(got), (u, got)


def test_a_batch_that_shrinks_keeps_its_scratch():
    store, kk, vv, sv = _store(*np.random.default_rng(5).standard_normal((2, 1, 64 * 64, 128)))
    store = store.expand(443, -1, -1).contiguous()
    q = torch.zeros((443, 8, 1, 128), dtype=torch.bfloat16, device="cuda")
    bytes_ = N.nosa_quant_scratch_bytes(443, 8, 64)
    scratch = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
    lens = torch.full((443,), 64 * 64, dtype=torch.int32, device="cuda")
    sel = torch.arange(64, dtype=torch.int32, device="cuda").repeat(443, 1)
    mean = vv[0].mean(0)
    tol = 2.0 ** -8 * np.abs(mean) + 2.0 ** -9 * sv[0].max()
    for units in (443, 442, 305, 304, 152, 20, 1):
        for listed in (False, True):
            out = torch.full_like(q, float("nan"))
            if listed:
                N.nosa_quant_attend(q, store, sel, None, units, 8, 1, 64, 64, lens, out, scratch, bytes_, stream=_stream())
            else:
                N.nosa_quant_dense_attend(q, store, units, 8, 1, 64, lens, 64 * 64, out, scratch, bytes_, stream=_stream())
            torch.cuda.synchronize()
            got = out.double().cpu().numpy()
            assert (np.abs(got[:units] - mean) <= tol).all()
            assert np.isnan(got[units:]).all()


@pytest.mark.parametrize("group,nq", FORMS)
def test_small_values_of_q_are_exact(group, nq):
    """Values of 2^-22 of their row's largest in odd and in even dims give exactly the same logits (about 1400, where the
    last of a value's eight bits is worth 10): two tokens share the weight."""
    small = 2.0 ** -22 * (1 + 2.0 ** -7)
    k, v = np.zeros((2, 1, 2 + nq, 128))
    k[0, 0, 33] = k[0, 1, 64] = 57344.0  # the same code and scale in an odd and in an even dim
    v[0, 0], v[0, 1] = 1.0, 2.0
    k[0, 2:] = -1.0  # the query tokens' own: no weight
    store, kk, _, _ = _store(k, v)
    assert kk[0, 0, 33] == kk[0, 1, 64] > 57000 and kk[0, 0, 0] == kk[0, 1, 0] == 0
    q = torch.zeros((1, group, nq, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 33], q[..., 64] = 1.0, small, small
    out = _dense(q, store, [2 + nq], scale=1e5)
    # groups of one value: weights alike, the sum and the minima exact
    assert (out == 1.5).all()


@pytest.mark.parametrize("group,nq", FORMS)
@pytest.mark.parametrize("q_size", [1.0, 1e6, 1e10, 1e20])
def test_equal_scores_share_the_weight_whatever_their_scales(group, nq, q_size):
    """Two tokens with the same key, far above the others, in different warps' shares; the V scales beside one of them are
    large.  Logits of 13 to 1e21."""
    rng = np.random.default_rng(53)
    n = 64 * 8 - 5
    k, v = rng.standard_normal((2, 1, n, 128))
    v[0, 64 * 5:64 * 5 + 64] *= 3000.0
    k[0, 64 * 5 + 9] = k[0, 20]
    k[0, [20, 64 * 5 + 9], 5] = 300.0
    store, kk, vv, sv = _store(k, v)
    a, b = 20, 64 * 5 + 9
    assert np.array_equal(kk[0, a], kk[0, b])
    q = torch.zeros((1, group, nq, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = q_size
    out = _dense(q, store, [n])
    ref = (vv[0, a] + vv[0, b]) / 2
    # weights, products with s and maxima rounded to f16, 2^-11 each of at most 16 |x^|'s parts, and the result to bf16
    err = np.abs(out[0] - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * 16 * (sv[0, a] + sv[0, b]) / 2).all(), np.nanmax(err / np.abs(ref))
