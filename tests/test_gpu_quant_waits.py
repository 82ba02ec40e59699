"""The 4-bit attention when its waits for staged tiles give up: the error bit, NaN outputs, and nothing left behind for
the next call.  The waits are made to give up by a limit of none (nosa_debug_quant_wait); what they waited for is
waited for again before its place is used."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from offloadable_block_sparse_gb300 import nosa as N  # noqa: E402


@pytest.fixture(autouse=True)
def limit():
    yield N.nosa_debug_quant_wait
    N.nosa_debug_quant_wait(0)


@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
@pytest.mark.parametrize("group,nq", [(8, 1), (8, 2), (8, 4)])
@pytest.mark.parametrize("units,nb", [(2, 30), (12, 200), (600, 9), (20, 1)],
                         ids=["cluster", "pieces", "unit-a-cta", "one-block"])
def test_waits_that_give_up_are_reported(limit, units, nb, group, nq, listed):
    torch.manual_seed(units)
    n = 64 * nb - 5
    store = torch.zeros((units, nb, N.NOSA_QUANT_BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    k = torch.randn((units, n, 128), device="cuda").to(torch.bfloat16)
    stream = torch.cuda.current_stream().cuda_stream
    N.nosa_quant_append(k, k, store, units, n, nb, stream=stream)
    q = torch.randn((units, group, nq, 128), device="cuda").to(torch.bfloat16)
    lens = torch.full((units,), n, dtype=torch.int32, device="cuda")
    lens[units // 2] = 0  # a unit without tokens waits for nothing
    sel = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(units, 1)
    size = N.nosa_quant_scratch_bytes(units, group * nq, nb)
    scratch = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def attend():
        out = torch.ones_like(q)
        scratch[:4] = 0
        if listed:
            N.nosa_quant_attend(q, store, sel, None, units, group, nq, nb, nb, lens, out, scratch, size, stream=stream)
        else:
            N.nosa_quant_dense_attend(q, store, units, group, nq, nb, lens, n, out, scratch, size, stream=stream)
        torch.cuda.synchronize()
        return out, int(scratch[:4].view(torch.int32).item())

    good, err = attend()
    assert err == 0 and torch.isfinite(good).all() and not good[units // 2].any()
    limit(-1)
    out, err = attend()
    assert err == 2
    some = lens > 0
    assert out[some].isnan().all()
    limit(0)
    again, err = attend()
    assert err == 0 and torch.equal(again, good)
