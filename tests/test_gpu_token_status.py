"""GPU: the device status word, with the token operators' errors beside the optimizer's."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def bad_id(dm):
    dm.embedding(torch.zeros(4, 8, device="cuda"), torch.tensor([1, 4], device="cuda"))


def overflow(dm):
    """An fp16 output that no fp16 number holds."""
    a = torch.full((128, 128), 200.0, dtype=torch.float16, device="cuda")
    dm.gemm_f16(a, a, torch.empty(128, 128, dtype=torch.float16, device="cuda"), b_trans=True)


def raised(dm):
    with pytest.raises(dm.DmuonError) as e:
        dm.check_status()
    return e.value.status


@pytest.mark.parametrize("order", [(bad_id, overflow), (overflow, bad_id)], ids=["index first", "overflow first"])
def test_an_index_does_not_hide_a_nonfinite_value(dm, order):
    """Both are reported, one check after the other, and then none."""
    dm.check_status()
    for make in order:
        make(dm)
    assert raised(dm) == dm.ERR_NONFINITE
    assert raised(dm) == dm.ERR_INDEX
    dm.check_status()
    bad_id(dm)
    assert raised(dm) == dm.ERR_INDEX
    dm.check_status()
