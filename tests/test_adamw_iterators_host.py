"""Moments for parameters that come by an iterator, as a model gives them."""
import pytest
import torch


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_of_parameters_from_an_iterator(bits):
    """Every kind of moment for every one: the second kind found the iterator used up."""
    from verifiable_repops_gemm_gb300 import ADAMW_GROUP, adamw_state
    params = [torch.zeros(3, 5), torch.zeros(300), torch.zeros(0)]
    st = adamw_state((p for p in params), bits)
    want = adamw_state(params, bits)
    assert sorted(st) == sorted(want)
    for k in want:
        assert [t.shape for t in st[k]] == [t.shape for t in want[k]] and len(st[k]) == 3
        assert all(not t.any() for t in st[k])
    if bits == 8:
        assert [t.numel() for t in st["m_scales"]] == [-(-p.numel() // ADAMW_GROUP) for p in params]
