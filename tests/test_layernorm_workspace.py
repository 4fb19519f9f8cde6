"""The bytes that rowops_layernorm_bwd's binding tells the library of a workspace."""
import pytest
import torch

from row_wise_softmax_warp_gb300 import binding


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float32])
def test_no_bytes_behind_the_storage(dtype):
    whole = torch.empty(512, dtype=dtype)
    size = whole.element_size()
    assert binding._bytes_behind(whole) == 512 * size
    assert binding._bytes_behind(whole[100:]) == 412 * size
    assert binding._bytes_behind(whole[::2]) == 256 * size  # as before: no more than its values
    for few in (torch.empty(1, dtype=dtype), whole[-1:]):
        assert binding._bytes_behind(few.expand(1 << 20)) == size  # too little for any call: refused by the library
    assert binding._bytes_behind(torch.empty(0, dtype=dtype)) == 0


@pytest.mark.gpu
def test_an_expanded_workspace_is_refused(ro):
    x = torch.randn(64, 768, device="cuda")
    gamma, inv = torch.ones(768, device="cuda"), torch.ones(64, device="cuda")
    view = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24)
    with pytest.raises(ro.RowopsError) as e:
        ro.rowops_layernorm_bwd(x, gamma, x, inv, workspace=view)
    assert e.value.status == 4
    room = torch.empty(ro.rowops_layernorm_bwd_workspace(64, 768), dtype=torch.uint8, device="cuda")
    want = ro.rowops_layernorm_bwd(x, gamma, x, inv)
    assert all(torch.equal(a, b) for a, b in zip(ro.rowops_layernorm_bwd(x, gamma, x, inv, workspace=room), want))
