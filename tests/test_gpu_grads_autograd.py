"""GPU checks that autograd notices tensors which clipping has changed."""
import pytest
import torch

import fp32_gemm_05_amd as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("into", [False, True])
def test_a_saved_tensor_that_is_clipped(dtype, into):
    x, other = torch.ones(9, device="cuda", dtype=dtype), torch.ones(3, 5, device="cuda")
    y = torch.full_like(x, 3.0)
    w = torch.ones(9, device="cuda", dtype=dtype, requires_grad=True)
    saved = y if into else x
    product = (w * saved).sum()  # saves it
    tensors, out = [x, other.t()], [y, torch.empty(3, 5, device="cuda").t()]
    versions = [t._version for t in tensors]
    sg.grad_norm(tensors)
    assert [t._version for t in tensors] == versions  # reads alone
    sg.clip_grad_norm(tensors, 0.5, out=out if into else None)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.backward()
    changed, kept = (out, tensors) if into else (tensors, [])
    assert all(t._version > 0 for t in changed) and all(t._version == v for t, v in zip(kept, versions))


def test_tensors_without_a_version():
    """Of inference mode: clipped like others."""
    with torch.inference_mode():
        x = torch.ones(4, device="cuda")
        norm = sg.clip_grad_norm([x], 1.0)
    assert float(norm) == 2 and bool(((x - 0.5).abs() < 1e-6).all())


def test_a_refused_call_changes_no_version():
    x = torch.ones(4, device="cuda")
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([x], -1.0)
    assert x._version == 0
