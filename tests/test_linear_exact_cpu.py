"""CPU check that the exact results of linear_exact.py show what is lost, at the sizes where a tolerance may hide it."""
import pytest
import torch

import linear_exact as e


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,H", [(515, 700, 1), (1000, 72, 2000), (2000, 1500, 777), (1030, 2056, 1032)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_plants(T, N, H, dtype, name):
    p = e.inputs(T, N, H, dtype, "cpu", 3)
    right = e.gradients(p, name)
    for w in right:
        e.equal(w.to(dtype), w)

    def without(keys, axis):
        """The gradients without the last token (axis 0) or the last output feature (1)."""
        q = dict(p)
        q["dY"] = p["dY"].clone()
        q["dY"].select(axis, -1).zero_()
        return [e.gradients(q, name)[k] for k in keys]

    for k, lost in ((1, without([1], 0)[0]), (2, without([2], 0)[0]), (0, without([0], 1)[0])):
        with pytest.raises(AssertionError):
            e.equal(lost.to(dtype), right[k])
    y, z = e.forward(p, "none")
    q = dict(p, X=p["X"].clone())
    q["X"][:, -1] = 0
    with pytest.raises(AssertionError):
        e.equal(e.forward(q, "none")[1].to(dtype), z)
    e.equal(y.to(dtype), y)
    bad = z.to(dtype)
    bad[-1, -1] = float("nan")
    with pytest.raises(AssertionError):
        e.equal(bad, z)
