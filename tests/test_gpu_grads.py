"""GPU checks of the gradients' norm and clipping against 64 bits.

Squares are exact or nearly so in 64 bits and their sum is off by less than n 2^-52 of itself; the norm's root halves
that and its rounding to fp32 is 2^-24.  The factor is computed from the unrounded norm and rounded once (2^-24), each
product once more (fp32 2^-24, bf16 2^-8), or by half of the type's smallest step below its normal range.
"""
import math

import pytest
import torch

import fp32_gemm_05_amd as sg

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16


def exact(tensors, max_norm=None, eps=1e-6):
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in tensors))
    if max_norm is None:
        return norm
    scale = min(1.0, float(torch.tensor(max_norm)) / (norm + float(torch.tensor(eps)))) if not math.isnan(norm) else math.nan
    return norm, [t.double() * scale for t in tensors]


def close(norm, want):
    assert norm.dtype == F32 and norm.shape == ()
    assert abs(float(norm) - want) <= (U + 2.0 ** -30) * want + 1e-45, (float(norm), want)


def same(got, want):
    for g, w in zip(got, want):
        step = 2 * U if g.dtype == F32 else U + B
        tol = w.abs() * step * (1 + step) + (2.0 ** -149 if g.dtype == F32 else 2.0 ** -133)
        bad = ~((g.double() - w).abs() <= tol)
        assert not bool(bad.any()), int(bad.sum())


def check(tensors, max_norm=1.0):
    close(sg.grad_norm(tensors), exact(tensors))
    norm, want = exact(tensors, max_norm)
    before = [t.clone() for t in tensors]
    out = [torch.full_like(t, float("nan")) for t in tensors]  # dense, in the order of its tensor
    close(sg.clip_grad_norm(tensors, max_norm, out=out), norm)
    same(out, want)
    for t, b in zip(tensors, before):
        assert torch.equal(t, b)
    close(sg.clip_grad_norm(tensors, max_norm), norm)
    for t, o in zip(tensors, out):
        assert torch.equal(t, o)


def some(shapes, g, scale=1.0):
    out = []
    for i, shape in enumerate(shapes):
        x = torch.randn(shape, generator=g, device="cuda") * scale * 10 ** (-(i % 5) / 2)
        out.append(x.to(BF16 if i % 3 == 1 else F32))
    return out


@pytest.mark.parametrize("shapes", [
    [(1,)], [(7,)], [(0,), (3,)], [(5, 0), (0, 5), (4, 4)], [(1000, 1000)], [(3, 5, 7, 11), (2,)], [(1 << 21,)] * 2,
    [(i % 17 + 1, i % 31 + 1) for i in range(500)], [(4097, 33), (33, 4097), (1, 70000), (70000, 1)], [()], [(9, 100003)]])
@pytest.mark.parametrize("max_norm", [1.0, 0.0, 1e30])
def test_shapes(shapes, max_norm):
    check(some(shapes, torch.Generator(device="cuda").manual_seed(len(shapes))), max_norm)


def test_views():
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn(300, 205, generator=g, device="cuda")
    b = torch.randn(71, 1003, generator=g, device="cuda").to(BF16)
    big = [t.clone() for t in (a, b)]
    views = [a[:, 3:200], b[5:60, 1:1002], torch.randn(33, 50, generator=g, device="cuda").t(),
             torch.randn(40, 60, generator=g, device="cuda")[1:, 2:31].t(), torch.randn(100, generator=g, device="cuda")[1:]]
    check(views, 0.5)
    # what lies between the views' rows is left as it was
    for now, then, rows, cols in ((a, big[0], slice(0, 300), slice(3, 200)), (b, big[1], slice(5, 60), slice(1, 1002))):
        rest = torch.ones_like(now, dtype=torch.bool)
        rest[rows, cols] = False
        assert torch.equal(now[rest], then[rest])


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 1e18, 1e37])
def test_range(scale):
    """Squares of these leave fp32's range, their norms do not."""
    g = torch.Generator(device="cuda").manual_seed(1)
    tensors = [(torch.rand(1000, generator=g, device="cuda") * scale), (torch.rand(50, generator=g, device="cuda") * scale).to(BF16)]
    check(tensors, scale)


@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_no_number(what):
    tensors = [torch.ones(10, device="cuda"), torch.ones(10, device="cuda", dtype=BF16)]
    tensors[0][3] = what
    norm = sg.grad_norm(tensors)
    assert float(norm) == what or math.isnan(float(norm)) == math.isnan(what) is True
    sg.clip_grad_norm(tensors, 1.0)
    # NaN everywhere, or a factor of 0, of which an infinity makes NaN
    assert bool(tensors[0][3].isnan())
    rest = torch.cat([tensors[0][:3], tensors[1].float()])
    assert bool(rest.isnan().all()) if math.isnan(what) else bool((rest == 0).all())


def test_nothing_to_clip_by_nothing():
    """norm + eps is 0: the tensors stay, whatever max_norm is."""
    for max_norm in (0.0, 1.0):
        x, y = torch.zeros(70, device="cuda"), torch.zeros(5, device="cuda", dtype=BF16)
        out = [torch.ones_like(x), torch.ones_like(y)]
        assert float(sg.clip_grad_norm([x, y], max_norm, eps=0.0, out=out)) == 0
        assert not out[0].any() and not out[1].any()
        sg.clip_grad_norm([x, y], max_norm, eps=0.0)
        assert not x.any() and not y.any()


def test_a_factor_of_one_leaves_the_bits():
    t = torch.tensor([math.nan], device="cuda")
    x = torch.randn(1000, device="cuda").to(BF16)
    y = x.clone()
    sg.clip_grad_norm([x], 1e9)
    assert torch.equal(x, y)
    out = torch.zeros_like(x)
    sg.clip_grad_norm([x], 1e9, out=[out])
    assert torch.equal(out, y) and bool(t.isnan())


def test_refusals():
    a, b = torch.ones(10, 10, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(sg.SgemmArgumentError):  # the same tensor twice
        sg.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([a, a.view(-1)[50:]], 1.0)
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([a, b], 1.0, out=[torch.empty_like(a), a.view(-1)[:4]])
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([a.view(-1)[:50]], 1.0, out=[a.view(-1)[1:51]])
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([a], -1.0)
    with pytest.raises(sg.SgemmArgumentError):
        sg.clip_grad_norm([a], math.nan)
    with pytest.raises(ValueError):
        sg.grad_norm([a.expand(3, 10, 10)])
    with pytest.raises(ValueError):
        sg.clip_grad_norm([a], 1.0, out=[torch.empty(10, 20, device="cuda")[:, ::2]])
    with pytest.raises(ValueError):
        sg.clip_grad_norm([torch.ones(10, 20, device="cuda").t()], 1.0, out=[torch.empty(20, 10, device="cuda")])
    with pytest.raises(ValueError):
        sg.grad_norm([])
    with pytest.raises(TypeError):
        sg.grad_norm([a.double()])
    with pytest.raises(ValueError):
        sg.grad_norm([a.cpu()])
    close(sg.grad_norm([a, a]), math.sqrt(200))  # a norm may count a tensor twice
    assert bool((a == 1).all())
