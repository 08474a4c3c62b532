"""GPU checks of the vocabulary head's calls on a stream that their operands were not made on."""
import pytest
import torch

import fp32_gemm_05_amd as sg

pytestmark = pytest.mark.gpu
T, V, H, K = 100, 1000, 512, 4


def operands():
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(V, H, generator=g, device="cuda") / H ** 0.5
    index = torch.randint(0, V, (T, K), generator=g, device="cuda")
    return {"X": X, "W": W, "target": index[:, 0].contiguous(), "index": index,
            "teacher": torch.randn(T, K, generator=g, device="cuda"),
            "dloss": torch.rand(T, generator=g, device="cuda")}


CALLS = {
    "vocab_ce": ("X", "W", "target"),
    "vocab_ce_grad": ("X", "W", "target", "lse", "dloss"),
    "vocab_distill": ("X", "W", "index", "teacher"),
    "vocab_distill_grad": ("X", "W", "index", "teacher", "lse", "picked", "dloss"),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_operands_are_kept_until_the_stream_has_read_them(name, handle):
    side = torch.cuda.Stream()
    given = operands()
    if "picked" in CALLS[name]:
        _, given["lse"], given["picked"] = sg.vocab_distill(given["X"], given["W"], given["index"], given["teacher"])
    else:
        _, given["lse"] = sg.vocab_ce(given["X"], given["W"], given["target"])
    want = getattr(sg, name)(*[given[a] for a in CALLS[name]])
    args = [given[a].clone() for a in CALLS[name]]
    del given
    places = {(a.data_ptr(), a.numel() * a.element_size()) for a in args}
    shapes = [(a.shape, a.dtype) for a in args]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # of the order of 0.1 s: the call's work waits behind it
    got = getattr(sg, name)(*args, stream=side.cuda_stream if handle else side)
    assert not side.query()
    del args
    # what the current stream allocates now is other memory
    again = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
    assert not side.query()
    assert not any(p < a.data_ptr() + a.numel() * a.element_size() and a.data_ptr() < p + n for a in again for p, n in places)
    for a in again:
        a.fill_(1)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
