"""Matrices that start off a 16-byte boundary: copied for the tensor cores as odd
widths are, with the same results bit for bit as on a boundary."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def off(t):
    """The same values one element later than a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def launches(ro, call):
    before = ro.rowops_kernel_launches()
    out = call()
    return out, ro.rowops_kernel_launches() - before


SIZES = [700, 0, 33, 300]
SHIFTS = [(True, False), (False, True), (True, True)]


def matrices(cin, cout, dtype):
    g = torch.Generator(device="cuda").manual_seed(cin)
    rows = sum(SIZES)
    at = torch.from_numpy(np.cumsum([0, *SIZES]).astype(np.int32)).cuda()
    make = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(dtype)  # noqa: E731
    return make(rows, cin), make(len(SIZES), cout, cin), make(rows, cout), at


@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("widths", [(768, 256), (136, 72), (64, 77), (77, 64)])
def test_products(ro, widths, shift):
    x, w, dy, at = matrices(*widths, torch.bfloat16)
    move = [off if s else (lambda t: t) for s in shift]
    for a, b, call in ((x, w, lambda a, b: ro.rowops_expert_matmul(a, b, at)),
                       (dy, w, lambda a, b: ro.rowops_expert_matmul(a, b, at, transposed=True)),
                       (dy, x, lambda a, b: ro.rowops_expert_matmul_wgrad(a, b, at))):
        want = call(a, b)
        got, n = launches(ro, lambda: call(move[0](a), move[1](b)))
        assert n == 2  # the copies and the product; one alone would be the kernel for any alignment
        assert torch.equal(got, want)


@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("widths", [(768, 256), (144, 77)])
def test_8bit(ro, widths, shift):
    x, w, _, at = matrices(*widths, torch.bfloat16)
    move = [off if s else (lambda t: t) for s in shift]
    xq, xs = ro.rowops_quantize_blocks(x)
    wq, ws = ro.rowops_quantize_blocks(w, block_rows=128)
    want = ro.rowops_expert_matmul_fp8(xq, xs, wq, ws, at)
    got, n = launches(ro, lambda: ro.rowops_expert_matmul_fp8(move[0](xq), xs, move[1](wq), ws, at))
    assert n == 2 and torch.equal(got, want)


def test_the_documented_bytes_are_enough(ro):
    """A matrix off a boundary takes its own bytes and 512 more, between guard bytes."""
    x, w, dy, at = matrices(136, 72, torch.float16)
    want = ro.rowops_expert_matmul(x, w, at)
    need = 2 * (x.numel() + w.numel()) + 2 * 512
    buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    for skip in (0, 16, 240):  # 16-byte aligned is enough
        got, n = launches(ro, lambda: ro.rowops_expert_matmul(off(x), off(w), at, workspace=buf[256 + skip:256 + need]
                                                              if skip == 0 else buf[256 - skip:256 - skip + need]))
        assert n == 2 and torch.equal(got, want)
    assert (buf[:16] == 77).all() and (buf[256 + need:] == 77).all()
