"""The experts' products against plain 64-bit forms.

Two kinds of inputs.  Small whole numbers, whose sums every type here holds
exactly, so outputs must be equal: this shows a wrong index.  Normal numbers, with
the bound of the arithmetic: an fp32 sum of K products, taken in any order and
rounded or cut at every step, is off by at most (K + 8) 2^-23 sum |products|; the
result is rounded to its type once (u_t |value|)."""
import numpy as np
import pytest
import torch

import expert_ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}

# group sizes; in, out.  The first of each pair of widths are multiples of 8.
GROUPS = {
    "one": [1],
    "dense": [300],
    "empty ends": [0, 0, 5, 0, 17, 0],
    "ragged": [1, 33, 0, 64, 127, 129, 2, 31, 32],
    "wide": [257, 0, 700, 255],
    "many": [3, 0, 1, 9, 0, 20] * 12,
    "nothing": [0, 0, 0],
}
WIDTHS = [(64, 128), (768, 256), (8, 8), (136, 72), (200, 328), (16, 512), (1, 1), (33, 50), (77, 130)]


def f64(t):
    return t.double().cpu().numpy()


def offsets_of(sizes, lead=0):
    return np.cumsum([lead] + list(sizes)).astype(np.int32)


def whole(rng, shape, k):
    """Numbers of -2..2, thinned so that a sum of k products of two of them stays below 256."""
    keep = min(1.0, (30.0 / max(k, 1)) ** 0.5)
    return rng.integers(-2, 3, shape) * (rng.random(shape) < keep)


def tensor(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(TYPES[dtype])


def bound(terms, want, k, out):
    return UNIT[out] * np.abs(want) + (1 + UNIT[out]) * (k + 8) * 2.0 ** -23 * terms + TINY[out]


def inputs(rng, kind, sizes, cin, cout, dtype, extra):
    """x, w, dy (with `extra` rows behind the last group holding NaN), as tensors and in 64 bits."""
    rows = sum(sizes)
    make = (lambda s, k: whole(rng, s, k)) if kind == "whole" else (lambda s, k: rng.normal(size=s))
    x = np.concatenate([make((rows, cin), cin), np.full((extra, cin), np.nan)])
    dy = np.concatenate([make((rows, cout), max(cout, max(sizes))), np.full((extra, cout), np.nan)])
    w = make((len(sizes), cout, cin), max(cin, cout))
    t = [tensor(a, dtype) for a in (x, w, dy)]
    return t, [f64(a) for a in t]


@pytest.mark.parametrize("kind", ["whole", "normal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("widths", WIDTHS)
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_products(ro, groups, widths, dtype, kind):
    sizes, (cin, cout), extra = GROUPS[groups], widths, 3
    rng = np.random.default_rng(len(groups) + cin)
    (x, w, dy), (x64, w64, dy64) = inputs(rng, kind, sizes, cin, cout, dtype, extra)
    offsets = offsets_of(sizes)
    at = torch.from_numpy(offsets).cuda()
    rows = int(offsets[-1])

    def check(got, want, terms, k, out=dtype):
        got = f64(got)
        if kind == "whole":
            assert (got == want).all()
        else:
            assert (np.abs(got - want) <= bound(terms, want, k, out)).all()

    y = torch.full((rows + extra, cout), 5.0, dtype=x.dtype, device="cuda")
    ro.rowops_expert_matmul(x, w, at, y=y)
    check(y[:rows], expert_ref.matmul(x64, w64, offsets)[:rows], expert_ref.matmul(abs(x64), abs(w64), offsets)[:rows],
          cin)
    assert (y[rows:] == 5).all()  # rows behind the last group stay

    dx = torch.full((rows + extra, cin), 5.0, dtype=x.dtype, device="cuda")
    ro.rowops_expert_matmul(dy, w, at, y=dx, transposed=True)
    wt = w64.transpose(0, 2, 1)
    check(dx[:rows], expert_ref.matmul(dy64, wt, offsets)[:rows], expert_ref.matmul(abs(dy64), abs(wt), offsets)[:rows],
          cout)
    assert (dx[rows:] == 5).all()

    want, terms = expert_ref.wgrad(dy64, x64, offsets), expert_ref.wgrad(abs(dy64), abs(x64), offsets)
    for out in (dtype, "f32"):
        dw = torch.full(want.shape, 5.0, dtype=TYPES[out], device="cuda")
        ro.rowops_expert_matmul_wgrad(dy, x, at, dw=dw)
        check(dw, want, terms, max(sizes), out)  # experts without rows: zeros


@pytest.mark.parametrize("widths", [(768, 256), (77, 130)])
def test_long_sums(ro, widths):
    """Enough rows and steps that every buffer of the pipeline is used many times."""
    cin, cout = widths
    sizes = [2000, 1, 0, 1500, 531]
    rng = np.random.default_rng(5)
    (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", sizes, cin, cout, "f16", 0)
    offsets = offsets_of(sizes)
    at = torch.from_numpy(offsets).cuda()
    assert (f64(ro.rowops_expert_matmul(x, w, at)) == expert_ref.matmul(x64, w64, offsets)).all()
    assert (f64(ro.rowops_expert_matmul_wgrad(dy, x, at, dtype=torch.float32))
            == expert_ref.wgrad(dy64, x64, offsets)).all()


@pytest.mark.parametrize("widths", [(33, 50), (77, 136), (136, 77), (1, 1)])
@pytest.mark.parametrize("groups", sorted(GROUPS))
def test_without_a_workspace(ro, groups, widths):
    """Rows off 16-byte boundaries with too little room for a copy: the kernel that takes any alignment."""
    sizes, (cin, cout) = GROUPS[groups], widths
    rng = np.random.default_rng(13)
    little = torch.empty(16, dtype=torch.uint8, device="cuda")
    for dtype in ("bf16", "f16"):
        (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", sizes, cin, cout, dtype, 0)
        offsets = offsets_of(sizes)
        at = torch.from_numpy(offsets).cuda()
        y = ro.rowops_expert_matmul(x, w, at, workspace=little)
        assert (f64(y) == expert_ref.matmul(x64, w64, offsets)).all()
        dx = ro.rowops_expert_matmul(dy, w, at, transposed=True, workspace=little)
        assert (f64(dx) == expert_ref.matmul(dy64, w64.transpose(0, 2, 1), offsets)).all()
        for out in (dtype, "f32"):
            dw = ro.rowops_expert_matmul_wgrad(dy, x, at, dtype=TYPES[out], workspace=little)
            assert (f64(dw) == expert_ref.wgrad(dy64, x64, offsets)).all()


def test_a_workspace_of_the_callers(ro):
    """Exactly the bytes that are asked for, with guard bytes around them."""
    rng = np.random.default_rng(14)
    sizes, cin, cout = [40, 0, 70], 33, 50
    (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", sizes, cin, cout, "f16", 0)
    offsets = offsets_of(sizes)
    at = torch.from_numpy(offsets).cuda()

    def room(need):
        buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + need]

    calls = [(ro.rowops_expert_matmul_workspace(110, cin, cout, 3),
              lambda ws: ro.rowops_expert_matmul(x, w, at, workspace=ws), expert_ref.matmul(x64, w64, offsets)),
             (ro.rowops_expert_matmul_workspace(110, cout, cin, 3, True),
              lambda ws: ro.rowops_expert_matmul(dy, w, at, transposed=True, workspace=ws),
              expert_ref.matmul(dy64, w64.transpose(0, 2, 1), offsets)),
             (ro.rowops_expert_matmul_wgrad_workspace(110, cin, cout),
              lambda ws: ro.rowops_expert_matmul_wgrad(dy, x, at, workspace=ws), expert_ref.wgrad(dy64, x64, offsets))]
    for need, call, want in calls:
        buf, ws = room(need)
        assert need > 0 and (f64(call(ws)) == want).all()
        assert (buf[:256] == 77).all() and (buf[256 + need:] == 77).all()
        buf, ws = room(need)
        assert (f64(call(ws[16:])) == want).all()  # 16 bytes fewer: another kernel or the slack


@pytest.mark.parametrize("widths", [(64, 128), (33, 50)])
def test_dense_without_offsets(ro, widths):
    cin, cout = widths
    rng = np.random.default_rng(6)
    (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", [200], cin, cout, "bf16", 0)
    assert (f64(ro.rowops_expert_matmul(x, w)) == expert_ref.matmul(x64, w64, None)).all()
    assert (f64(ro.rowops_expert_matmul_wgrad(dy, x)) == expert_ref.wgrad(dy64, x64, None)).all()


@pytest.mark.parametrize("widths", [(64, 128), (136, 72), (33, 50)])
def test_groups_that_start_late(ro, widths):
    """Rows before the first group are not read (NaN) and not written."""
    cin, cout = widths
    rng = np.random.default_rng(7)
    sizes, lead = [5, 40, 9], 11
    (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", [lead] + sizes, cin, cout, "f16", 2)
    w, w64 = w[1:].contiguous(), w64[1:]
    x[:lead], dy[:lead] = float("nan"), float("inf")
    offsets = offsets_of(sizes, lead)
    at = torch.from_numpy(offsets).cuda()
    y = torch.full((x.shape[0], cout), 5.0, dtype=x.dtype, device="cuda")
    ro.rowops_expert_matmul(x, w, at, y=y)
    end = offsets[-1]
    assert (f64(y[lead:end]) == expert_ref.matmul(x64, w64, offsets)[lead:end]).all()
    assert (y[:lead] == 5).all() and (y[end:] == 5).all()
    assert (f64(ro.rowops_expert_matmul_wgrad(dy, x, at)) == expert_ref.wgrad(dy64, x64, offsets)).all()


@pytest.mark.parametrize("widths", [(64, 128), (72, 136), (33, 50)])
def test_non_finite_stays_in_its_row_and_expert(ro, widths):
    cin, cout = widths
    rng = np.random.default_rng(8)
    sizes = [20, 30, 50]
    (x, w, dy), _ = inputs(rng, "normal", sizes, cin, cout, "bf16", 0)
    at = torch.from_numpy(offsets_of(sizes)).cuda()
    x[25, 3], w[2, 1, :] = float("nan"), float("inf")
    y = ro.rowops_expert_matmul(x, w, at)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[25], want[50:, 1] = True, True
    assert torch.equal(bad, want)
    dx = ro.rowops_expert_matmul(dy, w, at, transposed=True)
    assert torch.isfinite(dx[:50]).all() and not torch.isfinite(dx[50:]).any()
    dw = ro.rowops_expert_matmul_wgrad(dy, x, at)
    bad = ~torch.isfinite(dw)
    assert bad[1, :, 3].all() and bad.sum() == cout


def test_bad_offsets_stay_in_bounds(ro):
    """Offsets out of range or falling: clamped, so nothing outside y and dw is written."""
    for cin, cout in ((64, 128), (33, 50)):
        x = torch.randn(100, cin, device="cuda").bfloat16()
        dy = torch.randn(100, cout, device="cuda").bfloat16()
        w = torch.randn(4, cout, cin, device="cuda").bfloat16()
        for bad in ([-50, 2 ** 31 - 1, 30, 10, 200], [0, 40, 20, 90, 100], [100] * 5, [-2 ** 31] * 5, [5, 0, 100, 0, 100]):
            at = torch.tensor(bad, dtype=torch.int32, device="cuda")
            guard = torch.full((300, cout), 9.0, dtype=torch.bfloat16, device="cuda")
            ro.rowops_expert_matmul(x, w, at, y=guard[100:200])
            wide = torch.full((6, cout, cin), 9.0, dtype=torch.bfloat16, device="cuda")
            ro.rowops_expert_matmul_wgrad(dy, x, at, dw=wide[1:5])
            torch.cuda.synchronize()
            assert (guard[:100] == 9).all() and (guard[200:] == 9).all()
            assert (wide[0] == 9).all() and (wide[5] == 9).all()


@pytest.mark.parametrize("shift", ["x", "w", "y"])
def test_unaligned_buffers(ro, shift):
    """A buffer one element past a 16-byte boundary, the others on one."""
    rng = np.random.default_rng(10)
    sizes = [40, 0, 70]
    (x, w, dy), (x64, w64, dy64) = inputs(rng, "whole", sizes, 64, 128, "f16", 0)
    offsets = offsets_of(sizes)
    at = torch.from_numpy(offsets).cuda()

    def moved(t, there):
        if not there:
            return t
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    y = moved(torch.zeros(110, 128, dtype=x.dtype, device="cuda"), shift == "y")
    ro.rowops_expert_matmul(moved(x, shift == "x"), moved(w, shift == "w"), at, y=y)
    assert (f64(y) == expert_ref.matmul(x64, w64, offsets)).all()
    dw = moved(torch.zeros(3, 128, 64, dtype=x.dtype, device="cuda"), shift == "w")
    ro.rowops_expert_matmul_wgrad(moved(dy, shift == "y"), moved(x, shift == "x"), at, dw=dw)
    assert (f64(dw) == expert_ref.wgrad(dy64, x64, offsets)).all()


def test_gradients_by_differences(ro):
    """The product is bilinear: differences of a whole-number loss are exact."""
    rng = np.random.default_rng(12)
    sizes = [9, 0, 14]
    (x, w, dy), _ = inputs(rng, "whole", sizes, 16, 24, "f16", 0)
    at = torch.from_numpy(offsets_of(sizes)).cuda()

    def loss(x, w):
        return (ro.rowops_expert_matmul(x, w, at).double() * dy.double()).sum()

    dx = ro.rowops_expert_matmul(dy, w, at, transposed=True)
    dw = ro.rowops_expert_matmul_wgrad(dy, x, at)
    for s, c in ((0, 0), (8, 15), (9, 3), (22, 7)):
        x2 = x.clone()
        x2[s, c] += 1
        assert loss(x2, w) - loss(x, w) == dx[s, c].double()
    for e, n, c in ((0, 0, 0), (0, 23, 15), (1, 2, 2), (2, 5, 9)):
        w2 = w.clone()
        w2[e, n, c] += 1
        assert loss(x, w2) - loss(x, w) == dw[e, n, c].double()


def test_refusals(ro):
    x = torch.zeros(8, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(2, 24, 16, device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: ro.rowops_expert_matmul(x, w), lambda: ro.rowops_expert_matmul(x, w, at[:2]),
                 lambda: ro.rowops_expert_matmul(x, w, at, transposed=True),
                 lambda: ro.rowops_expert_matmul(x[:, :8], w[:, :, :8].contiguous(), at),
                 lambda: ro.rowops_expert_matmul(x, w, at, y=torch.zeros(8, 23, device="cuda", dtype=x.dtype)),
                 lambda: ro.rowops_expert_matmul_wgrad(x[:4], x, at)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ro.rowops_expert_matmul(x, w.half(), at), lambda: ro.rowops_expert_matmul(x.float(), w, at),
                 lambda: ro.rowops_expert_matmul(x, w, at.long()),
                 lambda: ro.rowops_expert_matmul_wgrad(x, x, at, dw=torch.zeros(2, 16, 16, device="cuda").half())):
        with pytest.raises(TypeError):
            call()
