"""Residual addition + RMS norm, forward and backward, against the formulas in
64 bits (GPU only).

Tolerances.  u = 2^-24 is the unit roundoff of fp32, half = eps(dtype) / 2 that
of the stored type.  A row's sum of squares adds positive terms over at most 32
sequential steps of a thread and 10 levels of a tree, so its relative error is
below 42 u and that of s = 1/sqrt(...) below 27 u with its own operations; y
takes two more products and the store's rounding.  In the backward the dot product
has signed terms: its error is below 44 u times the sum of their magnitudes.
"""
import pytest
import torch

import dropless_top_moe_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).tiny


def forward64(x, r, w, eps):
    h = x.double() if r is None else (x.float() + r.float()).to(x.dtype).double()
    s = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    return h * s * w.double(), h


def backward64(dy, h, w, dh, eps):
    dy, h, w = dy.double(), h.double(), w.double()
    s = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    g, xhat = dy * w, h * s
    dot = (g * xhat).mean(dim=1, keepdim=True)
    dx = s * (g - xhat * dot)
    size = s * (g.abs() + xhat.abs() * (g * xhat).abs().mean(dim=1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    terms = dy * xhat
    return dx, size, terms.sum(dim=0), terms.abs().sum(dim=0)


def check_forward(y, h, x, r, w, eps=EPS):
    y64, h64 = forward64(x, r, w, eps)
    assert torch.equal(h.double(), h64)
    tol = y64.abs() * (half(y.dtype) + 32 * U) + tiny(y.dtype)
    assert bool(((y.double() - y64).abs() <= tol).all())


def check_backward(dx, dw, dy, h, w, dh, eps=EPS):
    N = dy.shape[0]
    dx64, size, dw64, terms = backward64(dy, h, w, dh, eps)
    # 27 u on s twice, 44 u on the dot product, four operations: below 128 u of the terms' sizes
    tol = dx64.abs() * half(dx.dtype) + size * 128 * U + tiny(dx.dtype)
    assert bool(((dx.double() - dx64).abs() <= tol).all())
    # a block's rows in sequence (at least 148 blocks once there are as many rows), then at most
    # 148 * 16 / 16 + 16 partial sums; each term carries s's 27 u and a product
    steps = N // 148 + 1 + 148 + 16 + 32
    tol = dw64.abs() * half(dw.dtype) + terms * steps * U + tiny(dw.dtype)
    assert bool(((dw.double() - dw64).abs() <= tol).all())


SHAPES = [(1, 8), (1, 2048), (2, 128), (3, 136), (7, 1000), (147, 256), (149, 2048), (300, 4096), (1021, 7168),
          (33, 8192), (5000, 512), (40000, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES)
def test_forward(N, H, dtype):
    dt = DT[dtype]
    x, r, w = rand((N, H), dt, 1), rand((N, H), dt, 2), rand((H,), dt, 3)
    y, h = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS)
    check_forward(y, h, x, r, w)
    y, h = moe.moe_add_rms_norm(x, w, eps=EPS)
    assert h is x
    check_forward(y, h, x, None, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H", SHAPES)
def test_backward(N, H, dtype):
    dt = DT[dtype]
    dy, h, dh, w = (rand((N, H), dt, s) for s in (4, 5, 6, 7))
    w = w[0].contiguous()
    for extra in (dh, None):
        dx, dw = moe.moe_add_rms_norm_bwd(dy, h, w, dh=extra, eps=EPS)
        check_backward(dx, dw, dy, h, w, extra)
        again = moe.moe_add_rms_norm_bwd(dy, h, w, dh=extra, eps=EPS)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_widest_rows():
    for dt, H in ((torch.bfloat16, 16384), (torch.float32, 8192), (torch.bfloat16, 8200)):
        x, r, w, dy = rand((9, H), dt, 1), rand((9, H), dt, 2), rand((H,), dt, 3), rand((9, H), dt, 4)
        y, h = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS)
        check_forward(y, h, x, r, w)
        dx, dw = moe.moe_add_rms_norm_bwd(dy, h, w, dh=r, eps=EPS)
        check_backward(dx, dw, dy, h, w, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    dt = DT[dtype]
    x, w = rand((0, 256), dt, 1), rand((256,), dt, 2)
    y, h = moe.moe_add_rms_norm(x, w, residual=x.clone())
    assert y.shape == h.shape == (0, 256)
    dx, dw = moe.moe_add_rms_norm_bwd(x, x, w)
    assert dx.shape == (0, 256) and torch.equal(dw, torch.zeros_like(w))


def test_zero_and_large_rows_and_values_that_are_not_finite():
    x = rand((6, 512), torch.float32, 1)
    r = torch.zeros_like(x)
    x[1] = 0.0
    x[2] *= 1e-20             # squares underflow: the row is divided by sqrt(eps)
    x[3] *= 1e15
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    w = rand((512,), torch.float32, 2)
    y, h = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS)
    check_forward(y[:4], h[:4], x[:4], r[:4], w)
    assert bool((y[1] == 0).all())
    assert bool(y[4].isnan().all())               # the row's own values only
    assert bool(y[5, 9].isnan()) and bool((y[5, :9] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    dt = DT[dtype]
    N, H = 1500, 1024
    x, r, w = rand((N, H), dt, 1), rand((N, H), dt, 2), rand((H,), dt, 3)
    y0, h0 = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS)
    xs, rs = x.clone(), r.clone()
    y, h = moe.moe_add_rms_norm(xs, w, residual=rs, eps=EPS, y=xs, h=rs)
    assert y is xs and h is rs and torch.equal(y, y0) and torch.equal(h, h0)
    dy, dh = rand((N, H), dt, 4), rand((N, H), dt, 5)
    dx0, dw0 = moe.moe_add_rms_norm_bwd(dy, h0, w, dh=dh, eps=EPS)
    for which in range(3):
        t = [dy.clone(), h0.clone(), dh.clone()]
        dx, dw = moe.moe_add_rms_norm_bwd(t[0], t[1], w, dh=t[2], eps=EPS, dx=t[which])
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_more_than_32_bits_of_elements():
    N, H = (1 << 32) // 8192 + 77, 8192
    x = torch.empty((N, H), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    w = rand((H,), torch.bfloat16, 2)
    rows = [0, 1, (1 << 31) // H, (1 << 32) // H - 1, (1 << 32) // H, N - 1]
    keep = x[rows].clone()
    y, h = moe.moe_add_rms_norm(x, w, eps=EPS, y=x)
    assert y is x
    check_forward(y[rows], keep, keep, None, w)
    dx, _ = moe.moe_add_rms_norm_bwd(y, y, w, eps=EPS, dx=None)
    for i in rows:
        dx64, size, _, _ = backward64(y[i:i + 1], y[i:i + 1], w, None, EPS)
        tol = dx64.abs() * half(dx.dtype) + size * 128 * U + tiny(dx.dtype)
        assert bool(((dx[i:i + 1].double() - dx64).abs() <= tol).all()), i


def test_gradient_against_differences():
    """Directional derivatives of sum(y * dy) + sum(h * dh) by central differences of the
    formula in 64 bits.  With a step of 1e-4 the cubic term is below 1e-6 relative."""
    N, H = 5, 256
    x, r, w, dy, dh = (rand((N, H), torch.float32, s) for s in range(1, 6))
    w = w[0].contiguous()
    y, h = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS)
    dx, dw = moe.moe_add_rms_norm_bwd(dy, h, w, dh=dh, eps=EPS)

    def value(h64, w64):
        s = 1.0 / torch.sqrt((h64 * h64).mean(dim=1, keepdim=True) + EPS)
        return (h64 * s * w64 * dy.double()).sum() + (h64 * dh.double()).sum()

    t = 1e-4
    v, vw = rand((N, H), torch.float32, 8).double(), rand((H,), torch.float32, 9).double()
    hd, wd = h.double(), w.double()
    num = (value(hd + t * v, wd) - value(hd - t * v, wd)) / (2 * t)
    size = (dx.double() * v).abs().sum()
    assert abs(float((dx.double() * v).sum() - num)) <= 1e-5 * float(size)
    num = (value(hd, wd + t * vw) - value(hd, wd - t * vw)) / (2 * t)
    assert abs(float((dw.double() * vw).sum() - num)) <= 1e-5 * float((dw.double() * vw).abs().sum())


def test_replays_from_a_graph_and_on_another_stream():
    N, H = 700, 2048
    x, r, w, dy = (rand((N, H), torch.bfloat16, s) for s in range(1, 5))
    w = w[0].contiguous()
    y, h = moe.moe_add_rms_norm(x, w, residual=r)
    dx, dw = moe.moe_add_rms_norm_bwd(dy, h, w, dh=r)
    want = [t.clone() for t in (y, h, dx, dw)]
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        moe.moe_add_rms_norm(x, w, residual=r, y=y, h=h)
        moe.moe_add_rms_norm_bwd(dy, h, w, dh=r, dx=dx, dweight=dw, ws=ws)
    for _ in range(2):
        for t in (y, h, dx, dw):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, h, dx, dw), want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_without_a_residual_has_no_h_to_give(dtype):
    """h is x there, and y has taken its place: what came back as h would be y, and the
    backward pass of it another function's."""
    dt = DT[dtype]
    x, w, dy = rand((37, 256), dt, 1), rand((256,), dt, 2), rand((37, 256), dt, 3)
    keep = x.clone()
    y, h = moe.moe_add_rms_norm(x, w, eps=EPS, y=x)
    assert y is x and h is None
    check_forward(y, keep, keep, None, w)
    x = keep.clone()
    y, h = moe.moe_add_rms_norm(x, w, eps=EPS, y=x.view(37, 256))      # another tensor of the same memory
    assert h is None and torch.equal(x, y)
    y, h = moe.moe_add_rms_norm(keep, w, eps=EPS, y=torch.empty_like(keep))
    assert h is keep
    dx, dw = moe.moe_add_rms_norm_bwd(dy, h, w, eps=EPS)
    check_backward(dx, dw, dy, keep, w, None)
    r = rand((37, 256), dt, 4)
    x = keep.clone()
    y, h = moe.moe_add_rms_norm(x, w, residual=r, eps=EPS, y=x)        # with a residual h has a buffer of its own
    check_forward(y, h, keep, r, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_way_in_place(dtype):
    """h over x or residual, y over the other, either alone, x and residual the same tensor."""
    dt = DT[dtype]
    N, H = 700, 1024
    x0, r0, w = rand((N, H), dt, 1), rand((N, H), dt, 2), rand((H,), dt, 3)
    want = moe.moe_add_rms_norm(x0, w, residual=r0, eps=EPS)
    for hs, ys in (("x", "r"), ("r", "x"), ("x", None), ("r", None), (None, "x"), (None, "r")):
        t = {"x": x0.clone(), "r": r0.clone(), None: None}
        y, h = moe.moe_add_rms_norm(t["x"], w, residual=t["r"], eps=EPS, y=t[ys], h=t[hs])
        assert torch.equal(y, want[0]) and torch.equal(h, want[1]), (hs, ys)
    want = moe.moe_add_rms_norm(x0, w, residual=x0, eps=EPS)
    check_forward(*want, x0, x0, w)
    for which in ("h", "y"):
        t = x0.clone()
        y, h = moe.moe_add_rms_norm(t, w, residual=t, eps=EPS, **{which: t})
        assert torch.equal(y, want[0]) and torch.equal(h, want[1]), which
    dy = rand((N, H), dt, 4)
    want = moe.moe_add_rms_norm_bwd(dy, x0, w, dh=dy, eps=EPS)
    check_backward(*want, dy, x0, w, dy)
    got = moe.moe_add_rms_norm_bwd(dy, x0, w, dh=dy, eps=EPS, dx=dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
