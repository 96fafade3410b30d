"""The few-token layer against the float64 oracle (GPU only).

Tolerance of y, from the formulas.  u = 2^-24; D(n) = n + 64 roundings for a sum
of n products (a tensor-core step over 16 of them counted as 16 additions).
  g, u' carry D(H) u (|x| |W1|), D(H) u (|x| |W3|); silu' is below 1.1, so
  da <= (1.1 G |u'| + |silu(g)| U) D(H) u + 8 u |a| + half |a|,
half the rounding of bf16 activations: 2^-16 as two bf16 numbers (up to 64 tokens an
expert), 2^-8 as one,
  dout <= da |W2| + D(F) u |a| |W2|,
  dy <= sum_k w_k dout_k + 2 (K + 2) u sum_k w_k |a| |W2| + routing's error on w + half |y|.
"""
import numpy as np
import pytest
import torch

import dropless_top_moe_b200 as moe
from dropless_top_moe_b200._lib import MOE_DEVERR_TIMEOUT
from oracle import moe_oracle as om
from tests._cases import assert_routing, make_case, routing_tol, small_shape

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def reference(c, ids, w, K):
    """y in 64 bits on the device and the bound of its error, for the given routing."""
    x, W1, W3, W2 = (c[k].double() for k in ("x", "W1", "W3", "W2"))
    bf16 = c["x"].dtype == torch.bfloat16
    H, F = W1.shape[1], W1.shape[2]
    N = x.shape[0]
    y = torch.zeros(N, H, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(y)
    lr = om.router_logits(c["x_cpu"], c["W_r_cpu"])
    dw = routing_tol(H, float(np.sqrt(np.mean(lr * lr)))) / 2
    for e in torch.unique(ids).tolist():
        n, k = torch.nonzero(ids == e, as_tuple=True)
        half_act = (2.0 ** -16 if len(n) <= 64 else 2.0 ** -8) if bf16 else 0.0
        g, u = x[n] @ W1[e], x[n] @ W3[e]
        G, Ub = x[n].abs() @ W1[e].abs(), x[n].abs() @ W3[e].abs()
        s = g * torch.sigmoid(g)
        a = s * u
        da = (1.1 * G * u.abs() + s.abs() * Ub) * (H + 64) * U + a.abs() * (8 * U + half_act)
        out, size = a @ W2[e], a.abs() @ W2[e].abs()
        wk = w[n, k].double().unsqueeze(1)
        y.index_add_(0, n, wk * out)
        tol.index_add_(0, n, wk * (da @ W2[e].abs() + size * ((F + 64) + 2 * (K + 2)) * U) + dw * out.abs())
    half_y = torch.finfo(c["x"].dtype).eps / 2
    return y, tol * (1 + half_y) + half_y * y.abs()


def check(layer, c, K, y):
    ref = om.route(c["x_cpu"], c["W_r_cpu"], K)
    assert layer.status() == 0
    np.testing.assert_array_equal(layer.top_experts.cpu().numpy(), ref["top_experts"])
    assert_routing(layer.weights, ref["weights"], c["x"].shape[1], om.router_logits(c["x_cpu"], c["W_r_cpu"]),
                   "weights")
    ids = torch.as_tensor(np.asarray(ref["top_experts"]), device="cuda").long()
    w = torch.as_tensor(np.asarray(ref["weights"]), device="cuda")
    y64, tol = reference(c, ids, w, K)
    err = (y.double() - y64).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def run(shape, seed=0, N_max=None):
    c = make_case(shape, seed=seed, with_dy=False)
    layer = moe.MoEDecodeLayer(N_max or shape.N, shape.H, shape.E, shape.K, shape.F, dtype=shape.torch_dtype)
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    torch.cuda.synchronize()
    check(layer, c, shape.K, y)
    first = y.clone()
    for _ in range(3):
        y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert torch.equal(y, first)
    return layer, c


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 33, 64, 100, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_counts(N, dtype):
    run(small_shape("n", N=N, H=256, E=16, K=4, F=384, dtype=dtype), seed=N)


BF16 = [(5, 128, 1, 1, 128), (9, 128, 2, 1, 256), (3, 256, 5, 5, 128), (40, 384, 7, 3, 640), (20, 512, 256, 8, 128),
        (2, 640, 40, 32, 256), (11, 2048, 64, 6, 1408), (1, 1152, 64, 6, 2944), (128, 128, 3, 2, 1280),
        (64, 1024, 8, 2, 2048), (1, 1024, 16, 16, 2944), (1, 1024, 32, 32, 2944), (2, 1152, 30, 15, 2816),
        (3, 2048, 64, 8, 1408), (4, 1024, 40, 10, 2944), (4, 256, 4, 4, 4096), (3, 4096, 1, 1, 256)]
F32 = [(5, 128, 4, 2, 256), (1, 4, 1, 1, 1), (3, 8, 2, 2, 3), (9, 100, 5, 2, 33), (31, 132, 7, 7, 61), (64, 516, 130, 8, 100),
       (2, 1028, 40, 32, 257), (128, 64, 3, 1, 500), (17, 1000, 12, 3, 1500)]


@pytest.mark.parametrize("sizes", BF16, ids=str)
def test_bf16_shapes(sizes):
    N, H, E, K, F = sizes
    run(small_shape("s", N=N, H=H, E=E, K=K, F=F), seed=3)


@pytest.mark.parametrize("sizes", F32, ids=str)
def test_f32_shapes(sizes):
    N, H, E, K, F = sizes
    run(small_shape("s", N=N, H=H, E=E, K=K, F=F, dtype="f32"), seed=4)


@pytest.mark.parametrize("F", [63, 64, 205, 208, 443, 444])
@pytest.mark.parametrize("H", [188, 384, 388])
def test_f32_tile_widths(H, F):
    """Every pair of widths that gate and up, and down, may take, with and without aligned rows."""
    run(small_shape("w", N=64, H=H, E=30, K=6, F=F, dtype="f32"), seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("skew", [("zipf", 1.0), ("normal", 3.0), ("zipf", 6.0)])
def test_skewed_routing(dtype, skew):
    run(small_shape("z", N=128, H=256, E=32, K=2, F=256, dtype=dtype, skew=skew[0], skew_param=skew[1]), seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_token_on_the_same_experts(dtype):
    """Equal logits in every column but K: all tokens choose experts 3 and 5, 128 rows each."""
    shape = small_shape("same", N=128, H=128, E=8, K=2, F=256, dtype=dtype)
    c = make_case(shape, seed=6, with_dy=False)
    c["W_r"].zero_()
    c["W_r"][0, 3], c["W_r"][0, 5] = 2.0, 1.0
    c["x"][:, 0] = 1.0
    c["x_cpu"], c["W_r_cpu"] = c["x"].cpu(), c["W_r"].cpu()
    layer = moe.MoEDecodeLayer(128, 128, 8, 2, 256, dtype=shape.torch_dtype)
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    check(layer, c, 2, y)


def test_ties_go_to_the_lowest_id():
    shape = small_shape("ties", N=9, H=128, E=100, K=7, F=128)
    c = make_case(shape, seed=7, with_dy=False)
    c["W_r"].zero_()
    layer = moe.MoEDecodeLayer(9, 128, 100, 7, 128)
    layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert torch.equal(layer.top_experts.cpu(), torch.arange(7, dtype=torch.int32).expand(9, 7))
    assert torch.equal(layer.weights, torch.full((9, 7), 1.0, device="cuda") / 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fewer_tokens_than_the_layer_holds(dtype):
    shape = small_shape("part", N=50, H=256, E=16, K=4, F=256, dtype=dtype)
    layer, c = run(shape, seed=8, N_max=128)
    full = layer.y.clone()
    for n in (1, 0, 13, 50, 3):
        layer.y.fill_(7.0)
        part = {k: (v[:n].contiguous() if k in ("x", "x_cpu") else v) for k, v in c.items()}
        y = layer.forward(part["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
        assert y.shape == (n, 256) and layer.top_experts.shape == (n, 4)
        assert bool((layer.y[n:] == 7.0).all())
        if n:
            check(layer, part, 4, y)
    assert full.shape == (128, 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,bad1,bad2", [(12, 2, 7), (4, 1, 2), (2, 0, 1), (1, 0, 0)])
def test_values_that_are_not_finite_stay_in_their_rows(N, bad1, bad2, dtype):
    shape = small_shape("nan", N=N, H=256, E=16, K=2, F=256, dtype=dtype)
    layer, c = run(shape, seed=9)
    clean = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone()
    top = layer.top_experts.clone()
    bad = c["x"].clone()
    bad[bad2, 5] = float("inf")
    bad[bad1] = float("nan")
    y = layer.forward(bad, c["W_r"], c["W1"], c["W3"], c["W2"])
    torch.cuda.synchronize()
    assert layer.status() == 0
    keep = [i for i in range(N) if i not in (bad1, bad2)]
    assert torch.equal(layer.top_experts[keep], top[keep])
    assert bool(y[bad1].isnan().all()) and not bool(torch.isfinite(y[bad2]).all())
    assert bool((layer.top_experts >= 0).all()) and bool((layer.top_experts < 16).all())
    for row in layer.top_experts.tolist():
        assert len(set(row)) == 2
    if keep:
        err = (y[keep].double() - clean[keep].double()).abs()
        assert bool((err <= 2.0 ** -7 * clean[keep].double().abs().amax()).all())
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])      # nothing of it is left behind
    assert torch.equal(y, clean) and layer.status() == 0


def test_output_over_the_input_and_into_a_given_buffer():
    shape = small_shape("alias", N=21, H=256, E=8, K=2, F=512)
    layer, c = run(shape, seed=10)
    want = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone()
    out = torch.empty_like(want)
    assert layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"], y=out) is out
    assert torch.equal(out, want)
    x = c["x"].clone()
    layer.forward(x, c["W_r"], c["W1"], c["W3"], c["W2"], y=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_agrees_with_the_full_layer(dtype):
    """moe_layer_fwd on the same tokens: each is within its bound of the same function."""
    shape = small_shape("full", N=64, H=256, E=16, K=4, F=384, dtype=dtype)
    layer, c = run(shape, seed=11)
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    full = moe.MoELayer(64, 256, 16, 4, 384, dtype=shape.torch_dtype)
    yf = full.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert torch.equal(full.top_experts, layer.top_experts)
    scale = float(yf.double().abs().max())
    # the full layer also rounds each expert's output to the type
    assert float((y.double() - yf.double()).abs().max()) <= (2.0 ** -5 if dtype == "bf16" else 2.0 ** -15) * scale


def test_two_layers_on_two_streams():
    """Overlapping calls on two workspaces, many times; each gives its own result."""
    shapes = [small_shape("a", N=30, H=512, E=32, K=4, F=512), small_shape("b", N=7, H=256, E=8, K=2, F=1024),
              small_shape("c", N=64, H=256, E=16, K=2, F=300, dtype="f32")]
    work = [run(s, seed=12 + i) for i, s in enumerate(shapes)]
    want = [l.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone() for l, c in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(20):
        for (l, c), s in zip(work, streams):
            with torch.cuda.stream(s):
                l.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    torch.cuda.synchronize()
    for (l, c), w in zip(work, want):
        assert l.status() == 0 and torch.equal(l.y, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_replays_from_a_graph_with_new_tokens(dtype):
    shape = small_shape("graph", N=10, H=256, E=16, K=4, F=256, dtype=dtype)
    layer, c = run(shape, seed=15)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    for seed in (16, 17):
        d = make_case(shape, seed=seed, with_dy=False)
        for k in ("x", "W_r", "W1", "W3", "W2"):
            c[k].copy_(d[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(layer, d, 4, y)


def test_serving_and_training_steps_together():
    """Norm, few-token layer and full layer, their gradients and the clipping, as a program runs them:
    one step of a block h = x + r, y = layer(norm(h)) on both paths."""
    N, H, E, K, F = 48, 256, 16, 4, 256
    shape = small_shape("step", N=N, H=H, E=E, K=K, F=F, training=True)
    c = make_case(shape, seed=18, with_dy=True, repair=False)
    r = c["x"].flip(0).contiguous()
    w = torch.linspace(0.5, 1.5, H, device="cuda").to(torch.bfloat16)
    y, h = moe.moe_add_rms_norm(c["x"], w, residual=r)
    few = moe.MoEDecodeLayer(N, H, E, K, F)
    out = few.forward(y, c["W_r"], c["W1"], c["W3"], c["W2"])
    full = moe.MoELayer(N, H, E, K, F, training=True)
    ref = full.forward(y, c["W_r"], c["W1"], c["W3"], c["W2"])
    same = (full.top_experts == few.top_experts).all(dim=1)     # a tie in rounding may order two experts differently
    assert int(same.sum()) >= N - 2
    scale = float(ref.double().abs().max())
    assert float((out.double() - ref.double())[same].abs().max()) <= 2.0 ** -5 * scale
    g = full.backward(c["dy"], y, c["W_r"], c["W1"], c["W3"], c["W2"])
    dx, dw = moe.moe_add_rms_norm_bwd(g["dx"], h, w, dh=c["dy"])
    grads = [g["dW_r"], g["dW1"], g["dW3"], g["dW2"], dw]
    keep = [t.clone() for t in grads]
    norm = moe.moe_clip_grad_norm(grads, 1.0)
    n = float(sum(t.double().square().sum() for t in keep)) ** 0.5
    assert abs(float(norm) - n) <= 17 * U * n and n > 1.0
    after = float(sum(t.double().square().sum() for t in grads)) ** 0.5
    assert abs(after - 1.0) <= 2.0 ** -8 + 1e-6            # each element rounds to bf16 once
    assert full.status() == 0 and few.status() == 0 and bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("H,F", [(128, 128), (256, 512), (1024, 1280)])
@pytest.mark.parametrize("E", [1, 2])
def test_precision_does_not_depend_on_the_other_tokens(E, H, F):
    """The same rows while their experts' tokens grow past 64: every count has the bound of
    activations carried as two numbers (2^-16), which reference() gives to parts of 64."""
    shape = small_shape("split", N=128, H=H, E=E, K=E, F=F)
    c = make_case(shape, seed=20, with_dy=False)
    layer = moe.MoEDecodeLayer(128, H, E, E, F)
    ref = om.route(c["x_cpu"], c["W_r_cpu"], E)
    ids = torch.as_tensor(np.asarray(ref["top_experts"]), device="cuda").long()
    w = torch.as_tensor(np.asarray(ref["weights"]), device="cuda")
    parts = [{k: (v[s:s + 64] if k in ("x", "x_cpu") else v) for k, v in c.items()} for s in (0, 64)]
    y64, tol = (torch.cat(t) for t in zip(*(reference(p, ids[s:s + 64], w[s:s + 64], E)
                                            for p, s in zip(parts, (0, 64)))))
    for n in (64, 65, 72, 80, 81, 96, 97, 112, 127, 128):
        y = layer.forward(c["x"][:n], c["W_r"], c["W1"], c["W3"], c["W2"])
        err = (y.double() - y64[:n]).abs()
        assert layer.status() == 0
        assert bool((err <= tol[:n]).all()), (n, float((err / tol[:n]).max()))


@pytest.mark.parametrize("sizes", [(128, 128, 4, 2, 1280), (100, 128, 16, 8, 4096), (96, 4096, 12, 6, 128),
                                   (128, 128, 8, 8, 8192)], ids=str)
def test_many_tokens_on_many_short_tiles(sizes):
    """Tiles of two units, shorter than the length asked of a ticket for that many tokens."""
    N, H, E, K, F = sizes
    run(small_shape("short", N=N, H=H, E=E, K=K, F=F), seed=28)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 21])
def test_output_over_the_input(N, dtype):
    """y over x in every kernel: other blocks may still read tokens while some write y."""
    shape = small_shape("over", N=N, H=256, E=8, K=2, F=512, dtype=dtype)
    layer, c = run(shape, seed=21)
    want = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone()
    for _ in range(20):
        x = c["x"].clone()
        layer.forward(x, c["W_r"], c["W1"], c["W3"], c["W2"], y=x)
        assert torch.equal(x, want)
    assert layer.status() == 0


def test_layers_of_every_kernel_on_their_own_streams():
    """Overlapping calls of the direct variant (up to four tokens) with the other kernels."""
    shapes = [small_shape("a", N=3, H=1024, E=16, K=4, F=1024), small_shape("b", N=1, H=512, E=32, K=6, F=512),
              small_shape("c", N=30, H=512, E=32, K=4, F=512), small_shape("d", N=4, H=256, E=16, K=2, F=300, dtype="f32")]
    work = [run(s, seed=22 + i) for i, s in enumerate(shapes)]
    want = [l.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone() for l, c in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(30):
        for (l, c), s in zip(work, streams):
            with torch.cuda.stream(s):
                l.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    torch.cuda.synchronize()
    for (l, c), w in zip(work, want):
        assert l.status() == 0 and torch.equal(l.y, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_one_of_the_most_experts_is_used(dtype):
    """256 experts, each with tokens: token n's logits are largest at experts 32 n .. 32 n + 31 (mod 256)."""
    N, H, E, K, F = 24, 128, 256, 32, 128
    shape = small_shape("all", N=N, H=H, E=E, K=K, F=F, dtype=dtype)
    c = make_case(shape, seed=26, with_dy=False, repair=False)
    c["x"].zero_()
    for n in range(N):
        c["x"][n, n % 8] = 1.0
        c["x"][n, 8:] = torch.randn(H - 8, generator=torch.Generator().manual_seed(n)).to(c["x"])
    c["W_r"].zero_()
    for j in range(8):
        c["W_r"][j, 32 * j:32 * j + 32] = 4.0 + torch.arange(32, device="cuda") / 16
    c["x_cpu"], c["W_r_cpu"] = c["x"].cpu(), c["W_r"].cpu()
    layer = moe.MoEDecodeLayer(N, H, E, K, F, dtype=shape.torch_dtype)
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert torch.unique(layer.top_experts).numel() == E
    check(layer, c, K, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 8, 40])
def test_nothing_of_the_workspace_but_its_head_passes_from_call_to_call(N, dtype):
    """Whatever an earlier call, or one that gave up, left behind the workspace's first 256 bytes."""
    shape = small_shape("dirty", N=N, H=256, E=16, K=4, F=384, dtype=dtype)
    layer, c = run(shape, seed=27)
    want = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone()
    for byte in (0x00, 0x01, 0x7f, 0xff):
        layer.ws[256:].fill_(byte)
        y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
        assert layer.status() == 0 and torch.equal(y, want), byte
    assert not bool(layer.ws[:256].any())            # the counters between calls are back at zero


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 20])
def test_waits_on_other_blocks_give_up_and_the_workspace_serves_the_next_call(N, dtype):
    """Every wait on a handed-over value is bounded: it ends with the status bit and tells the others."""
    shape = small_shape("giveup", N=N, H=256, E=16, K=4, F=384, dtype=dtype)
    layer, c = run(shape, seed=29)
    want = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"]).clone()
    seen = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.selftest_handover_timeout(layer.ws, seen, 5_000_000)       # 5 ms each
    torch.cuda.synchronize()
    assert int(seen) == 7 and layer.status() == MOE_DEVERR_TIMEOUT
    # the status stays for whoever asks, and the next call is right all the same
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert layer.status() == MOE_DEVERR_TIMEOUT and torch.equal(y, want)
    moe.ops.call("moe_workspace_init", layer.ws.data_ptr(), layer.ws.numel(), torch.cuda.current_stream().cuda_stream)
    y = layer.forward(c["x"], c["W_r"], c["W1"], c["W3"], c["W2"])
    assert layer.status() == 0 and torch.equal(y, want)


def test_two_graphs_share_a_workspace():
    """Two captured calls of one layer, of different sizes and kernels, replayed in turn on one stream."""
    shape = small_shape("graphs", N=70, H=256, E=16, K=4, F=384)
    layer, c = run(shape, seed=30)
    args = (c["W_r"], c["W1"], c["W3"], c["W2"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = []
    for n in (3, 70, 20):
        x, y = c["x"][:n].clone(), torch.empty(n, 256, dtype=torch.bfloat16, device="cuda")
        want = layer.forward(x, *args).clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            layer.forward(x, *args, y=y)
        calls.append((graph, y, want, x))               # the graph reads x: it has to live
    for i in range(30):
        graph, y, want, _ = calls[(i * i + i // 4) % 3]
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    for call in calls * 5:                              # back to back
        call[0].replay()
    torch.cuda.synchronize()
    assert layer.status() == 0 and all(torch.equal(y, want) for _, y, want, _ in calls)
