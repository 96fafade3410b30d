"""Global gradient norm and clipping against the formula in 64 bits (GPU only).

Tolerances.  u = 2^-24.  A thread adds at most 32 positive squares in fp32 and
the rest runs in double: the sum is off by less than 33 u, the norm by less
than 17 u with its own rounding, the factor by less than 18 u; a scaled gradient by
one product's rounding more and the store's.
"""
import math

import pytest
import torch

import dropless_top_moe_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(norm, outs, grads, max_norm):
    n = norm64(grads)
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(float(norm) - n) <= 17 * U * n
    f = min(1.0, max_norm / (n + 1e-6))
    for o, g in zip(outs, grads):
        want = g.double() * f
        tol = want.abs() * (torch.finfo(g.dtype).eps / 2 + 20 * U) + torch.finfo(g.dtype).tiny
        assert o.dtype == g.dtype and bool(((o.double() - want).abs() <= tol).all())


LISTS = {
    "one": [(7,)],
    "layer": [(128, 4), (4, 128, 256), (4, 128, 256), (4, 256, 128), (128,)],
    "odd": [(1,), (3,), (8,), (9,), (4095,), (4096,), (4097,), (333, 1001), (0,), (5, 0, 2), (17,)],
    "large": [(64, 512, 300), (1 << 22,)],
    "many": [(i % 37 + 1, 19) for i in range(1700)],      # several launches of the longest table
    "hundred": [(513,)] * 100,
}


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("name", sorted(LISTS))
def test_clips_to_the_norm(name, kind):
    dts = {"f32": [torch.float32], "bf16": [torch.bfloat16], "mixed": [torch.float32, torch.bfloat16]}[kind]
    grads = [rand(s, dts[i % len(dts)], i) for i, s in enumerate(LISTS[name])]
    keep = [g.clone() for g in grads]
    n = norm64(grads)
    outs = [torch.empty_like(g) for g in grads]
    norm = moe.moe_clip_grad_norm(grads, 0.3 * n, outs=outs)
    check(norm, outs, keep, 0.3 * n)
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    again = [torch.empty_like(g) for g in grads]
    norm2 = moe.moe_clip_grad_norm(grads, 0.3 * n, outs=again)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(outs, again))
    norm3 = moe.moe_clip_grad_norm(grads, 0.3 * n)                   # in place
    assert torch.equal(norm, norm3) and all(torch.equal(a, b) for a, b in zip(outs, grads))


def test_below_the_limit_nothing_changes():
    grads = [rand((1000,), torch.bfloat16, 1), rand((77, 3), torch.float32, 2)]
    keep = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    for limit in (2 * norm64(grads), math.inf):
        norm = moe.moe_clip_grad_norm(grads, limit, outs=outs)
        check(norm, outs, keep, limit)
        assert all(torch.equal(o, k) for o, k in zip(outs, keep))
        moe.moe_clip_grad_norm(grads, limit)
        assert all(torch.equal(g, k) for g, k in zip(grads, keep))


def test_offset_views():
    """Views of one buffer that start and end off the 16-byte boundaries, the neighbours untouched."""
    for dt in (torch.float32, torch.bfloat16):
        flat = rand((40000,), dt, 3)
        keep = flat.clone()
        cuts = [(1, 2), (3, 4), (5, 12), (13, 5000), (5001, 5001 + 8191), (14001, 39999)]
        grads = [flat[a:b] for a, b in cuts]
        ref = [g.clone() for g in grads]
        n = norm64(ref)
        outflat = torch.full((40003,), 7.0, dtype=dt, device="cuda")
        outs = [outflat[a + 3:b + 3] for a, b in cuts]           # another offset than the inputs
        check(moe.moe_clip_grad_norm(grads, 0.5 * n, outs=outs), outs, ref, 0.5 * n)
        check(moe.moe_clip_grad_norm(grads, 0.5 * n), grads, ref, 0.5 * n)
        mask = torch.ones(40000, dtype=torch.bool, device="cuda")
        for a, b in cuts:
            mask[a:b] = False
        assert torch.equal(flat[mask], keep[mask])
        assert bool((outflat[3:][mask] == 7.0).all()) and bool((outflat[:3] == 7.0).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-12, 1e12, 1e22, 1e30])
def test_norms_whose_squares_leave_the_range(scale):
    grads = [rand((5000,), torch.float32, 1, scale), rand((5000,), torch.bfloat16, 2, scale),
             torch.zeros(9000, device="cuda")]
    n = norm64(grads)
    outs = [torch.empty_like(g) for g in grads]
    check(moe.moe_clip_grad_norm(grads, 0.25 * n, outs=outs), outs, grads, 0.25 * n)


def test_a_large_and_small_gradients_together():
    grads = [torch.full((3000,), 1e-25, device="cuda"), torch.full((3,), 1e20, device="cuda")]
    outs = [torch.empty_like(g) for g in grads]
    check(moe.moe_clip_grad_norm(grads, 1.0, outs=outs), outs, grads, 1.0)


def test_values_that_are_not_finite():
    g = rand((5000,), torch.float32, 1)
    g[17] = float("inf")
    out = torch.empty_like(g)
    norm = moe.moe_clip_grad_norm([g], 1.0, outs=[out])
    assert math.isinf(float(norm)) and bool(out[17].isnan()) and bool((out[:17] == 0).all())
    g[17] = float("nan")
    norm = moe.moe_clip_grad_norm([g], 1.0, outs=[out])
    assert math.isnan(float(norm)) and bool(out.isnan().all())


def test_empty_lists():
    assert float(moe.moe_clip_grad_norm([], 1.0)) == 0.0
    assert float(moe.moe_clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0


def test_a_limit_of_zero():
    g = rand((100,), torch.float32, 1)
    out = torch.ones_like(g)
    moe.moe_clip_grad_norm([g], 0.0, outs=[out])
    assert bool((out == 0).all())


def test_replays_from_a_graph_with_new_gradients():
    grads = [rand((300, 70), torch.bfloat16, 1), rand((9999,), torch.float32, 2)]
    outs = [torch.empty_like(g) for g in grads]
    ws = moe.clip_workspace(grads)
    norm = torch.zeros(1, device="cuda")
    moe.moe_clip_grad_norm(grads, 1.0, outs=outs, ws=ws, norm=norm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        moe.moe_clip_grad_norm(grads, 1.0, outs=outs, ws=ws, norm=norm)
    for k in range(3):
        for i, g in enumerate(grads):
            g.copy_(rand(g.shape, g.dtype, 10 * k + i, 0.1 + k))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(norm, outs, grads, 1.0)


def test_a_tensor_of_more_than_32_bits_of_elements():
    n = (1 << 32) + 4097
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    g.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    ref = math.sqrt(sum(float(p.double().square().sum()) for p in g.split(1 << 27)))
    keep = {k: g[k:k + 1000].clone() for k in (0, (1 << 31) - 500, (1 << 32) - 500, n - 1000)}
    norm = moe.moe_clip_grad_norm([g], 100.0)
    assert abs(float(norm) - ref) <= 17 * U * ref
    for k, v in keep.items():
        want = v.double() * (100.0 / (ref + 1e-6))
        tol = want.abs() * (torch.finfo(g.dtype).eps / 2 + 20 * U) + torch.finfo(g.dtype).tiny
        assert bool(((g[k:k + 1000].double() - want).abs() <= tol).all()), k


def test_the_data_parallel_reduction_clips(tmp_path):
    """allreduce_grads with a limit, on one rank: the reduction has nothing to add, the clipping runs."""
    import torch.distributed as dist
    from dropless_top_moe_b200.parallel import allreduce_grads

    dist.init_process_group("gloo", store=dist.FileStore(str(tmp_path / "store"), 1), rank=0, world_size=1)
    try:
        grads = [rand((100, 30), torch.bfloat16, 1), rand((77,), torch.float32, 2)]
        keep = [g.clone() for g in grads]
        assert allreduce_grads(grads) is None
        assert all(torch.equal(g, k) for g, k in zip(grads, keep))
        check(allreduce_grads(grads, max_norm=1.5), grads, keep, 1.5)
    finally:
        dist.destroy_process_group()


def test_a_factor_below_the_smallest_normal_float():
    """max_norm / norm below 2^-126: the factor has few bits as a float, and the scaled gradients do not."""
    for dt in (torch.float32, torch.bfloat16):
        for scale, limit in ((1e36, 1e-2), (1e37, 1e-6), (3e36, 2e-20)):
            grads = [rand((5000,), dt, 1, scale), rand((77,), dt, 2, scale)]
            keep = [g.clone() for g in grads]
            outs = [torch.empty_like(g) for g in grads]
            norm = moe.moe_clip_grad_norm(grads, limit, outs=outs)
            again = moe.moe_clip_grad_norm(grads, limit)                            # in place
            n = norm64(keep)
            assert torch.equal(norm, again)
            # a norm past the largest float is infinity as a float
            assert abs(float(norm) - n) <= 17 * U * n or (n > torch.finfo(torch.float32).max and math.isinf(float(norm)))
            f = limit / (n + 1e-6)
            assert f < 2.0 ** -126
            for o, p, g in zip(outs, grads, keep):
                want = g.double() * f
                tol = want.abs() * (torch.finfo(dt).eps / 2 + 20 * U) + torch.finfo(dt).tiny
                assert torch.equal(o, p) and bool(((o.double() - want).abs() <= tol).all())


def test_a_norm_past_the_largest_float():
    """The norm is written as infinity; finite gradients are scaled by its value all the same."""
    grads = [torch.full((400,), 3e38, device="cuda"), torch.full((9,), -1e30, device="cuda")]
    outs = [torch.empty_like(g) for g in grads]
    n = norm64(grads)
    assert n > torch.finfo(torch.float32).max
    for limit in (1e3, 1.0):
        assert math.isinf(float(moe.moe_clip_grad_norm(grads, limit, outs=outs)))
        for o, g in zip(outs, grads):
            want = g.double() * (limit / n)
            assert bool(((o.double() - want).abs() <= want.abs() * 20 * U + torch.finfo(g.dtype).tiny).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 5, 8, 9, 31, 4097, 16384, 300001])
def test_the_norm_does_not_depend_on_where_the_gradients_lie(n, dt):
    """Data-parallel ranks may hold the same gradients at other offsets from a 16-byte boundary,
    and have to scale them by the same bits."""
    values = [rand((n,), dt, 1), rand((2 * n + 3,), dt, 2), rand((n + 1,), torch.float32, 3)]
    ref = None
    for off in range(8):
        grads = []
        for i, v in enumerate(values):
            at = (off * (i + 1)) % 8
            flat = torch.full((v.numel() + 16,), float("nan"), dtype=v.dtype, device="cuda")   # the neighbours do not count
            flat[at:at + v.numel()] = v
            grads.append(flat[at:at + v.numel()])
        norm = moe.moe_clip_grad_norm(grads, 0.1 * n ** 0.5)
        check(norm, grads, values, 0.1 * n ** 0.5)
        got = [norm.clone()] + [g.clone() for g in grads]
        ref = ref or got
        assert all(torch.equal(a, b) for a, b in zip(ref, got)), off


def test_the_data_parallel_reduction_refuses_like_the_clipping():
    """check_clip, which allreduce_grads runs before it reduces, and the clipping agree on what they refuse."""
    from dropless_top_moe_b200.ops import check_clip

    flat = rand((64,), torch.float32, 1)
    keep = flat.clone()
    bad = [([flat[:8], flat[7:16]], 1.0), ([flat, flat], 1.0), ([flat], -0.5), ([flat], math.nan), ([flat[::2]], 1.0),
           ([flat.cpu()], 1.0), ([flat[:8], flat[8:].cpu()], 1.0), ([flat.half()], 1.0)]
    for grads, limit in bad:
        with pytest.raises((ValueError, TypeError)):
            check_clip(grads, limit)
        with pytest.raises((ValueError, TypeError, moe.MoEError)):
            moe.moe_clip_grad_norm(grads, limit)
    for grads, limit in [([], 1.0), ([flat[:8], flat[8:16], flat[0:0]], 0.0), ([flat], math.inf),
                         ([flat.bfloat16(), flat[1:]], 1.0)]:
        check_clip(grads, limit)
    assert torch.equal(flat, keep)


def test_some_outputs_in_place_and_others_not():
    grads = [rand((5000 + i,), [torch.float32, torch.bfloat16][i % 2], i) for i in range(6)]
    keep = [g.clone() for g in grads]
    outs = [g if i % 3 == 0 else torch.empty_like(g) for i, g in enumerate(grads)]
    n = norm64(keep)
    for limit in (0.2 * n, 2 * n):
        for g, k in zip(grads, keep):
            g.copy_(k)
        check(moe.moe_clip_grad_norm(grads, limit, outs=outs), outs, keep, limit)
        assert all(torch.equal(g, k) for i, (g, k) in enumerate(zip(grads, keep)) if i % 3)
