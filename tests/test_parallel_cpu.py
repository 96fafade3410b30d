"""Data-parallel gradient reduction across replicas: gloo ranks on CPU.

Each rank holds gradients of its own tokens; after allreduce_grads every rank
must hold the rank-ordered average, bitwise equal across ranks and runs.  The
library's rank-ordered sum kernel needs a GPU, so these CPU ranks exercise
the exchange (all-to-all of shards, all-gather, chunking and padding) with a
rank-ordered sum written here; the kernel itself is checked on the GPU."""
import os
import socket

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from dropless_top_moe_b200.parallel import allreduce_grads


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _cpu_ordered_sum(recv, world, scale, out):
    acc = torch.zeros(out.shape, dtype=torch.float32)
    for r in range(world):
        acc += recv[r].to(torch.float32)
    out.copy_((acc * scale).to(out.dtype))


def _worker(rank, world, port, q):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        out = []
        for dt in (torch.float32, torch.bfloat16):
            g = torch.Generator().manual_seed(100 + rank)
            ts = [torch.randn(3, 70, 33, generator=g).to(dt), torch.randn(1001, generator=g).to(dt)]
            allreduce_grads(ts, average=True, chunk_elems=512, local_sum=_cpu_ordered_sum)
            out.append([t.clone() for t in ts])
        q.put((rank, out))
    finally:
        dist.destroy_process_group()


def test_default_sum_refuses_cpu_tensors():
    from dropless_top_moe_b200.parallel import ordered_sum
    with pytest.raises(RuntimeError, match="CUDA"):
        ordered_sum(torch.zeros(2, 8), 2, 0.5, torch.zeros(8))


@pytest.mark.parametrize("world", [2, 3])
def test_allreduce_grads_gloo_ranks(world):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_worker, args=(r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=120) for _ in range(world))
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    # expected: rank-ordered fp32 sum of every rank's tensors, times 1/world
    for di, dt in enumerate((torch.float32, torch.bfloat16)):
        gens = [torch.Generator().manual_seed(100 + r) for r in range(world)]
        inputs = [[torch.randn(3, 70, 33, generator=g).to(dt), torch.randn(1001, generator=g).to(dt)]
                  for g in gens]
        for ti in range(2):
            acc = torch.zeros(inputs[0][ti].shape, dtype=torch.float32)
            for r in range(world):
                acc += inputs[r][ti].float()
            exp = (acc * (1.0 / world)).to(dt)
            for r in range(world):
                assert torch.equal(res[r][di][ti], exp), (dt, ti, r)


def _clip_worker(rank, world, port, q):
    """What the clipping refuses is refused before the exchange; what it takes is clipped after it."""
    from dropless_top_moe_b200 import parallel
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        g = torch.Generator().manual_seed(200 + rank)
        flat = torch.randn(400, generator=g)
        keep = flat.clone()
        ts = [flat[:100], flat[100:400]]
        bad = [(ts, -1.0, ValueError, "max_norm"), (ts, float("nan"), ValueError, "max_norm"),
               ([flat[:100], flat[99:300]], 1.0, ValueError, "share"), ([flat[:100], flat[:100]], 1.0, ValueError, "share"),
               (ts, 1.0, ValueError, "CUDA"), ([flat[:100], flat[100:200].double()], 1.0, TypeError, "dtype"),
               ([flat[:100], flat[100:400:2]], 1.0, ValueError, "contiguous")]
        for grads, limit, error, match in bad:
            with pytest.raises(error, match=match):
                allreduce_grads(iter(grads), local_sum=_cpu_ordered_sum, max_norm=limit)
            assert torch.equal(flat, keep), match
        # the clipping itself needs a GPU: a plain one in its place shows what it is given, and when
        order = []

        def clip(grads, limit):
            order.append("clip")
            norm = torch.stack([t.double().square().sum() for t in grads]).sum().sqrt()
            for t in grads:
                t.mul_(min(1.0, limit / (float(norm) + 1e-6)))
            return norm.float().reshape(1)
        check, parallel.moe_clip_grad_norm = parallel.check_clip, clip
        parallel.check_clip = lambda grads, limit: order.append("check")

        def local_sum(*a):
            order.append("sum")
            _cpu_ordered_sum(*a)
        norm = allreduce_grads(ts, local_sum=local_sum, max_norm=2.0)
        parallel.check_clip = check
        q.put((rank, order, norm, flat.clone()))
    finally:
        dist.destroy_process_group()


def test_allreduce_grads_with_a_limit_on_two_ranks():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_clip_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    res = {r: rest for r, *rest in (q.get(timeout=120) for _ in range(2))}
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    want = sum(torch.randn(400, generator=torch.Generator().manual_seed(200 + r)) for r in range(2)) * 0.5
    n = float(want.double().norm())
    assert n > 2.0
    for r in range(2):
        order, norm, flat = res[r]
        assert order == ["check", "sum", "sum", "clip"]
        assert abs(float(norm) - n) <= 2.0 ** -23 * n
        # one rounding of the sum, of the factor as a double and of the product
        assert torch.allclose(flat.double(), want.double() * (2.0 / (n + 1e-6)), rtol=2.0 ** -22, atol=0)
        assert torch.equal(flat, res[0][2])
