"""allreduce_and_clip on two gloo ranks: every rank holds its own gradients, and all hold the clipped sums afterwards.

The clipping itself runs on a GPU; here its definition in 64 bits stands in for it.
"""
import datetime
import math
import os
import socket

import numpy as np
import pytest

WORLD = 2
SHAPES = [(6, 9, 5), (6,), (0,), (11, 3)]


def _grads(rank):
    rng = np.random.default_rng(90 + rank)
    return [rng.standard_normal(s).astype(np.float32) for s in SHAPES]


def _rank_main(rank, world, port, max_norm, q):
    import torch
    import torch.distributed as dist

    from sparse_convolution_pruned_b200 import data_parallel, svconv

    def clip(grads, limit):
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
        for g in grads:
            g.mul_(min(1.0, limit / (norm + 1e-6)))
        return torch.tensor(norm, dtype=torch.float32)

    svconv.svconv_clip_grads = clip
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=60))
    try:
        grads = [torch.from_numpy(g) for g in _grads(rank)]
        norm = data_parallel.allreduce_and_clip((g for g in grads), max_norm)
        q.put((rank, float(norm), [g.numpy() for g in grads]))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("share", [0.25, 2.0])
def test_two_gloo_ranks_clip_the_sums(share):
    import torch.multiprocessing as mp

    sums = [a + b for a, b in zip(_grads(0), _grads(1))]
    total = math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in sums))
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    port = s.getsockname()[1]
    s.close()
    procs = [ctx.Process(target=_rank_main, args=(r, WORLD, port, share * total, q)) for r in range(WORLD)]
    for p in procs:
        p.start()
    res = sorted((q.get(timeout=120) for _ in range(WORLD)), key=lambda t: t[0])
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    f = min(1.0, share * total / (total + 1e-6))
    for _, norm, grads in res:
        assert abs(norm - total) <= 2.0 ** -23 * total
        for g, want in zip(grads, sums):
            np.testing.assert_allclose(g, want * f, rtol=2.0 ** -21, atol=0)  # fp32 roundings of the sum and the product
    for a, b in zip(res[0][2], res[1][2]):
        np.testing.assert_array_equal(a, b)
