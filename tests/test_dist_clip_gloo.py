"""Summing the adapters' gradients over ranks and clipping each adapter, two CPU processes over
gloo with a plain float64 clip in place of the GPU kernels: both ranks must hold the clipped
gradients and norms of all the ranks' tokens."""
import os
import socket

import torch
import torch.distributed as tdist
import torch.multiprocessing as mp

WORLD, N_AD = 2, 3
SHAPES = [(4, 16), (24, 4), (4, 24), (16, 4)]


def _local(rank):
    g = torch.Generator().manual_seed(60 + rank)
    return [torch.randn(N_AD, *s, generator=g) * (0.1 if i % 2 else 2.0) for i, s in enumerate(SHAPES)]


def _plain_clip(grads, max_norm, n):
    norm = torch.stack([t.double().reshape(n, -1).square().sum(1) for t in grads]).sum(0).sqrt()
    c = (max_norm / (norm + 1e-6)).clamp(max=1.0)
    for t in grads:
        t.mul_(c.to(t.dtype).view(n, *[1] * (t.dim() - 1)))
    return norm.float()


def _rank(rank, port, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    tdist.init_process_group("gloo", rank=rank, world_size=WORLD)
    from bit_nf4_quantized_04_b200 import dist
    grads = _local(rank)
    norm = dist.allreduce_clip_adapter_grads(grads, 1.5, N_AD, clip_fn=_plain_clip)
    torch.save((grads, norm), out + str(rank))
    tdist.destroy_process_group()


def test_two_ranks_hold_the_clipped_sums(tmp_path):
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    out = str(tmp_path / "r")
    mp.spawn(_rank, args=(port, out), nprocs=WORLD, join=True)
    want = [sum(ts) for ts in zip(*(_local(r) for r in range(WORLD)))]
    norm = _plain_clip(want, 1.5, N_AD)
    res = [torch.load(out + str(r)) for r in range(WORLD)]
    for grads, got in res:
        assert torch.equal(got, norm)
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_one_process_only_clips():
    from bit_nf4_quantized_04_b200 import dist
    grads, want = _local(0), _local(0)
    norm = dist.allreduce_clip_adapter_grads(grads, 1.5, N_AD, clip_fn=_plain_clip)
    assert torch.equal(norm, _plain_clip(want, 1.5, N_AD))
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
