"""A workspace that the binding makes itself is filled with zeros before any stream's first call, also one that is not the stream
of its making."""
import pytest
import torch

import mla_block_diffusion_gb300 as M
from synthetic import generate as gen
from synthetic.configs import TINY_STEP

pytestmark = pytest.mark.gpu


def qlinear():
    codes, scales = torch.zeros(128, 128, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda")
    return lambda: M.QLinear(codes, scales)


def qcache():
    codes, scales, table = torch.zeros(2, 64, 80, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda"), torch.zeros(
        1, 2, dtype=torch.int32, device="cuda")
    return lambda: M.QCache(64, 16, [codes], [scales], table, n_heads=8)


def drafter():
    W = {k: v.cuda() for k, v in gen.make_weights(TINY_STEP, "cpu").items()}
    return lambda: M.DSpark(TINY_STEP.geom, W)


@pytest.mark.parametrize("parts", [qlinear, qcache, drafter])
def test_first_call_on_another_stream(parts):
    make, made, used = parts(), torch.cuda.Stream(), torch.cuda.Stream()
    big = torch.ones(1 << 28, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(made):
        size = make().ws.numel()
        dirty = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]  # what the allocator gives next
        at = {t.data_ptr() for t in dirty}
        torch.cuda.synchronize()
        del dirty
        for _ in range(100):  # tens of milliseconds
            big.mul_(1.0)
        it = make()
    assert it.ws.data_ptr() in at
    with torch.cuda.stream(used):
        assert it.check() == 0
    torch.cuda.synchronize()
    assert not it.ws.any()


def test_made_in_a_capture():
    """In a capture nothing can be waited for: the fill is part of the graph."""
    codes, scales = torch.zeros(128, 128, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda")
    x, y = (torch.zeros(3, 128, dtype=torch.uint8, device="cuda"), torch.ones(1, 3, device="cuda")), torch.ones(3, 128, device="cuda")
    M.QLinear(codes, scales).matmul(*x, y)
    y.fill_(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin = M.QLinear(codes, scales)
        lin.matmul(*x, y)
    g.replay()
    assert lin.check() == 0 and not y.any()
