"""The order of no slots: offsets are zeros whatever the number of experts, and nothing else is touched."""
import pytest
import torch

import dense_gemm_09_amd as g

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [0, 1, 64, 2047, 2048, 5000, 8192])
def test_no_slots(G):
    assert g.route_order_workspace_size(0, G) == 0
    offsets = torch.full((G + 2,), 55, device="cuda", dtype=torch.int32)
    other = torch.full((4,), 55, device="cuda", dtype=torch.int32)
    for expert, position, order in ((None, None, None), (other, other, other), (other[:0], other[:0], other[:0])):
        offsets.fill_(55)
        g.route_order(0, G, expert, offsets, position, order)
        assert (offsets[:-1] == 0).all() and offsets[-1] == 55 and (other == 55).all()


def test_no_slots_captured():
    G = 4096
    offsets = torch.full((G + 1,), 55, device="cuda", dtype=torch.int32)
    g.route_order(0, G, None, offsets, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.route_order(0, G, None, offsets, None)
    for _ in range(3):
        offsets.fill_(7)
        graph.replay()
        assert (offsets == 0).all()
