"""The vector-state scan's status word: whatever the workspace held, a forward
starts it anew, and a timeout stays until it is read or the next forward."""
import pytest
import torch

import discrete_selective_ssm_b200 as naju

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture
def lost():
    """Within it the first block of a unit sends nothing: waits run out."""
    class Lost:
        def __enter__(self):
            naju.testing_set_wait_limit(200)
            naju.testing_set_skip_publish(True)

        def __exit__(self, *_):
            naju.testing_set_wait_limit(0)
            naju.testing_set_skip_publish(False)
    yield Lost()
    Lost().__exit__()


def case(units=1):
    g = torch.Generator().manual_seed(3)
    h, a, b = (torch.randn(units, 300, 32, generator=g).cuda() for _ in range(3))
    dims = naju.make_dims(units, 300, 32, 1, naju.F32)
    return h, a, b, naju.vscan_workspace(dims, h)


@pytest.mark.parametrize("byte", [0, 0x10, 0xff])
def test_any_workspace(byte, lost):
    h, a, b, ws = case()
    ws.fill_(byte)
    naju.vscan_fwd(h, a, b, workspace=ws)
    assert naju.last_device_status(ws) == 0
    ws.fill_(byte)
    with lost:
        naju.vscan_fwd(h, a, b, workspace=ws)
    assert naju.last_device_status(ws) == TIMEOUT and naju.last_device_status(ws) == 0


@pytest.mark.parametrize("units", [1, 40, 1000])
def test_from_any_unit(units, lost):
    """Timeouts of many clusters, most of them not the first block's (one block
    alone, as so many units would have, exchanges nothing: clusters of two)."""
    h, a, b, ws = case(units)
    naju.testing_set_vscan_cluster(2)
    try:
        for _ in range(5):
            with lost:
                naju.vscan_fwd(h, a, b, workspace=ws)
            assert naju.last_device_status(ws) == TIMEOUT
            naju.vscan_fwd(h, a, b, workspace=ws)
            assert naju.last_device_status(ws) == 0
    finally:
        naju.testing_set_vscan_cluster(0)


def test_a_forward_clears_a_backward_adds(lost):
    h, a, b, ws = case(3)
    with lost:
        naju.vscan_fwd(h, a, b, workspace=ws)
    naju.vscan_bwd(h, h, a, b, ws)
    assert naju.last_device_status(ws) == TIMEOUT  # the backward leaves the forward's
    with lost:
        naju.vscan_bwd(h, h, a, b, ws)
    assert naju.last_device_status(ws) == TIMEOUT
    with lost:
        naju.vscan_fwd(h, a, b, workspace=ws)
        naju.vscan_bwd(h, h, a, b, ws)
    naju.vscan_fwd(h, a, b, workspace=ws)
    assert naju.last_device_status(ws) == 0


def test_replays_keep_what_nobody_read(lost):
    h, a, b, ws = case()
    naju.vscan_fwd(h, a, b, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with lost, torch.cuda.graph(graph):
        naju.vscan_fwd(h, a, b, workspace=ws)
    graph.replay()
    graph.replay()
    assert naju.last_device_status(ws) == TIMEOUT and naju.last_device_status(ws) == 0
    graph.replay()
    assert naju.last_device_status(ws) == TIMEOUT
    graph.replay()
    naju.vscan_fwd(h, a, b, workspace=ws)
    assert naju.last_device_status(ws) == 0
