"""GPU tests of the plan above 8192 pairs: a workgroup's further rounds, a caller's workspace shared by calls in a
row, the two launches replayed from a graph. Plans have to be equal to the reference's."""
import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_act_amd as bf
from tests import _moe_ref as ref
from tests._gpu import DEV

pytestmark = pytest.mark.gpu


# pairs from 1048577 on give a workgroup a second round of 2048, from 2097153 on a third
@pytest.mark.parametrize("T,k,E", [(1048577, 1, 8), (140000, 8, 64), (131073, 8, 1024), (312507, 8, 64), (2097153, 1, 1), (52000, 64, 300)])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_plan_of_several_rounds(T, k, E, dropped):
    g = np.random.Generator(np.random.PCG64(T + E))
    ids = (E * g.random((T, k)) ** 2).astype(np.int32)          # experts unevenly liked
    bad = np.array([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=np.int64).astype(np.int32)
    ids = np.where(g.random((T, k)) < dropped, bad[g.integers(0, 4, (T, k))], ids).astype(np.int32)
    got = bf.moe_plan(torch.from_numpy(ids).to(DEV), E)
    for a, b, name in zip(got, ref.plan(ids, E), ("offsets", "slots", "rows")):
        assert np.array_equal(a.cpu().numpy(), b), name


def _plans(seed, T, k, E, n):
    g = np.random.Generator(np.random.PCG64(seed))
    return [g.integers(-1, E + 1, (T, k)).astype(np.int32) for _ in range(n)]


@pytest.mark.parametrize("where", ["current", "stream", "handle"])
def test_plans_in_a_row_share_a_workspace(where):
    """A caller's workspace, larger than needed and used by plans of several sizes one after the other on one
    stream; what lies past the bytes they need is not written."""
    sizes = [(1200, 8, 64), (9000, 1, 1024), (20000, 8, 8), (1100, 8, 300)]
    need = max(bf.moe_plan_workspace(*s) for s in sizes)
    assert min(bf.moe_plan_workspace(*s) for s in sizes) > 0
    workspace = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    inputs = [(E, ids) for i, (T, k, E) in enumerate(sizes) for ids in _plans(i, T, k, E, 2)]
    on_device = [(E, torch.from_numpy(ids).to(DEV)) for E, ids in inputs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    stream = {"current": None, "stream": s, "handle": s.cuda_stream}[where]
    got = [bf.moe_plan(ids, E, workspace=workspace, stream=stream) for E, ids in on_device]
    torch.cuda.synchronize()
    for (E, ids), plan in zip(inputs, got):
        for a, b, name in zip(plan, ref.plan(ids, E), ("offsets", "slots", "rows")):
            assert np.array_equal(a.cpu().numpy(), b), (E, name)
    assert torch.all(workspace[need:] == 0xA5)


@pytest.mark.parametrize("T,k,E", [(1200, 8, 64), (140000, 8, 128)])
@pytest.mark.parametrize("own", [True, False], ids=["own workspace", "allocated"])
def test_plan_of_two_launches_replays_from_a_graph(T, k, E, own):
    """More than 8192 pairs: counting launch, sorting launch, workspace between. Every replay, with eager
    plans of other ids between, equals the reference."""
    workspace = torch.empty(bf.moe_plan_workspace(T, k, E), dtype=torch.uint8, device=DEV) if own else None
    batches = _plans(T, T, k, E, 4)
    ids = torch.from_numpy(batches[0]).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bf.moe_plan(ids, E, workspace=workspace)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bf.moe_plan(ids, E, workspace=workspace)
    for batch in batches:
        bf.moe_plan(torch.from_numpy(batches[0][::-1].copy()).to(DEV), E)
        ids.copy_(torch.from_numpy(batch))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, name in zip(out, ref.plan(batch, E), ("offsets", "slots", "rows")):
            assert np.array_equal(a.cpu().numpy(), b), name
