"""A shared plan belongs to one build of its batch; steps padded to a size."""
import numpy as np
import pytest
import torch

from heterogeneous_adapters_amd import kv
from test_gpu_kv import host, i32
from test_gpu_shared import SharedStep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 8])  # 3 rows of a kv head, and 400
def test_a_plan_of_the_step_before_is_flagged(G, dtype):
    """Lengths that move on by a token leave rows and requests as many as they were."""
    n = 3 if G == 1 else 50
    s = SharedStep(G, [120 + i for i in range(n)], [1] * n, [0, n], [112], G, 1, 64, 16, dtype)
    want = s.run(0.125)
    s.check(want, 0.125)
    kv.lora_kv_build(i32(s.ctx), i32(s.new), s.T, s.tab, i32(s.free), s.num, s.bt, s.batch)
    out = torch.full_like(s.dq, 3.0)
    kv.lora_kv_attend_shared(s.dq, out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and int(s.batch.flags) == kv.FLAG_BATCH
    kv.lora_kv_build(i32(s.ctx - 1), i32(s.new), s.T, s.tab.clone(), i32(s.free), s.num, s.bt, s.batch)
    kv.lora_kv_attend_shared(s.dq, out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and int(s.batch.flags) == kv.FLAG_BATCH
    # planned again it is as before
    kv.lora_kv_build(i32(s.ctx), i32(s.new), s.T, s.tab, i32(s.free), s.num, s.bt, s.batch)
    s.again(0.125)
    assert int(s.batch.flags) == 0 and np.array_equal(host(s.out), want)


def test_a_build_that_serves_two_plans():
    s = SharedStep(2, [100, 130, 140], [1, 5, 1], [0, 3], [96], 4, 2, 64, 16, "bf16")
    want = s.run(0.125)
    other = kv.Shared(s.batch, 2)
    ws, out = kv.shared_workspace(s.batch, other), torch.empty_like(s.dq)
    kv.lora_kv_share(i32([0, 2]), i32([64]), s.batch, other)
    kv.lora_kv_attend_shared(s.dq, out, s.batch, other, s.tab, s.cache, 0.125, ws)
    s.out.zero_()
    kv.lora_kv_attend_shared(s.dq, s.out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert int(s.batch.flags) == 0 and np.array_equal(host(s.out), want)
    s.check(host(out), 0.125)


def test_plans_of_two_captured_steps_in_turn():
    """Two graphs build the same batch, each with a plan of its own; whichever is replayed finds its own."""
    s = SharedStep(5, [200, 220, 210, 30], [1] * 4, [0, 3], [192], 8, 2, 64, 16, "bf16")
    s.run(0.125)
    plans = [s.shared, kv.Shared(s.batch, 2)]
    wss = [s.ws, kv.shared_workspace(s.batch, plans[1])]
    ctxs = [i32(s.ctx), i32(s.ctx - 7)]
    outs = [torch.zeros_like(s.out) for _ in plans]
    new, free, groups, lens = i32(s.new), i32(s.free), i32(s.groups), i32(s.lens)

    def step(k):
        kv.lora_kv_build(ctxs[k], new, s.T, s.tab, free, s.num, s.bt, s.batch)
        kv.lora_kv_share(groups, lens, s.batch, plans[k])
        kv.lora_kv_attend_shared(s.dq, outs[k], s.batch, plans[k], s.tab, s.cache, 0.125, wss[k])

    want = []
    for k in (0, 1):
        step(k)
        torch.cuda.synchronize()
        want.append(outs[k].clone())
    graphs = []
    for k in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(k)
        graphs.append(g)
    for k in (0, 1, 1, 0, 0, 1):
        outs[k].fill_(9.0)
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k], want[k]) and int(s.batch.flags) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,G,D", [(3, 1, 64), (50, 8, 64), (11, 32, 160)])
def test_padded_steps_leave_the_rows_behind_alone(n, G, D, dtype):
    """More rows than the requests bring: a graph's size.  With T past B other classes of items come into play."""
    s = SharedStep(n, [120 + i for i in range(n)], [1] * n, [0, n], [112], G, 1, D, 16, dtype)
    s.check(s.run(0.125), 0.125)
    for pad in (1, 40):
        T = s.T + pad
        batch = kv.Batch(T, n, G, 1, D)
        shared = kv.Shared(batch, 1)
        ws = kv.shared_workspace(batch, shared)
        q = torch.full((T, G, D), float("nan"), dtype=s.dq.dtype, device=s.dq.device)
        q[:s.T] = s.dq
        out = torch.full_like(q, 3.0)
        kv.lora_kv_build(i32(s.ctx), i32(s.new), T, s.tab, i32(s.free), s.num, s.bt, batch)
        kv.lora_kv_share(i32(s.groups), i32(s.lens), batch, shared)
        kv.lora_kv_attend_shared(q, out, batch, shared, s.tab, s.cache, 0.125, ws)
        torch.cuda.synchronize()
        s.check(host(out[:s.T]), 0.125)
        assert torch.all(out[s.T:] == 3.0) and int(batch.flags) == 0
