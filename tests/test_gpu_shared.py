"""Attention of requests that share a prefix against the plain 64-bit form,
which attends to every request by itself."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import kv
from test_gpu_kv import DEV, Step, host, i32, to_dev

pytestmark = pytest.mark.gpu


class SharedStep(Step):
    """A step whose groups' requests have the same first tokens: full blocks of
    them by the same ids (`by_id`) or all of them as copies."""

    def __init__(self, seed, ctx, new, groups, lens, hq, hkv, D, bt, dtype, by_id=True, same=None, **kw):
        super().__init__(seed, np.array(ctx), np.array(new), hq, hkv, D, bt, dtype, **kw)
        self.groups, self.lens = groups, lens
        at = np.concatenate([[0], np.cumsum(np.array(ctx) + np.array(new))])
        lead_of = same or {}
        for g in range(len(lens)):
            members = range(max(groups[g], 0), min(groups[g + 1], len(ctx)))
            if not len(members):
                continue
            lead = lead_of.get(g, members[0])
            for i in members:
                n = min(lens[g], ctx[i], ctx[lead])
                if i == lead or n <= 0:
                    continue
                full = n // bt if by_id else 0
                self.table[i, :full] = self.table[lead, :full]
                self.ref["table"][i, :full] = self.ref["table"][lead, :full]
                for x in (self.k, self.v):
                    x[at[i]:at[i] + n] = x[at[lead]:at[lead] + n]
                pos = np.arange(full * bt, n)
                slots = self.ref["table"][i, pos // bt] * bt + pos % bt
                R.put(self.data, slots, self.k[at[i] + pos], self.v[at[i] + pos], bt)

    def run(self, scale, max_groups=None, stream=None):
        self.cache = kv.Cache(torch.tensor(self.data, device=DEV), self.bt, self.hkv, self.D)
        self.batch = kv.Batch(self.T + 3, len(self.ctx) + 2, self.hq, self.hkv, self.D)
        self.shared = kv.Shared(self.batch, len(self.lens) if max_groups is None else max_groups)
        self.tab = i32(self.table)
        self.dq = to_dev(self.q, self.dtype)
        self.out = torch.full_like(self.dq, 5.0)
        self.ws = kv.shared_workspace(self.batch, self.shared)
        kv.lora_kv_build(i32(self.ctx), i32(self.new), self.T, self.tab, i32(self.free), self.num, self.bt, self.batch)
        self.again(scale)
        return host(self.out)

    def counts_of_prefixes(self):
        """The plan's first count: items of the groups' prefixes."""
        return int(self.shared.buf[:4].view(torch.int32))

    def again(self, scale):
        kv.lora_kv_share(i32(self.groups), i32(self.lens), self.batch, self.shared)
        kv.lora_kv_attend_shared(self.dq, self.out, self.batch, self.shared, self.tab, self.cache, scale, self.ws)
        torch.cuda.synchronize()


CASES = [
    # ctx, new, groups, shared_len, hq, hkv, D, bt
    ([40, 40], [1, 1], [0, 2], [32], 1, 1, 32, 16),
    ([100, 90, 133, 64], [1] * 4, [0, 4], [64], 4, 1, 64, 16),
    ([70, 70, 70, 9, 200, 260], [1] * 6, [0, 3, 3, 4, 6], [64, 10, 9, 199], 8, 2, 128, 32),  # an empty group, short ones, alone, odd lengths
    ([600, 650, 590, 700, 5, 0], [1] * 6, [1, 4], [577], 8, 8, 96, 16),  # requests before and behind the group
    ([1100] * 9 + [20], [1] * 10, [0, 9, 10], [1100, 16], 16, 2, 64, 16),  # all that is cached, 72 rows of a kv head
    ([300, 310, 320], [1, 1, 1], [0, 3], [300], 40, 1, 128, 64),  # 120 rows
    ([700, 705, 700], [1, 0, 3], [0, 3], [690], 6, 3, 160, 16),  # a request without tokens
    ([40, 900, 900, 1000], [0, 0, 40, 1], [0, 4], [880], 4, 2, 64, 32),  # the first ones without, a chunk
    ([260, 300, 256, 0], [20, 1, 33, 17], [0, 3], [250], 7, 1, 192, 256),
    ([64, 64, 64, 64, 64], [1] * 5, [0, 5], [63], 12, 4, 224, 16),
    ([520, 530], [1, 20], [0, 2], [515], 4, 2, 256, 32),
    ([1000, 30], [1, 1], [0, 2], [1000], 4, 4, 64, 16),  # cut by the shorter request to less than it says
    ([10, 10], [1, 1], [0, 2], [10], 2, 1, 64, 16),  # nothing to share: under 16 tokens
    ([90] * 70, [1] * 70, [0, 10, 40, 70], [80, 48, 90], 2, 1, 32, 16),
    ([50, 60], [1, 1], [0], [], 4, 2, 64, 16),  # no groups
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared_against_plain(case, dtype):
    ctx, new, groups, lens, hq, hkv, D, bt = CASES[case]
    same = {0: 2} if case == 7 else None  # the group's first request with tokens
    s = SharedStep(case, ctx, new, groups, lens, hq, hkv, D, bt, dtype, by_id=case % 2 == 0, same=same, pad=case % 3)
    scale = 1.0 / math.sqrt(D)
    s.check(s.run(scale), scale)
    assert int(s.batch.flags) == 0
    assert (s.counts_of_prefixes() == 0) == (case in (12, 14))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_peaked_scores(dtype):
    s = SharedStep(3, [600, 640, 610], [1, 1, 20], [0, 3], [592], 4, 2, 64, 16, dtype, k_scale=6.0)
    s.check(s.run(0.9), 0.9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 64), (16, 1, 128), (32, 1, 128), (8, 2, 256)])
def test_prefixes_in_several_chunks_and_tiles(hq, hkv, D, dtype):
    """2 000 shared tokens: several chunks; 6 to 192 rows of a kv head."""
    s = SharedStep(hq + D, [2000, 2030, 2000, 2011, 2500, 2001], [1] * 6, [0, 6], [2000], hq, hkv, D, 16, dtype)
    scale = 1.0 / math.sqrt(D)
    s.check(s.run(scale), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,P,bt", [(32, 70, 16), (64, 700, 32), (96, 320, 16), (128, 64, 16), (128, 615, 64), (160, 130, 16), (192, 304, 32),
                                    (224, 77, 16), (256, 560, 16)])
def test_groups_of_many_rows(D, P, bt, dtype):
    """32 query heads on one: 352 and 448 rows of a group up to 128 dims, 160 and 288 past them, in tiles of 256 and 128."""
    n = (11, 14) if D <= 128 else (5, 9)
    ctx = [P + 3 * i for i in range(n[0])] + [40 + P - i % 2 for i in range(n[1])] + [9]
    s = SharedStep(D + P, ctx, [1] * len(ctx), [0, n[0], sum(n)], [P, P + 39], 32, 1, D, bt, dtype, by_id=P % 2 == 0, pad=2)
    scale = 1.0 / math.sqrt(D)
    s.check(s.run(scale), scale)
    assert int(s.batch.flags) == 0 and s.counts_of_prefixes() > 0


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("power,D", [(20, 64), (100, 128), (60, 160)])
def test_scores_far_from_zero_in_tiles_of_many_rows(power, D, order):
    """Scores of up to 2^power, growing or falling along the keys: all weight on one key."""
    n, P = (11, 130) if D <= 128 else (5, 130)
    s = SharedStep(power, [P] * n, [1] * n, [0, n], [P], 32, 1, D, 16, "bf16")
    at = np.concatenate([[0], np.cumsum([P + 1] * n)])
    place = np.argsort(np.arange(P))[::order]
    for i in range(n):
        s.k[at[i]:at[i + 1]] = 0.0
        s.k[at[i]:at[i] + P, :, 0] = 2.0 ** (power // 2) * (1 + (place % 4) / 2)[:, None] * np.where(place >= P - 4, 1, 2.0 ** -20)[:, None]
        pos = np.arange(P + 1)
        slots = s.ref["table"][i, pos // 16] * 16 + pos % 16
        R.put(s.data, slots, s.k[at[i]:at[i + 1]], s.v[at[i]:at[i + 1]], 16)
        s.k[at[i]:at[i + 1]], s.v[at[i]:at[i + 1]] = R.get(s.data, slots, 1, D, 16)  # as 4 bits hold them
    s.q[:] = 0.0
    s.q[..., 0] = 2.0 ** (power - power // 2)
    got = s.run(1.0)
    for i in range(n):
        score = s.k[at[i]:at[i + 1], 0, 0] * s.q[i, 0, 0]
        best = np.flatnonzero(score == score.max())
        want = R.bf16(s.v[at[i] + best].mean(0))  # the others' weights are 0, these are equal
        assert np.all(np.abs(got[i] - want) <= 2.0 ** -8 * np.abs(s.v[at[i] + best]).mean(0) + 2.0 ** -8 * np.abs(want))


def test_bad_blocks_and_ends_in_tiles_of_many_rows():
    """A block outside the cache in the middle, bytes of NaN scales behind the last token, two chunks."""
    n, P = 11, 592
    s = SharedStep(7, [P] * n, [1] * n, [0, n], [P], 32, 1, 128, 16, "bf16")
    s.run(0.1)
    s.tab[0, 5] = -9
    s.again(0.1)
    assert int(s.batch.flags) == kv.FLAG_BLOCK_RANGE
    got, at = host(s.out), np.concatenate([[0], np.cumsum([P + 1] * n)])
    for i in range(n):
        keep = np.r_[at[i]:at[i] + 80, at[i] + 96:at[i + 1]]
        o, a, sa = R.attend_rows(s.q[i:i + 1], s.k[keep], s.v[keep], [len(keep)], 0.1)
        assert np.all(np.abs(got[i] - o[0]) <= R.attend_bound(o, a, sa, len(keep), 128, "bf16")[0])


def test_strided_queries_and_outputs():
    s = SharedStep(2, [100, 130, 140], [1, 5, 1], [0, 3], [96], 4, 2, 64, 16, "bf16")
    s.run(0.125)
    want = s.out.clone()
    wide = torch.zeros((s.T, 9, 128), dtype=torch.bfloat16, device=DEV)
    q, out = wide[:, 1:5, :64], torch.full((4, s.T, 72), 7.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    q.copy_(s.dq)
    kv.lora_kv_attend_shared(q, out[..., :64], s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.equal(out[..., :64], want) and torch.all(out[..., 64:] == 7.0)


@pytest.mark.parametrize("groups,lens,flag", [([-1, 2], [32], True), ([0, 4], [32], True), ([2, 1, 3], [32, 32], True), ([0, 3], [-5], True),
                                              ([0, 3], [1 << 30], False), ([3, 3], [64], False)])
def test_groups_out_of_range_are_not_shared(groups, lens, flag):
    """Results stay right where all requests have their own tokens only if nothing, or what they have in common, is shared."""
    ctx = [100, 100, 100]
    s = SharedStep(1, ctx, [1, 1, 1], [0, 3], [100], 4, 2, 64, 16, "bf16")
    s.groups, s.lens = groups, lens
    s.check(s.run(0.125), 0.125)
    assert int(s.batch.flags) == (kv.FLAG_GROUPS if flag else 0)


def test_blocks_outside_the_cache_are_not_attended():
    s = SharedStep(4, [200, 210], [1, 1], [0, 2], [192], 4, 2, 64, 16, "bf16")
    s.run(0.125)
    s.tab[0, 3] = s.num + 5  # of the prefix
    s.again(0.125)
    assert int(s.batch.flags) == kv.FLAG_BLOCK_RANGE
    at = np.concatenate([[0], np.cumsum([201, 211])])
    for i in range(2):
        keep = np.r_[at[i]:at[i] + 48, at[i] + 64:at[i + 1]]
        o, a, sa = R.attend_rows(s.q[i:i + 1], s.k[keep], s.v[keep], [len(keep)], 0.125)
        assert np.all(np.abs(host(s.out)[i] - o[0]) <= R.attend_bound(o, a, sa, len(keep), 64, "bf16")[0])


def test_a_plan_that_was_not_built_for_the_call_writes_nothing():
    s = SharedStep(4, [100, 110], [1, 1], [0, 2], [96], 4, 2, 64, 16, "bf16")
    s.run(0.125)
    fresh = kv.Shared(s.batch, 2)  # never built
    out = torch.full_like(s.dq, 3.0)
    fresh.groups = 1
    kv.lora_kv_attend_shared(s.dq, out, s.batch, fresh, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and int(s.batch.flags) & kv.FLAG_BATCH
    s.batch.flags.zero_()
    s.shared.groups = 0  # another number of groups than the plan's
    kv.lora_kv_attend_shared(s.dq, out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and int(s.batch.flags) & kv.FLAG_BATCH
    # a batch that was never built
    b = kv.Batch(8, 4, 4, 2, 64)
    sh = kv.Shared(b, 1)
    b._resize(2, 2)
    kv.lora_kv_share(i32([0, 2]), i32([96]), b, sh)
    kv.lora_kv_attend_shared(s.dq, out, b, sh, s.tab, s.cache, 0.125, kv.shared_workspace(b, sh))
    torch.cuda.synchronize()
    assert torch.all(out == 3.0) and int(b.flags) & kv.FLAG_BATCH


def test_a_batch_built_again_after_its_plan_stays_in_its_buffers():
    """Rows that another plan's results do not cover are flagged, not read."""
    s = SharedStep(4, [100, 110], [1, 3], [0, 2], [96], 4, 2, 64, 16, "bf16")
    s.run(0.125)
    kv.lora_kv_build(i32([100, 110]), i32([3, 1]), s.T, s.tab, i32(s.free), s.num, s.bt, s.batch)
    kv.lora_kv_attend_shared(s.dq, s.out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert int(s.batch.flags) & kv.FLAG_BATCH


def test_the_same_bits_every_time_and_on_other_streams():
    s = SharedStep(6, [1500] * 8, [1] * 8, [0, 8], [1490], 16, 2, 64, 16, "bf16")
    s.run(0.125)
    want = s.out.clone()
    for _ in range(5):
        s.out.fill_(0)
        s.again(0.125)
        assert torch.equal(s.out, want)
    side = torch.cuda.Stream()
    s.out.fill_(0)
    torch.cuda.synchronize()
    kv.lora_kv_share(i32(s.groups), i32(s.lens), s.batch, s.shared, stream=side)
    kv.lora_kv_attend_shared(s.dq, s.out, s.batch, s.shared, s.tab, s.cache, 0.125, s.ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(s.out, want)


def test_captured_steps_replay_as_lengths_and_groups_move():
    B, hq, hkv, D, bt = 6, 8, 2, 64, 16
    ctx0 = np.array([640, 655, 700, 33, 40, 1])
    s = SharedStep(9, ctx0, [1] * B, [0, 3, 5], [640, 32], hq, hkv, D, bt, "bf16")
    scale = 0.125
    s.run(scale)
    ctx, new, free = i32(ctx0), torch.ones(B, dtype=torch.int32, device=DEV), i32(s.free)
    groups, lens = i32(s.groups), i32(s.lens)

    def step():
        kv.lora_kv_build(ctx, new, B, s.tab, free, s.num, bt, s.batch)
        kv.lora_kv_share(groups, lens, s.batch, s.shared)
        kv.lora_kv_attend_shared(s.dq, s.out, s.batch, s.shared, s.tab, s.cache, scale, s.ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        if k == 1:
            lens.copy_(i32([512, 0]))
        if k == 2:
            ctx.copy_(i32(ctx0 - np.array([5, 0, 0, 1, 1, 0])))
        if k == 3:
            groups.copy_(i32([0, 2, 2]))
        s.dq.normal_()
        s.out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        got = s.out.clone()
        s.out.fill_(9.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, s.out) and not torch.any(got == 9.0)
        ws = kv.attend_workspace(s.batch)
        plain = torch.empty_like(s.out)
        kv.lora_kv_attend(s.dq, plain, s.batch, s.tab, s.cache, scale, ws)
        torch.cuda.synchronize()
        # each within its roundings of the same sums: weights (2^-8 of sums of |V|) and outputs in bf16, and a little in fp32
        tol = 2 * 2.0 ** -8 * (float(np.abs(s.v).max()) * 1.01 + plain.float().abs()) + 2.0 ** -12
        assert torch.all((got.float() - plain.float()).abs() <= tol)


def test_far_offsets_of_a_large_cache():
    """Blocks behind 4 GiB, by a wide stride between blocks."""
    bt, hkv, D = 16, 1, 64
    s = SharedStep(5, [60, 60], [1, 1], [0, 2], [60], 4, hkv, D, bt, "bf16")
    nb = R.block_bytes(bt, hkv, D)
    stride = (1 << 29) + 16
    big = torch.empty(s.num * stride, dtype=torch.uint8, device=DEV).view(s.num, stride)
    assert s.num * stride > (1 << 32)
    big[:, :nb] = torch.tensor(s.data, device=DEV)
    want = s.run(0.125)
    s.check(want, 0.125)
    cache = kv.Cache(big, bt, hkv, D)
    out = torch.empty_like(s.out)
    kv.lora_kv_attend_shared(s.dq, out, s.batch, s.shared, s.tab, cache, 0.125, s.ws)
    torch.cuda.synchronize()
    assert torch.equal(out, s.out)


def test_many_requests_and_groups():
    rng = np.random.default_rng(9)
    B = 1300
    cuts = np.unique(rng.integers(0, B + 1, 400))
    groups = np.concatenate([[3], cuts[cuts > 3]])
    lens = rng.integers(0, 60, len(groups) - 1)
    ctx = rng.integers(0, 70, B)
    s = SharedStep(11, ctx, np.ones(B, np.int64), list(groups), list(lens), 2, 1, 32, 16, "bf16")
    s.check(s.run(0.3, max_groups=B), 0.3)
    assert int(s.batch.flags) == 0


def test_more_groups_than_lds_holds():
    rng = np.random.default_rng(3)
    B = 1500
    groups = np.sort(np.concatenate([[0, B], rng.choice(np.arange(1, B), 1148, replace=False)]))
    lens = rng.integers(0, 40, len(groups) - 1)
    assert len(lens) > 1024
    ctx, new = rng.integers(0, 50, B), np.where(rng.random(B) < 0.1, 0, 1)
    # a group is read through its first request with tokens
    first = {g: next((i for i in range(groups[g], groups[g + 1]) if new[i]), int(groups[g])) for g in range(len(lens))}
    s = SharedStep(12, ctx, new, list(groups), list(lens), 2, 1, 32, 16, "bf16", same=first)
    s.check(s.run(0.3), 0.3)
    assert int(s.batch.flags) == 0


def test_nothing_to_do():
    b = kv.Batch(4, 4, 4, 2, 64)
    sh = kv.Shared(b, 2)
    cache = kv.Cache(torch.zeros((2, R.block_bytes(16, 2, 64)), dtype=torch.uint8, device=DEV), 16, 2, 64)
    table = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    kv.lora_kv_build(i32([5, 0, 9]), i32([0, 0, 0]), 2, table, i32([]), 2, 16, b)
    kv.lora_kv_share(i32([0, 3]), i32([5]), b, sh)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    kv.lora_kv_attend_shared(q, out, b, sh, table, cache, 0.125, kv.shared_workspace(b, sh))
    torch.cuda.synchronize()
    assert torch.all(out == 3.0)
