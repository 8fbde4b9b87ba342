"""Beam search's operators on the GPU against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import beam_reference as BR
import kv_reference as R
from heterogeneous_adapters_amd import beam, kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MIN = {"bf16": torch.finfo(torch.bfloat16).min, "f32": torch.finfo(torch.float32).min}


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def logits_of(x, dtype, offset=0, pad=0):
    """x (rows, V) on the GPU: rows V + pad apart, the first `offset` elements behind a 16-byte border."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows, V = x.shape
    flat = torch.full((offset + rows * (V + pad) + 16,), float("nan"), dtype=t, device=DEV)
    y = flat[offset:offset + rows * (V + pad)].view(rows, V + pad)[:, :V]
    y.copy_(torch.tensor(x))
    return y, y.double().cpu().numpy()


class Select:
    def __init__(self, x, W, score, length, done, eos, penalty, dtype, offset=0, pad=0):
        self.W, self.eos, self.penalty = W, eos, penalty
        self.logits, self.x = logits_of(np.asarray(x), dtype, offset, pad)
        self.score = np.asarray(score, np.float32).astype(np.float64)
        self.length, self.done = np.asarray(length), np.asarray(done)
        rows, V = self.x.shape
        self.state = beam.Beams(torch.tensor(self.score, dtype=torch.float32, device=DEV), i32(length), i32(done))
        e = lambda t: torch.full((rows,), 77, dtype=t, device=DEV)  # noqa: E731
        self.parent, self.token = e(torch.int32), e(torch.int32)
        self.out = beam.Beams(e(torch.float32), e(torch.int32), e(torch.int32))
        self.flags = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = beam.select_workspace(rows // W, W, V)

    def run(self, out=None, flags=True):
        beam.lora_beam_select(self.logits, self.W, self.state, self.parent, self.token, out or self.out, self.ws,
                              length_penalty=self.penalty, eos=self.eos, flags=self.flags if flags else None)
        torch.cuda.synchronize()
        o = out or self.out
        return [t.cpu().numpy() for t in (self.parent, self.token, o.score, o.length, o.done)]

    def check(self, got, same=True):
        """Sums of exponentials: each exponent is off by one rounding of d log2(e), whose mean over the weights is below
        ln(V) 1.45 < 24, exp2 by two, the sum of 32 by 31 more: 2^-24 each, 64 of them; the total's own rounding."""
        parent, token, total, length, done, ranks = BR.select(self.x, self.W, self.score, self.length, self.done, self.eos, self.penalty)
        fine = np.isfinite(total)
        tol = np.where(fine, 2.0 ** -24 * np.abs(total) + 64 * 2.0 ** -24, 0)
        for b, best in enumerate(ranks):
            at = {(c[1], c[3]): c for c in best}
            rows = range(b * self.W, (b + 1) * self.W)
            chosen = set()
            for i, r in enumerate(rows):
                if i >= len(best):
                    assert (got[0][r], got[1][r], got[2][r], got[3][r], got[4][r]) == (-1, -1, -np.inf, 0, 1)
                    continue
                c = at[(int(got[0][r]) - b * self.W, int(got[1][r]))]
                n = max(c[5], 1) ** self.penalty
                assert abs(c[0] - best[i][0]) <= 2 * (2.0 ** -50 * abs(c[4]) + 64 * 2.0 ** -24) / n, (b, i)
                assert (c[1], c[3]) not in chosen
                chosen.add((c[1], c[3]))
                assert abs(float(got[2][r]) - c[4]) <= 2.0 ** -24 * abs(c[4]) + 64 * 2.0 ** -24
                assert got[3][r] == c[5]
                assert got[4][r] == int(bool(self.done[b * self.W + c[1]]) or (self.eos >= 0 and c[3] == self.eos))
        if same:
            assert np.array_equal(got[0], parent) and np.array_equal(got[1], token) and np.array_equal(got[4], done)
            assert np.all(np.abs(got[2][fine] - total[fine]) <= tol[fine])


def random_case(seed, B, W, V, done=0.2, spread=2.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, 1, V)) * spread + rng.standard_normal((B, W, V)) * 0.5
    score = -np.cumsum(rng.random((B, W)), 1) - 2
    return (x.reshape(B * W, V).astype(np.float32), score.flatten(), rng.integers(0, 50, B * W), (rng.random(B * W) < done).astype(np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,penalty,offset,pad", [
    (1, 1, 1, 0.0, 0, 0), (1, 4, 3, 0.0, 1, 0), (2, 1, 2048, 0.5, 0, 0), (3, 5, 2047, 1.0, 3, 0), (1, 4, 2049, 0.0, 5, 7), (2, 3, 4096, -0.7, 0, 8),
    (5, 8, 5003, 0.6, 7, 0), (1, 2, 32000, 0.0, 0, 0), (2, 16, 10007, 1.3, 2, 5), (1, 32, 3001, 0.0, 0, 1), (3, 32, 20, 0.9, 0, 0),
    (40, 3, 1000, 0.0, 0, 0), (1, 31, 40000, 0.4, 6, 0)])
def test_select_against_plain(B, W, V, penalty, offset, pad, dtype):
    x, score, length, done = random_case(B + W + V, B, W, V)
    s = Select(x, W, score, length, done, V // 2, penalty, dtype, offset, pad)
    s.check(s.run(), same=dtype == "f32" or penalty == 0.0)
    assert int(s.flags) == 0


def test_select_many_rows_and_more_chunks_than_waves():
    x, score, length, done = random_case(1, 1, 2, 60001)
    x, score = np.tile(x, (2100, 1)), np.tile(score, 2100)
    s = Select(x, 2, score, np.tile(length, 2100), np.tile(done * 0, 2100), -1, 0.0, "bf16")
    got = s.run()
    one = Select(x[:2], 2, score[:2], length, done * 0, -1, 0.0, "bf16")
    want = one.run()
    one.check(want)
    step = np.repeat(np.arange(2100) * 2, 2)
    assert np.array_equal(got[0], np.tile(want[0], 2100) + step) and np.array_equal(got[1], np.tile(want[1], 2100))
    # cut into other pieces, so summed in another order
    assert np.all(np.abs(got[2] - np.tile(want[2], 2100)) <= 2 * (64 * 2.0 ** -24 + 2.0 ** -24 * np.abs(got[2])))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,V", [(4, 3000), (8, 2048), (32, 6001)])
def test_equal_logits_go_by_row_and_token(W, V, dtype):
    for fill in (0.0, -7.5, MIN[dtype]):
        s = Select(np.full((W, V), fill), W, np.full(W, -1.5), np.full(W, 3), np.zeros(W), -1, 0.0, dtype)
        got = s.run()
        assert np.all(got[0] == 0) and np.array_equal(got[1], np.arange(W))
        assert np.all(np.abs(got[2] - (-1.5 - math.log(V))) <= 2.0 ** -24 * 12 + 64 * 2.0 ** -24)
        assert int(s.flags) == 0


def test_zeros_of_either_sign_are_equal():
    x = np.full((2, 100), -4.0)
    x[:, 10], x[:, 20], x[:, 5] = 0.0, -0.0, -0.0
    s = Select(x, 2, [-1.0, -9.0], [1, 1], [0, 0], -1, 0.0, "f32")
    got = s.run()
    assert list(got[0]) == [0, 0] and list(got[1]) == [5, 10]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_without_value(dtype):
    V, W = 4100, 4
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5 * W, V))
    x[:, ::3] = -np.inf  # masked
    x[0:W] = -np.inf  # a request without candidates
    x[W:2 * W, :] = MIN[dtype]  # masked with the lowest number, all of it
    x[2 * W:3 * W] = MIN[dtype]
    x[2 * W, 4000], x[2 * W + 1, 7] = 1.0, 0.5  # one candidate that counts per row
    x[3 * W] = -np.inf
    x[3 * W + 1, :] = -np.inf
    x[3 * W + 1, 2500] = -3.0  # a row with one token
    s = Select(x, W, np.tile([-1.0, -1.1, -1.2, -1.3], 5), np.arange(5 * W), np.zeros(5 * W), -1, 0.0, dtype)
    s.check(s.run())
    assert int(s.flags) == 0
    x[4 * W + 1, 17], x[4 * W + 1, 18], x[4 * W + 2, 0], x[4 * W + 3, V - 1] = np.nan, np.inf, np.nan, np.inf
    s = Select(x, W, np.tile([-1.0, -1.1, -1.2, -1.3], 5), np.arange(5 * W), np.zeros(5 * W), -1, 0.0, dtype)
    s.check(s.run())
    assert int(s.flags) == beam.FLAG_LOGITS
    s.check(s.run(flags=False))


def test_logits_at_the_ends_of_fp32():
    x = np.zeros((3, 50))
    x[0, 3], x[0, 9] = 3.3e38, 3.4e38
    x[1] = -3.0e38
    x[1, 4] = 3.0e38
    x[2, 1] = 1e-40
    s = Select(x, 3, [-1.0, -2.0, -3.0], [1, 1, 1], [0, 0, 0], -1, 0.0, "f32")
    got = s.run()
    assert list(got[0][:2]) == [0, 1] and list(got[1][:2]) == [9, 4]
    assert abs(got[2][0] + 1.0) < 1e-6 and abs(got[2][1] + 2.0) < 1e-6
    assert (got[0][2], got[1][2]) == (2, 1)


def test_beams_that_are_done_or_dead():
    x, score, length, _ = random_case(4, 3, 4, 500)
    score[1] = -np.inf
    score[2] = np.nan
    done = np.array([0, 1, 0, 1, 1, 1, 1, 1, 0, 0, 0, 1])
    score[11] = -0.01  # far ahead, stays first
    x[4:8] = np.nan  # rows that are done are not read
    s = Select(x, 4, score, length, done, 123, 0.0, "f32")
    got = s.run()
    s.check(got)
    assert int(s.flags) == 0
    assert sorted(got[0][4:8]) == [4, 5, 6, 7] and np.all(got[1][4:8] == 123) and got[0][8] == 11
    for p, c in zip(got[0], range(12)):
        if p >= 0 and done[p]:
            assert got[2][c] == np.float32(score[p]) and got[3][c] == length[p]


@pytest.mark.parametrize("penalty", [16.0, -16.0])
def test_steep_powers_of_length_next_to_dead_rows(penalty):
    x, score, length, done = random_case(8, 4, 3, 60)
    score[[1, 5]] = -np.inf
    length = np.array([2 ** 30, 5, 0, 1, 2, 3] * 2)
    s = Select(x, 3, score, length, done, 7, penalty, "f32")
    s.check(s.run(), same=False)


def test_start_and_in_place_steps():
    B, W, V = 3, 4, 700
    rng = np.random.default_rng(2)
    state = beam.Beams.start(B, W, device=DEV)
    score, length, done = state.score.cpu().numpy().astype(np.float64), np.zeros(B * W, np.int64), np.zeros(B * W, np.int64)
    for step in range(4):
        x = rng.standard_normal((B * W, V)).astype(np.float32) * 3
        x[:, 5] += 4.0  # ends some
        s = Select(x, W, score, length, done, 5, 0.8, "f32")
        s.state = state
        got = s.run(out=state)
        s.check(got)
        score, length, done = got[2].astype(np.float64), got[3], got[4]
        if step == 0:
            assert np.array_equal(got[0], np.repeat(np.arange(B) * W, W))
    assert done.any()


def test_select_of_nothing():
    s = beam.Beams(torch.zeros(0, device=DEV), i32([]), i32([]))
    beam.lora_beam_select(torch.zeros((0, 10), device=DEV), 4, s, i32([]), i32([]), s, beam.select_workspace(0, 4, 10))


# ------------------------------------------------------------------- reorder
def descent(rng, B, W, lens, prompt, bt, slack=3):
    """Tables whose rows share blocks as a search leaves them, free ids, number of blocks."""
    width = -(-max(lens) // bt) + slack
    table, used = np.full((B * W, width), -1), 0
    for b in range(B):
        blocks = -(-lens[b] // bt)
        line = np.arange(W)
        for j in range(blocks - 1, -1, -1):
            if j < prompt[b] // bt:
                line = np.zeros(W, np.int64)
            elif j < blocks - 1:
                line = np.sort(rng.integers(0, W, W))[line]
            names, mine = np.unique(line, return_inverse=True)
            table[b * W:(b + 1) * W, j] = used + mine
            used += len(names)
    num = used + B * W + 2
    ids = rng.permutation(num)
    return np.where(table >= 0, ids[table], -1), ids[used:], num


class Reorder:
    def __init__(self, parent, W, kv_len, table, free, num, bt, rows=None, width=None):
        self.args = parent, W, np.asarray(kv_len), np.asarray(table), free, num, bt
        self.moves = beam.Moves(rows or max(len(parent), 1), width or table.shape[1])
        self.moves.freed.fill_(-9)
        self.table = i32(table)
        self.new = torch.full_like(self.table, 55)
        self.new_len = torch.full((len(parent),), 55, dtype=torch.int32, device=DEV)
        self.parent, self.kv_len, self.free = i32(parent), i32(kv_len), i32(free)

    def run(self):
        _, W, _, _, _, num, bt = self.args
        beam.lora_beam_reorder(self.parent, W, self.kv_len, self.table, self.new_len, self.new, self.free, num, bt, self.moves)
        torch.cuda.synchronize()

    def check(self):
        want = BR.reorder(*self.args)
        m = self.moves
        n, f = len(want["copies"]), len(want["freed"])
        assert np.array_equal(self.new.cpu().numpy(), want["table"]) and np.array_equal(self.new_len.cpu().numpy(), want["new_len"])
        assert (int(m.copies), int(m.given_back), int(m.flags)) == (n, f, want["flags"])
        got = np.stack([t.cpu().numpy() for t in (m.source, m.target, m.tokens)], 1)
        assert got[:n].tolist() == [list(c) for c in want["copies"]] and np.all(got[n:] == -1)
        freed = m.freed.cpu().numpy()
        assert freed[:f].tolist() == want["freed"] and np.all(freed[f:] == -9)
        return want


@pytest.mark.parametrize("B,W,bt,hi", [(1, 1, 16, 40), (1, 4, 16, 100), (3, 2, 32, 200), (7, 5, 16, 90), (2, 32, 64, 500), (30, 8, 128, 900),
                                       (300, 3, 16, 60), (2, 16, 16, 9000), (1, 31, 256, 300)])
def test_reorder_against_plain(B, W, bt, hi):
    rng = np.random.default_rng(B * W + bt)
    lens = rng.integers(1, hi, B)
    lens[0] = hi // bt * bt or bt  # a last block that is full
    prompt = [int(rng.integers(0, n + 1)) for n in lens]
    table, free, num = descent(rng, B, W, lens, prompt, bt)
    for kind in range(3):
        parent = (rng.integers(0, W, (B, W)) if kind == 0 else np.tile(np.arange(W), (B, 1)) if kind == 1 else np.zeros((B, W), int))
        parent = (parent + np.arange(B)[:, None] * W).flatten()
        if kind == 0 and W > 2:
            parent[rng.random(B * W) < 0.1] = -1
        r = Reorder(parent, W, np.repeat(lens, W), table, free, num, bt, rows=B * W + 5, width=table.shape[1] + 1)
        r.run()
        want = r.check()
        assert want["flags"] == 0
        if kind == 1:
            assert not want["copies"] and not want["freed"]
        r.run()  # the same again: nothing of the inputs has changed
        r.check()


def test_reorder_of_rows_of_different_lengths_and_empty_requests():
    rng = np.random.default_rng(3)
    W, bt, num = 4, 16, 400
    kv_len = np.array([0, 16, 17, 40, 100, 0, 33, 33, 0, 0, 0, 0])
    ids = rng.permutation(num)
    table = np.full((12, 9), -1)
    at = 0
    for i, n in enumerate(kv_len):
        k = -(-n // bt)
        table[i, :k] = ids[at:at + k]
        at += k
    for parent in ([0, 1, 2, 3, 4, 4, 4, 6, 8, 9, -1, -1], [3, 3, 2, 2, -1, -1, -1, -1, 8, 8, 8, 8], [1, 1, 1, 0, 7, 6, 7, 6, -1, 8, 9, 10]):
        r = Reorder(np.array(parent), W, kv_len, table, ids[at:], num, bt)
        r.run()
        assert r.check()["flags"] == 0


@pytest.mark.parametrize("W,bt,prompt", [(2, 16, 5), (4, 16, 40), (8, 64, 100), (32, 128, 200), (3, 16, 32)])
def test_beams_on_one_prompts_open_block_part(W, bt, prompt):
    """All rows begin with the prompt's blocks, the last of them among these, and go on from different parents."""
    rng = np.random.default_rng(W)
    B, blocks = 2, -(-prompt // bt)
    ids = rng.permutation(B * blocks + B * W + 2)
    table = np.full((B * W, blocks + 1), -1)
    table[:, :blocks] = np.repeat(ids[:B * blocks].reshape(B, blocks), W, 0)
    base = np.arange(B)[:, None] * W
    for parent in (np.arange(W) + np.zeros((B, 1), int), np.arange(W)[::-1] + np.zeros((B, 1), int), rng.integers(0, W, (B, W))):
        r = Reorder((parent + base).flatten(), W, np.full(B * W, prompt), table, ids[B * blocks:], len(ids), bt)
        r.run()
        want = r.check()
        assert want["flags"] == 0 and not want["freed"] and len(want["copies"]) == (B * (W - 1) if prompt % bt else 0)
        last = r.new.cpu().numpy()[:, blocks - 1]
        assert not prompt % bt or len(set(last)) == B * W  # every row writes to a block of its own


@pytest.mark.parametrize("case", ["parent", "length", "free", "free_id", "table_id", "no_free"])
def test_reorder_flags(case):
    rng = np.random.default_rng(5)
    B, W, bt = 3, 4, 16
    lens = [40, 50, 20]
    table, free, num = descent(rng, B, W, lens, [20, 0, 16], bt)
    parent, kv_len = np.array([0, 0, 1, 1, 5, 5, 5, 6, 8, 8, 9, 9]), np.repeat(lens, W)
    if case == "parent":
        parent[1], parent[6], parent[11] = 4, -2, 12
    if case == "length":
        kv_len[0], kv_len[9] = -3, 5000
    if case == "free":
        free = free[:2]
    if case == "free_id":
        free[1] = num + 3
    if case == "table_id":
        table[2, 0], table[5, 1] = num, -4
    if case == "no_free":
        free = free[:0]
    r = Reorder(parent, W, kv_len, table, free, num, bt)
    r.run()
    assert r.check()["flags"] == {"parent": 2, "length": 4, "free": 8, "free_id": 16, "table_id": 16, "no_free": 8}[case]


def test_reorder_of_nothing_empties_the_lists():
    rng = np.random.default_rng(5)
    table, free, num = descent(rng, 1, 4, [40], [0], 16)
    r = Reorder(np.zeros(4, int), 4, np.full(4, 40), table, free, num, 16)
    r.run()
    assert int(r.moves.copies) == 3 and int(r.moves.given_back) > 0
    none = i32([])
    wide = torch.zeros((0, table.shape[1]), dtype=torch.int32, device=DEV)
    beam.lora_beam_reorder(none, 4, none, wide, none.clone(), wide.clone(), r.free, num, 16, r.moves)
    torch.cuda.synchronize()
    assert (int(r.moves.copies), int(r.moves.given_back), int(r.moves.flags)) == (0, 0, 0) and torch.all(r.moves.source == -1)


@pytest.mark.parametrize("layers,hkv,D,bt,extra", [(1, 1, 32, 16, 0), (3, 2, 96, 64, 32), (5, 3, 128, 256, 16), (70, 1, 64, 32, 0), (2, 8, 256, 16, 0)])
def test_copies_in_every_layer(layers, hkv, D, bt, extra):
    rng = np.random.default_rng(layers)
    B, W = 4, 3
    lens = [3 * bt + 1, 5, 2 * bt, bt + bt // 2 + 1]
    table, free, num = descent(rng, B, W, lens, [bt, 0, bt, 0], bt)
    parent = np.array([0, 0, 0, 3, 4, 3, 6, 6, 7, 10, 9, 10])
    r = Reorder(parent, W, np.repeat(lens, W), table, free, num, bt)
    r.run()
    want = r.check()
    nb = R.block_bytes(bt, hkv, D)
    data = [torch.tensor(rng.integers(0, 256, (num, nb + extra)).astype(np.uint8), device=DEV) for _ in range(layers)]
    before = [d.cpu().numpy() for d in data]
    beam.lora_beam_copy(r.moves, beam.Layers([kv.Cache(d, bt, hkv, D) for d in data]))
    torch.cuda.synchronize()
    for b, d in zip(before, data):
        rec = b[:, :nb].reshape(num, hkv, bt // 16, -1)
        for source, target, tokens in want["copies"]:
            rec[target, :, :-(-tokens // 16)] = rec[source, :, :-(-tokens // 16)]
        assert np.array_equal(d.cpu().numpy(), b)


def test_copies_outside_the_cache_and_without_target_are_left_out():
    rng = np.random.default_rng(1)
    table, free, num = descent(rng, 1, 4, [20], [0], 16)
    free = free.copy()
    free[0], table[0, 1] = num + 1, num + 9
    r = Reorder(np.array([0, 0, 1, 1]), 4, np.full(4, 20), table, free[:1], num, 16)
    r.run()
    r.check()
    data = torch.randint(0, 256, (num, R.block_bytes(16, 1, 32)), dtype=torch.uint8, device=DEV)
    before = data.clone()
    beam.lora_beam_copy(r.moves, beam.Layers([kv.Cache(data, 16, 1, 32)]))
    beam.lora_beam_copy(beam.Moves(4, 4), beam.Layers([kv.Cache(data, 16, 1, 32)]))  # no reorder yet
    beam.lora_beam_copy(r.moves, beam.Layers([]))
    torch.cuda.synchronize()
    assert torch.equal(data, before)


# ------------------------------------------------------------ a whole search
@pytest.mark.parametrize("W,bt,graphed", [(4, 16, False), (3, 32, False), (4, 16, True)])
def test_a_search_over_the_cache(W, bt, graphed):
    """Prompts, then steps of select, reorder, copy, build, append and shared attention: each beam's cached tokens are its
    history's, its attention is over them, and every block is in a table or free."""
    B, hq, hkv, D, V, steps, layers = 2, 4, 2, 64, 300, 9, 2
    rng = np.random.default_rng(W)
    prompt = [37, 70]
    rows = B * W
    width = -(-(max(prompt) + steps + 2) // bt)
    num = rows * width + 5
    nb = R.block_bytes(bt, hkv, D)
    caches = [kv.Cache(torch.zeros((num, nb), dtype=torch.uint8, device=DEV), bt, hkv, D) for _ in range(layers)]
    stack = beam.Layers(caches)
    # a token's K and V are its own at its place in the text: [token][position]
    kt = torch.randn((V, 100, hkv, D), dtype=torch.float64).to(torch.bfloat16).to(DEV)
    vt = torch.randn((V, 100, hkv, D), dtype=torch.float64).to(torch.bfloat16).to(DEV)
    text = [[list(rng.integers(0, V, n))] + [[] for _ in range(W - 1)] for n in prompt]
    history = [t for g in text for t in g]
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    other = torch.full_like(table, -1)
    free = list(rng.permutation(num))
    batch = kv.Batch(rows * 80, rows, hq, hkv, D)
    shared = kv.Shared(batch, B)
    ws, sws = kv.attend_workspace(batch), kv.shared_workspace(batch, shared)
    moves = beam.Moves(rows, width)
    state, nxt = beam.Beams.start(B, W, device=DEV), beam.Beams.start(B, W, device=DEV)
    parent, token = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(rows, dtype=torch.int32, device=DEV)
    select_ws = beam.select_workspace(B, W, V)
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    groups, shared_len = i32([0, W, 2 * W]), i32(prompt)
    sm = 1.0 / math.sqrt(D)

    def append(new):
        """Caches the last new[r] tokens of every row."""
        T = int(sum(new))
        tok = [t for r in range(rows) for t in history[r][len(history[r]) - new[r]:]]
        kv.lora_kv_build(lens, i32(new), T, table, i32(free), num, bt, batch)
        pos = batch.positions.long()
        for layer, c in enumerate(caches):
            kv.lora_kv_append(None, None, (kt[tok, pos] * (1 + layer)).contiguous(), vt[tok, pos].contiguous(), None, batch.slots, None, c, batch)
        torch.cuda.synchronize()
        assert int(batch.flags) == 0
        del free[:int(batch.new_blocks)]
        lens.add_(i32(new))

    append([len(h) for h in history])
    reused = False
    for step in range(steps):
        x = rng.standard_normal((rows, V)).astype(np.float32) * 2
        x[:, 7] += 3.0  # the end of a text
        if step == 0:
            logits = torch.empty((rows, V), device=DEV)
        logits.copy_(torch.tensor(x))
        want = BR.select(x.astype(np.float64), W, *[t.cpu().numpy().astype(np.float64 if i == 0 else np.int64)
                                                    for i, t in enumerate((state.score, state.length, state.done))], 7, 0.0)
        free_dev = i32(free + [0] * (num - len(free)))[:rows]

        def move():
            beam.lora_beam_select(logits, W, state, parent, token, nxt, select_ws, eos=7)
            beam.lora_beam_reorder(parent, W, lens, table, new_len, other, free_dev, num, bt, moves)
            beam.lora_beam_copy(moves, stack)

        new_len = torch.zeros_like(lens)
        if graphed and step > 2:  # captured: run twice, the same both times
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                move()
            torch.cuda.current_stream().wait_stream(side)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                move()
            g.replay()
            torch.cuda.synchronize()
            g.replay()
        else:
            move()
        torch.cuda.synchronize()
        par, tok = parent.cpu().numpy(), token.cpu().numpy()
        assert np.array_equal(par, want[0]) and np.array_equal(tok, want[1])
        assert int(moves.flags) == 0
        ended = [bool(state.done[p]) for p in par]
        history = [list(history[p]) for p in par]
        table, other = other, table
        lens = new_len.clone()
        state, nxt = nxt, state
        taken = int(moves.copies)
        back = moves.freed[:int(moves.given_back)].tolist()
        reused = reused or bool(back)
        free = free[taken:] + back
        new = [0 if e else 1 for e in ended]
        for r in range(rows):
            if new[r]:
                history[r].append(int(tok[r]))
        append(new)
        assert lens.tolist() == [len(h) for h in history]
        # blocks: each in a table or free, once
        t = table.cpu().numpy()
        held = {int(t[r, j]) for r in range(rows) for j in range(-(-len(history[r]) // bt))}
        assert not held & set(free) and len(set(free)) == len(free) and len(held) + len(free) == num
        # the cached tokens of every beam, and its attention
        for layer, c in enumerate(caches):
            data = c.data.cpu().numpy()
            for r in range(rows):
                L = len(history[r])
                slots = [int(t[r, p // bt]) * bt + p % bt for p in range(L)]
                k, _ = R.get(data, slots, hkv, D, bt)
                w = (kt[history[r], list(range(L))] * (1 + layer)).double().cpu().numpy()
                assert np.array_equal(k, R.values(*R.quantise(w.reshape(L, hkv, -1, 32))).reshape(L, hkv, D)), (step, layer, r)
        T = int(sum(new))
        if T == 0:
            continue
        q = torch.randn((T, hq, D), device=DEV).to(torch.bfloat16)
        out, plain = torch.empty_like(q), torch.empty_like(q)
        kv.lora_kv_share(groups, shared_len, batch, shared)
        kv.lora_kv_attend_shared(q, out, batch, shared, table, caches[0], sm, sws)
        kv.lora_kv_attend(q, plain, batch, table, caches[0], sm, ws)
        torch.cuda.synchronize()
        assert int(batch.flags) == 0
        data, qh, oh, ph = caches[0].data.cpu().numpy(), q.double().cpu().numpy(), out.double().cpu().numpy(), plain.double().cpu().numpy()
        at = 0
        for r in range(rows):
            if not new[r]:
                continue
            L = len(history[r])
            k, v = R.get(data, [int(t[r, p // bt]) * bt + p % bt for p in range(L)], hkv, D, bt)
            o, a, s = R.attend_rows(qh[at:at + 1], k, v, [L], sm)
            bound = R.attend_bound(o, a, s, L, D, "bf16")
            assert np.all(np.abs(oh[at:at + 1] - o) <= bound) and np.all(np.abs(ph[at:at + 1] - o) <= bound)
            at += 1
    assert reused and bool((state.done != 0).any())
