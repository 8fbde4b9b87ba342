"""Rows that go on from a parent whose open block is missing: nothing that a
block's last owner left there may become a beam's tokens."""
import numpy as np
import pytest
import torch

import kv_reference as R
from heterogeneous_adapters_amd import beam, kv
from test_gpu_beam import DEV, Reorder

pytestmark = pytest.mark.gpu


def caches(num, bt, layers=2, hkv=2, D=64):
    return [torch.randint(0, 256, (num, R.block_bytes(bt, hkv, D)), dtype=torch.uint8, device=DEV) for _ in range(layers)]


def copy(moves, data, bt, hkv=2, D=64):
    beam.lora_beam_copy(moves, beam.Layers([kv.Cache(d, bt, hkv, D) for d in data]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("requests", [1, 2])
def test_heirs_of_a_row_that_lost_its_open_block(requests):
    """Two steps: the free list is empty, then rows go on from those that got nothing; a second request copies as ever."""
    W, bt, num = 3, 16, 30
    ids = np.random.default_rng(requests).permutation(num)
    table = np.full((requests * W, 4), -1)
    table[:, :2] = ids[:requests * W * 2].reshape(-1, 2)
    lens = np.full(requests * W, 20)
    first = Reorder(np.array([0, 0, 0, 3, 4, 5][:requests * W]), W, lens, table, ids[:0], num, bt)
    first.run()
    assert int(first.moves.flags) == beam.FLAG_FREE_LIST and int(first.moves.copies) == 2
    now = first.new.cpu().numpy()
    a, b = table[0, :2]
    assert now[:3].tolist() == [[a, b, -1, -1], [a, -1, -1, -1], [a, -1, -1, -1]]

    free = ids[requests * W * 2:]
    r = Reorder(np.array([1, 1, 2, 4, 4, 3][:requests * W]), W, first.new_len.cpu().numpy(), now, free, num, bt)
    r.run()
    m = r.moves
    assert int(m.flags) == beam.FLAG_BLOCK_RANGE and r.new_len.tolist() == [20] * (requests * W)
    assert r.new[:3].tolist() == [[a, -1, -1, -1]] * 3
    back = [b]
    if requests == 2:  # the next block of the list is still the first
        (p, o), (c, d) = table[3, :2].tolist(), table[4, :2].tolist()
        assert r.new[3:].tolist() == [[c, d, -1, -1], [c, free[0], -1, -1], [p, o, -1, -1]]
        back += table[5, :2].tolist()
    n = requests - 1
    assert int(m.copies) == n and torch.all(m.source[n:] == -1) and torch.all(m.target[n:] == -1) and torch.all(m.tokens[n:] == -1)
    assert m.freed[:int(m.given_back)].tolist() == back
    data = caches(num, bt)
    before = [x.cpu().numpy() for x in data]
    copy(m, data, bt)
    for x, y in zip(data, before):
        if requests == 2:
            y[free[0]] = y[table[4, 1]]  # 4 tokens: the block's one unit
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("tokens,bt", [(4, 16), (20, 64), (33, 64)])
def test_copies_from_outside_the_cache_clear_their_target(tokens, bt):
    """The heir's block holds zeros, as many records as the row has tokens there, and not what was in it."""
    W, num = 3, 20
    ids = np.random.default_rng(tokens).permutation(num)
    table = np.full((W, 3), -1)
    table[:, :2] = ids[:6].reshape(3, 2)
    table[0, 1] = num + 9
    free = ids[6:]
    r = Reorder(np.array([0, 0, 1]), W, np.full(W, bt + tokens), table, free, num, bt)
    r.run()
    m = r.moves
    assert int(m.flags) == beam.FLAG_BLOCK_RANGE and int(m.copies) == 1
    assert [int(t[0]) for t in (m.source, m.target, m.tokens)] == [num + 9, free[0], tokens]
    assert r.new[1].tolist() == [table[0, 0], free[0], -1]
    data = caches(num, bt, hkv=2, D=96)
    before = [x.cpu().numpy() for x in data]
    copy(m, data, bt, hkv=2, D=96)
    for x, y in zip(data, before):
        y.reshape(num, 2, bt // 16, -1)[free[0], :, :-(-tokens // 16)] = 0
        assert np.array_equal(x.cpu().numpy(), y)
