"""clo_paged_plan on the GPU against the reference's loop over the requests
(whole numbers: equal)."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())


def run(length, keep, add, table, ring, state, max_new, in_place=False, keep_none=False):
    t = {n: gpu(x) for n, x in dict(length=length, keep=keep, add=add, table=table, ring=ring, state=state).items()}
    B = len(length)
    len_out = t["length"] if in_place else gpu(np.full(B, -7))
    ring_out = t["state"] if in_place else gpu([-7, -7])
    start, offsets, slots = gpu(np.full(B, -7)), gpu(np.full(B + 1, -7)), gpu(np.full(max_new, -7))
    err = gpu([0])
    clo.clo_paged_plan(t["length"], t["add"], t["table"], t["ring"], t["state"], ring_out, len_out, start, offsets,
                       slots, keep=None if keep_none else t["keep"], err_flag=err)
    torch.cuda.synchronize()
    got = dict(len_out=len_out, start=start, offsets=offsets, slot_map=slots, block_table=t["table"],
               free_ring=t["ring"], ring_out=ring_out)
    return {n: x.cpu().numpy() for n, x in got.items()}, int(err.item())


def compare(*a, **kw):
    want, werr = ref.plan(*a)
    got, err = run(*a, **kw)
    for n, x in want.items():
        assert np.array_equal(got[n], x), n
    assert err == werr
    return got, err


def draw(rng, B, mb, add_hi, spare):
    """A consistent state: every block is in one table entry or free."""
    length = rng.integers(0, mb * 16 - add_hi + 1, B)
    ended = rng.random(B) < 0.1
    keep = np.where(ended, 0, np.maximum(length - rng.integers(0, 40, B) * (rng.random(B) < 0.3), 0))
    add = np.where(ended, 0, rng.integers(0, add_hi + 1, B))
    used = np.arange(mb)[None] < -(-length // 16)[:, None]
    n = int(used.sum()) + spare
    ids = rng.permutation(n)
    table = np.full((B, mb), -1)
    table[used] = ids[:int(used.sum())]
    size = n + int(rng.integers(0, 5))
    size = max(size, 1)
    head = int(rng.integers(0, size))
    ring = np.full(size, -1)
    ring[(head + np.arange(spare)) % size] = ids[int(used.sum()):]
    return length, keep, add, table, ring, np.array([head, spare])


@pytest.mark.parametrize("seed", range(12))
def test_random_states(seed):
    rng = np.random.Generator(np.random.PCG64(100 + seed))
    B = int(rng.choice([1, 2, 31, 33, 200, 1025, 4096]))
    mb = int(rng.integers(2, 40))
    add_hi = int(rng.choice([1, 5, 30]))
    spare = int(rng.choice([0, B // 2, 4 * B]))
    length, keep, add, table, ring, state = draw(rng, B, mb, add_hi, spare)
    total = int(add.sum())
    max_new = int(rng.choice([0, total // 2, total, total + 37]))
    compare(length, keep, add, table, ring, state, max_new, in_place=bool(seed % 2))


def test_many_new_tokens():
    """More slots than one CTA writes."""
    rng = np.random.Generator(np.random.PCG64(7))
    length, keep, add, table, ring, state = draw(rng, 60, 400, 6000, 40000)
    compare(length, keep, add, table, ring, state, int(add.sum()) + 1000)
    compare(length, keep, add, table, ring, state, int(add.sum()) + 1001, in_place=True)


def test_keep_defaults_to_the_length():
    rng = np.random.Generator(np.random.PCG64(8))
    length, _, add, table, ring, state = draw(rng, 50, 6, 3, 100)
    want, _ = ref.plan(length, length, add, table, ring, state, 200)
    got, err = run(length, length, add, table, ring, state, 200, keep_none=True)
    assert err == 0 and all(np.array_equal(got[n], want[n]) for n in want)


def test_bad_numbers_leave_a_request_as_it_was():
    mb = 3
    length = np.array([5, 49, -1, 10, 10, 10, 48, 10])
    keep = np.array([6, 49, -1, -1, 10, 10, 48, 2])
    add = np.array([1, 0, 0, 1, -1, 2 ** 31 - 1, 1, 40])
    table = np.arange(8 * mb).reshape(8, mb)
    ring = np.arange(100, 120)
    got, err = compare(length, keep, add, table, ring, np.array([18, 5]), 64)
    assert err == ref.BAD_CTX
    assert got["start"].tolist() == [-1] * 7 + [2] and got["offsets"][-1] == 40


def test_no_room():
    """The first request that does not fit, and every later one with new
    tokens, gets nothing; one that only drops tokens is still served."""
    length, keep = np.array([16, 16, 32, 3]), np.array([16, 16, 10, 3])
    add = np.array([1, 17, 0, 1])
    table = np.array([[1, -1, -1], [2, -1, -1], [3, 4, -1], [5, -1, -1]])
    got, err = compare(length, keep, add, table, np.array([8, 9, -1, -1]), np.array([0, 2]), 50)
    assert err == ref.NO_ROOM and got["start"].tolist() == [16, -1, 10, -1]
    got, err = compare(length, keep, add, table, np.array([8, 9, 6, 7]), np.array([0, 4]), 3)
    assert err == ref.NO_ROOM | ref.BAD_INDEX  # a full ring takes nothing back


def test_bad_ring_states_and_entries():
    length, keep, add = np.array([16, 20]), np.array([16, 3]), np.array([1, 0])
    table = np.array([[1, -1], [2, 3]])
    for state in ([-1, 2], [4, 2], [0, -1], [0, 5]):
        _, err = compare(length, keep, add, table, np.array([8, 9, -1, -1]), np.array(state), 4)
        assert err & ref.BAD_INDEX
    for entry in (-1, 1 << 27, -(1 << 31)):  # a free block that is none
        got, err = compare(length, keep, add, table, np.array([entry, 9, 4, 4, 5]), np.array([0, 2]), 4)
        assert err == ref.BAD_INDEX and got["slot_map"][0] == -1


def test_no_requests():
    got, err = compare(np.zeros(0, int), np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), int), np.arange(6),
                       np.array([2, 3]), 10)
    assert err == 0 and got["offsets"].tolist() == [0] and got["ring_out"].tolist() == [2, 3]


def test_a_run_of_steps_never_shares_a_block():
    """Steps in place, with prompts, drafts dropped and requests ended, each
    against the reference; every block stays in exactly one place."""
    rng = np.random.Generator(np.random.PCG64(11))
    B, mb, size = 40, 12, 300
    length, table = np.zeros(B, int), np.full((B, mb), -1)
    ring, state = np.arange(size), np.array([0, size])
    for step in range(25):
        ended = rng.random(B) < 0.15
        keep = np.where(ended, 0, np.maximum(length - rng.integers(0, 5, B), 0))
        add = np.where(length == 0, rng.integers(0, 100, B), np.where(ended, 0, rng.integers(0, 6, B)))
        add = np.minimum(add, mb * 16 - keep)
        got, _ = compare(length, keep, add, table, ring, state, 600, in_place=True)
        length, table, ring, state = got["len_out"], got["block_table"], got["free_ring"], got["ring_out"]
        held = table[np.arange(mb)[None] < -(-length // 16)[:, None]]
        free = ring[(state[0] + np.arange(state[1])) % size]
        assert sorted(np.concatenate([held, free]).tolist()) == list(range(size))


def test_captured_and_replayed():
    """In place in a graph: each replay is one more step."""
    B, mb = 20, 8
    length, table = gpu(np.arange(B) * 3), gpu(np.full((B, mb), -1))
    for r in range(B):
        table[r, :-(-(3 * r) // 16)] = torch.arange(-(-(3 * r) // 16), dtype=torch.int32, device=dev()) + 10 * r
    ring, state = gpu(np.arange(300, 400)), gpu([95, 60])
    add, start, offsets, slots = gpu(np.ones(B)), gpu(np.zeros(B)), gpu(np.zeros(B + 1)), gpu(np.zeros(B + 4))
    call = clo.prepare_paged_plan(length, add, table, ring, state, state, length, start, offsets, slots)
    h = [x.cpu().numpy().copy() for x in (length, table, ring, state)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        want, err = ref.plan(h[0], h[0], np.ones(B, int), h[1], h[2], h[3], B + 4)
        assert err == 0
        h = [want[n] for n in ("len_out", "block_table", "free_ring", "ring_out")]
        for a, b in zip((length, table, ring, state, slots), h + [want["slot_map"]]):
            assert np.array_equal(a.cpu().numpy(), b)


def test_refused_tensors():
    i = gpu(np.zeros(4))
    args = [i, i.clone(), gpu(np.zeros((4, 2))), gpu(np.zeros(8)), gpu([0, 0]), gpu([0, 0]), i.clone(), i.clone(),
            gpu(np.zeros(5)), gpu(np.zeros(4))]
    for at, bad in ((0, i.long()), (1, i[:3]), (2, gpu(np.zeros((3, 2)))), (4, gpu([0])), (6, i[:2]), (8, i),
                    (9, i.float()), (3, i.cpu())):
        a = list(args)
        a[at] = bad
        with pytest.raises(clo.CloError):
            clo.clo_paged_plan(*a)
    with pytest.raises(clo.CloError):
        clo.clo_paged_plan(*args, keep=i[:3])
    with pytest.raises(clo.CloError):
        clo.clo_paged_plan(*args, block_size=32)
