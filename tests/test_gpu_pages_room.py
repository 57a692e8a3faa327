"""Room for new tokens where free pages run out, by the words of include/q4.h: one that the free pages
do not suffice for gets nothing, nor does any after it that needs some; who needs none is served."""
import random

import pytest

from tests.gpu_util import announce, torch_mod

torch = torch_mod()
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def books(requests, width, pages, ps):
    import gptq_bit_weight_amd as q4
    return q4.Pages(q4.PagedCache(*torch.zeros(2, pages, 1, ps, 8, dtype=torch.float16, device="cuda")), requests, width)


def extend(p, news):
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    return p.extend(ints(starts), starts[-1]).tolist()


def room(table, lengths, counts, ps, news):
    """The same on the host, request by request; returns the slots of each."""
    free, ended, slots = sorted(p for p, c in enumerate(counts) if c <= 0), False, []
    for r, n in enumerate(news):
        have, want = -(-lengths[r] // ps), -(-(lengths[r] + n) // ps)
        if want > len(table[r]):                    # the row is too short: nothing, and nobody else is held up
            slots.append([-1] * n)
            continue
        if want > have and (ended or want - have > len(free)):
            ended = True
            slots.append([-1] * n)
            continue
        for e in range(have, want):
            table[r][e] = free.pop(0)
            counts[table[r][e]] = 1
        slots.append([table[r][i // ps] * ps + i % ps for i in range(lengths[r], lengths[r] + n)])
        lengths[r] += n
    return slots


def test_room_on_the_last_page():
    announce("extend: one request without a free page, one that needs none")
    p = books(2, 4, 2, 16)
    assert extend(p, [16, 3]) == list(range(16)) + [16, 17, 18]
    assert extend(p, [1, 1]) == [-1, 19]
    assert p.lengths.tolist() == [16, 4]
    # (more tokens than a lane writes by itself)
    assert extend(p, [1, 9]) == [-1] + list(range(20, 29))
    assert extend(p, [7, 3]) == [-1] * 7 + [29, 30, 31]
    assert p.lengths.tolist() == [16, 16] and p.counts.tolist() == [1, 1] and p.table.tolist() == [[0, -1, -1, -1], [1, -1, -1, -1]]
    assert extend(p, [1, 1]) == [-1, -1]
    p.free(ints([0]))
    assert extend(p, [0, 1]) == [0] and p.lengths.tolist() == [0, 17]


@pytest.mark.parametrize("seed", range(8))
def test_full_pools(seed):
    """Pools that are nearly always full."""
    rng = random.Random(seed)
    R, ps = rng.choice([5, 70, 1300]), rng.choice([2, 8, 16])
    P = rng.randint(R, 2 * R)
    announce(f"extend in full pools seed={seed} R={R} ps={ps} P={P}")
    p = books(R, 6, P, ps)
    table, lengths, counts = [[-1] * 6 for _ in range(R)], [0] * R, [0] * P
    refused = served = 0
    for _ in range(12):
        if rng.random() < 0.3:
            gone = rng.sample(range(R), max(R // 5, 1))
            p.free(ints(gone))
            for r in gone:
                for e in range(-(-lengths[r] // ps)):
                    counts[table[r][e]] -= 1
                    table[r][e] = -1
                lengths[r] = 0
        news = [rng.choice([0, 1, 1, 1, 2, rng.randint(1, 2 * ps)]) for _ in range(R)]
        before = list(lengths)
        want = room(table, lengths, counts, ps, news)
        assert extend(p, news) == [s for x in want for s in x]
        assert p.lengths.tolist() == lengths and p.counts.tolist() == counts and p.table.tolist() == table
        ended = False
        for r, n in enumerate(news):
            ended |= n > 0 and lengths[r] == before[r]
            refused += ended and n > 0 and lengths[r] == before[r]
            served += ended and lengths[r] > before[r]
    assert refused and served
