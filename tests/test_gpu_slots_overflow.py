"""dsa_assign_slots in a step that does not fit: the pages that leave the stack
are the ones that the table has, and lengths count the tokens that have a place,
so that the next step goes on from a whole table."""
import pytest
import torch

from dsa_sparse_attention_index_gb300 import binding as B
from test_gpu_slots import Step

pytestmark = pytest.mark.gpu

MIXES = {"small": ([10, 64, 100, 0, 63], [60, 3, 200, 0, 70]), "empty contexts": ([0] * 5, [100] * 5),
         "many": ([(7 * i) % 300 for i in range(2500)], [(3 * i) % 31 for i in range(2500)])}


def placed(s, max_rows, pages):
    """One token after another while there are rows and pages: (table, lengths, pages left)."""
    table, lens, count, rows = [list(r) for r in s.table0], list(s.cached), pages, 0
    for i, (c, n) in enumerate(zip(s.cached, s.new)):
        short = False
        for p in range(c, c + min(n, max_rows - rows)):
            if p % 64 == 0:
                short = short or count == 0
                if not short:
                    count -= 1
                    table[i][p // 64] = s.free0[count]
            lens[i] += not short
        rows += min(n, max_rows - rows)
    return table, lens, count


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("part", [0.0, 0.3, 0.55, 0.999])
@pytest.mark.parametrize("what", ["rows", "pages", "both"])
def test_assign_of_a_step_that_does_not_fit(mix, in_place, part, what):
    s = Step(*MIXES[mix], pad=0)
    taken = sum(-(-(c + n) // 64) - -(-c // 64) for c, n in zip(s.cached, s.new))
    most = int(part * s.rows) if what != "pages" else s.rows
    pages = int(part * taken) if what != "rows" else taken
    s.free0 = s.free0[:pages]
    s.reset()
    s.pos, s.slots = s.pos[:most], s.slots[:most]
    if in_place:
        s.lens, s.left = s.c, s.count
    s.call()
    table, lens, left = placed(s, most, pages)
    assert s.st.item() == B.ERR_BOUNDS
    assert s.table.tolist() == table and s.lens.tolist() == lens and s.left.item() == left
    # rows have slots in the order of the requests; those without a page have none
    want, row = [], 0
    for i, (c, n) in enumerate(zip(s.cached, s.new)):
        n = min(n, most - row)
        want += [table[i][p // 64] * 64 + p % 64 if p < lens[i] else -1 for p in range(c, c + n)]
        row += n
        assert s.starts[i + 1].item() == row
    assert s.slots.tolist() == want
