"""The plan of a batch, by loops: pages given and taken back, and where each new token goes.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``). Written from the statement in include/moe4.h.

Parity: pinned (invariants and a worked example in tests/test_oracle_plan_rope.py).
"""
import numpy as np

CAPACITY, BAD_INDEX = 1, 2


def batch_plan(new, lens, table, free, count, page, T, rows_each=0):
    """All as lists or arrays -> dict of slots, positions, seq_ids, offsets, lens, count, table, free, and the errors (a
    sum of CAPACITY and BAD_INDEX)."""
    new, lens = [int(x) for x in new], [int(x) for x in lens]
    table, free = np.array(table, dtype=np.int64), np.array(free, dtype=np.int64)
    B, cols, pages = len(lens), table.shape[1], len(free)
    errors = set()
    if count < 0 or count > pages:
        errors.add(BAD_INDEX)
        count = min(max(count, 0), pages)
    valid = [0 <= n <= cols * page for n in lens]
    if not all(valid):
        errors.add(BAD_INDEX)
    out_lens = list(lens)
    for b in range(B):
        if new[b] < 0 and valid[b]:
            for j in range(-(-lens[b] // page)):
                if count < pages:
                    free[count] = table[b, j]
                    count += 1
                else:
                    errors.add(BAD_INDEX)
            out_lens[b] = 0
    slots, positions, seqs = np.full(T, -1), np.zeros(T, dtype=np.int64), np.full(T, -1)
    offsets, top, asked, left, row = [0], count, 0, count, 0
    for b in range(B):
        n = max(new[b], 0)
        if rows_each:
            row = b * rows_each
        shown = min(n, rows_each) if rows_each else n  # tokens that have rows of their own
        seqs[min(row, T):min(row + shown, T)] = b
        if n > 0 and valid[b]:
            if lens[b] + n <= cols * page and (not rows_each or (n <= rows_each and row + n <= T)):
                held = -(-lens[b] // page)
                need = -(-(lens[b] + n) // page) - held
                asked += need
                if (need == 0 or asked <= top) and row + n <= T:
                    for j in range(need):
                        left -= 1
                        p = free[left]
                        if not 0 <= p < pages:
                            errors.add(BAD_INDEX)
                            p = -1
                        table[b, held + j] = p
                    for i in range(n):
                        pos = lens[b] + i
                        p = table[b, pos // page]
                        if not 0 <= p < pages:
                            errors.add(BAD_INDEX)
                        else:
                            slots[row + i] = p * page + pos % page
                        positions[row + i] = pos
                    out_lens[b] = lens[b] + n
                else:
                    errors.add(CAPACITY)
            else:
                errors.add(CAPACITY)
        row += rows_each or n
        offsets.append(min(row, 2 ** 31 - 1))
    return dict(slots=slots, positions=positions, seq_ids=seqs, offsets=np.array(offsets), lens=np.array(out_lens, dtype=np.int64),
                count=left, table=table, free=free, errors=sum(errors))
