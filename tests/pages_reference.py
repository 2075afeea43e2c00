"""Pages of a cache by plain Python: what dllm_pages_* do, on lists and numpy
arrays.  Contents are arrays whose first dimension counts the pages."""
import numpy as np


def free_pages(refs):
    return [p for p in range(len(refs)) if refs[p] <= 0]


def fork(pools, refs, table, held, lens, src, dst, page):
    """Returns (fresh, error); everything else in place."""
    free = free_pages(refs)
    fresh, error, served, old = [], False, 0, refs.copy()
    rows, tokens = table.copy(), lens.copy()
    broke = False
    for s, d in zip(src, dst):
        if not (0 <= s < len(table) and 0 <= d < len(table)):
            fresh.append(-2)
            error = True
            if 0 <= d < len(table):
                held[d] = lens[d] = 0
            continue
        n = int(tokens[s])
        full, tail = n // page, n % page != 0
        if tail and (broke or served == len(free)):
            fresh.append(-2)
            broke = error = True
            held[d] = lens[d] = 0
            continue
        for j in range(full):
            table[d, j] = rows[s, j]
            refs[rows[s, j]] += 1
        if tail:
            new = free[served]
            served += 1
            table[d, full] = new
            refs[new] = 1
            for a in pools:
                a[new] = a[rows[s, full]]
        fresh.append(new if tail else -1)
        held[d], lens[d] = full + tail, n
    assert (old[free] == 0).all()
    return fresh, error


def grow(refs, table, held, lens, rows, extra, page):
    free = free_pages(refs)
    taken, error, at, broke = [], False, 0, False
    for b in rows:
        if not 0 <= b < len(table):
            taken.append(-1)
            error = True
            continue
        want = -(-(int(lens[b]) + extra) // page)
        if want > table.shape[1]:
            taken.append(-1)
            error = True
            continue
        more = max(0, want - int(held[b]))
        if more and (broke or at + more > len(free)):
            taken.append(-1)
            broke = error = True
            continue
        for k in range(more):
            table[b, held[b] + k] = free[at + k]
            refs[free[at + k]] = 1
        at += more
        held[b] += more
        taken.append(more)
    return taken, error


def release(refs, table, held, rows):
    error = False
    for b in rows:
        if not 0 <= b < len(table):
            error = True
            continue
        for j in range(held[b]):
            if refs[table[b, j]] <= 0:
                error = True
            else:
                refs[table[b, j]] -= 1
        held[b] = 0
    return error


def compact(pools, refs, table, held):
    used = [p for p in range(len(refs)) if refs[p] > 0]
    U = len(used)
    new = np.full(len(refs), -1, dtype=np.int64)
    new[used] = used
    movers = [p for p in used if p >= U]
    holes = [p for p in range(U) if refs[p] <= 0]
    for a, b in zip(movers, holes):
        new[a] = b
        refs[b], refs[a] = refs[a], 0
        for x in pools:
            x[b] = x[a]
    for b in range(len(table)):
        for j in range(held[b]):
            table[b, j] = new[table[b, j]]
    return U, new
