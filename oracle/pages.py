"""Oracle of the page operations, on plain Python lists.

State: refs (count of each page), table (rows of entries), lens. A page is
free when its count is not positive; pages are handed out lowest first, in
list order. Each function changes copies and returns them, with the set of
flags raised ("row", "page", "nopage", "len").
"""

PAGE = 64


def held(length, width):
    return -(-min(max(length, 0), PAGE * width) // PAGE)


def _copy(refs, table, lens):
    return list(refs), [list(r) for r in table], list(lens)


def _free(refs):
    return [p for p, c in enumerate(refs) if c <= 0]


def pages_free(refs, table, lens, rows):
    refs, table, lens = _copy(refs, table, lens)
    flags = set()
    for r in rows:
        if r < 0:
            continue
        if r >= len(table):
            flags.add("row")
            continue
        for j in range(held(lens[r], len(table[r]))):
            p = table[r][j]
            table[r][j] = -1
            if p == -1:
                continue
            if not 0 <= p < len(refs) or refs[p] <= 0:
                flags.add("page")
                continue
            refs[p] -= 1
        lens[r] = 0
    return refs, table, lens, flags


def pages_fork(refs, table, lens, parents, children):
    """Also returns the page copies [(src, dst)]."""
    before = _copy(refs, table, lens)
    refs, table, lens = _copy(refs, table, lens)
    free = _free(refs)
    flags, copies, seen = set(), [], set()
    rank = 0
    for a, c in zip(parents, children):
        if a < 0 or c < 0:
            continue
        again = c in seen
        seen.add(c)
        if a >= len(table) or c >= len(table) or again or before[2][c] > 0:
            flags.add("row")
            continue
        width = len(table[a])
        length = min(max(before[2][a], 0), PAGE * width)
        full = length // PAGE
        if length % PAGE:
            src = before[1][a][full]
            if 0 <= src < len(refs):
                mine, rank = rank, rank + 1
                if mine >= len(free):
                    flags.add("nopage")
                    continue
                table[c][full] = free[mine]
                refs[free[mine]] = 1
                copies.append((src, free[mine]))
            else:
                table[c][full] = src
                flags.add("page")
        for j in range(full):
            p = before[1][a][j]
            table[c][j] = p
            if 0 <= p < len(refs):
                refs[p] += 1
            else:
                flags.add("page")
        lens[c] = length
    return refs, table, lens, flags, copies


def pages_extend(refs, table, lens, rows, new_lens):
    refs, table, lens = _copy(refs, table, lens)
    free = _free(refs)
    flags, seen = set(), set()
    rank = 0
    for r, want in zip(rows, new_lens):
        if r < 0:
            continue
        again = r in seen
        seen.add(r)
        if r >= len(table) or again:
            flags.add("row")
            continue
        width = len(table[r])
        length = min(max(lens[r], 0), PAGE * width)
        if want < length or want > PAGE * width:
            flags.add("len")
            continue
        have, need = -(-length // PAGE), -(-want // PAGE) - -(-length // PAGE)
        mine, rank = rank, rank + need
        if rank > len(free) and need > 0:
            flags.add("nopage")
            continue
        for j in range(need):
            table[r][have + j] = free[mine + j]
            refs[free[mine + j]] = 1
        lens[r] = want
    return refs, table, lens, flags


def pages_compact(refs, table, lens):
    """Also returns num_live and the page moves [(src, dst)]."""
    live = [p for p, c in enumerate(refs) if c > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    moved = [p for p in live if p >= n]
    moves = list(zip(moved, holes))
    to = dict(moves)
    flags = set()
    new_refs = [c if i < n else 0 for i, c in enumerate(refs)]
    for s, d in moves:
        new_refs[d] = refs[s]
    new_table = []
    for row, length in zip(table, lens):
        row = list(row)
        for j in range(held(length, len(row))):
            p = row[j]
            if 0 <= p < len(refs) and refs[p] > 0:
                row[j] = to.get(p, p)
            else:
                flags.add("page")
        new_table.append(row)
    return new_refs, new_table, flags, n, moves


def pages_shrink(refs, table, lens, rows, new_lens):
    refs, table, lens = _copy(refs, table, lens)
    before = list(lens)
    flags, seen = set(), set()
    for r, want in zip(rows, new_lens):
        if r < 0:
            continue
        again = r in seen
        seen.add(r)
        if r >= len(table) or again:
            flags.add("row")
            continue
        width = len(table[r])
        if want == before[r]:
            continue
        if want < 0 or want > min(max(before[r], 0), PAGE * width):
            flags.add("len")
            continue
        for j in range(held(want, width), held(before[r], width)):
            p = table[r][j]
            table[r][j] = -1
            if p == -1:
                continue
            if not 0 <= p < len(refs) or refs[p] <= 0:
                flags.add("page")
                continue
            refs[p] -= 1
        lens[r] = want
    return refs, table, lens, flags
