"""The page pool (free, fork, reserve) as a program on the host would keep it:
plain lists, one sequence after another. Arrays are changed in place; every call
returns the status bits."""
from __future__ import annotations

PAGE = 16
BAD_SEQ, IN_USE, NO_PAGES, ROW_FULL, BAD_TABLE = 1, 2, 4, 8, 16


def free(table, used, count, refs, seqs):
    status = 0
    for s in seqs:
        if not 0 <= s < len(table):
            status |= BAD_SEQ
            continue
        if not 0 <= count[s] <= len(table[s]):
            status |= BAD_TABLE
            continue
        for page in list(table[s])[:count[s]]:
            if not 0 <= page < len(refs):
                status |= BAD_TABLE
            elif refs[page] <= 0:
                status |= BAD_TABLE
            else:
                refs[page] -= 1
        used[s] = count[s] = 0
    return status


def fork(table, used, count, refs, parents, children):
    status = 0
    before = list(count)
    for i, (p, c) in enumerate(zip(parents, children)):
        if not (0 <= p < len(table) and 0 <= c < len(table)) or c in parents or c in children[:i]:
            status |= BAD_SEQ
            continue
        n = -(-used[p] // PAGE)
        if before[c]:
            status |= IN_USE
            continue
        if used[p] < 0 or n > before[p] or n > len(table[p]):
            status |= BAD_TABLE
            continue
        for j in range(n):
            page = table[p][j]
            table[c][j] = page
            if 0 <= page < len(refs):
                refs[page] += 1
            else:
                status |= BAD_TABLE
        used[c], count[c] = used[p], n
    return status


def reserve(table, used, count, refs, new_tokens):
    """Returns (status, src, dst, room)."""
    status = 0
    n = len(table)
    src, dst, room = [-1] * n, [-1] * n, [PAGE * min(max(c, 0), len(table[s])) for s, c in enumerate(count)]
    before = list(refs)
    free_pages = [i for i, r in enumerate(refs) if r == 0]
    wanted = 0
    for s, add in enumerate(new_tokens):
        if add <= 0:
            continue
        width = len(table[s])
        want, first = -(-(used[s] + add) // PAGE), used[s] // PAGE
        if used[s] < 0 or not 0 <= count[s] <= width or (want <= width and -(-used[s] // PAGE) > count[s]):
            status |= BAD_TABLE
            continue
        if want > width:
            status |= ROW_FULL
            continue
        held = [table[s][j] for j in range(first, min(count[s], want))]
        if any(not 0 <= page < len(refs) for page in held):
            status |= BAD_TABLE
            continue
        places = [first + k for k, page in enumerate(held) if before[page] > 1] + list(range(count[s], want))
        wanted += len(places)
        if places and wanted > len(free_pages):
            status |= NO_PAGES
            continue
        for k, j in enumerate(places):
            page = free_pages[wanted - len(places) + k]
            if j < count[s]:
                refs[table[s][j]] -= 1
                if j == first and used[s] % PAGE:
                    src[s], dst[s] = table[s][j], page
            refs[page] = 1
            table[s][j] = page
        count[s] = max(count[s], want)
        room[s] = PAGE * count[s]
    return status, src, dst, room
