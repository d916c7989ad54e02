"""The books of a paged cache, row by row and page by page.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain Python lists: refs [pages] (how
many places of the table hold each page), table [B][P], lens [B]; changed in place.
"""


def places(length, page, width):
    return min(-(-max(length, 0) // page), width)


def count(table, lens, page, pages):
    """The references that a table stands for."""
    refs = [0] * pages
    for row, n in zip(table, lens):
        for p in row[:places(n, page, len(row))]:
            if 0 <= p < pages:
                refs[p] += 1
    return refs


def copy_pages(caches, src, dst):
    for s, d in zip(src, dst):
        for c in caches:
            if 0 <= s < len(c) and 0 <= d < len(c):
                c[d] = c[s]


def fork(refs, table, lens, parents, page):
    rows, sizes = [list(r) for r in table], list(lens)
    for b, a in enumerate(parents):
        if a == b or not 0 <= a < len(parents):
            continue
        width = len(rows[b])
        for p in rows[b][:places(sizes[b], page, width)]:
            if 0 <= p < len(refs):
                refs[p] -= 1
        held = rows[a][:places(sizes[a], page, width)]
        for p in held:
            if 0 <= p < len(refs):
                refs[p] += 1
        table[b][:len(held)] = held
        lens[b] = sizes[a]


def append(refs, table, lens, q_starts, tokens, page):
    """Returns (slots, src, dst)."""
    before = list(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    slots, src, dst = [-1] * tokens, [-1] * len(lens), [-1] * len(lens)
    taken = 0
    for b in range(len(lens)):
        n, old, width = q_starts[b + 1] - q_starts[b], max(lens[b], 0), len(table[b])
        if n == 0 or old + n > width * page:
            continue
        have, want = places(old, page, width), places(old + n, page, width)
        own = 0
        if old % page:
            last = table[b][have - 1]
            own = int(0 <= last < len(refs) and before[last] > 1)
        need = want - have + own
        mine = free[taken:taken + need]
        taken += need
        if len(mine) < need:
            continue
        if own:
            src[b], dst[b] = table[b][have - 1], mine[0]
            refs[src[b]] -= 1
            table[b][have - 1] = mine[0]
        table[b][have:want] = mine[own:]
        for p in mine:
            refs[p] += 1
        for i in range(n):
            p = table[b][(old + i) // page]
            if 0 <= p < len(refs):
                slots[q_starts[b] + i] = p * page + (old + i) % page
        lens[b] = old + n
    return slots, src, dst


def truncate(refs, table, lens, new_lens, page):
    for b, n in enumerate(new_lens):
        n = max(n, 0)
        if n < lens[b]:
            for p in table[b][places(n, page, len(table[b])):places(lens[b], page, len(table[b]))]:
                if 0 <= p < len(refs):
                    refs[p] -= 1
            lens[b] = n


def compact(refs, table, lens, page, max_moves):
    """Returns (src, dst)."""
    src, dst, to = [-1] * max_moves, [-1] * max_moves, {}
    low, high = 0, len(refs) - 1
    for i in range(max_moves):
        while low < len(refs) and refs[low] > 0:
            low += 1
        while high >= 0 and refs[high] <= 0:
            high -= 1
        if low >= high:
            break
        src[i], dst[i], to[high] = high, low, low
        refs[low], refs[high] = refs[high], 0
    for b, row in enumerate(table):
        for i in range(places(lens[b], page, len(row))):
            row[i] = to.get(row[i], row[i])
    return src, dst
