"""The cache in 8 bits and its pages, one value, one block and one sequence at a
time, in 64 bits."""
import numpy as np

# every E4M3 code's value: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f and 0xff are NaN
CODES = np.array([(-1.0) ** (c >> 7) * ((c & 7) / 8 * 2.0 ** -6 if c & 0x78 == 0
                                        else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                  if c & 0x7F != 0x7F else np.nan for c in range(256)])
POSITIVE = CODES[:0x7F]  # rising


def power(e):
    """What codes of a block with exponent e are multiplied by."""
    return np.where(np.asarray(e) == 0, 0.0, 2.0 ** (np.asarray(e, np.float64) - 127))


def encode(x):
    """The code nearest to x (of two as near the even one); beyond the largest, the largest."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, np.where(np.isnan(a), 0, a)), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    up, down = POSITIVE[hi] - a, a - POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (a <= 0), hi, lo)
    code = np.where(a == POSITIVE[hi], hi, code)
    return np.where(np.isnan(x), 0x7F, code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(top):
    """The smallest e of at least 1 with top <= 448 * 2^(e - 127); 0 of 0."""
    if top == 0:
        return 0
    e = 1
    while top > 448 * 2.0 ** (e - 127):
        e += 1
    return e


def append(x, codes, exps, counts, lengths, table, block):
    """Stores x[n][heads][d] in codes [pages][page][heads][d] (bytes) and exps [pages][blocks][heads], in place."""
    page, first = codes.shape[1], 0
    for s, (c, length) in enumerate(zip(counts, lengths)):
        old = length - c
        p = old
        while p < length:
            begin = p // block * block
            end = min(begin + block, length)
            pg, slot = int(table[s, p // page]), begin % page
            new = x[first + p - old:first + end - old].astype(np.float64)
            size = np.where(np.isfinite(new), np.abs(new), 0)
            for h in range(x.shape[1]):
                e = exponent(size[:, h].max())
                if p > begin:
                    was = int(exps[pg, slot // block, h])
                    e = max(e, was)
                    if e > was:
                        held = codes[pg, slot:slot + p - begin, h]
                        codes[pg, slot:slot + p - begin, h] = encode(CODES[held] * 2.0 ** (was - e))
                codes[pg, slot + p - begin:slot + end - begin, h] = encode(new[:, h] * 2.0 ** (127 - max(e, 1)))
                exps[pg, slot // block, h] = e
            p = end
        first += c


def values(codes, exps):
    """The values of a cache's codes."""
    block = codes.shape[1] // exps.shape[1]
    return CODES[codes] * power(exps).repeat(block, 1)[..., None]


def reserve(counts, lengths, table, page, ring, state, n):
    """(offsets, new lengths, table, ring, state, slots, positions, who is left out)."""
    table, ring, pages, width = table.copy(), ring.copy(), len(ring), table.shape[1]
    head, tail = (int(x) for x in state)
    free = tail - head
    offsets, new, slots, positions, out = [0], [], [-1] * n, [-1] * n, []
    taken, given, wanted = 0, 0, 0
    before = ring.copy()
    for s, (c, length) in enumerate(zip(counts, lengths)):
        length = ~length if length < 0 else length
        first = offsets[-1]
        offsets.append(first + max(c, 0))
        held = -(-length // page)
        if c < 0:
            for k in range(held):
                ring[(tail + given) % pages] = table[s, k]
                given += 1
            new.append(0)
            continue
        need = -(-(length + c) // page) - held
        if held + need > width:
            new.append(~length)
            out.append(s)
            continue
        wanted += need
        if (need > 0 and wanted > free) or (c > 0 and offsets[-1] > n):
            new.append(~length)
            out.append(s)
            continue
        for k in range(need):
            table[s, held + k] = before[(head + wanted - need + k) % pages]
        taken = wanted if need else taken
        for i in range(c):
            at = length + i
            slots[first + i] = int(table[s, at // page]) * page + at % page
            positions[first + i] = at
        new.append(length + c)
    return offsets, new, table, ring, [head + taken, tail + given], slots, positions, out
