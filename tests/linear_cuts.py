"""How linear attention cuts a call into segments of chunks (csrc/gdn_linear.hip), for tests that mean a certain form.
test_linear_cuts.py holds these against the source's own functions."""
MAX_SEG_CHUNKS = 16


def up(a, b):
    return -(-a // b)


def forward_cut(pairs, chunks, ncu):
    """(chunks of a segment, segments) of the forward pass."""
    best, least = chunks, 10 * (10 * chunks + 10)
    for a_cu in (1, 2):
        most = a_cu * ncu // pairs
        if most < 2 or chunks < 2:
            continue
        s = up(chunks, most)
        cost = (10 * s + 30) * (10 if pairs * up(chunks, s) <= ncu else 14)
        if cost < least:
            least, best = cost, s
    return best, up(chunks, best)


def grad_cut(pairs, chunks, ncu):
    """(chunks of a segment, segments) of the gradient."""
    best, seg = -1, MAX_SEG_CHUNKS
    for s in range(min(MAX_SEG_CHUNKS, up(pairs * chunks, 4 * ncu)), MAX_SEG_CHUNKS + 1):
        n, length = up(chunks, s), min(s, chunks)
        cost = 2 * up(pairs * n, ncu) * (length + 1)
        if n > 1:
            cost += up(pairs * (n - 1), 2 * ncu) * length + 2
        if best < 0 or cost <= best:
            best, seg = cost, s
    return seg, up(chunks, seg)
