"""The attention planner's rules (csrc/gk_plan.cuh) in plain Python: the work units of one call
from the context lengths alone.  Shares no code with the library."""
from __future__ import annotations

MIN_SPLIT, CANDS, MAX_SPLITS, UNITS_PER_WARP, MIN_PIECE, SHORT = 512, 22, 64, 8, 512, 1024


def plan(lengths, pos_w, window, planes, warps, cap, short_merge, force=None):
    """lengths: keys of a row's full layers (0: no work).  Returns a dict: split (chunk length),
    full, small (full-layer entries: whole chunks in order; pieces and remainders in any order),
    swa (window entries in row order), pieces, records, split_rows.  An entry is (row, first key,
    end, index, chunks)."""
    live = [b for b, L in enumerate(lengths) if L > 0]
    longest, total = max(lengths, default=0), sum(lengths)
    sizes = [MIN_SPLIT << k for k in range(CANDS)]

    def units(S):
        return sum(-(-lengths[b] // S) for b in live)

    def need(S):
        return sum(-(-lengths[b] // S) for b in live if lengths[b] > S)

    if force is None:
        # near a quarter of a warp's share of the full-layer work ...
        share = total * planes // (4 * warps)
        k = next((i for i, S in enumerate(sizes) if S >= share), CANDS - 1)
        # ... enough units for the warps ...
        while k > 0 and (units(sizes[k]) + len(live)) * planes < UNITS_PER_WARP * warps:
            k -= 1
        # ... and no short chunks that would give a row many partials
        while k < CANDS - 1 and sizes[k] <= SHORT and -(-longest // sizes[k]) > short_merge:
            k += 1
    else:
        k = sizes.index(force)
    while k < CANDS - 1 and sizes[k] * MAX_SPLITS < longest:
        k += 1
    while k < CANDS - 1 and need(sizes[k]) > cap:
        k += 1
    S = sizes[k]

    whole = {b: lengths[b] // S for b in live}
    rest = {b: lengths[b] % S for b in live}
    long_rows = [b for b in live if whole[b] >= 2]
    cut, parts = {b: 0 for b in live}, 0
    # last wave: chunks beyond the whole waves of the warps are cut into pieces
    n = sum(whole.values()) * planes
    if force is None and long_rows and n >= warps and n % warps:
        idle = (warps - n % warps) * S
        if (sum(rest.values()) + len(live) * window) * planes < idle:
            beyond = sum(whole.values()) - n // warps * warps // planes
            pp = min(8, S // MIN_PIECE)
            while pp >= 2:
                per_row = (MAX_SPLITS - 1 - max(whole.values())) // (pp - 1) \
                    if MAX_SPLITS - 1 >= max(whole.values()) else -1
                room = (cap - need(S)) // (pp - 1)
                c = min(beyond, per_row * len(long_rows), room)
                if c >= 1:
                    each, more = divmod(c, len(long_rows))
                    for i, b in enumerate(long_rows):
                        cut[b] = min(each + (i < more), whole[b])
                    parts = pp
                    break
                pp //= 2

    full, small, swa, records, split_rows, pieces = [], [], [], 0, [], 0
    for b in live:
        keep = whole[b] - cut[b]
        ns = keep + cut[b] * parts + (rest[b] > 0)
        full += [(b, s * S, (s + 1) * S, s, ns) for s in range(keep)]
        for i in range(cut[b] * parts):
            t = keep * S + i * (S // parts)
            small.append((b, t, t + S // parts, keep + i, ns))
        pieces += cut[b] * parts
        if rest[b]:
            small.append((b, whole[b] * S, lengths[b], ns - 1, ns))
        if ns > 1:
            records += ns
            split_rows.append((b, ns))
        swa.append((b, max(0, pos_w[b] - window + 1), pos_w[b] + 1, 0, 1))
    return dict(split=S, full=full, small=small, swa=swa, pieces=pieces, records=records,
                split_rows=split_rows, live=len(live))
