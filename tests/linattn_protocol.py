"""The mbarrier hand-offs of the tensor-core linear attention kernels (xlstm_mlstm_matrix_b200/csrc/linattn_tc.cu) in
the model of barrier_protocol: each role's waits and arrivals in program order, checked for deadlock, for a phase that
completes twice before its consumer waits, and for a wait that starts while the phase before is still open.

A group of warps that acts as one (each warp arrives, each waits) is one role here.  A TMA copy is a role of its own:
it is issued in the producer's order but completes when it likes, so two copies' completions are not ordered.
"""
from barrier_protocol import Protocol


def _copy(P, bar: str, tag: int):
    """The producer issues a copy that completes `tag` of `bar`."""
    issue = f"ISSUE_{bar}_{tag}_"
    P.arrive("load", issue, 0)
    P.wait(f"copy {bar} {tag}", issue, 0)
    P.arrive(f"copy {bar} {tag}", bar, tag)


def tile_protocol(items, nslots: int, stages: int, nx: int, z_relay: bool = True) -> Protocol:
    """tile_tc_kernel.  items: one list per item (128 tokens of a head) of its tiles, each (units, entry): how many score
    units the tile has and whether a state enters; nslots: ring slots of Y (and of the state); nx: X buffers.
    z_relay=False gives the earlier form, in which the warp of the scores skipped Z's slots."""
    P = Protocol()
    u = k = i = 0
    for xi, tiles in enumerate(items):
        xb = xi % nx
        if xi >= nx:
            P.wait("load", f"XFREE{xb}", xi - nx)
        _copy(P, f"XFULL{xb}", xi)
        P.wait("scores", f"XFULL{xb}", xi)
        P.arrive("weights", "TABLE", xi)
        P.wait("weights", "TABLE", xi)
        for ti, (units, entry) in enumerate(tiles):
            b = i & 1
            for j in range(units):
                s = k & 1
                slots_y = list(range(u, u + nslots))
                u += nslots
                slots_e = list(range(u, u + nslots)) if j == 0 and entry else []
                u += len(slots_e)
                z = u
                u += 1
                for v in slots_y + slots_e + [z]:
                    if v >= stages:
                        P.wait("load", f"EMPTY{v % stages}", v - stages)
                    _copy(P, f"FULL{v % stages}", v)
                # scores and the state's part
                if k >= 2:
                    P.wait("scores", f"PRODUCT{s}", k - 2)
                for v in slots_y:
                    P.wait("scores", f"FULL{v % stages}", v)
                    P.arrive("scores", f"EMPTY{v % stages}", v)
                P.arrive("scores", f"SCORES{s}", k)
                if j == 0:
                    if i >= 2:
                        P.wait("scores", f"TAKEN{b}", i - 2)
                    for v in slots_e:
                        P.wait("scores", f"FULL{v % stages}", v)
                        P.arrive("scores", f"EMPTY{v % stages}", v)
                    P.arrive("scores", f"ENTRY{b}", i)
                if j == units - 1 and ti == len(tiles) - 1:
                    P.arrive("scores", f"XFREE{xb}", xi)
                if z_relay:
                    P.wait("scores", f"FULL{z % stages}", z)
                    P.arrive("scores", f"ZREADY{s}", k)
                # weighted scores against Z
                if j == 0:
                    P.wait("products", f"SCALED{b}", i)
                if z_relay:
                    P.wait("products", f"ZREADY{s}", k)
                P.wait("products", f"FULL{z % stages}", z)
                P.wait("products", f"WEIGHTS{s}", k)
                P.arrive("products", f"EMPTY{z % stages}", z)
                P.arrive("products", f"PRODUCT{s}", k)
                # weights
                P.wait("weights", f"SCORES{s}", k)
                P.arrive("weights", f"WEIGHTS{s}", k)
                k += 1
            P.arrive("products", f"DONE{b}", i)
            # scaling and read-out: the storer frees the staging memory and stores from it
            P.wait("read-out", f"ENTRY{b}", i)
            P.arrive("read-out", f"SCALED{b}", i)
            P.wait("read-out", f"DONE{b}", i)
            P.arrive("read-out", "OUT_FREE", i)
            P.wait("read-out", "OUT_FREE", i)
            P.arrive("read-out", f"TAKEN{b}", i)
            P.arrive("read-out", "OUT_FULL", i)
            P.wait("read-out", "OUT_FULL", i)
            i += 1
    return P


def state_protocol(segments, stages: int, parts: int, accs: int, skip_last: bool = False) -> Protocol:
    """state_tc_kernel.  segments: per tile, the stages of each of its segments in chain order; skip_last: the last
    segment's sum is not formed.  Two groups of warps weight every other stage."""
    P = Protocol()
    c = g = stores = 0
    for tile in segments:
        for si, n in enumerate(tile):
            if si:                      # the state entering this segment leaves through the staging memory
                P.arrive("fold", "OUT_FREE", stores)
                P.wait("fold", "OUT_FREE", stores)
                P.arrive("fold", "OUT_FULL", stores)
                P.wait("fold", "OUT_FULL", stores)
                stores += 1
            if skip_last and si == len(tile) - 1:
                continue
            if g >= accs:
                P.wait("products", f"TAKEN{g % accs}", g - accs)
            for _ in range(n):
                st = c % stages
                if c >= stages:
                    P.wait("load", f"EMPTY{st}", c - stages)
                _copy(P, f"FULL{st}", c)
                w = f"weights{c & 1}"
                P.wait(w, f"FULL{st}", c)
                if c >= parts:
                    P.wait(w, f"EMPTY{(c - parts) % stages}", c - parts)
                P.arrive(w, f"SCALED{st}", c)
                P.wait("products", f"SCALED{st}", c)
                P.arrive("products", f"EMPTY{st}", c)
                c += 1
            P.arrive("products", f"ACC{g % accs}", g)
            P.wait("fold", f"ACC{g % accs}", g)
            P.arrive("fold", f"TAKEN{g % accs}", g)
            g += 1
    return P
