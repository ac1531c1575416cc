"""The order in which the roles of one block of the tensor-core attention forward (csrc/attn_tc.cu) wait for
one another, as coroutines on the host: the copy warp, the two issuers and the rows of the two query tiles.
Every wait is a condition on counts of what has happened. Products and copies end as soon as they are
issued and every row moves its reference in every step: what completes here completes whenever fewer rows
do, since that only takes waits away, and in whatever time the products take, since no wait is for something
not to have happened yet."""
import dataclasses

STAGES, KEYS, ROWS = 4, 64, 128


@dataclasses.dataclass
class Walk:
    n: int
    ns: int
    first: int

    def tile(self, i):
        return i if i < self.ns else self.first + i - self.ns


def key_walk(p0, p1, kv, window, sinks):
    end = min(p1 + 1, kv)
    if end <= 0:
        return Walk(0, 0, 0)
    lo = p0 - window + 1 if window > 0 and p0 >= window else 0
    s = min(sinks, end)
    ns = (s - 1) // KEYS + 1 if s > 0 else 0
    first = max(ns, lo // KEYS)
    return Walk(ns + max(0, (end - 1) // KEYS - first + 1), ns, first)


def blocks(nq, kv, G, window, sinks, splits=1):
    """The walks of a sequence's blocks: (steps of the block, [active steps of tile 0, of tile 1])."""
    tok = ROWS // G
    pos = kv - nq
    for t0 in range(0, nq, 2 * tok):
        spans = [(t0, min(tok, nq - t0)), (t0 + tok, max(0, min(tok, nq - t0 - tok)))]
        whole = key_walk(pos + t0, pos + t0 + spans[0][1] + spans[1][1] - 1, kv, window, sinks)
        place = {whole.tile(i): i for i in range(whole.n)}
        for split in range(splits):
            w0, w1 = whole.n * split // splits, whole.n * (split + 1) // splits
            act = []
            for first, n in spans:
                w = key_walk(pos + first, pos + first + n - 1, kv, window, sinks) if n else Walk(0, 0, 0)
                steps = [place[w.tile(i)] for i in range(w.n)]
                act.append([i - w0 for i in steps if w0 <= i < w1])
            yield w1 - w0, act, 2 if spans[1][1] else 1


class Bar:
    """An mbarrier: completed phases, and a wait by parity, which can tell only neighbouring phases apart."""

    def __init__(self, count=1):
        self.count, self.arrived, self.phases = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phases = 0, self.phases + 1

    def done(self, phase):
        assert phase <= self.phases + 1 and self.phases <= phase + 1, "the parity names two phases"
        return self.phases > phase


def completes(n, act, ntiles, paged, own_wait):
    """Whether every role ends. own_wait: a row that moves its reference waits for its own tile's products;
    otherwise for the unit of the ring that carries them, which both tiles' issuers let go of."""
    full, empty = [Bar() for _ in range(STAGES)], [Bar(ntiles) for _ in range(STAGES)]
    s_full, p_full = [[Bar(), Bar()] for _ in "01"], [[Bar(), Bar()] for _ in "01"]
    o_done, fin = [Bar(), Bar()], [Bar(), Bar()]
    turns = [0, 0]  # passed to tile t

    def copies():
        for c in range(n + 2):
            if c >= STAGES:
                yield lambda: empty[c % STAGES].done(c // STAGES - 1)
            full[c % STAGES].arrive()

    def issuer(t):
        ns = np = 0
        for c in range(n + 2 if n and t < ntiles else 0):
            yield lambda: full[c % STAGES].done(c // STAGES)
            if c - 2 in act[t]:
                yield lambda: p_full[t][np & 1].done(np >> 1)
                o_done[t].arrive()
                np += 1
            if c in act[t]:
                s_full[t][ns & 1].arrive()
                ns += 1
            empty[c % STAGES].arrive()
        fin[t].arrive()

    def rows(t):
        mine, theirs = len(act[t]), len(act[1 - t])
        for k, i in enumerate(act[t]):
            yield lambda: s_full[t][k & 1].done(k >> 1)
            if paged:
                yield lambda: full[(i + 2) % STAGES].done((i + 2) // STAGES)
            if k:
                u = act[t][k - 1] + 2
                yield (lambda: o_done[t].done(k - 1)) if own_wait else (lambda: empty[u % STAGES].done(u // STAGES))
            if (k < theirs) if t else (0 < k <= theirs):
                yield lambda: turns[t] > 0
                turns[t] -= 1
            if (k + 1 < theirs) if t else (k < theirs):
                turns[1 - t] += 1
            p_full[t][k & 1].arrive()
        if mine:
            yield lambda: fin[t].done(0)

    roles = [copies(), issuer(0), issuer(1), rows(0), rows(1)]
    waits = [lambda: True] * len(roles)
    while True:
        moved = False
        for r, role in enumerate(roles):
            while role is not None and waits[r]():
                moved = True
                try:
                    waits[r] = next(role)
                except StopIteration:
                    role = roles[r] = None
        if not any(roles):
            return True
        if not moved:
            return False
