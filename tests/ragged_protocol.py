"""A model on the host of how the warps of the prefill attention kernel (csrc/ragged_attn_tc.cu) hand
work to one another: the item queue, the ring of key and value tiles, Q, the score buffers, O and the
joined halves, with copies and products that end at times of their own.  Every step takes its turn
at random, at speeds that change, and the model raises Broken where

* an arrival goes past a barrier's count,
* a wait by parity passes for the wrong phase, or can no longer pass,
* a product, a softmax step or an epilogue finds something else in its operand than it came for,
* the block ends with copies or products in flight.

`without` leaves one rule out: "q_read" (the second half of a joined item waits for the first one's last
product with Q), "pass" (an issuer lets go of a tile that only the other one uses itself, after having
seen it), "drain" (the producer sees its last copies land before it leaves)."""
import random


class Broken(Exception):
    pass


class GaveUp(Exception):
    pass


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.bytes, self.phase = name, count, count, 0, 0

    def arrive(self, expect=0):
        if self.pending < 1:
            raise Broken(f"{self.name}: arrival past its count")
        self.pending -= 1
        self.bytes += expect
        self._turn()

    def landed(self):
        self.bytes -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def blocks(self, k):
        return (self.phase & 1) == (k & 1)


class Block:
    """One CTA.  items: (key tiles, solo, tiles of row tile 0, of 1, whether each one's last half is unseen).
    f8: copies land in two staged tiles, and four warps widen them into a ring of three."""

    def __init__(self, items, seed, f8=False, without=()):
        slots = 3 if f8 else 4
        self.rng, self.items, self.slots, self.without = random.Random(seed), items, slots, without
        two = range(2)
        self.q_full, self.q_empty = Barrier("q_full", 1), Barrier("q_empty", 2 + 4)      # a warp arrives as one
        self.kv_full = [Barrier(f"kv_full {i}", 4 if f8 else 1) for i in range(slots)]
        self.kv_empty = [Barrier(f"kv_empty {i}", 2) for i in range(slots)]
        self.st_full = [Barrier(f"st_full {i}", 1 + 1) for i in two]                     # the tile; its scales
        self.st_empty = [Barrier(f"st_empty {i}", 4) for i in two]
        self.stage, self.f8 = [None, None], f8
        self.s_full = [[Barrier(f"s_full {w}{b}", 1) for b in two] for w in two]
        self.p_full = [[Barrier(f"p_full {w}{b}", 4) for b in two] for w in two]
        self.pv_done = [Barrier(f"pv_done {w}", 1) for w in two]
        self.o_full = [Barrier(f"o_full {w}", 1) for w in two]
        self.o_empty = [Barrier(f"o_empty {w}", 4) for w in two]
        self.work_full = [Barrier(f"work_full {i}", 1) for i in two]
        self.work_empty = [Barrier(f"work_empty {i}", 15 if f8 else 11) for i in two]
        self.side_full, self.q_read = Barrier("side_full", 4), Barrier("q_read", 1)
        self.work, self.ring, self.q = [None, None], [None] * slots, None
        self.s, self.p = [[None, None], [None, None]], [[set(), set()], [set(), set()]]
        self.o, self.read_out = [None, None], [0, 0]
        self.pipe, self.copies, self.abort = [[], []], [], False
        self.agents = {"finder": self._role(self._finder()), "producer": self._role(self._producer(), self._copies_landed)}
        if f8:
            for i in range(4):
                self.agents[f"widen {i}"] = self._role(self._widen(i))
        for w in two:
            self.agents[f"issuer {w}"] = self._role(self._issuer(w), lambda w=w: not self.pipe[w])
            for i in range(4):
                self.agents[f"softmax {w}{i}"] = self._role(self._softmax(w, i))

    # ---- what an agent does at its end, whether it got there or gave up
    def _role(self, steps, ended=None):
        try:
            yield from steps
        except GaveUp:
            pass
        while ended is not None and not ended():
            yield None

    def _copies_landed(self):
        # without the rule it looks only when a wait has been given up already
        return not self.copies or ("drain" in self.without and not self.abort)

    def _wait(self, bar, k):
        """The k-th phase, by parity as the kernel does."""
        while bar.blocks(k):
            if self.abort:
                raise GaveUp
            yield bar, k
        if bar.phase != k + 1:
            raise Broken(f"{bar.name}: a wait for phase {k} passed in phase {bar.phase}")

    def _wait_free(self, bar, k):
        if k > 0:
            yield from self._wait(bar, k - 1)

    def _next(self, at):
        i = at[0]
        at[0] += 1
        yield from self._wait(self.work_full[i & 1], i >> 1)
        item = self.work[i & 1]
        yield None
        self.work_empty[i & 1].arrive()
        return item

    # ---- the warps
    def _finder(self):
        for i in range(len(self.items) + 1):
            yield from self._wait_free(self.work_empty[i & 1], i >> 1)
            self.work[i & 1] = (i, *self.items[i]) if i < len(self.items) else None
            self.work_full[i & 1].arrive()
            yield None

    def _producer(self):
        at, q_loads, pos = [0], 0, 0
        while True:
            item = yield from self._next(at)
            if item is None:
                return
            i, n, solo = item[:3]
            if n == 0:
                continue
            yield from self._wait_free(self.q_empty, q_loads)
            q_loads += 1
            self.q_full.arrive(expect=1)
            self.q = None
            self.copies.append((None, i, self.q_full))
            yield None
            order = [(j, v) for j in range(n) for v in (False, True)]
            if solo:              # K0 K1 V0 K2 V1 ... V(n-1)
                order = [(0, False)] + [x for j in range(n) for x in ([(j + 1, False)] if j + 1 < n else []) + [(j, True)]]
            full, empty, to = (self.st_full, self.st_empty, self.stage) if self.f8 else (self.kv_full, self.kv_empty, self.ring)
            for j, v in order:
                slot = pos % len(to)
                yield from self._wait_free(empty[slot], pos // len(to))
                full[slot].arrive(expect=1)
                to[slot] = None
                self.copies.append(((to, slot), (i, j, v), full[slot]))
                if self.f8:
                    yield None
                    self.copies.append(((to, None), None, full[slot]))
                    full[slot].bytes += 1             # the scales' arrival comes when they land
                    full[slot].pending -= 1
                pos += 1
                yield None

    def _widen(self, warp):
        at, pos = [0], 0
        while True:
            item = yield from self._next(at)
            if item is None:
                return
            for _ in range(2 * item[1]):
                st, kv = pos % 2, pos % self.slots
                yield from self._wait(self.st_full[st], pos // 2)
                yield from self._wait_free(self.kv_empty[kv], pos // self.slots)
                tile = self.stage[st]
                yield None
                if self.stage[st] != tile or tile is None:
                    raise Broken(f"a staged tile is {self.stage[st]}, was {tile}")
                parts = self.ring[kv] if isinstance(self.ring[kv], dict) and len(self.ring[kv]) < 4 else {}
                self.ring[kv] = {**parts, warp: tile}
                self.kv_full[kv].arrive()
                self.st_empty[st].arrive()
                pos += 1
                yield None

    def _issuer(self, w):
        at, q_loads, o_uses, p_uses, pos, pipe = [0], 0, 0, 0, 0, self.pipe[w]

        def see():
            yield from self._wait(self.kv_full[pos % self.slots], pos // self.slots)

        def commit(bar):
            pipe.append(bar.arrive)

        def release(slot, alone):
            commit(self.kv_empty[slot])
            if alone and "pass" in self.without:
                commit(self.kv_empty[slot])

        def let_go(slot):
            if "pass" not in self.without:
                self.kv_empty[slot].arrive()

        while True:
            item = yield from self._next(at)
            if item is None:
                return
            i, n, solo, n0, n1, unseen = item
            if n == 0:
                continue
            nw = (n0, n1)[w]
            stop = 1 if nw > 0 and unseen[w] else 0
            left = qk_left = 2 * nw

            def qk(slot, h, j):
                nonlocal qk_left
                if qk_left != stop:
                    pipe.append(lambda i=i: self._product_qk(w, i, slot, h, j))
                qk_left -= 1
                commit(self.s_full[w][h])

            def release_q():
                commit(self.q_empty)
                if solo and w == 0 and n > 1 and "q_read" not in self.without:
                    commit(self.q_read)

            yield from self._wait(self.q_full, q_loads)
            q_loads += 1
            for j in range(min(n, 2) if solo else 1):
                yield from see()
                slot = pos % self.slots
                pos += 1
                if solo and j != w:
                    let_go(slot)
                    continue
                if nw > 0:
                    qk(slot, 0, j)
                    yield None
                    qk(slot, 1, j)
                release(slot, solo)
            yield None
            if nw <= 1:
                release_q()
            if nw > 0:
                yield from self._wait_free(self.o_empty[w], o_uses)
                o_uses += 1
            done, ahead = 0, 2 if solo else 1
            for j in range(n):
                mine = (j & 1) == w if solo else j < nw
                yield from see()
                v = pos % self.slots
                pos += 1
                k = None
                if mine:
                    done += 1
                    for h in range(2):
                        yield from self._wait(self.p_full[w][h], p_uses >> 1)
                        p_uses += 1
                        if left != stop:
                            pipe.append(lambda i=i, v=v, h=h, j=j, first=(done == 1 and h == 0):
                                        self._product_pv(w, i, v, h, j, first))
                        commit(self.pv_done[w])
                        left -= 1
                        if left == 0:
                            commit(self.o_full[w])
                        yield None
                        if done < nw:
                            if k is None:
                                yield from see()
                                k = pos % self.slots
                                pos += 1
                            qk(k, h, j + ahead)
                            yield None
                    if done + 1 == nw:
                        release_q()
                give = let_go if solo and not mine else lambda slot: release(slot, solo)
                give(v)
                if j + ahead < n:
                    if k is None:
                        yield from see()
                        k = pos % self.slots
                        pos += 1
                    give(k)
                yield None

    def _softmax(self, w, warp):
        at, steps, items, joins = [0], 0, 0, 0
        while True:
            item = yield from self._next(at)
            if item is None:
                return
            i, n, solo, n0, n1, unseen = item
            nw, join = (n0, n1)[w], solo and n > 1
            skip = 1 if nw > 0 and unseen[w] else 0
            for u in range(2 * nw - skip):
                buf, j = steps & 1, (u & ~1) + w if solo else u >> 1
                yield from self._wait(self.s_full[w][buf], steps >> 1)
                if u == 0 and not join and w == (0 if solo else 1):
                    self.q_empty.arrive()
                yield None
                if self.s[w][buf] != (i, j, buf):
                    raise Broken(f"a softmax step for {(i, j, buf)} reads S of {self.s[w][buf]}")
                if u > 0 and self.rng.random() < 0.4:             # the running maximum moves
                    yield from self._wait(self.pv_done[w], steps - 1)
                    if self.o[w] is None or len(self.o[w][1]) != u:
                        raise Broken(f"O is rescaled at step {u} while it holds {self.o[w]}")
                    yield None
                self.p[w][buf].add((i, j, buf, warp))
                self.p_full[w][buf].arrive()
                steps += 1
                yield None
            if skip:
                yield from self._wait(self.s_full[w][1], steps >> 1)
                self.p_full[w][1].arrive()
                steps += 1
            if nw > 0:
                yield from self._wait(self.o_full[w], items)
                items += 1
                if self.o[w] is None or self.o[w][0] != i or len(self.o[w][1]) != 2 * nw - skip:
                    raise Broken(f"the epilogue of item {i} reads O of {self.o[w]}")
            yield None
            if join and w == 1:
                if "q_read" not in self.without:
                    yield from self._wait(self.q_read, joins)
                self.q = ("half", i)
                yield None
                self.side_full.arrive()
            elif join:
                yield from self._wait(self.side_full, joins)
                yield None
                if self.q != ("half", i):
                    raise Broken(f"the join of item {i} reads {self.q}")
                self.q_empty.arrive()
            joins += join
            if nw > 0:
                self.read_out[w] += 1
                if self.read_out[w] % 4 == 0:
                    self.o[w] = None
                self.o_empty[w].arrive()
            yield None

    # ---- what ends at a time of its own
    def _holds(self, slot, tile):
        return self.ring[slot] == (dict.fromkeys(range(4), tile) if self.f8 else tile)

    def _product_qk(self, w, i, slot, h, j):
        if not self._holds(slot, (i, j, False)) or self.q != i:
            raise Broken(f"Q K^T of item {i} tile {j} reads {self.ring[slot]} and Q of {self.q}")
        if self.p[w][h]:
            raise Broken(f"Q K^T of item {i} tile {j} overwrites P")
        self.s[w][h] = (i, j, h)

    def _product_pv(self, w, i, slot, h, j, first):
        if not self._holds(slot, (i, j, True)) or self.p[w][h] != {(i, j, h, x) for x in range(4)}:
            raise Broken(f"P V of item {i} tile {j} reads {self.ring[slot]} and P of {self.p[w][h]}")
        self.p[w][h] = set()
        if first:
            if self.o[w] is not None:
                raise Broken(f"item {i} overwrites O before it has been read out")
            self.o[w] = (i, [])
        self.o[w][1].append((j, h))

    def _copy_lands(self):
        place, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
        if place is None:
            self.q = what
        elif place[1] is not None:
            place[0][place[1]] = what
        bar.landed()

    def run(self, give_up=None):
        """give_up(self, running): whether a wait is given up now."""
        running, blocked = dict(self.agents), {}
        speed = dict.fromkeys([*running, 0, 1, "copy"], 1.0)
        turn = 0
        while running:
            turn += 1
            if turn % self.rng.choice([30, 100, 400]) == 0:
                speed = {n: self.rng.choice([0.002, 0.05, 1, 1, 5]) for n in speed}
            if give_up is not None and give_up(self, running):
                self.abort = True
            able = [n for n in running if blocked.get(n) is None or self.abort or not blocked[n][0].blocks(blocked[n][1])]
            able += [w for w in range(2) if self.pipe[w]] + (["copy"] if self.copies else [])
            if not able:
                raise Broken("nobody can go on: " + ", ".join(f"{n} waits for {blocked[n][0].name}" for n in running))
            n = self.rng.choices(able, [speed[x] for x in able])[0]
            if n == "copy":
                self._copy_lands()
            elif isinstance(n, int):
                self.pipe[n].pop(0)()
            else:
                try:
                    blocked[n] = next(running[n])
                except StopIteration:
                    del running[n]
        if self.copies or self.pipe[0] or self.pipe[1]:
            raise Broken("the block ends with copies or products in flight")


def random_items(rng):
    items = []
    for _ in range(rng.randint(1, 14)):
        n, unseen = rng.choice([0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9]), [rng.random() < 0.5 for _ in range(2)]
        if rng.random() < 0.5:
            items.append((n, True, (n + 1) // 2, n // 2, unseen))
        else:
            items.append((n, False, rng.choice([n, n, max(n - 1, 0), 0]), n, unseen))
    return items
