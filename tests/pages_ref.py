"""A page table in plain Python: lists of pages per slot and a stack of free ones."""


class Table:
    def __init__(self, n_slots, n_pages, page, max_pages):
        self.page, self.max_pages, self.n_pages = page, max_pages, n_pages
        self.free = list(range(n_pages))[::-1]
        self.pages = [[] for _ in range(n_slots)]
        self.lens = [0] * n_slots
        self.word = set()

    def _slots(self, slots):
        """Slots, None for those out of range or named before; BAD_SLOT noted."""
        seen, out = set(), []
        for s in slots:
            ok = 0 <= s < len(self.lens) and s not in seen
            if not ok:
                self.word.add("slot")
            seen.add(s)
            out.append(s if ok else None)
        return out

    def holders(self, page):
        return sum(page in p for p in self.pages)

    def extend(self, slots, counts, n_rows):
        rows, offsets, lens, wanted, left = [], [0], [], 0, len(self.free)
        state = [self.holders(p[-1]) if p else 0 for p in self.pages]
        for s, c in zip(self._slots(slots), counts):
            places = c if 0 <= c <= self.max_pages * self.page else 0
            ok = s is not None
            if ok:
                held = self.lens[s]
                ok = 0 <= c and held + c <= self.max_pages * self.page
                ok = ok and not (c and held % self.page and state[s] > 1)
                if not ok:
                    self.word.add("position")
            if ok:
                need = -(-(held + c) // self.page) - len(self.pages[s])
                wanted += need
                if need and wanted > left:
                    ok = False
                    self.word.add("pages")
            if ok:
                for _ in range(need):
                    self.pages[s].append(self.free.pop())
                rows += [self.pages[s][r // self.page] * self.page + r % self.page for r in range(held, held + c)]
                self.lens[s] = held + c
            else:
                rows += [-1] * places
            offsets.append(offsets[-1] + places)
            lens.append(0 if s is None else self.lens[s])
        rows = (rows + [-1] * n_rows)[:n_rows]
        return rows, offsets, lens

    def share(self, slots, source, n_pages):
        full = self.lens[source] // self.page
        before = list(self.lens)
        for s in self._slots(slots):
            if s is None:
                continue
            if s == source or before[s] or full < n_pages:
                self.word.add("position")
                continue
            self.pages[s] = self.pages[source][:n_pages]
            self.lens[s] = n_pages * self.page

    def truncate(self, slots, lens=None):
        gone = []
        for i, s in enumerate(self._slots(slots)):
            if s is None:
                continue
            m = 0 if lens is None else lens[i]
            if m < 0:
                self.word.add("position")
            elif m < self.lens[s]:
                keep = -(-m // self.page)
                gone += self.pages[s][keep:]
                self.pages[s], self.lens[s] = self.pages[s][:keep], m
        back = []
        for p in gone:
            if p not in back and not self.holders(p):
                back.append(p)
        self.free += back[::-1]

    def table(self):
        return [p + [-1] * (self.max_pages - len(p)) for p in self.pages]
