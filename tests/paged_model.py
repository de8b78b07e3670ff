"""The paged cache's rules in plain Python (test helper): the model the CUDA calls are held to."""
import numpy as np


class Model:
    def __init__(self, k, v, max_seqs, max_pages):
        self.k, self.v = k.copy(), v.copy()  # [layers, pages, page, heads, hd]
        self.page = k.shape[2]
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(max_seqs, np.int32)
        self.refs = np.zeros(k.shape[1], np.int32)
        self.status = 0

    def held(self, n):
        return -(-int(n) // self.page)

    def hand_out(self, needs):
        """Pages for each entry in order, lowest first; an entry the free pages do not reach gets None, as does
        every later one that needs pages."""
        free = [int(p) for p in np.flatnonzero(self.refs == 0)]
        out, at = [], 0
        for n in needs:
            if n is None:
                out.append(None)
                continue
            if n and at + n > len(free):
                self.status |= 2
                out.append(None)
                at += n
                continue
            out.append(free[at:at + n])
            at += n
        for pages in out:
            for p in pages or []:
                self.refs[p] = 1
        return out

    def extend(self, seqs, add):
        needs, named = [], set()
        for s, a in zip(seqs, add):
            if not 0 <= s < len(self.lens) or s in named or a < 0:
                self.status |= 1
                needs.append(None)
                named.add(s)
                continue
            named.add(s)
            if self.lens[s] + a > self.table.shape[1] * self.page:
                self.status |= 16
                needs.append(None)
                continue
            needs.append(self.held(self.lens[s] + a) - self.held(self.lens[s]))
        for s, a, pages in zip(seqs, add, self.hand_out(needs)):
            if pages is None:
                continue
            h = self.held(self.lens[s])
            self.table[s, h:h + len(pages)] = pages
            self.lens[s] += a

    def append(self, layer, seqs, counts, k, v):
        at = 0
        for s, n in zip(seqs, counts):
            for i in range(n):
                p = int(self.lens[s]) - n + i
                page = self.table[s, p // self.page]
                if self.refs[page] > 1:
                    self.status |= 8
                else:
                    self.k[layer, page, p % self.page] = k[at]
                    self.v[layer, page, p % self.page] = v[at]
                at += 1

    def fork(self, src, dst, share):
        needs, named, size = [], set(), self.lens.copy()
        n = len(self.lens)
        for s, d in zip(src, dst):
            if not 0 <= s < n or not 0 <= d < n or d in named or size[d] != 0:
                self.status |= 1
                needs.append(None)
                if 0 <= s < n:
                    named.add(d)
                continue
            named.add(d)
            needs.append(self.held(size[s]) - (size[s] // self.page if share else 0))
        for s, d, pages in zip(src, dst, self.hand_out(needs)):
            if pages is None:
                continue
            kept = size[s] // self.page if share else 0
            for j in range(self.held(size[s])):
                old = self.table[s, j]
                if j < kept:
                    self.table[d, j] = old
                    self.refs[old] += 1
                else:
                    new = pages[j - kept]
                    self.table[d, j] = new
                    there = min(self.page, size[s] - j * self.page)
                    self.k[:, new, :there] = self.k[:, old, :there]
                    self.v[:, new, :there] = self.v[:, old, :there]
            self.lens[d] = size[s]

    def free(self, seqs):
        for s in seqs:
            if not 0 <= s < len(self.lens):
                self.status |= 1
                continue
            for j in range(self.held(self.lens[s])):
                self.refs[self.table[s, j]] -= 1
            self.table[s] = -1
            self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        high = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = np.arange(len(self.refs), dtype=np.int32)
        for a, b in zip(high, holes):
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            to[a] = b
        self.table = np.where(self.table >= 0, to[self.table], self.table).astype(np.int32)
        return live

    def sequence(self, layer, s):
        """Keys and values of sequence s: [len, heads, hd]."""
        n = int(self.lens[s])
        p = np.arange(n)
        at = self.table[s, p // self.page], p % self.page
        return self.k[layer][at], self.v[layer][at]
