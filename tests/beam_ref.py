"""Plain definitions of the page and beam-search operators, for the tests: the
pool as Python lists, one sequence after the other; the selection in 64 bits by
sorting all continuations."""
import math

import torch

PAGE, CAPACITY, ARG = 0x04, 0x08, 0x10


class Pool:
    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = list(refs), [list(r) for r in table], list(lens), page
        self.status = 0

    @classmethod
    def of(cls, pool):
        return cls(pool.refs.tolist(), pool.page_table.tolist(), pool.lens.tolist(), pool.page_size)

    def pages(self, n):
        return -(-n // self.page)

    def fits(self, n):
        return n >= 0 and self.pages(n) <= len(self.table[0])

    def hold(self, p):
        if not 0 <= p < len(self.refs):
            self.status |= PAGE
        elif self.refs[p] >= 0:
            self.refs[p] += 1

    def give_up(self, p):
        if not 0 <= p < len(self.refs) or self.refs[p] == 0:
            self.status |= PAGE
        elif self.refs[p] > 0:
            self.refs[p] -= 1

    def resize(self, new):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        todo, writers = [], {}
        for b, n in enumerate(new):
            if n < 0 or not self.fits(self.lens[b]):
                self.status |= ARG
                continue
            if not self.fits(n):
                self.status |= CAPACITY
                continue
            inside = self.lens[b] % self.page if n > self.lens[b] else 0
            last = self.table[b][self.pages(self.lens[b]) - 1] if inside else None
            if last is not None and not 0 <= last < len(self.refs):
                self.status |= PAGE
                last = None
            elif last is not None and self.refs[last] == 0:
                self.status |= PAGE
                last = None
            if last is not None:
                writers.setdefault(last, []).append(b)
            todo.append((b, n, inside, last))
        plan, taken = [], 0
        for b, n, inside, last in todo:
            copy = False
            if last is not None:
                others = self.refs[last] - len(writers[last])  # holders that do not grow
                copy = self.refs[last] < 0 or (self.refs[last] > 1 and (others > 0 or b != writers[last][0]))
            need = max(self.pages(n) - self.pages(self.lens[b]), 0)
            plan.append((b, n, inside, last, copy))
            taken += need + copy
        moves = []
        if taken > len(free):
            self.status |= CAPACITY
            return moves
        free = iter(free)
        drop = []
        for b, n, inside, last, copy in plan:
            had, has = self.pages(self.lens[b]), self.pages(n)
            if copy:
                p = next(free)
                moves.append((last, p, inside))
                self.table[b][had - 1] = p
                self.refs[p] = 1
                drop.append(last)
            for i in range(had, has):
                self.table[b][i] = p = next(free)
                self.refs[p] = 1
            for i in range(has, had):
                drop.append(self.table[b][i])
                self.table[b][i] = -1
            self.lens[b] = n
        for p in drop:
            self.give_up(p)
        return moves

    def fork(self, parents):
        table, lens = [list(r) for r in self.table], list(self.lens)
        drop = []
        for b, src in enumerate(parents):
            if src == b:
                continue
            if not -1 <= src < len(lens) or not self.fits(lens[b]) or (src >= 0 and not self.fits(lens[src])):
                self.status |= ARG
                continue
            n = lens[src] if src >= 0 else 0
            had, has = self.pages(lens[b]), self.pages(n)
            for i in range(max(had, has)):
                old = table[b][i] if i < had else None
                new = table[src][i] if i < has else None
                self.table[b][i] = -1 if new is None else new
                if old == new:
                    continue
                if new is not None:
                    self.hold(new)
                if old is not None:
                    drop.append(old)
            self.lens[b] = n
        for p in drop:
            self.give_up(p)

    def compact(self):
        used = sum(r != 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= used]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < used][:len(src)]
        remap = [p if r else -1 for p, r in enumerate(self.refs)]
        for s, d in zip(src, dst):
            remap[s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
        for b, n in enumerate(self.lens):
            if not self.fits(n):
                self.status |= ARG
                continue
            for i in range(self.pages(n)):
                p = self.table[b][i]
                if not 0 <= p < len(remap) or remap[p] < 0:
                    self.status |= PAGE
                else:
                    self.table[b][i] = remap[p]
        return [(s, d, self.page) for s, d in zip(src, dst)], remap

    def check(self):
        """The counts are those of the held entries (no page is pinned or held from outside)."""
        count = [0] * len(self.refs)
        for row, n in zip(self.table, self.lens):
            for p in row[:self.pages(n)]:
                count[p] += 1
        assert count == self.refs


def continuations(logits, scores, done=None, done_token=0):
    """The scores of all continuations [batch, beams, vocab] in 64 bits, -inf where none is offered."""
    batch, beams = scores.shape
    logits, scores = logits.double().cpu().view(batch, beams, -1), scores.double().cpu()
    flat = torch.full(logits.shape, -math.inf, dtype=torch.float64)
    for b in range(batch):
        for k in range(beams):
            if not math.isfinite(scores[b, k]):
                continue
            if done is not None and done[b, k]:
                flat[b, k, done_token] = scores[b, k]
                continue
            x = logits[b, k].clone()
            x[~(x <= torch.finfo(torch.float64).max)] = -math.inf
            top = x.max()
            if top > -math.inf:
                flat[b, k] = scores[b, k] + ((x - top) - torch.log(torch.exp(x - top).sum()))
    return flat


def select(logits, scores, n, done=None, done_token=0, flat=None):
    """Per request the n best (score, row, token); fewer where fewer are offered.  Equal scores: the lowest beam, of
    it the largest logit (64 bits lose what is below 2^-53 of a score), of equal ones the lowest token."""
    batch, beams = scores.shape
    flat = continuations(logits, scores, done, done_token) if flat is None else flat
    vocab = flat.shape[-1]
    logits = logits.double().cpu().view(flat.shape)
    out = []
    for b in range(batch):
        token = torch.sort(logits[b].nan_to_num(nan=-math.inf), dim=-1, descending=True, stable=True).indices
        ordered = flat[b].gather(1, token).flatten()
        order = torch.sort(ordered, descending=True, stable=True)
        out.append([(v, b * beams + i // vocab, token[i // vocab, i % vocab].item())
                    for v, i in zip(order.values[:n].tolist(), order.indices[:n].tolist()) if v > -math.inf])
    return out


def select_tolerance(score, terms):
    """A score is start + (logit - lse), and the sum of exponentials behind lse is off, relative to itself, by at most:
    the exponents' two roundings, 2 ln 2 * 2^-24 |t| with |t| <= 32 for terms that matter (what lies below adds less
    than 2^-31 a term); the exponential's 2^-22; `terms` additions of a thread in two accumulators, 2^-24 each; the
    joins' 2^-27 and the logarithm's 2^-27.  Then one rounding of the score to 32 bits."""
    return 2 * 0.6932 * 32 * 2.0 ** -24 + 2.0 ** -22 + (terms / 2 + 1) * 2.0 ** -24 + 2.0 ** -26 + 2.0 ** -24 * abs(score)
