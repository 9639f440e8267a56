"""Plain 64-bit restatements of the paged KV cache operators, written from
their definitions: page assignment, cache write, tree attention with the
error a correct kernel may have, and the move of an accepted path."""
import numpy as np

HEAD_DIM = 128
U32 = 2.0 ** -24          # half a step of fp32, relative
HALF_BF16 = 2.0 ** -8
HALF_F16 = 2.0 ** -11


class Pool:
    """Block tables, pages held and the free list, with lists and loops."""

    def __init__(self, rows, width, num_pages, page_size, free=None):
        self.page = page_size
        self.num_pages = num_pages
        self.tables = np.full((rows, width), -1, dtype=np.int32)
        self.owned = [0] * rows
        self.free = list(range(num_pages)) if free is None else list(free)

    def assign(self, seq, new, max_tokens):
        """One step, or None if it is refused (nothing changes then)."""
        rows, width = self.tables.shape
        for b in range(rows):
            if new[b] < 0 or new[b] > seq[b] or seq[b] > width * self.page:
                return None
        want = [-(-int(s) // self.page) for s in seq]
        grow = sum(max(0, w - o) for w, o in zip(want, self.owned))
        back = []
        for b in range(rows):
            back += [int(self.tables[b, i]) for i in range(want[b], self.owned[b])]
        if grow > len(back) + len(self.free) or int(np.sum(new)) > max_tokens:
            return None
        # the free list's end after the dropped pages were put there, the
        # first dropped one last
        stack = self.free + back[::-1]
        for b in range(rows):
            for i in range(self.owned[b], want[b]):
                self.tables[b, i] = stack.pop()
        self.free = stack
        self.owned = want
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        slots = np.full(max_tokens, -1, dtype=np.int64)
        positions = np.zeros(max_tokens, dtype=np.int32)
        t = 0
        for b in range(rows):
            for pos in range(int(seq[b]) - int(new[b]), int(seq[b])):
                slots[t] = int(self.tables[b, pos // self.page]) * self.page + pos % self.page
                positions[t] = pos
                t += 1
        return cu, slots, positions


def gather(cache, table, length):
    """Rows 0..length of a request: [length, heads, 128] (cache as values)."""
    page = cache.shape[1]
    return np.stack([cache[table[p // page], p % page] for p in range(length)]) if length else \
        np.zeros((0,) + cache.shape[2:], dtype=cache.dtype)


def tree_attention(q, k_cache, v_cache, tables, seq, cu, mask=None, scale=None, ds=(1.0, 1.0, 1.0),
                   fp8=False):
    """(out, tolerance) in fp64: q [T, Hq, 128], caches as values [pages, page,
    Hkv, 128].  The tolerance is what a kernel may differ by that multiplies
    exactly, accumulates in fp32 and rounds P to f16 (E4M3 cache) or bf16:
      - score: fp32 accumulation of 128 products, at most 16 u sum |q k| (the
        bound the library's score self-test checks), four more roundings of
        the score and of the reference it is taken against, and, for an E4M3
        cache, Q represented to 2^-17 of its row's largest element (a row is
        scaled to a largest element of 2^3 at least with remainders rounded to
        2^-14, or of 2^7 at least with remainders rounded to 2^-10);
      - a weight w_j moves by the score's error (twice: its own and the
        maximum's), by P's rounding, by the exponential's 2^-21;
      - P V: fp32 accumulation over the key tiles;
      - the output's own rounding to bf16."""
    T, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    scale = 1 / np.sqrt(D) if scale is None else scale
    out = np.zeros((T, Hq, D))
    tol = np.zeros((T, Hq, D))
    for b in range(len(seq)):
        a, z, L = int(cu[b]), int(cu[b + 1]), int(seq[b])
        n = z - a
        if n == 0:
            continue
        k = gather(k_cache, tables[b], L)
        v = gather(v_cache, tables[b], L)
        for i in range(n):
            sees = np.zeros(L, dtype=bool)
            sees[:L - n] = True
            if mask is None:
                sees[L - n:L - n + i + 1] = True
            else:
                for m in range(n):
                    sees[L - n + m] = (int(mask[a + i, m // 64]) >> (m % 64)) & 1
            if not sees.any():
                continue
            for h in range(Hq):
                kk, vv = k[sees, h // G] * ds[1], v[sees, h // G] * ds[2]
                qi = q[a + i, h]
                with np.errstate(all="ignore"):
                    s = kk @ qi * scale
                    w = np.exp(s - s.max())
                    total = w.sum()
                    w = w / total
                    out[a + i, h] = w @ vv
                    mag = np.abs(w) @ np.abs(vv)
                    ds_score = 16 * U32 * (np.abs(kk) @ np.abs(qi)) * scale + \
                        4 * U32 * (np.abs(s) + np.abs(s).max())
                    if fp8:
                        ds_score = ds_score + 2.0 ** -17 * np.abs(qi).max() * \
                            np.abs(kk).sum(1) * scale
                    per_weight = 2 * ds_score.max() + (HALF_F16 if fp8 else HALF_BF16) + 2.0 ** -20 + \
                        (16 + L / 128) * U32
                    tol[a + i, h] = HALF_BF16 * np.abs(out[a + i, h]) + \
                        per_weight * mag * (1 + 2 * HALF_BF16) + 2.0 ** -30 * np.abs(vv).max()
    return out, tol


def keep_path(cache, tables, seq, cu, paths, keep):
    """The cache after every request's accepted path moved to its tail."""
    new = cache.copy()
    page = cache.shape[1]
    for b in range(len(seq)):
        first = int(seq[b]) - (int(cu[b + 1]) - int(cu[b]))
        for i in range(int(keep[b])):
            s, d = first + int(paths[b][i]), first + i
            new[tables[b][d // page], d % page] = cache[tables[b][s // page], s % page]
    return new
