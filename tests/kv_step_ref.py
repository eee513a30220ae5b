"""A page pool's steps, and head norms with rotary positions, plainly (Python lists, binary64 numpy).

Shares no code with the library."""
import numpy as np

PI = 3.141592653589793


class Pool:
    """Sequences as lists of pages (None: given back), and a list of free ones, the last on top."""

    def __init__(self, pages, page, batch, max_pages, window=0, sinks=0):
        self.free = list(range(pages - 1, -1, -1))
        self.page, self.max_pages, self.window, self.sinks = page, max_pages, window, sinks
        self.lens, self.held = [0] * batch, [[] for _ in range(batch)]

    def plan(self, q_lens, tokens, advance=True):
        """cu_q, kv_lens, served, positions, slots, and the pages that each sequence has with the step."""
        cu, kv, served, positions, slots, have = [0], [], [], [0] * tokens, [-1] * tokens, []
        row, left, asked, taken = 0, len(self.free), 0, 0
        for b, n in enumerate(max(0, q) for q in q_lens):
            end = row + n
            after = self.lens[b] + n
            fits = end <= tokens and after <= self.max_pages * self.page
            need = -(-after // self.page) - len(self.held[b]) if fits else 0
            first = asked
            asked += need
            ok = fits and (need == 0 or asked <= left)
            pages = self.held[b] + ([self.free[left - 1 - first - i] for i in range(need)] if ok else [])
            taken += need if ok else 0
            for i in range(n):
                if row + i < tokens:
                    at = self.lens[b] + i
                    positions[row + i] = at
                    if ok and pages[at // self.page] is not None:
                        slots[row + i] = pages[at // self.page] * self.page + at % self.page
            row = end
            cu.append(min(row, tokens))
            kv.append(after if ok else self.lens[b])
            served.append(int(ok))
            have.append(pages)
        if advance:
            self.lens, self.held = list(kv), have
            del self.free[left - taken:]
        return cu, kv, served, positions, slots, have

    def release(self, keep=None):
        back = []
        for b, pages in enumerate(self.held):
            n = self.lens[b] if keep is None else min(max(keep[b], 0), self.lens[b])
            stay = -(-n // self.page)
            for i, page in enumerate(pages):
                past = i >= stay
                slid = self.window and (i + 1) * self.page <= n - self.window + 1 and i * self.page >= self.sinks
                if (past or slid) and page is not None:
                    back.append(page)
                    pages[i] = None
            del pages[stay:]
            self.lens[b] = n
        self.free += back[::-1]


def turn(x, weight, positions, freqs, interleaved=False, eps=1e-6, offset=0.0):
    """Rows x [T][heads][D] normed (weight not None) and rotated by positions * freqs (Python ints, 2^-64 turns), in binary64."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (offset + np.asarray(weight, np.float64))
    half = len(freqs)
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    turns = np.array([[(int(p) * f) % 2 ** 64 / 2 ** 64 for f in freqs] for p in positions]).reshape(len(positions), 1, half)
    c, s = np.cos(2 * PI * turns), np.sin(2 * PI * turns)
    out = y.copy()
    p, q = a * c - b * s, a * s + b * c
    if interleaved:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = p, q
    else:
        out[..., :half], out[..., half:2 * half] = p, q
    return out
