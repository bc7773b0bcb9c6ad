"""Token streams of the paged cache (oracle; test infrastructure only).

A token stream stores position j in slot j % page_size of its page j / page_size.
TokenStreamsOracle is the page state machine written with explicit page ids per
position: a stack of free pages (popped from its end), each stream's dict of page
index -> page id. With a retention window, evict() frees every page none of whose
positions a later query can see (a query at p sees j > p - window, and j < sinks);
a page is freed as a whole. causal_attend_fp64 is softmax attention with the
visible set spelled out per query; tree_attend_fp64 the same for trees of drafted tokens, whose
nodes' paths are walked; rotate_fp64 the rotation of rows by positions.
"""

import numpy as np

TWO_PI = "6.2831853071795864769252867665590057683943387987502"


class TokenError(Exception):
    def __init__(self, code):
        super().__init__(code)
        self.code = code


class TokenStreamsOracle:
    def __init__(self, pool_pages, page_size):
        self.page_size = page_size
        self.free = list(range(pool_pages))[::-1]
        self.streams = {}

    def open(self, sid, max_tokens, window=0, sinks=0):
        self.streams[sid] = dict(max=max_tokens, window=window, sinks=sinks, len=0, pages={}, last=None)

    def _sees(self, st, length, j):
        """Whether some query at a position >= length sees position j."""
        return st["window"] == 0 or j >= length or j > length - st["window"] or j < st["sinks"]

    def append(self, sids, counts):
        S = self.page_size
        need = []
        for sid, n in zip(sids, counts):
            st = self.streams[sid]
            if st["len"] + n > st["max"]:
                raise TokenError("INVALID")
            have = -(-st["len"] // S)
            need.append(range(have, -(-(st["len"] + n) // S)))
        if sum(map(len, need)) > len(self.free):
            raise TokenError("OOM")
        for sid, n, new in zip(sids, counts, need):
            if n == 0:
                continue
            st = self.streams[sid]
            for i in new:
                st["pages"][i] = self.free.pop()
            st["len"] += n
            st["last"] = n

    def drop(self, sids, counts):
        S = self.page_size
        for sid, n in zip(sids, counts):
            st = self.streams[sid]
            if n < 0 or n > st["len"]:
                raise TokenError("INVALID")
            end = st["len"] - n
            gone = [i for i in range(-(-st["len"] // S)) if i not in st["pages"]]
            if gone and any(self._sees(st, end, j) for i in gone for j in range(i * S, i * S + S)):
                raise TokenError("STATE")
        for sid, n in list(zip(sids, counts))[::-1]:
            if n == 0:
                continue
            st = self.streams[sid]
            end = st["len"] - n
            for i in range(-(-st["len"] // S) - 1, -(-end // S) - 1, -1):
                self.free.append(st["pages"].pop(i))
            st["len"] = end
            st["last"] = None

    def keep(self, sids, counts, kept):
        """Of each stream's last counts[i] tokens kept[i] (a number) stay."""
        S = self.page_size
        for sid, n, m in zip(sids, counts, kept):
            st = self.streams[sid]
            if not 0 <= m <= n or n > st["len"]:
                raise TokenError("INVALID")
            if any(p // S not in st["pages"] for p in range(st["len"] - n, st["len"])):
                raise TokenError("STATE")
        self.drop(sids, [n - m for n, m in zip(counts, kept)])
        for sid, n in zip(sids, counts):
            if n:
                self.streams[sid]["last"] = None

    def rollback(self, sid):
        st = self.streams[sid]
        if st["last"] is None:
            raise TokenError("STATE")
        self.drop([sid], [st["last"]])

    def evict(self, sid):
        st, S = self.streams[sid], self.page_size
        for i in sorted(st["pages"]):
            held = range(i * S, i * S + S)
            if (i + 1) * S <= st["len"] and not any(self._sees(st, st["len"], j) for j in held):
                self.free.append(st["pages"].pop(i))
        st["last"] = None

    def release(self, sid):
        st = self.streams[sid]
        for i in sorted(st["pages"]):
            self.free.append(st["pages"].pop(i))
        st["len"], st["last"] = 0, None

    def table(self, sid):
        st, S = self.streams[sid], self.page_size
        idx = [st["pages"][i] for i in sorted(st["pages"])]
        lens = [min(S, st["len"] - i * S) for i in sorted(st["pages"])]
        return idx, lens


def visible(p, n_keys, window, sinks):
    j = np.arange(n_keys)
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def causal_attend_fp64(q, k, v, pos0, window, sinks, sm_scale):
    """q [rows][q_heads][64] at positions pos0 .., k and v [keys][heads][64], float64."""
    rows, q_heads, d = q.shape
    group = q_heads // k.shape[1]
    seen = np.stack([visible(pos0 + i, k.shape[0], window, sinks) for i in range(rows)])
    out = np.empty_like(q)
    for g in range(q_heads):
        s = sm_scale * (q[:, g] @ k[:, g // group].T)
        s = np.where(seen, s, -np.inf)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        out[:, g] = (p @ v[:, g // group]) / p.sum(axis=1, keepdims=True)
    return out


def tree_paths(parents):
    """Each node's path, itself first, walked from node to node."""
    paths = []
    for i, p in enumerate(parents):
        assert -1 <= p < i
        paths.append([i] + (paths[p] if p >= 0 else []))
    return paths


def tree_visible(parents, before, window, sinks):
    """[nodes][before + nodes]: what each node of a tree behind `before` tokens sees."""
    paths = tree_paths(parents)
    place = np.concatenate([np.arange(before), [before + len(p) - 1 for p in paths]]).astype(np.int64)
    seen = np.zeros((len(parents), before + len(parents)), dtype=bool)
    for i, path in enumerate(paths):
        seen[i, :before] = True
        seen[i, [before + a for a in path]] = True
        if window:
            seen[i] &= (place > before + len(path) - 1 - window) | (place < sinks)
    return seen


def tree_attend_fp64(q, k, v, parents, window, sinks, sm_scale):
    """q [nodes][q_heads][64], k and v [before + nodes][heads][64], float64."""
    seen = tree_visible(parents, len(k) - len(q), window, sinks)
    group = q.shape[1] // k.shape[1]
    out = np.empty_like(q)
    for g in range(q.shape[1]):
        s = np.where(seen, sm_scale * (q[:, g] @ k[:, g // group].T), -np.inf)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        out[:, g] = (p @ v[:, g // group]) / p.sum(axis=1, keepdims=True)
    return out


def rotate_fp64(x, positions, freq, axis, pair_distance):
    """Rows [rows][heads][64], positions [rows][axes]: each pair times e^(i freq position). The
    angle's whole turns are taken off in exact arithmetic (a double as a fraction)."""
    from fractions import Fraction
    out = np.empty_like(x, dtype=np.float64)
    tau = Fraction(TWO_PI)
    d = pair_distance
    for i in range(32):
        a = i // d * 2 * d + i % d
        angle = []
        for p in positions[:, axis[i]]:
            t = Fraction(float(freq[i])) * int(p)
            angle.append(float(t - round(t / tau) * tau))
        turn = np.exp(1j * np.array(angle))[:, None]
        z = (x[..., a] + 1j * x[..., a + d]) * turn
        out[..., a], out[..., a + d] = z.real, z.imag
    return out
