"""Token streams of the paged cache (oracle; test infrastructure only).

A token stream stores position j in slot j % page_size of its page j / page_size.
TokenStreamsOracle is the page state machine written with explicit page ids per
position: a stack of free pages (popped from its end), each stream's dict of page
index -> page id. With a retention window, evict() frees every page none of whose
positions a later query can see (a query at p sees j > p - window, and j < sinks);
a page is freed as a whole. causal_attend_fp64 is softmax attention with the
visible set spelled out per query.
"""

import numpy as np


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
