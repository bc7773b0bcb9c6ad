"""Token streams over the paged cache: causal attention of new tokens, the same with a sliding
window and sinks, and the cache's write (quantised or not) with its read-back.

A case's streams hold past tokens; each gets new ones. "attend" and "window" cases compute the new
tokens' attention, with the cache as it stands after their append; "write" cases append the new
tokens, read them back and drop them again. Where `own` is false the operators are computed in
elementary torch operations on plain tensors (pages, tables, codes), where it is true through the
package's public calls."""

import torch

own = False

D = 64                      # head_dim
E4M3_MAX = 448.0


def _case(name, op, **kw):
    c = dict(name=name, op=op, streams=1, past=0, new=1, ragged=False, heads=8, q_heads=32, page=256,
             e4m3=False, window=0, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token, short history: the latency of a call
        _case("decode_one", "attend", past=776, heads=16, q_heads=16),
        # a server's step: 32 users of different histories, one token each
        _case("decode_batch", "attend", streams=32, past=8191, ragged=True, page=64),
        # the same on 8-bit pages
        _case("decode_batch_e4m3", "attend", streams=32, past=8191, ragged=True, page=64, e4m3=True),
        # one user with a long document: the axis must be split to fill the card
        _case("decode_long", "attend", past=131071, q_heads=64),
        # five drafted tokens each to verify, small pages
        _case("verify_drafts", "attend", streams=16, past=4001, new=5, ragged=True, page=16),
        # a prompt from nothing, one query head per key head
        _case("prefill", "attend", new=8192, heads=16, q_heads=16),
        # a late chunk of a long prompt on 8-bit pages (1,374 new tokens of 43,968)
        _case("chunk_e4m3", "attend", past=42594, new=1374, e4m3=True),
        # a server's mixed step: some users decode, some bring a prompt's chunk; groups of 3
        _case("mixed_batch", "attend", streams=12, past=4500, new=1500, ragged=True, q_heads=24, page=64),
        # single tokens of long conversations under a sliding window with 4 sinks
        _case("window_decode", "window", streams=48, past=20000, ragged=True, q_heads=64, page=64, window=4096,
              sinks=4),
        # a prompt's chunk under a sliding window
        _case("window_chunk", "window", past=12288, new=4096, window=1024, sinks=4),
        # one token of 64 users stored in 8 bits and read back: latency
        _case("write_decode", "write", streams=64, past=500, e4m3=True, page=64),
        # prompts stored in 8 bits and read back: bandwidth
        _case("write_chunk", "write", streams=4, past=100, new=5501, ragged=True, heads=16, q_heads=16, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "window", "window", "write"])
    heads = rng.choice([2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    e4m3 = rng.random() < 0.5
    c = dict(op=op, streams=1, past=0, new=1, ragged=rng.random() < 0.7, heads=heads, q_heads=heads * group,
             page=page, e4m3=e4m3, window=0, sinks=0)
    if op == "write":
        c["new"] = _log(rng, 1, 6000)
        c["streams"] = _log(rng, 1, max(1, min(64, 20000 // c["new"])))
        c["past"] = rng.randrange(0, 800)
        return c
    kind = rng.choice(["decode", "few", "chunk"])
    if kind == "chunk":
        c["new"] = _log(rng, 40, 4000)
        c["streams"] = _log(rng, 1, max(1, min(8, 2000 // c["new"])))
        c["past"] = rng.choice([0, _log(rng, 10, 20000)])
    else:
        c["new"] = 1 if kind == "decode" else _log(rng, 2, 40)
        c["streams"] = _log(rng, 1, 48)
        c["past"] = _log(rng, 10, max(40, min(60000, 300000 // c["streams"])))
    if op == "window":
        c["window"] = _log(rng, 1, 5000)
        c["sinks"] = rng.choice([0, 1, 4, 5, 17, 100])
    return c


def _lengths(c):
    """(past, new) of each stream: ragged ones spread from an eighth of the longest to all of it."""
    n = c["streams"]
    past, new = [], []
    for i in range(n):
        f = ((i * 5 + 3) % n) / n if c["ragged"] else 0.0
        past.append(c["past"] - int(c["past"] * f * 7 / 8))
        new.append(max(1, c["new"] - int(c["new"] * f)) if c["ragged"] and c["new"] > 8 else c["new"])
    return past, new


def _pairs(c):
    """Visible (query, key) pairs and, per stream, the key positions that some query sees."""
    pairs = slots = 0
    w, s = c["window"], c["sinks"]
    for past, new in zip(*_lengths(c)):
        end = past + new
        if not w:
            pairs += new * past + new * (new + 1) // 2
            slots += end
            continue
        for p in range(past, end):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(s, lo)
        lo = max(0, past - w + 1)
        slots += end - lo + min(s, lo)
    return pairs, slots


def work(c):
    _, new = _lengths(c)
    row = D + 1 if c["e4m3"] else 2 * D
    if c["op"] == "write":
        n = sum(new) * c["heads"] * 2
        return {"bytes": n * (2 * D + row + row + 2 * D), "flops": 0}
    pairs, slots = _pairs(c)
    return {"bytes": slots * c["heads"] * 2 * row + 2 * sum(new) * c["q_heads"] * D * 2,
            "flops": 4 * D * c["q_heads"] * pairs}


def _inputs(c, seed):
    """k, v of every stream's past and new tokens ([rows][heads][64], streams back to back) and the
    new tokens' q. Keys carry a few strong channels, rows differ in size, as trained ones do."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    past, new = _lengths(c)

    def rows(n, heads, strong):
        x = torch.randn((n, heads, D), generator=g, device="cuda", dtype=torch.bfloat16)
        if strong:
            lift = torch.zeros((heads, D), device="cuda", dtype=torch.bfloat16)
            lift[:, :: 16] = torch.randn((heads, D // 16), generator=g, device="cuda").mul_(3).bfloat16()
            x += lift
        return x

    size = 1 + torch.rand((sum(past) + sum(new), 1, 1), generator=g, device="cuda").bfloat16()
    k = rows(sum(past) + sum(new), c["heads"], True)
    v = rows(sum(past) + sum(new), c["heads"], False) * size
    q = rows(sum(new), c["q_heads"], False) * 1.5
    return k, v, q


def _parts(c, x):
    """The past and the new rows of x, each packed over the streams."""
    past, new = _lengths(c)
    both = [t for i in range(len(past)) for t in (past[i], new[i])]
    pieces = torch.split(x, both)
    return torch.cat(pieces[0::2]), torch.cat(pieces[1::2])


def prepare(c, seed):
    past, new = _lengths(c)
    n, page = c["streams"], c["page"]
    k, v, q = _inputs(c, seed)
    k_past, k_new = _parts(c, k)
    v_past, v_new = _parts(c, v)
    pages = [-(-(a + b) // page) for a, b in zip(past, new)]
    state = {"case": c, "q": q, "k": k_new, "v": v_new}
    if own:
        # the program's cache: its streams opened, the past appended (and what left the window
        # evicted), and, where the call is the attention, the new tokens appended
        from paged_kv_cache_build_gb300 import PagedKVCache
        cache = PagedKVCache(sum(pages) + n, page, c["heads"], max_streams=n, fp8=c["e4m3"])
        sids = [cache.open_token_stream(a + b, window=c["window"], sinks=c["sinks"]) for a, b in zip(past, new)]
        held = [i for i in range(n) if past[i] > 0]
        if held:
            cache.append_tokens(cache.token_batch([sids[i] for i in held], [past[i] for i in held]), k_past, v_past)
        if c["window"]:
            for s in sids:
                cache.evict_window(s)
        batch = cache.token_batch(sids, new)
        if c["op"] != "write":
            cache.append_tokens(batch, k_new, v_new)
        state.update(cache=cache, batch=batch)
        return state
    # plain tensors: pages [pages][page][heads][64] (bf16, or codes with row exponents), each stream's
    # table of page ids in scrambled order, and the flat slot of every past and new token
    dev = k.device
    total = sum(pages)
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).to(dev)
    table = torch.zeros((n, max(pages)), dtype=torch.long, device=dev)
    at = [0]
    for i in range(n):
        table[i, : pages[i]] = ids[at[-1]: at[-1] + pages[i]]
        at.append(at[-1] + pages[i])
    t_past, t_new = torch.tensor(past, device=dev), torch.tensor(new, device=dev)

    def slots(count, first):
        who = torch.repeat_interleave(torch.arange(n, device=dev), count)
        start = torch.cumsum(count, 0) - count
        pos = torch.arange(int(count.sum()), device=dev) - start[who] + first[who]
        return who, pos, table[who, pos // page] * page + pos % page

    _, _, past_slot = slots(t_past, torch.zeros_like(t_past))
    who, pos, new_slot = slots(t_new, t_past)
    shape = (total * page, c["heads"], D)
    stores = []
    for old, fresh in ((k_past, k_new), (v_past, v_new)):
        if c["e4m3"]:
            store = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev),
                     torch.zeros(shape[:2], dtype=torch.int8, device=dev)]
        else:
            store = [torch.zeros(shape, dtype=torch.bfloat16, device=dev)]
        _store(store, past_slot, old)
        if c["op"] != "write":
            _store(store, new_slot, fresh)
        stores.append(store)
    state.update(stores=stores, table=table, who=who, pos=pos, new_slot=new_slot,
                 row=torch.arange(len(who), device=dev) - (torch.cumsum(t_new, 0) - t_new)[who], most=max(new))
    return state


def _quantise(x):
    """E4M3 codes (as their values) and the exponent of each row of 64."""
    x = x.float()
    big = x.abs().amax(-1)
    m, ex = torch.frexp(big)
    e = torch.where(big > 0, (ex - 9 + (m > E4M3_MAX / 512).int()).clamp(-126, 126), torch.zeros_like(ex))
    y = torch.ldexp(x, -e[..., None])
    _, ey = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (ey - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step, e


def _store(store, slot, x):
    if len(store) == 1:
        store[0][slot] = x
        return
    codes, e = _quantise(x)
    store[0].view(torch.uint8)[slot] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    store[1][slot] = e.to(torch.int8)


def _load(store, slot):
    if len(store) == 1:
        return store[0][slot].float()
    codes = store[0].view(torch.uint8)[slot].view(torch.float8_e4m3fn)
    return torch.ldexp(codes.float(), store[1][slot][..., None].int())


def run(state):
    c = state["case"]
    if own:
        cache, batch = state["cache"], state["batch"]
        if c["op"] == "write":
            cache.append_tokens(batch, state["k"], state["v"])
            out = cache.read_tokens(batch)
            cache.drop_tokens(batch)
            return out
        return cache.attend_tokens(batch, state["q"], window=c["window"], sinks=c["sinks"])
    ks, vs = state["stores"]
    if c["op"] == "write":
        slot = state["new_slot"]
        _store(ks, slot, state["k"])
        _store(vs, slot, state["v"])
        return _load(ks, slot).bfloat16(), _load(vs, slot).bfloat16()
    n, page, heads, group = c["streams"], c["page"], c["heads"], c["q_heads"] // c["heads"]
    slot = (state["table"][:, :, None] * page + torch.arange(page, device=state["q"].device)).reshape(n, -1)
    k, v = _load(ks, slot), _load(vs, slot)                               # [n][keys][heads][64]
    most, who, row = state["most"], state["who"], state["row"]
    q = torch.zeros((n, most, heads, group, D), device=k.device)
    q[who, row] = state["q"].float().reshape(-1, heads, group, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, heads, most * group, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5).reshape(n, heads, most, group, -1)
    pos = torch.zeros((n, most), dtype=torch.long, device=k.device)
    pos[who, row] = state["pos"]
    j = torch.arange(slot.shape[1], device=k.device)
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    s.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(n, heads, most * group, -1), v.permute(0, 2, 1, 3))
    o = (o.reshape(n, heads, most, group, D) / total).permute(0, 2, 1, 3, 4).reshape(n, most, -1, D)
    return o[who, row].bfloat16()


def _nearest_e4m3(x):
    """Rows of 64 in doubles to what their 8-bit form stands for: the nearest of the format's values
    (ties to the even code), scaled by the smallest power of two that holds the row."""
    code = torch.arange(127, device=x.device)
    value = torch.where(code < 8, (code % 8) / 8.0 * 2.0 ** -6, (1 + (code % 8) / 8.0) * 2.0 ** (code // 8 - 7.0)).double()
    big = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / E4M3_MAX))
    e = e + (big > E4M3_MAX * 2.0 ** e) - (big <= E4M3_MAX * 2.0 ** (e - 1)).double()
    e = torch.where(big > 0, e.clamp(-126, 126), torch.zeros_like(e))
    y = (x / 2.0 ** e)
    middle = (value[1:] + value[:-1]) / 2
    a = y.abs().contiguous()
    low = torch.bucketize(a, middle)                 # middles below a
    up = torch.bucketize(a, middle, right=True)      # and those equal to it
    i = torch.where(low % 2 == 0, low, up)
    return torch.sign(y) * value[i] * 2.0 ** e


def exact(c, seed):
    past, new = _lengths(c)
    pairs, slots = _pairs(c) if c["op"] != "write" else (0, 0)
    if 8 * D * c["q_heads"] * pairs > 4e12:
        return None
    k, v, q = _inputs(c, seed)
    if c["op"] == "write":
        k, v = _parts(c, k)[1], _parts(c, v)[1]
        if not c["e4m3"]:
            return k.double(), v.double()
        return tuple(torch.cat([_nearest_e4m3(b.double()) for b in x.split(4096)]) for x in (k, v))
    outs, r, t = [], 0, 0
    group = c["q_heads"] // c["heads"]
    for a, b in zip(past, new):
        out = torch.empty((b, c["q_heads"], D), dtype=torch.float64, device=k.device)
        for h in range(c["heads"]):
            kk, vv = k[r: r + a + b, h].double(), v[r: r + a + b, h].double()
            if c["e4m3"]:
                kk, vv = _nearest_e4m3(kk), _nearest_e4m3(vv)
            for b0 in range(0, b, 2048):
                nb = min(2048, b - b0)
                p = torch.arange(a + b0, a + b0 + nb, device=k.device)[:, None]
                j = torch.arange(a + b, device=k.device)[None]
                hide = j > p
                if c["window"]:
                    hide |= (j <= p - c["window"]) & (j >= c["sinks"])
                for g in range(group):
                    z = q[t + b0: t + b0 + nb, h * group + g].double() @ kk.T / 8.0
                    out[b0: b0 + nb, h * group + g] = torch.softmax(z.masked_fill(hide, float("-inf")), -1) @ vv
        outs.append(out)
        r, t = r + a + b, t + b
    return torch.cat(outs)
