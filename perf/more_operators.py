"""A tree of drafted tokens over the paged cache: rotary positions with several axes as tokens are
appended, the tree's attention, and the accepted tokens kept.

"rotary" cases append new tokens (k rotated, q rotated beside them), read them back and drop them
again. In "tree" cases a stream's last tokens are the nodes of a tree, and each node's query sees
what came before the tree, the node's ancestors and itself. "keep" cases append a tree's nodes on
every layer, keep some of them, read those back and drop them. Where `own` is false the operators
are computed in elementary torch operations on plain tensors (pages, tables, codes), where it is true
through the package's public calls."""

import functools

import torch

own = False

D = 64                      # head_dim
PAIRS = D // 2
E4M3_MAX = 448.0
MOST_NODES = 256            # of one stream's tree


def _case(name, op, **kw):
    c = dict(name=name, op=op, streams=1, past=0, new=1, ragged=False, heads=8, q_heads=32, page=256,
             e4m3=False)
    if op == "rotary":
        c.update(axes=3, distance=32, kind="text", start=0, base=10000.0)
    elif op == "tree":
        c.update(window=0, sinks=0)
    else:
        c.update(kept=1, layers=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token: the latency of a call
        _case("rotary_one", "rotary", past=776, start=776, heads=16, q_heads=16, axes=1),
        # a server's step: 64 users' next tokens, 8-bit pages, text behind images (three axes)
        _case("rotary_decode_e4m3", "rotary", streams=64, past=500, start=40000, page=64, e4m3=True),
        # prompts of images and text, far into a long conversation
        _case("rotary_prompt", "rotary", streams=4, past=100, new=5501, ragged=True, heads=16, q_heads=16,
              kind="video", start=900000, base=1000000.0),
        # eight frames of 5 + 37 x 37 tokens, two axes of half a row each, on 8-bit pages
        _case("rotary_frames_e4m3", "rotary", new=8 * 1374, heads=16, q_heads=16, axes=2, distance=16,
              kind="frames", e4m3=True),
        # one user's drafts: the latency of a call
        _case("tree_one", "tree", past=776, new=16, heads=16, q_heads=16),
        # a server's step: 16 users with trees of up to 32 drafts, small pages
        _case("tree_batch", "tree", streams=16, past=4001, new=32, ragged=True, page=16),
        # the same with 64 drafts on 8-bit pages
        _case("tree_batch_e4m3", "tree", streams=16, past=4001, new=64, ragged=True, page=64, e4m3=True),
        # one user with a long document and a large tree: the axis must be split to fill the card
        _case("tree_long", "tree", past=131071, new=64, q_heads=64),
        # trees of 7 drafts over long conversations under a sliding window with 4 sinks; groups of 3
        _case("tree_window", "tree", streams=48, past=20000, new=7, ragged=True, q_heads=24, page=64,
              window=4096, sinks=4),
        # one user's step in a one-layer model: 4 of 16 drafts accepted
        _case("keep_one", "keep", past=776, new=16, kept=4, heads=16, q_heads=16),
        # a server's step: 32 users, up to 5 of 32 drafts accepted, four layers
        _case("keep_batch", "keep", streams=32, past=500, new=32, kept=5, ragged=True, page=64, layers=4),
        # large trees on 8-bit pages, long accepted paths
        _case("keep_batch_e4m3", "keep", streams=64, past=300, new=200, kept=40, ragged=True, page=16, layers=2,
              e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "tree", "tree", "tree", "keep"])
    heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    c = dict(op=op, streams=1, past=0, new=1, ragged=rng.random() < 0.7, heads=heads, q_heads=heads * group,
             page=rng.choice([16, 32, 64, 128, 256]), e4m3=rng.random() < 0.5)
    if op == "rotary":
        planes = heads * (2 + group)
        most = max(1, min(11000, 500000 // planes))
        c["new"] = _log(rng, 1, most)
        c["streams"] = _log(rng, 1, max(1, min(64, most // c["new"])))
        c["past"] = rng.randrange(0, 800)
        c.update(axes=rng.choice([1, 2, 3, 3, 4]), distance=rng.choice([1, 2, 4, 8, 16, 32, 32]),
                 kind=rng.choice(["text", "video", "frames"]), start=rng.choice([0, _log(rng, 1, 4000000)]),
                 base=rng.choice([100.0, 10000.0, 1000000.0]))
        return c
    if op == "keep":
        c["new"] = _log(rng, 1, MOST_NODES)
        c["kept"] = rng.randrange(0, c["new"] + 1)
        c["layers"] = rng.choice([1, 2, 3, 4])
        c["streams"] = _log(rng, 1, max(1, min(64, 50000 // (c["new"] * heads * c["layers"]))))
        c["past"] = rng.randrange(0, 800)
        return c
    c["new"] = _log(rng, 1, MOST_NODES)
    c["streams"] = _log(rng, 1, max(1, min(48, 2000 // c["new"])))
    budget = 400000000 // (c["streams"] * c["new"] * c["q_heads"])
    keys = min(60000, 1500000 // (c["streams"] * heads), budget)
    c["past"] = 0 if keys < 20 else rng.choice([0] + [_log(rng, 10, keys)] * 7)
    c.update(window=0, sinks=0)
    if rng.random() < 0.4:
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


def _kept(c):
    """How many of each stream's drafts are accepted: ragged ones from none to all of them."""
    _, new = _lengths(c)
    n = c["streams"]
    return [min(m, (c["kept"] * ((i * 7) % n + 1)) // n if c["ragged"] and n > 1 else c["kept"])
            for i, m in enumerate(new)]


def _rotation(c):
    """Each pair's frequency and axis. Axes share a row's pairs in equal parts (the last takes the
    rest); "frames" start each axis' frequencies anew, as vision models do, the others run on."""
    per = PAIRS // c["axes"]
    axis = [min(i // per, c["axes"] - 1) for i in range(PAIRS)]
    if c["kind"] == "frames":
        count = [axis.count(a) for a in range(c["axes"])]
        freq = [c["base"] ** (-(i - axis.index(axis[i])) / count[axis[i]]) for i in range(PAIRS)]
    else:
        freq = [c["base"] ** (-i / PAIRS) for i in range(PAIRS)]
    return freq, axis


def _positions(c, seed):
    """[rows][axes] positions: text counts up on every axis at once; video tokens have a time, a row
    and a column of a 12 x 19 grid; frames are 5 tokens at 0 and 37 x 37 from 1 on."""
    g = torch.Generator().manual_seed(seed)
    parts = []
    for past, new in zip(*_lengths(c)):
        first = c["start"] + int(torch.randint(0, 1000, (1,), generator=g))
        i = torch.arange(new)
        if c["kind"] == "text":
            p = (first + i)[:, None].expand(new, c["axes"])
        elif c["kind"] == "video":
            p = first + torch.stack([i // 228, i % 228 // 19, i % 19, i], 1)[:, : c["axes"]]
        else:
            j = i % 1374 - 5
            cell = torch.stack([1 + j // 37, 1 + j % 37, i // 1374, i], 1)[:, : c["axes"]]
            p = torch.where(j[:, None] < 0, torch.zeros_like(cell), cell)
        parts.append(p)
    return torch.cat(parts).int().contiguous().cuda()


def _parents(c, seed):
    """Each node's parent among its stream's nodes (-1: none): wide trees with some long branches."""
    g = torch.Generator().manual_seed(seed)
    parts = []
    for new in _lengths(c)[1]:
        i = torch.arange(new)
        u, far = torch.rand(new, generator=g), torch.rand(new, generator=g) < 0.7
        parts.append(torch.where(far, (u * (i + 1)).long().clamp(max=i) - 1, i - 1))
    return torch.cat(parts).int().cuda()


def _choices(c, seed):
    """The accepted nodes of each stream, in order, and the tensor of all."""
    g = torch.Generator().manual_seed(seed)
    lists = [torch.randperm(m, generator=g)[:k].sort().values for m, k in zip(_lengths(c)[1], _kept(c))]
    return lists, torch.cat(lists).int().cuda()


def work(c):
    past, new = _lengths(c)
    row = D + 1 if c["e4m3"] else 2 * D
    n = sum(new)
    if c["op"] == "rotary":
        return {"bytes": n * (c["heads"] * 2 * (2 * D + row + row + 2 * D) + c["q_heads"] * 4 * D + 4 * c["axes"]),
                "flops": n * (c["heads"] + c["q_heads"]) * 3 * D}
    if c["op"] == "keep":
        k = sum(_kept(c))
        return {"bytes": c["layers"] * c["heads"] * 2 * (n * (2 * D + row) + k * (2 * row + row + 2 * D)), "flops": 0}
    # a wide tree's ancestors are few: a node's own pairs are counted as the whole tree's depth of 8
    pairs = slots = 0
    for a, b in zip(past, new):
        seen = a if not c["window"] else min(a, c["window"] + c["sinks"])
        pairs += b * (seen + min(b, 8))
        slots += seen + b
    return {"bytes": slots * c["heads"] * 2 * row + 2 * n * c["q_heads"] * D * 2 + 4 * n,
            "flops": 4 * D * c["q_heads"] * pairs}


def _inputs(c, seed):
    """k, v of every stream's past and new tokens ([layers * rows][heads][64], streams back to back) and
    the new tokens' q. Keys carry a few strong channels, rows differ in size, as trained ones do."""
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

    total = (sum(past) + sum(new)) * c.get("layers", 1)
    size = 1 + torch.rand((total, 1, 1), generator=g, device="cuda").bfloat16()
    k = rows(total, c["heads"], True)
    v = rows(total, c["heads"], False) * size
    q = rows(sum(new), c["q_heads"], False) * 1.5
    return k, v, q


def _parts(c, x):
    """The past and the new rows of x, each packed over the streams ([layers] first, if the case has
    them)."""
    past, new = _lengths(c)
    both = [t for i in range(len(past)) for t in (past[i], new[i])]
    layers = c.get("layers", 0)
    old, fresh = [], []
    for one in x.split(sum(both)):
        pieces = torch.split(one, both)
        old.append(torch.cat(pieces[0::2]))
        fresh.append(torch.cat(pieces[1::2]))
    return (torch.stack(old), torch.stack(fresh)) if layers else (old[0], fresh[0])


def prepare(c, seed):
    past, new = _lengths(c)
    n, page = c["streams"], c["page"]
    k, v, q = _inputs(c, seed)
    k_past, k_new = _parts(c, k)
    v_past, v_new = _parts(c, v)
    pages = [-(-(a + b) // page) for a, b in zip(past, new)]
    layers = c.get("layers", 1)
    state = {"case": c, "q": q, "k": k_new, "v": v_new}
    if c["op"] == "rotary":
        state["positions"] = _positions(c, seed)
    elif c["op"] == "tree":
        state["parents"] = _parents(c, seed)
    else:
        state["lists"], state["choices"] = _choices(c, seed)
    if own:
        # the program's cache: its streams opened, the past appended (and what left the window
        # evicted), and, where the call is the attention, the tree's nodes appended
        from paged_kv_cache_build_gb300 import PagedKVCache, Rotary
        cache = PagedKVCache(sum(pages) + n, page, c["heads"], layers=layers, max_streams=n, fp8=c["e4m3"])
        window, sinks = c.get("window", 0), c.get("sinks", 0)
        sids = [cache.open_token_stream(a + b, window=window, sinks=sinks) for a, b in zip(past, new)]
        held = [i for i in range(n) if past[i] > 0]
        if held:
            old = cache.token_batch([sids[i] for i in held], [past[i] for i in held])
            for layer in range(layers):
                rows = (k_past, v_past) if c["op"] != "keep" else (k_past[layer], v_past[layer])
                cache.append_tokens(old, *rows, layer=layer)
        if window:
            for s in sids:
                cache.evict_window(s)
        batch = cache.token_batch(sids, new)
        if c["op"] == "tree":
            cache.append_tokens(batch, k_new, v_new)
        elif c["op"] == "keep":
            state["accepted"] = cache.token_batch(sids, _kept(c))
        else:
            freq, axis = _rotation(c)
            state["rotary"] = Rotary(freq, axis, pair_distance=c["distance"])
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
        for layer in range(layers):
            if c["e4m3"]:
                store = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev),
                         torch.zeros(shape[:2], dtype=torch.int8, device=dev)]
            else:
                store = [torch.zeros(shape, dtype=torch.bfloat16, device=dev)]
            _store(store, past_slot, old[layer] if c["op"] == "keep" else old)
            if c["op"] == "tree":
                _store(store, new_slot, fresh)
            stores.append(store)
    state.update(stores=stores, new_slot=new_slot, table=table, who=who, past=t_past,
                 row=torch.arange(len(who), device=dev) - (torch.cumsum(t_new, 0) - t_new)[who], most=max(new))
    if c["op"] == "rotary":
        freq, axis = _rotation(c)
        state.update(freq=torch.tensor(freq, dtype=torch.float64, device=dev), axis=torch.tensor(axis, device=dev))
    if c["op"] == "keep":
        t_kept = torch.tensor(_kept(c), device=dev)
        state["kept_who"], _, state["kept_slot"] = slots(t_kept, t_past)
        state["first"] = torch.cumsum(t_new, 0) - t_new
    return state


@functools.lru_cache(None)
def _powers(dtype, device):
    return torch.tensor([2.0 ** i for i in range(-149, 128)], dtype=dtype, device=device)


def _power(e, like):
    """2^e, from a list: a power taken on the device may be an ulp off, which a value midway between
    two codes would show."""
    return _powers(like.dtype, like.device)[e.long() + 149]


def _quantise(x):
    """E4M3 codes (as their values) and the exponent of each row of 64."""
    big = x.abs().amax(-1)
    m, ex = torch.frexp(big)
    e = torch.where(big > 0, (ex - 9 + (m > E4M3_MAX / 512).int()).clamp(-126, 126), torch.zeros_like(ex))
    y = x * _power(-e[..., None], x)
    _, ey = torch.frexp(y)
    step = _power((ey - 1).clamp(min=-6) - 3, y)
    return (torch.round(y / step) * step).float(), e


def _store(store, slot, x):
    if len(store) == 1:
        store[0][slot] = x.bfloat16()
        return
    codes, e = _quantise(x if x.dtype == torch.float64 else x.float())
    store[0].view(torch.uint8)[slot] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    store[1][slot] = e.to(torch.int8)


def _load(store, slot):
    if len(store) == 1:
        return store[0][slot].float()
    codes = store[0].view(torch.uint8)[slot].view(torch.float8_e4m3fn)
    codes = codes.float()
    return codes * _power(store[1][slot][..., None], codes)


def _turn(x, cos, sin, distance):
    """Rows of 64 with the elements of each pair `distance` apart, turned by each pair's angle."""
    y = x.reshape(x.shape[:-1] + (D // (2 * distance), 2, distance))
    a, b = y[..., 0, :], y[..., 1, :]
    cos = cos.reshape(cos.shape[0], 1, D // (2 * distance), distance)
    sin = sin.reshape(cos.shape)
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -2).reshape(x.shape)


def run(state):
    c = state["case"]
    if own:
        cache, batch = state["cache"], state["batch"]
        if c["op"] == "rotary":
            q = cache.append_tokens_rotary(batch, state["k"], state["v"], state["positions"], state["rotary"],
                                           q=state["q"])
            k, v = cache.read_tokens(batch)
            cache.drop_tokens(batch)
            return q, k, v
        if c["op"] == "tree":
            return cache.attend_tree(batch, state["q"], state["parents"], window=c["window"], sinks=c["sinks"])
        for layer in range(c["layers"]):
            cache.append_tokens(batch, state["k"][layer], state["v"][layer], layer=layer)
        cache.keep_tokens(batch, state["choices"], state["accepted"])
        out = [cache.read_tokens(state["accepted"], layer=layer) for layer in range(c["layers"])]
        cache.drop_tokens(state["accepted"])
        return out
    if c["op"] == "rotary":
        angle = state["positions"][:, state["axis"]].double() * state["freq"]
        cos, sin = torch.cos(angle), torch.sin(angle)
        q = _turn(state["q"].float(), cos.float(), sin.float(), c["distance"]).bfloat16()
        if c["e4m3"]:                            # a code's border is met in 64 bits
            k = _turn(state["k"].double(), cos, sin, c["distance"])
        else:
            k = _turn(state["k"].float(), cos.float(), sin.float(), c["distance"])
        (ks, vs), slot = state["stores"], state["new_slot"]
        _store(ks, slot, k)
        _store(vs, slot, state["v"])
        return q, _load(ks, slot).bfloat16(), _load(vs, slot).bfloat16()
    if c["op"] == "keep":
        layers, slot = c["layers"], state["new_slot"]
        source = slot[state["first"][state["kept_who"]] + state["choices"].long()]
        outs = []
        for layer in range(layers):
            pair = []
            for rows, store in ((state["k"], state["stores"][layer]), (state["v"], state["stores"][layers + layer])):
                _store(store, slot, rows[layer])
                for part in store:
                    bits = part.view(torch.uint8) if part.dtype == torch.float8_e4m3fn else part
                    bits[state["kept_slot"]] = bits[source]
                pair.append(_load(store, state["kept_slot"]).bfloat16())
            outs.append(tuple(pair))
        return outs
    ks, vs = state["stores"]
    n, page, heads, group = c["streams"], c["page"], c["heads"], c["q_heads"] // c["heads"]
    dev = state["q"].device
    slot = (state["table"][:, :, None] * page + torch.arange(page, device=dev)).reshape(n, -1)
    k, v = _load(ks, slot), _load(vs, slot)                               # [n][keys][heads][64]
    most, who, row, past = state["most"], state["who"], state["row"], state["past"]
    q = torch.zeros((n, most, heads, group, D), device=dev)
    q[who, row] = state["q"].float().reshape(-1, heads, group, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, heads, most * group, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(D ** -0.5).reshape(n, heads, most, group, -1)
    # which nodes lead to which: the parents' steps, doubled until they are longer than any path
    parent = torch.full((n, most), -1, dtype=torch.long, device=dev)
    parent[who, row] = state["parents"].long()
    at = torch.arange(most, device=dev)
    lead = ((parent[:, :, None] == at) | (at[:, None] == at)).float()
    for _ in range(max(1, most - 1).bit_length()):
        lead = (torch.matmul(lead, lead) > 0).float()
    depth = lead.sum(-1).long() - 1                                       # [n][nodes]
    j = torch.arange(slot.shape[1], device=dev)
    node = (j - past[:, None])                                            # [n][keys]: the key's node
    in_tree = (node >= 0) & (node < most)
    node = node.clamp(0, most - 1)
    where = torch.where(in_tree, past[:, None] + depth.gather(1, node), j.expand(n, -1))
    seen = torch.where(in_tree[:, None], lead.gather(2, node[:, None].expand(n, most, -1)) > 0,
                       (j < past[:, None])[:, None])
    if c["window"]:
        p = past[:, None, None] + depth[:, :, None]
        seen = seen & ((where[:, None] > p - c["window"]) | (where[:, None] < c["sinks"]))
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
    value = torch.where(code < 8, (code % 8).double() / 8 * 2.0 ** -6,
                        (1 + (code % 8).double() / 8) * _power(code // 8 - 7, x))
    big = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / E4M3_MAX)).long().clamp(-148, 126)
    e = e + (big > E4M3_MAX * _power(e, x)).long() - (big <= E4M3_MAX * _power(e - 1, x)).long()
    e = torch.where(big > 0, e.clamp(-126, 126), torch.zeros_like(e))
    y = x / _power(e, x)
    middle = (value[1:] + value[:-1]) / 2
    a = y.abs().contiguous()
    low = torch.bucketize(a, middle)                 # middles below a
    up = torch.bucketize(a, middle, right=True)      # and those equal to it
    i = torch.where(low % 2 == 0, low, up)
    return torch.sign(y) * value[i] * _power(e, x)


def _stored(c, x):
    return torch.cat([_nearest_e4m3(b) for b in x.split(2048)]) if c["e4m3"] and len(x) else x


def exact(c, seed):
    past, new = _lengths(c)
    if c["op"] == "tree" and 8 * D * c["q_heads"] * sum(b * (a + b) for a, b in zip(past, new)) > 4e12:
        return None
    k, v, q = _inputs(c, seed)
    k_new, v_new = _parts(c, k)[1], _parts(c, v)[1]
    if c["op"] == "rotary":
        # a pair as a complex number times e^(i angle)
        freq, axis = _rotation(c)
        position = _positions(c, seed).double()
        d = c["distance"]
        first = [(i // d) * 2 * d + i % d for i in range(PAIRS)]
        turn = torch.stack([torch.polar(torch.ones_like(position[:, 0]), freq[i] * position[:, axis[i]])
                            for i in range(PAIRS)], 1)[:, None]
        out = []
        for x in (q, k_new):
            x = x.double()
            z = torch.complex(x[..., first], x[..., [a + d for a in first]]) * turn
            y = torch.empty_like(x)
            y[..., first], y[..., [a + d for a in first]] = z.real, z.imag
            out.append(y)
        return out[0], _stored(c, out[1]), _stored(c, v_new.double())
    if c["op"] == "keep":
        lists, _ = _choices(c, seed)
        at, rows = 0, []
        for m, chosen in zip(new, lists):
            rows += [at + int(i) for i in chosen]
            at += m
        rows = torch.tensor(rows, dtype=torch.long, device=k.device)
        return [tuple(_stored(c, x[layer][rows].double()) for x in (k_new, v_new)) for layer in range(c["layers"])]
    parents = _parents(c, seed).tolist()
    outs, r, t = [], 0, 0
    group = c["q_heads"] // c["heads"]
    for a, b in zip(past, new):
        # each node's path, walked from node to node
        hide = torch.zeros((b, a + b), dtype=torch.bool)
        hide[:, a:] = True
        deep = []
        for i in range(b):
            path, x = [i], parents[t + i]
            while x >= 0:
                path.append(x)
                x = parents[t + x]
            deep.append(len(path) - 1)
            for x in path:
                far = deep[i] - deep[x]
                if not c["window"] or far < c["window"] or a + deep[x] < c["sinks"]:
                    hide[i, a + x] = False
            if c["window"]:
                lo = max(0, a + deep[i] - c["window"] + 1)
                hide[i, min(c["sinks"], lo, a): min(lo, a)] = True
        hide = hide.to(k.device)
        out = torch.empty((b, c["q_heads"], D), dtype=torch.float64, device=k.device)
        for h in range(c["heads"]):
            kk, vv = _stored(c, k[r: r + a + b, h].double()), _stored(c, v[r: r + a + b, h].double())
            for g in range(group):
                z = q[t: t + b, h * group + g].double() @ kk.T / 8.0
                out[:, h * group + g] = torch.softmax(z.masked_fill(hide, float("-inf")), -1) @ vv
        outs.append(out)
        r, t = r + a + b, t + b
    return torch.cat(outs)
