"""More operators of the paged key/value cache, as they are measured: attention of requests that
share a long prefix (op "shared"), the attention weight that every cached key has got (op
"weights"), and eviction of the keys that got least (op "evict").

run() computes the plain form of an operator in torch, or, with `own` set, calls the library.
Every length of a case follows from the case itself; the values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def _weights(name, **kw):
    c = dict(name=name, op="weights", B=1, H=8, Hkv=8, d=64, P=16, dtype="bf16", new_lo=1, new_hi=1,
             cached_lo=0, cached_hi=0, clip_k=0, key_term=False, window=0, sinks=0, accumulate=True)
    c.update(kw)
    return c


def _evict(name, **kw):
    c = dict(name=name, op="evict", B=1, Hkv=8, d=64, P=16, dtype="bf16", len_lo=0, len_hi=0, budget=0,
             limit=0, sinks=4, recent=64)
    c.update(kw)
    return c


def _shared(name, **kw):
    c = dict(name=name, op="shared", groups=1, per_group=1, H=8, Hkv=8, d=64, P=16, dtype="bf16", new=1,
             prefix_lo=0, prefix_hi=0, own_lo=1, own_hi=1, clip_k=0, key_term=False, value_term=False)
    c.update(kw)
    return c


def listed():
    return [
        # the weights of one decoding step of the Transformer-big decoder, caches of 1K-2K
        _weights("weights_decode", B=32, H=16, Hkv=16, d=64, cached_lo=1023, cached_hi=2047, clip_k=16,
                 key_term=True),
        # one decoding step of 64 requests with long caches, eight query heads to a key head
        _weights("weights_grouped", B=64, H=16, Hkv=2, d=128, P=32, cached_lo=2047, cached_hi=16383),
        # the last 32 tokens of each prompt observe all of it, before the cache is cut down
        _weights("weights_observe", B=8, H=16, Hkv=4, d=128, new_lo=32, new_hi=32, cached_lo=4001,
                 cached_hi=32001, accumulate=False),
        # four whole prompts of 4096 tokens with the key-relative term
        _weights("weights_prompt", B=4, H=16, Hkv=16, d=128, new_lo=4096, new_hi=4096, clip_k=64,
                 key_term=True, accumulate=False),
        # single precision, as a model is checked before it is cast: short odd chunks
        _weights("weights_f32", B=3, H=8, Hkv=8, d=64, P=8, dtype="f32", new_lo=61, new_hi=127,
                 cached_lo=100, cached_hi=700, clip_k=16, key_term=True),
        # a handful of chats that have passed their limit
        _evict("evict_small", B=4, Hkv=4, d=64, len_lo=577, len_hi=700, budget=512, limit=576),
        # a batch whose caches are cut back every 256 tokens
        _evict("evict_batch", B=64, Hkv=4, d=128, len_lo=2000, len_hi=2304, budget=2048, limit=2048,
               recent=256),
        # one long document cut down to a quarter after its prompt
        _evict("evict_long", B=1, Hkv=4, d=128, P=64, len_lo=131071, len_hi=131071, budget=32768,
               limit=32768, sinks=16, recent=1024),
        # a decoding step of 32 chats behind one instruction text, both relative terms
        _shared("shared_decode", per_group=32, H=16, Hkv=16, d=64, prefix_lo=2048, prefix_hi=2048,
                own_lo=30, own_hi=500, clip_k=16, key_term=True, value_term=True),
        # a decoding step of 64 chats behind a long one, four query heads to a key head
        _shared("shared_grouped", per_group=64, H=16, Hkv=4, d=128, prefix_lo=8192, prefix_hi=8192,
                own_lo=100, own_hi=1000),
        # four proposed tokens each for eight groups of 16 requests (few-shot headers)
        _shared("shared_groups", groups=8, per_group=16, H=16, Hkv=4, d=128, P=32, new=4, prefix_lo=1000,
                prefix_hi=8000, own_lo=20, own_hi=700),
        # 256 samples that continue one long document
        _shared("shared_long", per_group=256, H=16, Hkv=2, d=128, P=64, prefix_lo=32768,
                prefix_hi=32768, own_lo=1, own_hi=300),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _fits(c):
    """No more work than the largest listed case, and a cache and scores that memory holds."""
    w = work(c)
    f32 = c["dtype"] == "f32"
    if w["bytes"] > 5e8 or w["flops"] > (4e9 if f32 else 1.3e11):
        return False
    if c["op"] == "evict":
        return sum(_evict_lens(c)) * c["Hkv"] * c["d"] * (4 if f32 else 2) * 2 < 1.5e9
    if c["H"] > 64:
        return False
    if c["op"] == "weights":
        cached, new = _lens(c)
        return (max(a * (a + b) for a, b in zip(new, cached)) * c["H"] < 4e8 and
                sum(a + b for a, b in zip(new, cached)) * c["Hkv"] * c["d"] < 8e8)
    prefix, tail = _shared_lens(c)
    n = sum(prefix) * c["per_group"] + sum(map(sum, tail))  # the plain form's keys
    return n * c["Hkv"] * c["d"] < 8e9 and len(prefix) * c["per_group"] <= 512


def draw(rng):
    while True:
        op = rng.choice(["weights", "evict", "shared"])
        f32 = rng.random() < 0.15
        dt = "f32" if f32 else "bf16"
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        P = rng.choice([8, 16, 32, 64, 128])
        d = rng.choice([64, 128, 128, 80] if f32 else [64, 128])
        if op == "evict":
            budget = _log(rng, 64, 65536)
            limit = budget + (0 if rng.random() < 0.5 else _log(rng, 1, budget))
            hi = limit + _log(rng, 1, 3 * budget)
            c = _evict("", B=_log(rng, 1, 256), Hkv=Hkv, d=d, P=P, dtype=dt, budget=budget, limit=limit,
                       len_lo=int(hi * rng.uniform(0.3, 1)), len_hi=hi,
                       sinks=min(rng.choice([0, 1, 4, 16, 130]), budget // 4), recent=_log(rng, 1, budget // 2))
        else:
            g = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
            key_term = rng.random() < 0.5
            clip_k = rng.choice([1, 4, 16, 64]) if key_term else 0
            if op == "weights":
                kind = rng.choice(["decode", "decode", "observe", "chunk", "prompt"])
                cached = 0 if kind == "prompt" else _log(rng, 1, 2048 if f32 else 65536)
                new = 1 if kind == "decode" else _log(rng, 2, 64 if kind == "observe" else 127 if f32 else 4096)
                windowed = rng.random() < 0.25
                c = _weights("", B=_log(rng, 1, 4 if f32 else 128), H=Hkv * g, Hkv=Hkv, d=d, P=P, dtype=dt,
                             new_lo=max(1, int(new * rng.uniform(0.3, 1))), new_hi=new,
                             cached_lo=int(cached * rng.uniform(0, 1)), cached_hi=cached, clip_k=clip_k,
                             key_term=key_term, window=_log(rng, 16, 8192) if windowed else 0,
                             sinks=rng.choice([0, 1, 4, 16, 130]) if windowed else 0,
                             accumulate=kind in ("decode", "chunk"))
            else:
                prefix = _log(rng, 100, 2048 if f32 else 65536)
                tail = _log(rng, 1, 256 if f32 else 2048)
                value_term = rng.random() < 0.3
                c = _shared("", groups=_log(rng, 1, 16), per_group=_log(rng, 1, 8 if f32 else 256), H=Hkv * g,
                            Hkv=Hkv, d=d, P=P, dtype=dt, new=rng.choice([1, 1, 1, 2, 4, 7]),
                            prefix_lo=int(prefix * rng.uniform(0.2, 1)), prefix_hi=prefix,
                            own_lo=max(1, int(tail * rng.uniform(0, 1))), own_hi=tail,
                            clip_k=clip_k or (16 if value_term else 0), key_term=key_term,
                            value_term=value_term)
        del c["name"]
        if _fits(c):
            return c


# ------------------------------------------------------------------------------ lengths
def _spread(i, step, lo, hi):
    """The i-th of lengths spread evenly over lo .. hi, odd and even ones alike."""
    return lo + int(((i + 1) * step % 1.0) * (hi - lo + 1))


def _lens(c):
    """Cached and new tokens of every request."""
    cached = [_spread(i, 0.7548776662466927, c["cached_lo"], c["cached_hi"]) for i in range(c["B"])]
    new = [_spread(i, 0.6180339887498949, c["new_lo"], c["new_hi"]) for i in range(c["B"])]
    return cached, new


def _evict_lens(c):
    return [_spread(i, 0.7548776662466927, c["len_lo"], c["len_hi"]) for i in range(c["B"])]


def _shared_lens(c):
    """Shared keys of every group (whole pages), and the own keys of its requests behind them, the
    new ones among them."""
    n = c["per_group"]
    prefix = [_spread(i, 0.7548776662466927, c["prefix_lo"], c["prefix_hi"]) // c["P"] * c["P"]
              for i in range(c["groups"])]
    tail = [[c["new"] - 1 + _spread(i * n + j, 0.6180339887498949, c["own_lo"], c["own_hi"])
             for j in range(n)] for i in range(c["groups"])]
    return prefix, tail


def _pages(n, P):
    return (n + P - 1) // P


def _visible(c, cached, new):
    """(query, key) pairs that a request's rows see, and the rows of the cache any of them sees."""
    w, s = c["window"], c["sinks"]
    pos = np.arange(cached, cached + new, dtype=np.int64)
    if not w:
        return int((pos + 1).sum()), cached + new
    behind = np.maximum(pos + 1 - w, 0)  # keys that the window leaves behind
    pairs = int((np.minimum(pos + 1, w) + np.minimum(behind, s)).sum())
    first = max(0, cached + 1 - w)
    return pairs, cached + new - first + min(s, first)


def work(c):
    es, P, d, Hkv = (2 if c["dtype"] == "bf16" else 4), c["P"], c["d"], c["Hkv"]
    if c["op"] == "evict":
        by = 4 * (2 * c["B"] + 2)
        for n in _evict_lens(c):
            if n > c["limit"]:
                moved = c["budget"] - c["sinks"]
                by += Hkv * (4 * n + moved * (4 * d * es + 4)) + 4 * _pages(n, P)
        return {"bytes": by, "flops": 0}
    H, k = c["H"], c["clip_k"]
    if c["op"] == "weights":
        cached, new = _lens(c)
        T = sum(new)
        by, fl = T * H * (d * es + 4) + 4 * (2 * c["B"] + 1), 0
        for a, n in zip(cached, new):
            pairs, rows = _visible(c, a, n)
            read = 4 * (rows - n) if c["accumulate"] else 0
            by += Hkv * (rows * (d * es + 4) + read) + 4 * _pages(rows, P)
            fl += 2 * d * H * pairs
        if c["key_term"]:
            by, fl = by + Hkv * (k + 1) * d * es, fl + 2 * d * T * H * (k + 1)
        return {"bytes": by, "flops": fl}
    prefix, tail = _shared_lens(c)
    B, n = c["groups"] * c["per_group"], c["new"]
    terms = int(c["key_term"]) + int(c["value_term"])
    by = 2 * B * n * H * d * es + 4 * (2 * B + 2 * c["groups"] + 2) + terms * Hkv * (k + 1) * d * es
    fl = 2 * d * B * n * H * (k + 1) * terms
    for L, own_keys in zip(prefix, tail):
        by += 2 * L * Hkv * d * es + 4 * _pages(L, P)
        for t in own_keys:
            by += 2 * t * Hkv * d * es + 4 * _pages(t, P)
            fl += 4 * d * H * sum(L + t - i for i in range(n))
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------------------ inputs
def _filled_table(lens, M, P, order, i32):
    """Block table whose rows hold the pages of `lens` tokens each, taken from `order`."""
    table = torch.full((len(lens), M), -1, **i32)
    filled = torch.arange(M, device=order.device)[None, :] < torch.tensor([_pages(x, P) for x in lens],
                                                                          device=order.device)[:, None]
    table[filled] = order[:sum(_pages(x, P) for x in lens)]
    return table


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device=dev)
    st = {"case": dict(c)}
    P, Hkv, d = c["P"], c["Hkv"], c["d"]

    def normal(*shape, std=1.0):
        x = torch.empty(shape, dtype=_DT[c["dtype"]], device=dev)
        return x.normal_(0.0, std, generator=g)

    def weight(*shape):  # what keys have got so far: a few much, most of them little
        x = torch.empty(shape, dtype=torch.float32, device=dev)
        return x.normal_(-1.0, 1.5, generator=g).exp_()

    if c["op"] == "evict":
        lens = _evict_lens(c)
        M = _pages(max(lens), P)
        used = sum(_pages(x, P) for x in lens)
        order = torch.randperm(used + 16, generator=g, device=dev).to(torch.int32)
        st["block_table"] = _filled_table(lens, M, P, order, i32)
        st["kv_len"] = torch.tensor(lens, **i32)
        st["lens"] = lens
        st["k_pages"], st["v_pages"] = normal(used + 16, Hkv, P, d), normal(used + 16, Hkv, P, d)
        st["mass"] = weight(used + 16, Hkv, P)
        st["free_pages"] = order
        st["free_head"] = torch.tensor([used], **i32)
        if own:
            import relative_position_representations_gb300 as rp
            st["kv_len_out"] = torch.empty(c["B"], **i32)
            st["free_head_out"] = torch.empty(1, **i32)
            st["workspace"] = torch.empty(rp.relattn_paged_evict_workspace_size(c["B"], Hkv, M * P),
                                          dtype=torch.uint8, device=dev)
        return st

    H, k = c["H"], c["clip_k"]
    if c["op"] == "weights":
        cached, new = _lens(c)
        total = [a + b for a, b in zip(cached, new)]
        M, n_pages = _pages(max(total), P), sum(_pages(t, P) for t in total) + 16
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        st["block_table"] = _filled_table(total, M, P, order, i32)
    else:
        prefix, tail = _shared_lens(c)
        n = c["per_group"]
        total = [L + t for L, ts in zip(prefix, tail) for t in ts]
        new = [c["new"]] * len(total)
        cached = [t - c["new"] for t in total]
        # the pages of the prefixes, then every request's own
        lens = prefix + [t for ts in tail for t in ts]
        M = _pages(max(prefix), P) + _pages(max(map(max, tail)), P)
        n_pages = sum(_pages(x, P) for x in lens) + 16
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        parts = _filled_table(lens, M, P, order, i32)
        head = parts[:len(prefix)].repeat_interleave(n, 0)
        tails = parts[len(prefix):]
        have = torch.tensor([L // P for L in prefix], device=dev).repeat_interleave(n)[:, None]
        j = torch.arange(M, device=dev)[None, :]
        st["block_table"] = torch.where(j < have, head, tails.gather(1, (j - have).clamp(min=0)))
        st["group_start"] = torch.arange(0, len(total) + 1, n, **i32)
        st["prefix_len"] = torch.tensor(prefix, **i32)
    T = sum(new)
    # the queries come out of one projection with the new keys and values
    st["q"] = normal(T, H + 2 * Hkv, d)[:, :H]
    st["k_pages"] = normal(n_pages, Hkv, P, d)
    st["aK"] = normal(Hkv, 2 * k + 1, d, std=0.02) if c["key_term"] else None
    st["kv_len"] = torch.tensor(total, **i32)
    st["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    st["cached"], st["new"] = cached, new
    st["scale"] = d ** -0.5
    if c["op"] == "weights":
        st["mass"] = weight(n_pages, Hkv, P)
        # the forward pass of the step has left each row's log-sum-exp
        st["lse"] = torch.empty((T, H), dtype=torch.float32, device=dev)
        for b, rows, h0, h1, s, j in _scores(st):
            st["lse"][rows, h0:h1] = torch.logsumexp(s, 3).permute(2, 0, 1).reshape(-1, h1 - h0)
        if own:
            import relative_position_representations_gb300 as rp
            st["workspace"] = torch.empty(rp.relattn_paged_weights_workspace_size(T, H), dtype=torch.uint8,
                                          device=dev)
        return st
    st["v_pages"] = normal(n_pages, Hkv, P, d)
    st["aV"] = normal(Hkv, 2 * k + 1, d, std=0.02) if c["value_term"] else None
    st["out"] = torch.empty((T, H, d), dtype=_DT[c["dtype"]], device=dev)
    if own:
        import relative_position_representations_gb300 as rp
        st["workspace"] = torch.empty(rp.relattn_paged_shared_workspace_size(T, H, Hkv, d),
                                      dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------------------ plain forms
def _keys_of(c, cached, new, dev):
    """The cache rows that some row of a request sees: the first tokens, then the window."""
    total, window = cached + new, c.get("window", 0)
    first = max(0, cached + 1 - window) if window else 0
    return torch.cat([torch.arange(min(c.get("sinks", 0), first), device=dev),
                      torch.arange(first, total, device=dev)])


def _scores(st):
    """Masked scores in single precision, a block of rows and key heads at a time: (request, rows
    of the block, first and last query head, scores [key heads, group, rows, keys], keys)."""
    c = st["case"]
    H, Hkv, d, P, k = c["H"], c["Hkv"], c["d"], c["P"], c["clip_k"]
    gsz, window, at = H // Hkv, c.get("window", 0), 0
    aK = None if st["aK"] is None else st["aK"][:, :k + 1].float()
    dev = st["q"].device
    for b in range(len(st["new"])):
        n, cached = st["new"][b], st["cached"][b]
        j = _keys_of(c, cached, n, dev)
        page, row = st["block_table"][b, j // P].long(), j % P
        hs = max(1, min(Hkv, int(4e8 / (n * gsz * len(j)))))   # key heads at a time
        for h in range(0, Hkv, hs):
            h1 = min(Hkv, h + hs)
            K = st["k_pages"][page, h:h1, row].float().transpose(0, 1)       # [heads, keys, d]
            q = st["q"][at:at + n, h * gsz:h1 * gsz].float().reshape(n, h1 - h, gsz, d).permute(1, 2, 0, 3)
            q = q.reshape(h1 - h, gsz * n, d)
            pos = (cached + torch.arange(n, device=dev)).repeat(gsz)
            off = j[None, :] - pos[:, None]                                  # j - i
            s = q @ K.transpose(1, 2)
            if aK is not None:
                lab = off.clamp(-k, 0) + k
                s += torch.gather(q @ aK[h:h1].transpose(1, 2), 2, lab.expand(h1 - h, -1, -1))
            s *= st["scale"]
            hide = off > 0
            if window:
                hide = hide | ((off <= -window) & (j >= c["sinks"])[None, :])
            s.masked_fill_(hide, float("-inf"))
            yield b, slice(at, at + n), h * gsz, h1 * gsz, s.reshape(h1 - h, gsz, n, len(j)), j
        at += n


def _plain_weights(st):
    c = st["case"]
    P, gsz = c["P"], c["H"] // c["Hkv"]
    for b, rows, h0, h1, s, j in _scores(st):
        lse = st["lse"][rows, h0:h1].reshape(-1, s.shape[0], gsz).permute(1, 2, 0)[..., None]
        got = (s - lse).exp_().sum((1, 2))                                   # [heads, keys]
        page, row = st["block_table"][b, j // P].long(), j % P
        heads = slice(h0 // gsz, h1 // gsz)
        if c["accumulate"]:
            old = st["mass"][page, heads, row].t()
            got = got + torch.where(j < st["cached"][b], old, 0.0)
        st["mass"][page, heads, row] = got.t()
    return st["mass"]


def _plain_evict(st):
    c = st["case"]
    P, Hkv, budget, sinks, recent = c["P"], c["Hkv"], c["budget"], c["sinks"], c["recent"]
    table, mass = st["block_table"], st["mass"]
    dev = table.device
    gone, new_len = [], []
    h = torch.arange(Hkv, device=dev)[:, None]
    for b, n in enumerate(st["lens"]):
        new_len.append(min(n, budget) if n > c["limit"] else n)
        if n <= c["limit"]:
            continue
        gone.append(table[b, _pages(budget, P):_pages(n, P)])
        j = torch.arange(n, device=dev)
        got = mass[table[b, j // P].long(), :, j % P].t()                    # [Hkv, n]
        rest = torch.sort(got[:, sinks:n - recent], dim=1, descending=True, stable=True).indices
        rest = torch.sort(rest[:, :budget - sinks - recent], 1).values + sinks
        kept = torch.cat([rest, torch.arange(n - recent, n, device=dev).expand(Hkv, -1)], 1)
        to = torch.arange(sinks, budget, device=dev)
        src = (table[b, kept // P].long(), h, kept % P)
        dst = (table[b, to // P].long()[None, :], h, to[None, :] % P)
        for x in (st["k_pages"], st["v_pages"], mass):
            x[dst] = x[src]
    head = st["free_head"] - sum(x.numel() for x in gone)
    if gone:
        gone = torch.cat(gone)
        st["free_pages"][head.long() + torch.arange(gone.numel(), device=dev)] = gone
    return [torch.tensor(new_len, dtype=torch.int32, device=dev), head.to(torch.int32), st["free_pages"],
            st["k_pages"], st["v_pages"], mass]


def _plain_shared(st):
    c = st["case"]
    H, Hkv, d, P, k = c["H"], c["Hkv"], c["d"], c["P"], c["clip_k"]
    gsz, out = H // Hkv, st["out"]
    aV = None if st["aV"] is None else st["aV"][:, :k + 1].float()
    for b, rows, h0, h1, s, j in _scores(st):
        heads, n = slice(h0 // gsz, h1 // gsz), s.shape[2]
        page, row = st["block_table"][b, j // P].long(), j % P
        V = st["v_pages"][page, heads, row].float().transpose(0, 1)
        p = (s - s.amax(3, keepdim=True)).exp_().reshape(s.shape[0], gsz * n, -1)
        z = p @ V
        if aV is not None:
            pos = (st["cached"][b] + torch.arange(n, device=out.device)).repeat(gsz)
            lab = (j[None, :] - pos[:, None]).clamp(-k, 0) + k
            bins = torch.zeros((s.shape[0], gsz * n, k + 1), device=out.device)
            z += bins.scatter_add_(2, lab.expand(s.shape[0], -1, -1), p) @ aV[heads]
        z /= p.sum(2, keepdim=True)
        z = z.reshape(-1, gsz, n, d).permute(2, 0, 1, 3).reshape(n, h1 - h0, d)
        out[rows, h0:h1] = z.to(out.dtype)
    return out


def run(state):
    st = state
    c = st["case"]
    op = c["op"]
    if not own:
        return {"weights": _plain_weights, "evict": _plain_evict, "shared": _plain_shared}[op](st)
    import relative_position_representations_gb300 as rp
    if op == "weights":
        return rp.relattn_paged_weights(st["q"], st["k_pages"], st["block_table"], st["q_start"], st["kv_len"],
                                        st["lse"], st["mass"], aK=st["aK"], clip_k=c["clip_k"],
                                        window=c["window"], sinks=c["sinks"], scale=st["scale"],
                                        accumulate=c["accumulate"], max_new=max(st["new"]),
                                        workspace=st["workspace"])
    if op == "evict":
        kv_len, head = rp.relattn_paged_evict(
            st["kv_len"], st["block_table"], st["k_pages"], st["v_pages"], st["mass"], c["budget"],
            limit=c["limit"], sinks=c["sinks"], recent=c["recent"], free_pages=st["free_pages"],
            free_head=st["free_head"], kv_len_out=st["kv_len_out"], free_head_out=st["free_head_out"],
            workspace=st["workspace"])
        return [kv_len, head, st["free_pages"], st["k_pages"], st["v_pages"], st["mass"]]
    return rp.relattn_paged_shared_fwd(st["q"], st["k_pages"], st["v_pages"], st["block_table"], st["q_start"],
                                       st["kv_len"], st["group_start"], st["prefix_len"], aK=st["aK"],
                                       aV=st["aV"], clip_k=c["clip_k"], scale=st["scale"], max_new=c["new"],
                                       out=st["out"], workspace=st["workspace"])


# ------------------------------------------------------------------------------ exact values
def _exact_evict(c, st):
    """Key by key, as lists: sorted by weight and place, the kept ones copied to the front."""
    P, Hkv = c["P"], c["Hkv"]
    table = st["block_table"].tolist()
    free, head = st["free_pages"].tolist(), int(st["free_head"])
    mass = st["mass"].double().cpu().numpy()
    lens, gone = [], []
    moves = [[], [], [], [], []]   # head, page and row from, page and row to
    for b, n in enumerate(_evict_lens(c)):
        if n <= c["limit"]:
            lens.append(n)
            continue
        lens.append(c["budget"])
        row = np.array(table[b])
        gone += table[b][-(-c["budget"] // P):-(-n // P)]
        j = np.arange(n)
        always = (j < c["sinks"]) | (j >= n - c["recent"])
        for h in range(Hkv):
            a = mass[row[j // P], h, j % P]
            order = np.lexsort((j, -a, ~always))     # the ones kept anyway first, then by weight, then place
            kept = np.sort(order[:c["budget"]])
            to = np.arange(c["budget"])
            for m, x in zip(moves, (np.full(len(to), h), row[kept // P], kept % P, row[to // P], to % P)):
                m.append(x)
    head -= len(gone)
    free[head:head + len(gone)] = gone
    res = [torch.tensor(x, dtype=torch.int32) for x in (lens, [head], free)]
    if moves[0]:
        h, p0, r0, p1, r1 = (torch.from_numpy(np.concatenate(m)).to(st["mass"].device) for m in moves)
    for x in (st["k_pages"], st["v_pages"], st["mass"]):
        x = x.clone()
        if moves[0]:
            x[p1, h, r1] = x[p0, h, r0]
        res.append(x.double() if x.numel() < 4e8 else x)
    return res


def exact(case, seed):
    """The definitions in 64 bits: the eviction as sorted lists, attention and its weights head by
    head and row block by row block."""
    c = case
    st = prepare(c, seed)
    P, Hkv, d = c["P"], c["Hkv"], c["d"]
    if c["op"] == "evict":
        return _exact_evict(c, st)
    H, k = c["H"], c["clip_k"]
    gsz, T = H // Hkv, sum(st["new"])
    window, sinks = c.get("window", 0), c.get("sinks", 0)
    dev = st["q"].device
    weights = c["op"] == "weights"
    res = st["mass"].double() if weights else torch.zeros((T, H, d), dtype=torch.float64, device=dev)
    at = 0
    for b, (n, cached) in enumerate(zip(st["new"], st["cached"])):
        total = cached + n
        idx = st["block_table"][b, :-(-total // P)].long()
        for h in range(Hkv):
            K = st["k_pages"][idx, h].reshape(-1, d)[:total].double()
            V = None if weights else st["v_pages"][idx, h].reshape(-1, d)[:total].double()
            got = torch.zeros(total, dtype=torch.float64, device=dev)
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                i = torch.arange(cached + r0, cached + r1, device=dev)
                dist = i[:, None] - torch.arange(total, device=dev)[None, :]
                seen = dist >= 0
                if window:
                    seen &= (dist < window) | (torch.arange(total, device=dev) < sinks)[None, :]
                r = k - dist.clamp(0, k)                 # table row of offset -dist, clipped
                for q_head in range(h * gsz, (h + 1) * gsz):
                    q = st["q"][at + r0:at + r1, q_head].double()
                    e = q @ K.T
                    if st["aK"] is not None:
                        e = e + (q @ st["aK"][h].double().T).gather(1, r)
                    e = torch.where(seen, e * st["scale"], -math.inf)
                    if weights:
                        got += torch.exp(e - st["lse"][at + r0:at + r1, q_head].double()[:, None]).sum(0)
                        continue
                    a = torch.softmax(e, 1)
                    o = a @ V
                    if st["aV"] is not None:
                        w = torch.zeros((r1 - r0, 2 * k + 1), dtype=torch.float64, device=dev)
                        o = o + w.scatter_add(1, r, a) @ st["aV"][h].double()
                    res[at + r0:at + r1, q_head] = o
            if weights:
                # keys that no row sees keep what they have
                j = torch.arange(total, device=dev)
                if window:
                    first = max(0, cached + 1 - window)
                    j = j[(j >= first) | (j < sinks)]
                old = res[idx[j // P], h, j % P]
                keep = (j < cached) if c["accumulate"] else torch.zeros_like(j, dtype=torch.bool)
                res[idx[j // P], h, j % P] = got[j] + torch.where(keep, old, 0.0)
        at += n
    return res
