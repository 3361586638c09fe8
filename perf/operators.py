"""The paged key/value cache operators, as they are measured: block tables and slot maps from
request lengths (op "plan"), new rows written to their pages (op "append"), and attention of
the new tokens over the pages with relative terms, grouped heads, a sliding window and first
tokens that stay visible (op "attend").

run() computes the plain form of an operator in torch, or, with `own` set, calls the library.
Every length of a case follows from the case itself; the values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def _attend(name, **kw):
    c = dict(name=name, op="attend", B=1, H=8, Hkv=8, d=64, P=16, dtype="bf16", new_lo=1,
             new_hi=1, chunk_every=1, cached_lo=0, cached_hi=0, clip_k=0, key_term=False,
             value_term=False, window=0, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # one generated token for each of 32 running requests: the smallest plan there is
        dict(name="plan_decode", op="plan", B=32, P=16, new_lo=1, new_hi=1, cached_lo=1024,
             cached_hi=2047),
        # a wave of prompts and of chunks of prompts admitted at once, about 65000 tokens
        dict(name="plan_prompts", op="plan", B=256, P=16, new_lo=1, new_hi=511, cached_lo=0,
             cached_hi=4096),
        # the new rows of one decoding step of 32 requests (16 heads of 64)
        dict(name="append_decode", op="append", T=32, Hkv=16, d=64, P=16, dtype="bf16"),
        # the rows of 16384 prompt tokens
        dict(name="append_prompts", op="append", T=16384, Hkv=8, d=128, P=16, dtype="bf16"),
        # one decoding step of the Transformer-big decoder, both relative terms, caches of 1K-2K
        _attend("decode_relative", B=32, H=16, Hkv=16, d=64, cached_lo=1023, cached_hi=2047,
                clip_k=16, key_term=True, value_term=True),
        # one decoding step of 64 requests with long caches, eight query heads to a key head
        _attend("decode_grouped", B=64, H=16, Hkv=2, d=128, P=32, cached_lo=2047,
                cached_hi=16383),
        # a single user far into a long document
        _attend("decode_one_long", B=1, H=16, Hkv=4, d=128, P=64, cached_lo=131070,
                cached_hi=131070),
        # many chats that keep a window and the first few tokens
        _attend("decode_window", B=128, H=16, Hkv=4, d=64, cached_lo=900, cached_hi=32767,
                window=1024, sinks=4),
        # four fresh prompts of 4096 tokens with the key-relative term: the work of a prefill
        _attend("prompt_relative", B=4, H=16, Hkv=16, d=128, new_lo=4096, new_hi=4096,
                clip_k=64, key_term=True),
        # a step that mixes generated tokens with chunks of prompts of odd sizes
        _attend("mixed_step", B=24, H=16, Hkv=4, d=128, new_lo=401, new_hi=613, chunk_every=6,
                cached_lo=1, cached_hi=8191),
        # chunks of a long document under a window, both relative terms
        _attend("chunk_window", B=2, H=16, Hkv=2, d=64, new_lo=2048, new_hi=2048,
                cached_lo=30001, cached_hi=32001, clip_k=16, key_term=True, value_term=True,
                window=4096, sinks=16),
        # single precision, as a model is checked before it is cast: short odd chunks
        _attend("chunk_f32", B=3, H=8, Hkv=8, d=64, P=8, dtype="f32", new_lo=61, new_hi=127,
                cached_lo=100, cached_hi=700, clip_k=16, key_term=True, value_term=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "attend"])
    if op == "plan":
        while True:
            hi = _log(rng, 1, 2048)
            c = dict(op="plan", B=_log(rng, 1, 1024), P=rng.choice([8, 16, 32, 64, 128]),
                     new_lo=_log(rng, 1, hi), new_hi=hi, cached_lo=0,
                     cached_hi=_log(rng, 1, 16384))
            if sum(_lens(c)[1]) <= 66000:
                return c
    if op == "append":
        while True:
            c = dict(op="append", T=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 4, 8, 12, 16]),
                     d=rng.choice([64, 80, 128]), P=rng.choice([8, 16, 32, 64, 128]),
                     dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
            if work(c)["bytes"] <= 135e6:
                return c
    while True:
        kind = rng.choice(["decode", "decode", "chunk", "chunk", "prompt", "mixed"])
        f32 = rng.random() < 0.125
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        g = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
        cached = 0 if kind == "prompt" else _log(rng, 1, 2048 if f32 else 65536)
        new = 1 if kind == "decode" else _log(rng, 2, 127 if f32 else 4096)
        terms = rng.choice([(False, False), (True, False), (True, True), (False, True)])
        windowed = rng.random() < 0.35
        c = _attend("", B=_log(rng, 1, 4 if f32 else 128), H=Hkv * g, Hkv=Hkv,
                    d=rng.choice([64, 128]), P=rng.choice([8, 16, 32, 64, 128]),
                    dtype="f32" if f32 else "bf16", new_lo=max(1, int(new * rng.uniform(0.3, 1))),
                    new_hi=new, chunk_every=rng.choice([3, 6, 9]) if kind == "mixed" else 1,
                    cached_lo=int(cached * rng.uniform(0, 1)), cached_hi=cached,
                    clip_k=rng.choice([1, 4, 16, 64]) if any(terms) else 0, key_term=terms[0],
                    value_term=terms[1], window=_log(rng, 16, 8192) if windowed else 0,
                    sinks=rng.choice([0, 1, 4, 16, 130]) if windowed else 0)
        del c["name"]
        w = work(c)
        cached_l, new_l = _lens(c)
        # the plain form's scores over all of a request's keys, and the caches in memory
        scores = max(a * (a + b if not windowed else min(a + b, a + c["window"] + c["sinks"]))
                     for a, b in zip(new_l, cached_l)) * c["H"]
        cache = sum(a + b + c["P"] for a, b in zip(new_l, cached_l)) * Hkv * c["d"] * 4
        if w["bytes"] > 6e8 or w["flops"] > (4e9 if f32 else 2.7e11):
            continue
        if scores > 1.2e9 or cache > 4e9 or c["H"] > 64:
            continue
        return c


# ------------------------------------------------------------------------------ lengths
def _spread(i, step, lo, hi):
    """The i-th of lengths spread evenly over lo .. hi, odd and even ones alike."""
    return lo + int(((i + 1) * step % 1.0) * (hi - lo + 1))


def _lens(c):
    """Cached and new tokens of every request."""
    cached = [_spread(i, 0.7548776662466927, c["cached_lo"], c["cached_hi"]) for i in range(c["B"])]
    new = [_spread(i, 0.6180339887498949, c["new_lo"], c["new_hi"])
           if i % c.get("chunk_every", 1) == 0 else 1 for i in range(c["B"])]
    return cached, new


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
    if c["op"] == "plan":
        cached, new = _lens(c)
        P = c["P"]
        taken = sum(_pages(a + b, P) - _pages(a, P) for a, b in zip(cached, new))
        part = sum(1 for a in cached if a % P)  # a partly filled page's entry is read
        return {"bytes": 4 * (4 * c["B"] + 3 + 2 * taken + part + sum(new)),
                "flops": 2 * sum(new)}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        return {"bytes": 4 * c["T"] * c["Hkv"] * c["d"] * es + 4 * c["T"], "flops": 0}
    cached, new = _lens(c)
    T, H, Hkv, d, k = sum(new), c["H"], c["Hkv"], c["d"], c["clip_k"]
    terms = int(c["key_term"]) + int(c["value_term"])
    by, fl = 2 * T * H * d * es + 4 * (2 * c["B"] + 1), 2 * d * T * H * (k + 1) * terms
    for a, n in zip(cached, new):
        pairs, rows = _visible(c, a, n)
        by += 2 * rows * Hkv * d * es + 4 * _pages(rows, c["P"])
        fl += 4 * d * H * pairs
    return {"bytes": by + terms * Hkv * (k + 1) * d * es, "flops": fl}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device=dev)
    st = {"case": dict(c)}

    def normal(*shape, std=1.0):
        x = torch.empty(shape, dtype=_DT[c["dtype"]], device=dev)
        return x.normal_(0.0, std, generator=g)

    if c["op"] == "append":
        T, Hkv, d, P = c["T"], c["Hkv"], c["d"], c["P"]
        pages = _pages(T, P) + 64
        # the new keys and values come out of one projection, side by side
        kv = normal(T, 2, Hkv, d)
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
        st["k_pages"], st["v_pages"] = normal(pages, Hkv, P, d), normal(pages, Hkv, P, d)
        order = torch.randperm(pages, generator=g, device=dev)
        if T <= 256:  # a decoding step: every token in a page of its own
            page = order[torch.arange(T, device=dev) % pages]
            row = torch.randint(0, P, (T,), generator=g, device=dev)
            if T > pages:
                t = torch.arange(T, device=dev)
                page, row = order[t // P], t % P
        else:
            t = torch.arange(T, device=dev)
            page, row = order[t // P], t % P
        st["slots"] = (page * P + row).to(torch.int32)
        return st

    cached, new = _lens(c)
    P, B = c["P"], c["B"]
    total = [a + b for a, b in zip(cached, new)]
    M = _pages(max(total), P)
    have = [_pages(a, P) for a in (cached if c["op"] == "plan" else total)]
    n_pages = sum(_pages(t, P) for t in total) + 16
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, M), -1, **i32)
    n_have = torch.tensor(have, device=dev)
    filled = torch.arange(M, device=dev)[None, :] < n_have[:, None]
    table[filled] = order[:sum(have)]
    st["block_table"] = table
    if c["op"] == "plan":
        st["cached_len"] = torch.tensor(cached, **i32)
        st["new_len"] = torch.tensor(new, **i32)
        # the pages handed out before come first in the list
        st["free_pages"] = order
        st["free_head"] = torch.tensor([sum(have)], **i32)
        st["tokens"] = sum(new)
        if own:
            st["kv_len"] = torch.empty(B, **i32)
            st["q_start"] = torch.empty(B + 1, **i32)
            st["slots"] = torch.empty(sum(new), **i32)
            st["free_head_out"] = torch.empty(1, **i32)
        return st

    T, H, Hkv, d, k = sum(new), c["H"], c["Hkv"], c["d"], c["clip_k"]
    # the queries come out of one projection with the new keys and values
    qkv = normal(T, H + 2 * Hkv, d)
    st["q"] = qkv[:, :H]
    st["k_pages"], st["v_pages"] = normal(n_pages, Hkv, P, d), normal(n_pages, Hkv, P, d)
    st["aK"] = normal(Hkv, 2 * k + 1, d, std=0.02) if c["key_term"] else None
    st["aV"] = normal(Hkv, 2 * k + 1, d, std=0.02) if c["value_term"] else None
    st["kv_len"] = torch.tensor(total, **i32)
    st["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    st["cached"], st["new"] = cached, new
    st["scale"] = d ** -0.5
    st["out"] = torch.empty((T, H, d), dtype=_DT[c["dtype"]], device=dev)
    if own:
        import relative_position_representations_gb300 as rp
        st["workspace"] = torch.empty(rp.relattn_paged_workspace_size(H, Hkv, d),
                                      dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_plan(st):
    P = st["case"]["P"]
    table, head = st["block_table"], st["free_head"]
    cached, new = st["cached_len"], st["new_len"]
    B, M = table.shape
    F = st["free_pages"].numel()
    dev = table.device
    old, tot = (cached + P - 1) // P, (cached + new + P - 1) // P
    bad = (cached < 0) | (new < 0) | (tot > M)
    need = torch.where(bad, 0, tot - old)
    incl = torch.cumsum(need, 0)
    placed = ~bad & ((need == 0) | (head + incl <= F))
    # new entries of every row of the table
    j = torch.arange(M, device=dev)[None, :]
    fresh = placed[:, None] & (j >= old[:, None]) & (j < tot[:, None])
    src = (head + incl - need - old)[:, None] + j
    table.copy_(torch.where(fresh, st["free_pages"][src.clamp(0, F - 1)], table))
    n_new = new.clamp(min=0)
    q_start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(n_new, 0).to(torch.int32)])
    kv_len = torch.where(placed, cached + new, cached)
    t = torch.arange(st["tokens"], device=dev, dtype=torch.int32)
    b = (t[:, None] >= q_start[None, 1:]).sum(1).clamp(max=B - 1)
    pos = cached[b] + t - q_start[b]
    ok = placed[b] & (t < q_start[B])
    page = table[b, (pos // P).clamp(0, M - 1)]
    slots = torch.where(ok, page * P + pos % P, -1).to(torch.int32)
    head_out = head + torch.where(placed, incl, 0).max().to(torch.int32)
    return [table, q_start, kv_len, slots, head_out.to(torch.int32)]


def _plain_append(st):
    P = st["case"]["P"]
    s = st["slots"].long()
    page, row = s // P, s % P
    st["k_pages"][page, :, row] = st["k"]
    st["v_pages"][page, :, row] = st["v"]
    return [st["k_pages"], st["v_pages"]]


def _keys_of(c, cached, new, dev):
    """The cache rows that some row of a request sees: the first tokens, then the window."""
    total = cached + new
    first = max(0, cached + 1 - c["window"]) if c["window"] else 0
    return torch.cat([torch.arange(min(c["sinks"], first), device=dev),
                      torch.arange(first, total, device=dev)])


def _plain_attend(st):
    c = st["case"]
    H, Hkv, d, P, k = c["H"], c["Hkv"], c["d"], c["P"], c["clip_k"]
    gsz = H // Hkv
    out, at = st["out"], 0
    aK = None if st["aK"] is None else st["aK"][:, :k + 1].float()
    aV = None if st["aV"] is None else st["aV"][:, :k + 1].float()
    for b in range(c["B"]):
        n, cached = st["new"][b], st["cached"][b]
        dev = out.device
        j = _keys_of(c, cached, n, dev)
        page, row = st["block_table"][b, j // P].long(), j % P
        K = st["k_pages"][page, :, row].float().transpose(0, 1)       # [Hkv, keys, d]
        V = st["v_pages"][page, :, row].float().transpose(0, 1)
        q = st["q"][at:at + n].float().reshape(n, Hkv, gsz, d).permute(1, 2, 0, 3)
        q = q.reshape(Hkv, gsz * n, d)
        pos = (cached + torch.arange(n, device=dev)).repeat(gsz)
        off = j[None, :] - pos[:, None]                               # j - i
        s = q @ K.transpose(1, 2)
        lab = off.clamp(-k, 0) + k
        if aK is not None:
            s += torch.gather(q @ aK.transpose(1, 2), 2, lab.expand(Hkv, -1, -1))
        s *= st["scale"]
        hide = off > 0
        if c["window"]:
            hide = hide | ((off <= -c["window"]) & (j >= c["sinks"])[None, :])
        s.masked_fill_(hide, float("-inf"))
        m = s.amax(2, keepdim=True)
        s -= torch.where(m.isinf(), torch.zeros_like(m), m)
        p = s.exp_()
        l = p.sum(2, keepdim=True)
        z = p @ V
        if aV is not None:
            bins = torch.zeros((Hkv, gsz * n, k + 1), device=dev)
            bins.scatter_add_(2, lab.expand(Hkv, -1, -1), p)
            z += bins @ aV
        z /= torch.where(l > 0, l, torch.ones_like(l))
        out[at:at + n] = z.reshape(Hkv, gsz, n, d).permute(2, 0, 1, 3).reshape(n, H, d).to(out.dtype)
        at += n
    return out


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[op](st)
    import relative_position_representations_gb300 as rp
    if op == "plan":
        kv_len, q_start, slots, head = rp.relattn_paged_plan(
            st["cached_len"], st["new_len"], st["block_table"], st["free_pages"],
            st["free_head"], st["case"]["P"], st["tokens"], kv_len=st["kv_len"],
            q_start=st["q_start"], slots=st["slots"], free_head_out=st["free_head_out"])
        return [st["block_table"], q_start, kv_len, slots, head]
    if op == "append":
        rp.relattn_paged_append(st["k"], st["v"], st["slots"], st["k_pages"], st["v_pages"])
        return [st["k_pages"], st["v_pages"]]
    c = st["case"]
    return rp.relattn_paged_fwd(st["q"], st["k_pages"], st["v_pages"], st["block_table"],
                                st["q_start"], st["kv_len"], aK=st["aK"], aV=st["aV"],
                                clip_k=c["clip_k"], window=c["window"], sinks=c["sinks"],
                                scale=st["scale"], max_new=max(st["new"]), out=st["out"],
                                workspace=st["workspace"])


# ------------------------------------------------------------------------------ exact values
def exact(case, seed):
    """The definitions in 64 bits: the plan as an allocator would do it page by page, the copy
    slot by slot, attention head by head and row block by row block."""
    c = case
    st = prepare(c, seed)
    P = c["P"]
    if c["op"] == "plan":
        table = st["block_table"].cpu().numpy().astype(np.int64)
        cached, new = st["cached_len"].tolist(), st["new_len"].tolist()
        free, head = st["free_pages"].tolist(), int(st["free_head"])
        starts, lens, slots = [0], [], []
        for b in range(c["B"]):
            for i in range(new[b]):
                p = cached[b] + i
                if p % P == 0:
                    table[b, p // P] = free[head]
                    head += 1
                slots.append(int(table[b, p // P]) * P + p % P)
            starts.append(starts[-1] + new[b])
            lens.append(cached[b] + new[b])
        return [torch.tensor(table, dtype=torch.int32)] + \
               [torch.tensor(x, dtype=torch.int32) for x in (starts, lens, slots, [head])]
    if c["op"] == "append":
        s = st["slots"].long()
        res = []
        for x, pages in ((st["k"], st["k_pages"]), (st["v"], st["v_pages"])):
            flat = pages.transpose(1, 2).reshape(-1, c["Hkv"], c["d"]).double()
            flat.index_copy_(0, s, x.double())
            res.append(flat.reshape(-1, P, c["Hkv"], c["d"]).transpose(1, 2).contiguous())
        return res
    H, Hkv, d, k = c["H"], c["Hkv"], c["d"], c["clip_k"]
    gsz = H // Hkv
    T = sum(st["new"])
    z = torch.zeros((T, H, d), dtype=torch.float64, device=st["q"].device)
    at = 0
    for b in range(c["B"]):
        n, cached = st["new"][b], st["cached"][b]
        n_pages = _pages(cached + n, P)
        idx = st["block_table"][b, :n_pages].long()
        for h in range(Hkv):
            K = st["k_pages"][idx, h].double().reshape(n_pages * P, d)
            V = st["v_pages"][idx, h].double().reshape(n_pages * P, d)
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                lo = 0
                if c["window"] and c["sinks"] == 0:
                    lo = max(0, cached + r0 + 1 - c["window"])
                hi = cached + r1
                j = torch.arange(lo, hi, device=z.device)
                if c["window"] and c["sinks"]:
                    j = j[(j < c["sinks"]) | (j > cached + r0 - c["window"])]
                Kj, Vj = K[j], V[j]
                i = torch.arange(cached + r0, cached + r1, device=z.device)
                dist = i[:, None] - j[None, :]
                seen = dist >= 0
                if c["window"]:
                    seen &= (dist < c["window"]) | (j < c["sinks"])[None, :]
                r = k - dist.clamp(0, k)                 # table row of offset -dist, clipped
                for q_head in range(h * gsz, (h + 1) * gsz):
                    q = st["q"][at + r0:at + r1, q_head].double()
                    e = q @ Kj.T
                    if st["aK"] is not None:
                        e = e + (q @ st["aK"][h].double().T).gather(1, r)
                    e = torch.where(seen, e * st["scale"], -math.inf)
                    a = torch.softmax(e, 1)
                    o = a @ Vj
                    if st["aV"] is not None:
                        w = torch.zeros((r1 - r0, 2 * k + 1), dtype=torch.float64, device=z.device)
                        o = o + w.scatter_add(1, r, a) @ st["aV"][h].double()
                    z[at + r0:at + r1, q_head] = o
        at += n
    return z
