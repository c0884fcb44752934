"""Cases, plain forms and exact values of the paged-cache operators.

Four operators, as a serving program calls them around the decode step:

* ``plan``    the block tables and slot map of one batch step, from request
              lengths (``paged_plan``);
* ``append``  the new tokens' key and value rows into their pages
              (``paged_append``);
* ``attn``    a chunk of new tokens of every sequence over its paged cache,
              causal (``paged_attn``);
* ``window``  the same with a sliding window and a few first tokens that stay
              visible (``paged_attn`` with ``window`` and ``sinks``).

With ``own`` false ``run`` computes the plain form: elementary torch
operations in fp32.  With ``own`` true it makes the package's calls.
``exact`` evaluates the definition in fp64, written apart from the plain form.

Sizes are those of this repository's workloads (32 query heads over 8 KV
heads at d = 128, caches of 32,768 / 65,536 / 131,072 tokens, the small fp32
shape of 8 heads over 2 at d = 64) or generic.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------

def _attn_case(name, B, ctx, new, lens, Hq, Hkv, d, page, dtype, window=0, sinks=0):
    """ctx: cached tokens of the longest sequence, the new ones included;
    new: new tokens of a sequence; lens: how both vary over the batch."""
    return {"name": name, "op": "window" if window else "attn", "B": B, "ctx": ctx, "new": new,
            "lens": lens, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "window": window, "sinks": sinks}


def listed():
    return [
        # a decode step of 256 running requests, each with a growing table
        {"name": "plan_decode_256", "op": "plan", "B": 256, "ctx": 32768, "new": 1,
         "lens": "ragged", "page": 16},
        # prompts arriving together: 24 ragged chunks of up to 4,096 tokens
        {"name": "plan_prompts_24x4k", "op": "plan", "B": 24, "ctx": 8192, "new": 4096,
         "lens": "ragged", "page": 64},
        # the new rows of one decode step of 16 sequences (latency)
        {"name": "append_decode_16", "op": "append", "B": 16, "ctx": 1024, "new": 1,
         "lens": "ragged", "Hkv": 8, "d": 128, "page": 64, "dtype": "bf16"},
        # a prompt batch's rows, read as slices of the fused q/k/v projection
        {"name": "append_prompts_16k", "op": "append", "B": 8, "ctx": 4096, "new": 2048,
         "lens": "ragged", "Hkv": 8, "d": 128, "page": 16, "dtype": "bf16"},
        # dense attention of one decode token over the headline's 128K cache
        _attn_case("attn_decode_1x128k", 1, 131072, 1, "same", 32, 8, 128, 64, "bf16"),
        # a ragged decode batch, caches of up to 64K tokens
        _attn_case("attn_decode_16x64k", 16, 65536, 1, "ragged", 32, 8, 128, 16, "bf16"),
        # a prompt's 2,048-token chunk over a 32K cache
        _attn_case("attn_chunk_2k_of_32k", 1, 32768, 2048, "same", 32, 8, 128, 64, "bf16"),
        # continuous batching: one prompt chunk among 31 decoding sequences
        _attn_case("attn_mixed_32", 32, 8192, 1000, "mixed", 32, 8, 128, 16, "bf16"),
        # the small fp32 shape: a chunk of its 4,096-token cache
        _attn_case("attn_chunk_f32", 1, 4096, 250, "same", 8, 2, 64, 32, "f32"),
        # one token of one short request under a window (latency)
        _attn_case("window_decode_1", 1, 4096, 1, "same", 32, 8, 128, 16, "bf16", 1024, 4),
        # a decode batch of the self-decoder's window layers
        _attn_case("window_decode_64", 64, 32768, 1, "ragged", 16, 2, 64, 16, "bf16", 4095, 4),
        # a long prompt's chunk through a window layer
        _attn_case("window_chunk_8k", 1, 16384, 8192, "same", 32, 8, 128, 64, "bf16", 4096, 4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "window", "window"])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "plan":
        if rng.random() < 0.5:
            return {"op": op, "B": _log(rng, 1, 512), "ctx": _log(rng, 64, 32768), "new": 1,
                    "lens": "ragged", "page": page}
        new = _log(rng, 16, 4096)
        return {"op": op, "B": _log(rng, 1, 24), "ctx": new + _log(rng, 1, 4096), "new": new,
                "lens": rng.choice(["ragged", "mixed"]), "page": page}
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 2048)])
        return {"op": op, "B": _log(rng, 1, 8 if new > 1 else 256), "ctx": new + _log(rng, 1, 2048),
                "new": new, "lens": rng.choice(["same", "ragged"]), "Hkv": rng.choice([1, 2, 8]),
                "d": rng.choice([64, 128]), "page": page, "dtype": rng.choice(["bf16", "f32"])}
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128])
    if rng.random() < 0.5:  # decode: up to 2^19 cached tokens in all
        B = _log(rng, 1, 128)
        ctx = _log(rng, 64, min(131072, (1 << 19) // B))
        new, lens = 1, rng.choice(["same", "ragged"])
    else:                   # chunks: up to 2^25 pairs of a new and a cached token
        B = _log(rng, 1, 32)
        new = _log(rng, 2, min(2048, 8192 // B))
        ctx = new + _log(rng, 1, min(32768, (1 << 25) // (B * new)))
        lens = rng.choice(["same", "ragged", "mixed"])
        if dtype == "f32":
            new = min(new, 256)
    window = sinks = 0
    if op == "window":
        window = _log(rng, 16, 8192)
        sinks = rng.choice([0, 1, 4, 16])
    c = _attn_case("", B, ctx, new, lens, Hq, Hkv, d, page, dtype, window, sinks)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of every sequence: the
    case's own numbers, whatever the seed of the data."""
    B, ctx, new = case["B"], case["ctx"], case["new"]
    if case["lens"] == "same":
        return [new] * B, [ctx] * B
    r = random.Random("%d/%d/%d" % (B, ctx, new))
    ns, cs = [], []
    for b in range(B):
        if case["lens"] == "mixed":     # one chunk, the others decode
            n = new if b == B // 2 else 1
        else:
            n = new if b == 0 else r.randint((new + 1) // 2, new)
        c = ctx if b == 0 else r.randint(max(n, ctx // 8), ctx)
        ns.append(n)
        cs.append(max(c, n))
    return ns, cs


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(g, shape, dtype):
    """A cache pool of normal rows, filled piece by piece."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        flat[i:i + (1 << 26)].normal_(generator=g)
    return t


def _blocks(n, page):
    return -(-n // page)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(g, case, lens):
    """Block tables of sequences of these lengths over shuffled pages."""
    page = case["page"]
    nb = [_blocks(n, page) for n in lens]
    pages = sum(nb) + 7
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(nb)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    g = _gen(seed)
    new, kv = _lengths(case)
    page, B = case["page"], case["B"]
    T = sum(new)
    st = {"case": case, "new": new, "kv": kv, "T": T}
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["starts"] = starts
    if case["op"] == "plan":
        past = [c - n for n, c in zip(new, kv)]
        nb_all = [_blocks(c, page) for c in kv]
        nb_old = [_blocks(c, page) for c in past]
        pages = sum(nb_all) + 64
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(nb_all) + 8), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(nb_old):
            table[b, :n] = perm[at:at + n]
            at += n
        st.update(table=table, pages=pages, new_lens=_i32(new), lens=_i32(past),
                  free_pages=perm[at:].contiguous(), free_count=_i32([pages - at]))
        return st
    if case["op"] == "append":
        # keys and values are column ranges of one projection's output rows
        dt, w = DTYPES[case["dtype"]], case["Hkv"] * case["d"]
        table, pages = _tables(g, case, kv)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        for b in range(B):
            pos = torch.arange(kv[b] - new[b], kv[b], device="cuda")
            slots[starts[b]:starts[b + 1]] = table[b].long()[pos // page] * page + pos % page
        qkv = _randn(g, (T, 6 * w), dt)
        shape = (pages, case["Hkv"], page, case["d"])
        st.update(K=_pool(g, shape, dt), V=_pool(g, shape, dt), slots=slots.to(torch.int32),
                  k_new=qkv[:, 4 * w:5 * w].unflatten(1, (case["Hkv"], case["d"])),
                  v_new=qkv[:, 5 * w:].unflatten(1, (case["Hkv"], case["d"])))
        return st
    dt = DTYPES[case["dtype"]]
    table, pages = _tables(g, case, kv)
    shape = (pages, case["Hkv"], page, case["d"])
    st.update(K=_pool(g, shape, dt), V=_pool(g, shape, dt), table=table,
              q=_randn(g, (T, case["Hq"], case["d"]), dt),
              q_start=_i32(starts), kv_lens=_i32(kv))
    return st


# ---- one pass -----------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        import token_sparse_attention_sm_b200 as sd
        if case["op"] == "plan":
            p = sd.paged_plan(state["new_lens"], state["lens"], state["table"],
                              state["free_pages"], state["free_count"], case["page"],
                              state["T"], state["pages"], check=False)
            return [state["table"], p["kv_lens"], p["q_start"], p["positions"], p["slots"],
                    p["free_left"]]
        if case["op"] == "append":
            sd.paged_append(state["K"], state["V"], state["k_new"], state["v_new"],
                            state["slots"], check=False)
            return [state["K"], state["V"]]
        out, lse = sd.paged_attn(state["q"], state["K"], state["V"], state["table"],
                                 state["q_start"], state["kv_lens"], window=case["window"],
                                 sinks=case["sinks"], max_new=max(state["new"]), check=False)
        return [out, lse]
    if case["op"] == "plan":
        return _plain_plan(state)
    if case["op"] == "append":
        return _plain_append(state)
    return _plain_attn(state)


def _plain_plan(st):
    page, T = st["case"]["page"], st["T"]
    table, new, past = st["table"], st["new_lens"].long(), st["lens"].long()
    B, cols = table.shape
    kv = past + new
    q_end = torch.cumsum(new, 0)
    q_start = torch.cat([q_end.new_zeros(1), q_end])
    nb_old = (past + page - 1) // page
    nb_new = (kv + page - 1) // page
    need = nb_new - nb_old
    taken = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device="cuda")[None, :]
    fresh = (col >= nb_old[:, None]) & (col < nb_new[:, None])
    at = st["free_count"].long() - 1 - (taken[:, None] + col - nb_old[:, None])
    page_id = st["free_pages"][at.clamp(0, st["free_pages"].numel() - 1)]
    table.copy_(torch.where(fresh, page_id, table))
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(q_end, row, right=True)
    pos = past[seq] + row - q_start[seq]
    slot = table[seq, pos // page].long() * page + pos % page
    left = st["free_count"] - need.sum().to(torch.int32)
    return [table, kv.to(torch.int32), q_start.to(torch.int32), pos.to(torch.int32),
            slot.to(torch.int32), left]


def _plain_append(st):
    page = st["case"]["page"]
    s = st["slots"].long()
    st["K"][s // page, :, s % page] = st["k_new"]
    st["V"][s // page, :, s % page] = st["v_new"]
    return [st["K"], st["V"]]


def _gather(cache, table, b, n, page):
    """The first n rows of sequence b: [Hkv, n, d]."""
    rows = cache[table[b, :_blocks(n, page)].long()]          # [blocks, Hkv, page, d]
    rows = rows.transpose(0, 1)
    return rows.reshape(rows.shape[0], -1, rows.shape[-1])[:, :n]


def _visible(case, q_pos, k_pos):
    q_pos, k_pos = q_pos[:, None], k_pos[None, :]
    see = k_pos <= q_pos
    if case["window"]:
        see = see & ((k_pos > q_pos - case["window"]) | (k_pos < case["sinks"]))
    return see


def _plain_attn(st):
    case = st["case"]
    q, page, Hkv, d = st["q"], case["page"], case["Hkv"], case["d"]
    G = case["Hq"] // Hkv
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    for b in range(case["B"]):
        n, c = st["new"][b], st["kv"][b]
        r0 = st["starts"][b]
        k = _gather(st["K"], st["table"], b, c, page).float()
        v = _gather(st["V"], st["table"], b, c, page).float()
        k_pos = torch.arange(c, device="cuda")
        step = max(1, (1 << 29) // (case["Hq"] * c))          # rows of scores held at once
        for i in range(0, n, step):
            m = min(step, n - i)
            x = q[r0 + i:r0 + i + m].float().unflatten(1, (Hkv, G))
            x = x.permute(1, 2, 0, 3).reshape(Hkv, G * m, d)
            z = (x @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
            see = _visible(case, torch.arange(c - n + i, c - n + i + m, device="cuda"), k_pos)
            z = z.view(Hkv, G, m, c).masked_fill_(~see, float("-inf"))
            top = z.amax(-1, keepdim=True)
            p = z.sub_(top).exp_()
            s = p.sum(-1, keepdim=True)
            o = (p.view(Hkv, G * m, c) @ v).view(Hkv, G, m, d) / s
            out[r0 + i:r0 + i + m] = o.permute(2, 0, 1, 3).reshape(m, -1, d).to(q.dtype)
            lse[r0 + i:r0 + i + m] = (top + s.log())[..., 0].permute(2, 0, 1).reshape(m, -1)
    return [out, lse]


# ---- what a pass cannot do without ------------------------------------------------

def _pairs_and_rows(case):
    """Visible (new token, cached token) pairs, and cached rows that some new
    token sees, over the batch."""
    pairs = rows = 0
    w, s = case["window"], case["sinks"]
    for n, c in zip(*_lengths(case)):
        first = c - n
        if not w:
            pairs += n * first + n * (n + 1) // 2
            rows += c
            continue
        for p in range(first, c):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(s, lo)
        lo = max(0, first - w + 1)
        rows += c - lo + min(s, lo)
    return pairs, rows


def work(case):
    new, kv = _lengths(case)
    T, page = sum(new), case["page"]
    if case["op"] == "plan":
        need = tails = 0
        for n, c in zip(new, kv):
            need += _blocks(c, page) - _blocks(c - n, page)
            tails += 1 if (c - n) % page else 0
        # lengths, tail pages and free pages read; tables, starts, lengths, maps written
        return {"bytes": 4 * (2 * case["B"] + tails + need + 1) +
                4 * (need + 2 * case["B"] + 2 + 2 * T), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        return {"bytes": 4 * T * case["Hkv"] * case["d"] * e + 4 * T, "flops": 0}
    pairs, rows = _pairs_and_rows(case)
    tables = sum(_blocks(c, page) for c in kv) if not case["window"] else _blocks(rows, page)
    return {"bytes": 2 * rows * case["Hkv"] * case["d"] * e + 2 * T * case["Hq"] * case["d"] * e +
            4 * T * case["Hq"] + 4 * (tables + 2 * case["B"] + 1),
            "flops": 4 * pairs * case["Hq"] * case["d"]}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    """Row by row of the definition: o = sum_j w_j v_j with
    w_j = exp(z_j - lse), lse = log sum_j exp(z_j), z_j = <q, k_j> / sqrt(d)
    over the tokens j the row sees; one query head at a time."""
    if case["op"] in ("plan", "append"):
        return None     # whole numbers and copies: compared as they are
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    q = st["q"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, c, r0 = st["new"][b], st["kv"][b], st["starts"][b]
        j = torch.arange(c, device="cuda")
        page_of = st["table"][b][j // case["page"]].long()
        for h in range(case["Hkv"]):
            k = st["K"][page_of, h, j % case["page"]].double()
            v = st["V"][page_of, h, j % case["page"]].double()
            for a in range(h * G, (h + 1) * G):
                for i in range(0, n, 2048):
                    rows = slice(r0 + i, r0 + min(n, i + 2048))
                    p = c - n + torch.arange(i, min(n, i + 2048), device="cuda")
                    z = torch.einsum("id,jd->ij", q[rows, a].double(), k) / case["d"] ** 0.5
                    hidden = j[None] > p[:, None]
                    if case["window"]:
                        old = j[None] < p[:, None] - case["window"] + 1
                        hidden = hidden | (old & (j[None] >= case["sinks"]))
                    z[hidden] = -math.inf
                    total = torch.logsumexp(z, 1)
                    w = torch.exp(z - total[:, None])
                    out[rows, a] = torch.einsum("ij,jd->id", w, v)
                    lse[rows, a] = total
    return [out, lse]
