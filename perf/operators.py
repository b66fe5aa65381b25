"""The attention operators and the cache-page operators on real sizes: cases,
inputs, plain forms and work counts.

Three families, told apart by a case's ``op``:

``prompt``  attention of a packed batch of prompts over per-head K and V, with
            q in BF16 or as INT8 codes with a scale per token or per head;
``cache``   one decoding token per sequence over the paged latent KV cache,
            with an optional prefix that the whole batch shares;
``pages``   one scheduling step of a page pool: sequences end, survivors are
            forked, every running sequence grows, the pool is compacted, and
            the pages that moved are copied in every layer's cache.

The plain forms are elementary torch operations in 32 bits, rounded once.
"""
from __future__ import annotations

import random

import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------ cases

def _prompt(name, lens, heads, kv_heads, dqk, dv, q="bf16", past="", pad=0):
    """lens: new tokens of each sequence; past: cached tokens before them
    (chunked prefill; "" for none); pad: rows behind the last sequence."""
    return {"name": name, "op": "prompt", "lens": lens, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dqk": dqk, "dv": dv, "q": q, "pad": pad}


def _cache(name, batch, heads, lkv, rope, page, shared, lo, hi, layout):
    """Own lengths are drawn in [lo, hi] by random.Random(layout)."""
    return {"name": name, "op": "cache", "batch": batch, "heads": heads, "lkv": lkv, "rope": rope, "page": page,
            "shared": shared, "lo": lo, "hi": hi, "layout": layout}


def _pages(name, layers, lkv, rope, page, seqs, pages, lo, hi, ends, forks, grow, layout):
    """seqs running sequences of lo..hi tokens; `ends` of them end, `forks`
    children are forked, every other one grows by `grow` tokens."""
    return {"name": name, "op": "pages", "layers": layers, "lkv": lkv, "rope": rope, "page": page, "seqs": seqs,
            "pages": pages, "lo": lo, "hi": hi, "ends": ends, "forks": forks, "grow": grow, "layout": layout}


def listed():
    return [
        # the smallest q-path dims, two short prompts: what a call costs
        _prompt("prompt_tiny_int8", "4,3", 2, 2, 48, 32, q="int8"),
        # one V2-Lite prompt of the benchmark's prefill length
        _prompt("prompt_v2lite_4096", "4096", 16, 16, 192, 128),
        # a ragged V2-Lite batch as a server packs it, rows left over in the buffer
        _prompt("prompt_v2lite_ragged", "1,7,100,513,129,2047,33,1000", 16, 16, 192, 128, pad=37),
        # grouped heads, chunks of prompts behind a cached past
        _prompt("prompt_grouped_chunk", "512,300,1", 32, 4, 128, 128, past="7680,4097,1023"),
        # V3 heads with the prolog's INT8 q, four prompts
        _prompt("prompt_v3_packed_int8", "4099,2048,1331,700", 128, 128, 192, 128, q="int8"),
        # V3 heads, the benchmark's prefill length, one scale per head
        _prompt("prompt_v3_16384_int8_per_head", "16384", 128, 128, 192, 128, q="int8_per_head"),
        # one user, one short context: latency
        _cache("cache_v2lite_single", 1, 16, 512, 64, 64, 0, 100, 100, 1),
        # the benchmark's V2-Lite decode batch over ragged contexts
        _cache("cache_v2lite_64", 64, 16, 512, 64, 64, 0, 1, 4096, 2),
        # long contexts without sharing, V3 heads
        _cache("cache_v3_long", 32, 128, 512, 64, 64, 0, 2000, 32768, 3),
        # the benchmark's V3 decode batch behind a long common prompt
        _cache("cache_v3_shared", 128, 128, 512, 64, 64, 8192, 1, 1024, 4),
        # a small pool, one layer: latency of a scheduling step
        _pages("pages_small", 1, 512, 64, 64, 8, 256, 40, 700, 2, 3, 1, 5),
        # a server's pool over 8 layers, fragmented by ended sequences
        _pages("pages_server", 8, 512, 64, 64, 256, 4096, 100, 1500, 64, 48, 17, 6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "cache", "cache", "pages"])
    if op == "prompt":
        heads, kv, dqk, dv = rng.choice([(16, 16, 192, 128), (128, 128, 192, 128), (32, 4, 128, 128), (2, 2, 48, 32),
                                         (8, 1, 64, 64), (12, 4, 80, 112)])
        lens, past, pairs = [], [], 0
        most = 16384 * 16384 * 128 // 4 // heads
        for _ in range(rng.randint(1, 9)):
            n, p = _log_int(rng, 1, 4096), rng.choice([0, 0, _log_int(rng, 1, 8192)])
            if sum(lens) + n > 8192 or pairs + n * (n + p) > most:
                continue
            lens.append(n), past.append(p)
            pairs += n * (n + p)
        if not lens:
            lens, past = [rng.randint(1, 64)], [0]
        case = _prompt("", ",".join(map(str, lens)), heads, kv, dqk, dv, q=rng.choice(["bf16", "int8", "int8_per_head"]),
                       past=",".join(map(str, past)) if any(past) else "", pad=rng.choice([0, 1, 50]))
    elif op == "cache":
        batch = _log_int(rng, 1, 128)
        heads, lkv, rope = rng.choice([(16, 512, 64), (128, 512, 64), (64, 512, 64), (5, 256, 32), (2, 64, 16)])
        hi = _log_int(rng, 1, min(16384, 400000 // batch))
        shared = rng.choice([0, _log_int(rng, 1, 8192)])
        case = _cache("", batch, heads, lkv, rope, rng.choice([16, 32, 48, 64, 128]), shared, rng.randint(0, hi), hi,
                      rng.randint(1, 10 ** 6))
    else:
        seqs = _log_int(rng, 2, 256)
        page = rng.choice([16, 32, 64, 128])
        hi = _log_int(rng, 1, 1500)
        layers = _log_int(rng, 1, 16)
        ends = rng.randint(0, seqs // 2)
        forks = rng.randint(0, seqs - ends)
        per = -(-(hi + 40) // page) + 1
        pages = seqs * per * 2 + rng.randint(8, 64)
        case = _pages("", layers, 512, 64, page, seqs, pages, rng.randint(0, hi), hi, ends, forks, rng.randint(1, 40),
                      rng.randint(1, 10 ** 6))
        while case["layers"] > 1 and case["layers"] * pages * page * 1152 > 5 * 10 ** 9:
            case["layers"] -= 1
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs

def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _prompt_lens(case):
    new = _ints(case["lens"])
    past = _ints(case["past"]) or [0] * len(new)
    return new, [p + n for p, n in zip(past, new)]


def _cache_lens(case):
    r = random.Random(case["layout"])
    return [case["shared"] + r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _pool_plan(case):
    """Host-side start of a pool: (rows of the page table, lengths, the
    sequences that end, parents, children)."""
    r = random.Random(case["layout"])
    order = list(range(case["pages"]))
    r.shuffle(order)
    n, page = case["seqs"], case["page"]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    rows = []
    for length in lens:
        k = -(-length // page)
        rows.append(order[:k])
        order = order[k:]
    ended = r.sample(range(n), case["ends"])
    live = [s for s in range(n) if s not in ended]
    parents = [r.choice(live) for _ in range(case["forks"])]
    children = list(range(n, n + case["forks"]))
    return rows, lens, ended, live, parents, children


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    if case["op"] == "prompt":
        new, total = _prompt_lens(case)
        tq, tk = sum(new) + case["pad"], sum(total)
        h, hk, dqk, dv = case["heads"], case["kv_heads"], case["dqk"], case["dv"]
        st = {"case": case, "cu_q": _offsets(new), "cu_k": _offsets(total), "scale": dqk ** -0.5, "q_scale": None,
              "k": _normal(g, (tk, hk, dqk)), "v": _normal(g, (tk, hk, dv)),
              "out": torch.zeros((tq, h, dv), dtype=torch.bfloat16, device=DEV),
              "lse": torch.zeros((tq, h), dtype=torch.float32, device=DEV)}
        if case["q"] == "bf16":
            st["q"] = _normal(g, (tq, h, dqk), 1.7)
        else:
            x = torch.randn((tq, h, dqk), generator=g, device=DEV) * 1.7
            amax = x.abs().amax(dim=-1) if case["q"] == "int8_per_head" else x.abs().amax(dim=(1, 2))
            st["q_scale"] = (amax / 127.0).contiguous()
            st["q"] = (x / st["q_scale"].reshape(tq, -1, 1)).round().clamp(-127, 127).to(torch.int8)
        return st
    if case["op"] == "cache":
        page, c = case["page"], case["lkv"] + case["rope"]
        lens = _cache_lens(case)
        shared_pages = case["shared"] // page
        width = max(1, -(-max(lens) // page))
        count = shared_pages + sum(max(0, -(-n // page) - shared_pages) for n in lens)
        order = torch.randperm(count + 3, generator=g, device=DEV)[:count].tolist()
        table = torch.full((case["batch"], width), -1, dtype=torch.int32)
        at = shared_pages
        for b, n in enumerate(lens):
            k = -(-n // page)
            row = order[:shared_pages] + order[at:at + k - shared_pages]
            at += k - shared_pages
            table[b, :k] = torch.tensor(row, dtype=torch.int32)
        st = {"case": case, "page_table": table.to(DEV),
              "seq_lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
              # whole pages are shared: the tokens of a page that is not full are each sequence's own
              "shared_len": torch.tensor([shared_pages * page], dtype=torch.int32, device=DEV),
              "cache": _normal(g, (count + 3, page, c)), "q": _normal(g, (case["batch"], case["heads"], c)),
              "scale": 192.0 ** -0.5,
              "out": torch.zeros((case["batch"], case["heads"], case["lkv"]), dtype=torch.bfloat16, device=DEV),
              "lse": torch.zeros((case["batch"], case["heads"]), dtype=torch.float32, device=DEV)}
        st["workspace"] = torch.empty(_cache_workspace(case), dtype=torch.uint8, device=DEV)
        return st
    rows, lens, ended, live, parents, children = _pool_plan(case)
    page, n = case["page"], case["seqs"] + case["forks"]
    width = -(-(case["hi"] + case["grow"]) // page) + 1
    table = torch.full((n, width), -1, dtype=torch.int32)
    refs = torch.zeros(case["pages"], dtype=torch.int32)
    for s, row in enumerate(rows):
        table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
        refs[torch.tensor(row, dtype=torch.long)] += 1
    growing = live + children
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    st = {"case": case, "table0": table.to(DEV), "lens0": i32(lens + [0] * case["forks"]), "refs0": refs.to(DEV),
          "ended": i32(ended), "parents": i32(parents), "children": i32(children), "growing": i32(growing),
          "counts": i32([case["grow"]] * len(growing)),
          "cache": _normal(g, (case["layers"], case["pages"], page, case["lkv"] + case["rope"]))}
    st["table"], st["lens"], st["refs"] = (st[k].clone() for k in ("table0", "lens0", "refs0"))
    st["src"], st["dst"] = (torch.full((max(1, case["forks"]),), -1, dtype=torch.int32, device=DEV) for _ in "ab")
    st["slots"], st["positions"] = (torch.zeros(case["grow"] * len(growing), dtype=torch.int32, device=DEV) for _ in "ab")
    st["moved_to"] = torch.zeros(case["pages"], dtype=torch.int32, device=DEV)
    return st


def _cache_workspace(case):
    if not own:
        return 16
    from mla_attention_prolog_gb300 import binding
    return binding.attend_cache_workspace_bytes(case["batch"], case["heads"], case["lkv"], case["rope"])


# ------------------------------------------------------------ plain forms

def _rows_of(cu, rows):
    """For each row of a packed buffer: its sequence, its place in it, and
    whether a sequence holds it."""
    at = torch.arange(rows, device=DEV)
    seq = torch.bucketize(at, cu[1:].long(), right=True)
    held = seq < cu.numel() - 1
    seq = seq.clamp(max=cu.numel() - 2)
    return seq, at - cu.long()[seq], held


def _plain_prompt(st):
    q, k, v, out, lse = st["q"], st["k"], st["v"], st["out"], st["lse"]
    (tq, h, _), hk = q.shape, k.shape[1]
    sq, iq, held = _rows_of(st["cu_q"], tq)
    sk, ik, _ = _rows_of(st["cu_k"], k.shape[0])
    nq, nk = (c[1:].long() - c[:-1].long() for c in (st["cu_q"], st["cu_k"]))
    allowed = (sq[:, None] == sk[None, :]) & held[:, None] & (ik[None, :] <= (iq + nk[sq] - nq[sq])[:, None])
    group = h // hk
    step = max(1, min(hk, (1 << 31) // max(1, group * allowed.numel())))
    qf = q.float()
    if st["q_scale"] is not None:
        qf = qf * st["q_scale"].reshape(tq, -1, 1)
    for a in range(0, hk, step):   # a slice of the heads at a time: the scores of all would not fit the card
        b = min(hk, a + step)
        s = torch.matmul(qf[:, a * group:b * group].reshape(tq, b - a, group, -1).permute(1, 2, 0, 3),
                         k[:, a:b].float().permute(1, 2, 0)[:, None]) * st["scale"]
        s.masked_fill_(~allowed, NEG)
        m = s.amax(dim=-1, keepdim=True).nan_to_num_(neginf=0.0)
        p = s.sub_(m).exp_()
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p, v[:, a:b].float().permute(1, 0, 2)[:, None]) / total.clamp(min=1e-37)
        o = o.reshape((b - a) * group, tq, -1).permute(1, 0, 2)
        z = (m + total.log()).reshape((b - a) * group, tq).t()
        out[:, a * group:b * group] = torch.where(held[:, None, None], o, out[:, a * group:b * group].float()).to(out.dtype)
        lse[:, a * group:b * group] = torch.where(held[:, None], z, lse[:, a * group:b * group])
    return {"out": out, "lse": lse}


def _plain_cache(st):
    case, lens = st["case"], st["seq_lens"].long()
    width = st["page_table"].shape[1] * case["page"]
    rows = st["cache"][st["page_table"].clamp(min=0).long()].float().reshape(case["batch"], width, -1)
    s = torch.matmul(st["q"].float(), rows.transpose(1, 2)) * st["scale"]
    s.masked_fill_((torch.arange(width, device=DEV)[None, :] >= lens[:, None])[:, None], NEG)
    m = s.amax(dim=-1, keepdim=True).nan_to_num_(neginf=0.0)
    p = s.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    st["out"].copy_(torch.matmul(p, rows[:, :, :case["lkv"]]) / total.clamp(min=1e-37))
    st["lse"].copy_((m + total.log())[..., 0])
    return {"out": st["out"], "lse": st["lse"]}


def _restore(st):
    for k in ("table", "lens", "refs"):
        st[k].copy_(st[k + "0"])


def _pages_out(st):
    return {k: st[k] for k in ("table", "lens", "refs", "slots", "positions", "moved_to", "cache")}


def _held(table, lens, page):
    """Which entries of a page table hold a page."""
    return torch.arange(table.shape[1], device=DEV)[None, :] < ((lens + page - 1) // page)[:, None]


def _take(st, need):
    """The pages of `need` sequences in order, each the lowest that are free:
    [sequence, place] -> page."""
    free = torch.argsort((st["refs"] != 0).to(torch.int32), stable=True)
    first = need.cumsum(0) - need
    at = first[:, None] + torch.arange(st["table"].shape[1], device=DEV)[None, :]
    return free[at.clamp(max=free.numel() - 1)]


def _count(refs, table, held, by):
    refs.index_add_(0, table.clamp(min=0).reshape(-1).long(), (held.reshape(-1).to(torch.int32) * by))


def _plain_pages(st):
    case, page = st["case"], st["case"]["page"]
    _restore(st)
    table, lens, refs, cache = st["table"], st["lens"], st["refs"], st["cache"]
    place = torch.arange(table.shape[1], device=DEV)[None, :]
    # the sequences that end give back their pages
    e = st["ended"].long()
    _count(refs, table[e], _held(table[e], lens[e], page), -1)
    table[e] = -1
    lens[e] = 0
    # children share their parent's full pages and get a copy of the last one
    a, c = st["parents"].long(), st["children"].long()
    part = (lens[a] % page != 0).to(torch.int64)
    full = lens[a] // page
    fresh = _take(st, part)[:, :1]
    last = table[a].gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))
    rows = torch.where(place < full[:, None], table[a], -1)
    rows = torch.where((place == full[:, None]) & (part[:, None] > 0), fresh.to(torch.int32), rows)
    table[c] = rows
    lens[c] = lens[a]
    _count(refs, rows, rows >= 0, 1)
    src, dst = last[:, 0].long(), torch.where(part > 0, fresh[:, 0], last[:, 0].long())
    some = part > 0
    cache[:, dst[some]] = cache[:, src[some]]
    # every running sequence grows
    w, grow = st["growing"].long(), case["grow"]
    old = lens[w].long()
    before, need = (old + page - 1) // page, (old + grow + page - 1) // page - (old + page - 1) // page
    got = _take(st, need)
    rows = torch.where((place >= before[:, None]) & (place < (before + need)[:, None]),
                       got.gather(1, (place - before[:, None]).clamp(min=0)).to(torch.int32), table[w])
    new = (rows >= 0) & (place >= before[:, None])
    table[w] = rows
    lens[w] = (old + grow).to(torch.int32)
    _count(refs, rows, new, 1)
    at = old[:, None] + torch.arange(grow, device=DEV)[None, :]
    st["positions"].copy_(at.reshape(-1))
    st["slots"].copy_((rows.gather(1, at // page).long() * page + at % page).reshape(-1))
    # live pages move down into the free ones below the count of live pages
    live = refs != 0
    count = live.sum()
    ids = torch.arange(refs.numel(), device=DEV)
    goes = live & (ids >= count)
    holes = torch.argsort((live | (ids >= count)).to(torch.int32), stable=True)
    rank = goes.to(torch.int64).cumsum(0) - 1
    moved = torch.where(goes, holes[rank.clamp(min=0)], torch.where(live, ids, -1))
    st["moved_to"].copy_(moved)
    held = table >= 0
    table.copy_(torch.where(held, moved[table.clamp(min=0).long()].to(torch.int32), table))
    kept = refs.clone()
    refs.masked_fill_(goes, 0)
    refs[moved[goes]] = kept[goes]
    cache[:, moved[goes]] = cache[:, ids[goes]]
    return _pages_out(st)


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"prompt": _plain_prompt, "cache": _plain_cache, "pages": _plain_pages}[op](state)
    from mla_attention_prolog_gb300 import binding
    if op == "prompt":
        binding.attend_prompt(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], state["out"],
                              state["lse"], scale=state["scale"], causal=True, q_scale=state["q_scale"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "cache":
        binding.attend_cache(state["q"], state["cache"], state["page_table"], state["seq_lens"], state["out"],
                             state["lse"], state["workspace"], scale=state["scale"], shared_len=state["shared_len"])
        return {"out": state["out"], "lse": state["lse"]}
    _restore(state)
    pool = binding.PagePool(state["table"], state["lens"], state["refs"], state["case"]["page"])
    pool.release(state["ended"])
    pool.fork(state["parents"], state["children"], state["src"][:state["parents"].numel()],
              state["dst"][:state["parents"].numel()])
    binding.copy_pages(state["cache"], state["src"], state["dst"])
    pool.extend(state["growing"], state["counts"], state["slots"], state["positions"])
    pool.compact(state["moved_to"])
    binding.copy_pages(state["cache"], None, state["moved_to"])
    return _pages_out(state)


# ------------------------------------------------------------------- work

def work(case):
    if case["op"] == "prompt":
        new, total = _prompt_lens(case)
        pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
        h, hk, dqk, dv, tq, tk = case["heads"], case["kv_heads"], case["dqk"], case["dv"], sum(new), sum(total)
        q = tq * h * dqk * (2 if case["q"] == "bf16" else 1)
        q += {"bf16": 0, "int8": 4 * tq, "int8_per_head": 4 * tq * h}[case["q"]]
        return {"bytes": q + 2 * tk * hk * (dqk + dv) + 2 * tq * h * dv + 4 * tq * h + 8 * (len(new) + 1),
                "flops": 2 * h * (dqk + dv) * pairs}
    if case["op"] == "cache":
        lens, page, h, c = _cache_lens(case), case["page"], case["heads"], case["lkv"] + case["rope"]
        shared = case["shared"] // page * page
        keys = shared + sum(n - shared for n in lens)
        rows = case["batch"] * h
        table = 4 * sum(-(-n // page) for n in lens)
        return {"bytes": 2 * rows * c + 2 * keys * c + 2 * rows * case["lkv"] + 4 * rows + table + 4 * case["batch"],
                "flops": 2 * h * (c + case["lkv"]) * sum(lens)}
    page = case["page"]
    rows, lens, _, live, parents, children = _pool_plan(case)
    copies = 0
    refs = [0] * case["pages"]
    for s in live:
        for p in rows[s]:
            refs[p] += 1
    lengths = {s: lens[s] for s in live}
    for p in parents:
        copies += lens[p] % page != 0
    lengths.update({c: lens[p] for p, c in zip(parents, children)})
    fresh = sum(-(-(n + case["grow"]) // page) - -(-n // page) for n in lengths.values()) + copies
    free = [i for i, r in enumerate(refs) if r == 0]
    taken = set(free[:fresh]) | {i for i, r in enumerate(refs) if r}
    used = sum(i >= len(taken) for i in taken)
    width = -(-(case["hi"] + case["grow"]) // page) + 1
    entries = width * (case["seqs"] + case["forks"])
    book = 4 * (2 * entries + 3 * case["pages"]) + 8 * case["grow"] * len(lengths)
    return {"bytes": 2 * (copies + used) * case["layers"] * page * 2 * (case["lkv"] + case["rope"]) + book,
            "flops": entries + case["pages"]}


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    if case["op"] == "pages":
        return None   # whole numbers and copies: nothing is computed
    st = prepare(case, seed)
    if case["op"] == "prompt":
        new, total = _prompt_lens(case)
        if case["heads"] * sum(n * t for n, t in zip(new, total)) > 128 * 6000 ** 2:
            return None
        h, group = case["heads"], case["heads"] // case["kv_heads"]
        out, lse = st["out"].double(), st["lse"].double()
        a = b = 0
        for n, t in zip(new, total):
            i, j = torch.arange(n, device=DEV)[:, None], torch.arange(t, device=DEV)[None, :]
            hidden = j - (t - n) > i
            for head in range(h):
                q = st["q"][a:a + n, head].double()
                if st["q_scale"] is not None:
                    by = st["q_scale"][a:a + n].double()
                    q = q * (by[:, head] if by.dim() == 2 else by)[:, None]
                s = (q @ st["k"][b:b + t, head // group].double().t()) * st["scale"]
                s[hidden] = NEG
                z = torch.logsumexp(s, dim=1)
                out[a:a + n, head] = torch.exp(s - z[:, None]) @ st["v"][b:b + t, head // group].double()
                lse[a:a + n, head] = z
            a, b = a + n, b + t
        return {"out": out, "lse": lse}
    out, lse = st["out"].double(), st["lse"].double()
    flat = st["cache"].reshape(-1, st["cache"].shape[-1])
    for b, n in enumerate(_cache_lens(case)):
        at = torch.arange(n, device=DEV)
        rows = flat[st["page_table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]].double()
        if n == 0:
            lse[b] = NEG
            continue
        s = (st["q"][b].double() @ rows.t()) * st["scale"]
        z = torch.logsumexp(s, dim=1)
        out[b] = torch.exp(s - z[:, None]) @ rows[:, :case["lkv"]]
        lse[b] = z
    return {"out": out, "lse": lse}
