"""Cases of the paged latent cache and of the attention that reads it.

A rollout samples many answers to one prompt: the prompt's cache is filled once,
forked for every answer, read by all of them at each step, grown by the new
tokens, and given back when an answer ends.  Two kinds of operator:

* attention for a batch whose sequences share a long prefix (absorbed latent
  form: the 512-wide latent rows are keys and values), over a paged cache;
* the pages' own upkeep: copying pages, forking sequences, growing them by new
  rows, and retiring them (freeing, then compacting what is left).

`run` computes each in plain torch operations, or, where `own` is true, with the
framework's calls.  Lengths follow from the case alone; the seed sets the values
and where the pages lie.
"""
import math

import numpy as np
import torch

own = False

WIDTH = 512            # latent width
POOL = 4               # tokens of a pooled key; a page holds page / POOL of them
POOL_WIDTH = 128


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # the first steps of a short chat with four samples: latency counts
        {"name": "attend_small", "op": "attend", "groups": 1, "seqs": 4, "queries": 1, "heads": 64,
         "prefix": 203, "tail_lo": 1, "tail_hi": 17, "page": 16},
        # rollouts of a few prompts, fewer heads, drafted tokens verified two at a time, ragged lengths
        {"name": "attend_ragged", "op": "attend", "groups": 7, "seqs": 5, "queries": 3, "heads": 16,
         "prefix": 2311, "tail_lo": 3, "tail_hi": 777, "page": 32},
        # an ordinary rollout step: two prompts of 8K tokens, eight samples each
        {"name": "attend_rollout", "op": "attend", "groups": 2, "seqs": 8, "queries": 1, "heads": 64,
         "prefix": 8191, "tail_lo": 100, "tail_hi": 1024, "page": 64},
        # a large one: two prompts of 32K tokens, 32 samples each
        {"name": "attend_large", "op": "attend", "groups": 2, "seqs": 32, "queries": 1, "heads": 64,
         "prefix": 32768, "tail_lo": 500, "tail_hi": 2048, "page": 64},
        # a handful of pages moved, one layer
        {"name": "copy_small", "op": "copy", "groups": 1, "seqs": 2, "prefix": 333, "tail_lo": 5, "tail_hi": 60,
         "page": 16, "layers": 1, "count": 5, "spare": 40},
        # a prompt's worth of pages moved in four layers
        {"name": "copy_large", "op": "copy", "groups": 4, "seqs": 4, "prefix": 4096, "tail_lo": 100, "tail_hi": 900,
         "page": 64, "layers": 4, "count": 300, "spare": 320},
        # one prompt forked for four samples
        {"name": "fork_small", "op": "fork", "groups": 1, "seqs": 1, "prefix": 205, "tail_lo": 0, "tail_hi": 0,
         "page": 16, "layers": 1, "count": 4, "spare": 16},
        # a batch of prompts forked for sixteen samples each
        {"name": "fork_batch", "op": "fork", "groups": 16, "seqs": 1, "prefix": 2500, "tail_lo": 0, "tail_hi": 63,
         "page": 64, "layers": 4, "count": 256, "spare": 300},
        # one decoded token in each of 48 sequences
        {"name": "grow_decode", "op": "grow", "groups": 6, "seqs": 8, "prefix": 1111, "tail_lo": 1, "tail_hi": 300,
         "page": 64, "layers": 1, "count": 1, "spare": 64},
        # a chunk of prompt written in each of eight sequences
        {"name": "grow_chunk", "op": "grow", "groups": 8, "seqs": 1, "prefix": 2000, "tail_lo": 0, "tail_hi": 777,
         "page": 64, "layers": 2, "count": 1025, "spare": 200},
        # a few finished samples given back
        {"name": "retire_small", "op": "retire", "groups": 2, "seqs": 4, "prefix": 333, "tail_lo": 5, "tail_hi": 90,
         "page": 16, "layers": 1, "count": 3, "spare": 20},
        # a step that ends many samples, after which the pool is packed
        {"name": "retire_large", "op": "retire", "groups": 8, "seqs": 16, "prefix": 4099, "tail_lo": 50, "tail_hi": 1500,
         "page": 64, "layers": 2, "count": 64, "spare": 100},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "copy", "fork", "grow", "retire"])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        heads = rng.choice([1, 8, 16, 32, 64, 64, 128])
        while True:
            groups, seqs, queries = _log(rng, 1, 12), _log(rng, 1, 40), rng.choice([1, 1, 1, 2, 3, 5])
            prefix, tail = _log(rng, 1, 40000), _log(rng, 5, 2500)
            rows = groups * seqs * queries * heads
            # no dearer than the largest listed one, in work and in rows
            if rows * (prefix + tail) <= 4096 * 34000 and rows <= 16384 and groups * prefix <= 70000 and groups * seqs * tail <= 140000:
                break
        return {"op": op, "groups": groups, "seqs": seqs, "queries": queries, "heads": heads, "prefix": prefix,
                "tail_lo": rng.randint(min(tail, queries), tail), "tail_hi": tail, "page": page}
    while True:
        case = {"op": op, "groups": _log(rng, 1, 16), "seqs": _log(rng, 1, 16), "prefix": _log(rng, 1, 5000),
                "tail_lo": 0, "tail_hi": _log(rng, 1, 1500), "page": page, "layers": rng.choice([1, 1, 2, 3, 4])}
        live = case["groups"] * case["seqs"]
        if op == "copy":
            case["count"] = _log(rng, 1, 300)
            case["spare"] = case["count"] + rng.randint(0, 30)
        elif op == "fork":
            case["count"] = _log(rng, 1, 256)
            case["spare"] = case["count"] + rng.randint(0, 30)
        elif op == "grow":
            case["count"] = _log(rng, 1, 1100)
            case["spare"] = live * (case["count"] // page + 1) + rng.randint(0, 30)
        else:
            case["count"] = rng.randint(1, live)
            case["spare"] = rng.randint(0, 100)
        lens = _lens(case)
        tokens = int(lens.sum())
        if op == "copy" and case["count"] > case["groups"] * (case["prefix"] // page):
            continue
        if (tokens + case["spare"] * page) * case["layers"] <= 300000 and live * case["count"] <= (9000 if op == "grow" else 1 << 30):
            return case


# ---- lengths and pages (from the case; `rng` places the pages) ---------------

def _spread(n, lo, hi):
    """n whole numbers over lo..hi, uneven, from the case alone."""
    return lo + np.floor((hi - lo + 1) * ((np.arange(n) + 1) * 0.6180339887498949 % 1.0)).astype(np.int64)


def _prefixes(case):
    """Shared tokens of each group: the case's length, a little less from group to group."""
    return np.maximum(1, case["prefix"] - _spread(case["groups"], 0, case["prefix"] // 5) * (np.arange(case["groups"]) > 0))


def _lens(case):
    """Length of each sequence, its group's prefix included."""
    n = case["groups"] * case["seqs"]
    return np.repeat(_prefixes(case), case["seqs"]) + _spread(n, case["tail_lo"], case["tail_hi"])


def _ceil(a, b):
    return -(-a // b)


def _pool(case, rng, rows, spare, room):
    """Page table [rows, wide], lengths, references and free pages of sequences that share their groups' whole pages."""
    page, seqs = case["page"], case["seqs"]
    lens, shared = _lens(case), _prefixes(case) // page          # whole pages that a group shares
    wide = int(_ceil(lens.max() + room, page))
    own_pages = _ceil(lens, page) - np.repeat(shared, seqs)
    used = int(shared.sum() + own_pages.sum())
    n_pages = used + spare
    ids = rng.permutation(n_pages)
    col = np.arange(wide)[None, :]
    first_s = np.concatenate([[0], np.cumsum(shared)[:-1]])
    first_o = shared.sum() + np.concatenate([[0], np.cumsum(own_pages)[:-1]])
    sh, fs = np.repeat(shared, seqs)[:, None], np.repeat(first_s, seqs)[:, None]
    at = np.where(col < sh, fs + col, first_o[:, None] + col - sh)
    table = np.full((rows, wide), -1, np.int32)
    n = len(lens)
    live = col < _ceil(lens, page)[:, None]
    table[:n] = np.where(live, ids[np.where(live, at, 0)], -1)
    length = np.zeros(rows, np.int32)
    length[:n] = lens
    refs = np.bincount(table[:n][live], minlength=n_pages).astype(np.int32)
    free = np.full(n_pages, -1, np.int32)
    free[:spare] = ids[used:]
    return table, length, refs, free, spare


def _normal(shape, gen):
    """bf16 normals, drawn on the GPU."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return out.normal_(generator=gen)


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    page, lens = case["page"], _lens(case)
    n = len(lens)
    if case["op"] == "attend":
        table, length, refs, _, _ = _pool(case, rng, n, 3, 0)
        n_pages = len(refs)
        st = {"op": "attend", "scale": WIDTH ** -0.5, "heads": case["heads"], "queries": case["queries"],
              "groups": case["groups"], "seqs": case["seqs"], "page": page,
              "longest_prefix": int(_prefixes(case).max()), "longest_tail": int((lens - np.repeat(_prefixes(case), case["seqs"])).max())}
        rows = n * case["queries"]
        # sharper than unit scores, as trained queries are
        st["q"] = _normal((rows, case["heads"], WIDTH), gen) * 2
        st["kv"] = _normal((n_pages, page, WIDTH), gen)
        # a prefix that ends inside a page: each sequence has a copy of that page's rows, as forking leaves it
        cut = np.repeat(_prefixes(case), case["seqs"])
        b, first = np.flatnonzero(cut % page > 0), np.arange(n) // case["seqs"] * case["seqs"]
        ids, at = table[b, cut[b] // page], table[first[b], cut[b] // page]
        ids, at, part = (torch.from_numpy(a.astype(np.int64)).cuda() for a in (ids, at, cut[b] % page))
        copied = torch.arange(page, device="cuda") < part[:, None]
        st["kv"][ids] = torch.where(copied[:, :, None], st["kv"][at], st["kv"][ids])
        st["table"] = torch.from_numpy(table).cuda()
        st["lens"] = torch.from_numpy(length).cuda()
        st["prefix"] = torch.from_numpy(_prefixes(case).astype(np.int32)).cuda()
        st["cu_q"] = torch.arange(0, rows + 1, case["queries"], dtype=torch.int32, device="cuda")
        st["cu_groups"] = torch.arange(0, n + 1, case["seqs"], dtype=torch.int32, device="cuda")
        return st
    count, layers = case["count"], case["layers"]
    rows = n + (count if case["op"] == "fork" else 2)
    room = count if case["op"] == "grow" else 0
    table, length, refs, free, n_free = _pool(case, rng, rows, case["spare"], room)
    n_pages = len(refs)
    # all of the pool's whole numbers in one buffer, so that a pass can begin from the same pool again
    parts = [table.reshape(-1), length, refs, free, np.array([n_free], np.int32)]
    st = {"op": case["op"], "page": page, "n_pages": n_pages, "rows": rows, "wide": table.shape[1]}
    st["start"] = torch.from_numpy(np.concatenate(parts).astype(np.int32)).cuda()
    st["meta"] = st["start"].clone()
    cut = np.cumsum([0] + [len(p) for p in parts])
    st["table"] = st["meta"][cut[0]:cut[1]].view(rows, -1)
    st["lens"], st["refs"], st["free"], st["n_free"] = (st["meta"][cut[i]:cut[i + 1]] for i in range(1, 5))
    st["latents"] = _normal((layers, n_pages, page, WIDTH), gen)
    st["pooled"] = _normal((layers, n_pages, page // POOL, POOL_WIDTH), gen)
    as_int = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()  # noqa: E731
    if case["op"] == "copy":
        st["src"] = as_int(rng.permutation(np.flatnonzero(refs > 0))[:count])
        st["dst"] = as_int(rng.permutation(free[:n_free])[:count])
    elif case["op"] == "fork":
        st["parents"] = as_int(np.sort(rng.randint(0, n, count)))
        st["children"] = as_int(n + rng.permutation(count))
    elif case["op"] == "grow":
        st["which"] = as_int(rng.permutation(n))
        # each sequence by `count` tokens, all but the first a little less
        more = np.maximum(1, count - _spread(n, 0, count // 3) * (np.arange(n) > 0))
        st["more"], st["cu_new"] = as_int(more), as_int(np.concatenate([[0], np.cumsum(more)]))
        st["total"] = int(more.sum())
        st["new"] = _normal((layers, st["total"], WIDTH), gen)
    else:
        st["which"] = as_int(rng.permutation(n)[:count])
    if own:
        # the handle that a program makes once for its pool: the same tensors, checked
        import sparse_attention_kpool_compress_gb300 as K
        st["pages"] = K.KPoolPages(st["table"], st["lens"], st["refs"], st["free"], st["n_free"], page)
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    if st["op"] == "attend":
        return _attend_own(st) if own else _attend(st)
    st["meta"].copy_(st["start"])        # the pool as it was before the last pass
    extra = (_upkeep_own if own else _upkeep)(st)
    # (behind its first n_free entries the free list stays as it was)
    return {k: st[k] for k in ("table", "lens", "refs", "n_free", "free", "latents", "pooled")} | extra


def _attend_own(st):
    import sparse_attention_kpool_compress_gb300 as K
    return K.kpool_shared_prefix_mla_fwd(st["q"], st["kv"], st["table"], st["lens"], st["cu_q"], st["cu_groups"],
                                         st["prefix"], st["scale"])


def _upkeep_own(st):
    import sparse_attention_kpool_compress_gb300 as K
    stores = [st["latents"], st["pooled"]]
    if st["op"] == "copy":
        K.kpool_pages_copy(st["src"], st["dst"], stores)
    elif st["op"] == "fork":
        K.kpool_pages_fork(st["pages"], st["parents"], st["children"], stores)
    elif st["op"] == "grow":
        begin = K.kpool_pages_extend(st["pages"], st["which"], st["more"])
        K.kpool_pages_write(st["pages"], st["which"], begin, st["cu_new"], st["new"], st["latents"])
        return {"begin": begin}
    else:
        K.kpool_pages_free(st["pages"], st["which"])
        K.kpool_pages_compact(st["pages"], stores)
    return {}


def _attend(st):
    """Scores of the shared tokens once for a group's queries, of the rest for each sequence; one softmax over both."""
    G, S, Q, H, page = st["groups"], st["seqs"], st["queries"], st["heads"], st["page"]
    B = G * S
    flat = st["kv"].reshape(-1, WIDTH)
    table, lens = st["table"].long(), st["lens"].long()
    prefix = st["prefix"].long()
    q = st["q"].float() * st["scale"]
    seen = lens[:, None] - Q + 1 + torch.arange(Q, device="cuda")              # [B, Q]: tokens a query sees
    at = torch.arange(st["longest_prefix"], device="cuda")
    t = table[::S]                                                            # a group's first sequence
    ids = t.gather(1, (at // page).expand(G, -1).clamp(max=t.shape[1] - 1)).clamp(min=0)
    k1 = flat[ids * page + at % page].float()                                 # [G, P, 512]
    s1 = torch.matmul(q.view(G, S * Q * H, WIDTH), k1.transpose(1, 2)).view(B, Q, H, -1)
    end = torch.minimum(prefix.repeat_interleave(S, output_size=B)[:, None], seen)
    s1.masked_fill_((at >= end[:, :, None])[:, :, None, :], -math.inf)
    at2 = prefix.repeat_interleave(S, output_size=B)[:, None] + torch.arange(max(1, st["longest_tail"]), device="cuda")
    ids = table.gather(1, (at2 // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
    k2 = flat[ids * page + at2 % page].float()                                # [B, R, 512]
    s2 = torch.matmul(q.view(B, Q * H, WIDTH), k2.transpose(1, 2)).view(B, Q, H, -1)
    s2.masked_fill_((at2[:, None, :] >= seen[:, :, None])[:, :, None, :], -math.inf)
    top = torch.maximum(s1.amax(-1), s2.amax(-1))
    ref = torch.where(top.isinf(), 0.0, top)[..., None]
    s1.sub_(ref).exp_()
    s2.sub_(ref).exp_()
    total = s1.sum(-1) + s2.sum(-1)
    o = torch.matmul(s1.view(G, S * Q * H, -1), k1).view(B, Q * H, WIDTH) + torch.matmul(s2.view(B, Q * H, -1), k2)
    o = o.view(B * Q, H, WIDTH) / torch.where(total > 0, total, 1.0).view(B * Q, H, 1)
    return o.to(torch.bfloat16), (ref[..., 0] + total.log()).view(B * Q, H)


def _upkeep(st):
    return {"copy": _copy, "fork": _fork, "grow": _grow, "retire": _retire}[st["op"]](st)


def _copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    st["latents"].index_copy_(1, dst, st["latents"].index_select(1, src))
    st["pooled"].index_copy_(1, dst, st["pooled"].index_select(1, src))
    return {}


def _copy_rows(store, src, dst, rows):
    """The first `rows[i]` rows of page src[i] to dst[i], in all layers."""
    part = torch.arange(store.shape[2], device="cuda") < rows[:, None]
    store.index_copy_(1, dst, torch.where(part[None, :, :, None], store.index_select(1, src), store.index_select(1, dst)))


def _fork(st):
    page, parents, children = st["page"], st["parents"].long(), st["children"].long()
    length = st["lens"][parents].long()
    part = length % page
    need = part > 0
    rank = need.cumsum(0) - 1
    fresh = torch.where(need, st["free"][(st["n_free"].long() - 1 - rank).clamp(0, st["n_pages"] - 1)].long(), 0)
    rows = st["table"][parents].long()
    col = torch.arange(st["wide"], device="cuda")[None, :]
    whole = col < (length // page)[:, None]
    last = (length // page).clamp(max=st["wide"] - 1)[:, None]
    src = rows.gather(1, last)[:, 0]
    st["refs"].index_add_(0, rows.clamp(min=0).view(-1), whole.view(-1).int())
    st["refs"].index_add_(0, fresh, need.int())
    made = torch.where(whole, rows, torch.where((col == last) & need[:, None], fresh[:, None], -1))
    # columns behind a child's last page stay as they were
    st["table"][children] = torch.where(col < _ceil(length, page)[:, None], made, st["table"][children].long()).int()
    st["lens"][children] = length.int()
    st["n_free"] -= need.sum().int()
    src, dst, part = src[need], fresh[need], part[need]
    _copy_rows(st["latents"], src, dst, part)
    _copy_rows(st["pooled"], src, dst, _ceil(part, POOL))
    return {}


def _grow(st):
    page, which, more = st["page"], st["which"].long(), st["more"].long()
    begin = st["lens"][which].long()
    had, has = _ceil(begin, page), _ceil(begin + more, page)
    base = (has - had).cumsum(0) - (has - had)
    col = torch.arange(st["wide"], device="cuda")[None, :]
    new = (col >= had[:, None]) & (col < has[:, None])
    at = st["n_free"].long() - 1 - (base[:, None] + col - had[:, None])
    got = torch.where(new, st["free"][at.clamp(0, st["n_pages"] - 1)].long(), 0)
    table = torch.where(new, got, st["table"][which].long())
    st["table"][which] = table.int()
    st["refs"].index_add_(0, got.view(-1), new.view(-1).int())
    st["n_free"] -= (has - had).sum().int()
    st["lens"][which] = (begin + more).int()
    seq = torch.repeat_interleave(torch.arange(len(which), device="cuda"), more, output_size=st["total"])
    pos = begin[seq] + torch.arange(st["total"], device="cuda") - st["cu_new"].long()[seq]
    where = table[seq, pos // page] * page + pos % page
    st["latents"].view(st["latents"].shape[0], -1, WIDTH).index_copy_(1, where, st["new"])
    return {"begin": begin.int()}


def _retire(st):
    page, n, which = st["page"], st["n_pages"], st["which"].long()
    # free: one reference less for each page (which pages that leaves free, the compaction below sees)
    col = torch.arange(st["wide"], device="cuda")[None, :]
    held = col < _ceil(st["lens"][which].long(), page)[:, None]
    st["refs"].index_add_(0, st["table"][which].long().clamp(min=0).view(-1), -held.view(-1).int())
    st["table"][which] = torch.where(held, -1, st["table"][which])
    st["lens"][which] = 0
    # compact: the live pages above their count move, in order, into the free pages below it
    live = st["refs"] > 0
    k = live.sum()
    i = torch.arange(n, device="cuda")
    src, dst = (live & (i >= k)).nonzero()[:, 0], (~live & (i < k)).nonzero()[:, 0]
    to = i.index_copy(0, src, dst)
    used = col < _ceil(st["lens"].long(), page)[:, None]
    st["table"].copy_(torch.where(used, to[st["table"].long().clamp(min=0)], st["table"].long()))
    st["refs"].index_copy_(0, dst, st["refs"][src])
    st["refs"].index_fill_(0, src, 0)
    st["latents"].index_copy_(1, dst, st["latents"].index_select(1, src))
    st["pooled"].index_copy_(1, dst, st["pooled"].index_select(1, src))
    st["free"].copy_(torch.where(i < n - k, n - 1 - i, st["free"]))
    st["n_free"].copy_((n - k).view(1))
    return {}


# ---- what a pass cannot do without ---------------------------------------------

def _page_bytes(case):
    return case["layers"] * (case["page"] * WIDTH * 2 + case["page"] // POOL * POOL_WIDTH * 2)


def work(case):
    lens, page = _lens(case), case["page"]
    if case["op"] == "attend":
        pre = _prefixes(case)
        rows = len(lens) * case["queries"] * case["heads"]
        # the query at place i of the last `queries` sees all but the queries - 1 - i last tokens
        seen = sum(int(np.maximum(lens - i, 0).sum()) for i in range(case["queries"])) * case["heads"]
        tokens = int(pre.sum() + (lens - np.repeat(pre, case["seqs"])).sum())
        return {"bytes": rows * (4 * WIDTH + 4) + tokens * 2 * WIDTH + 4 * tokens // page, "flops": 4 * WIDTH * seen}
    if case["op"] == "copy":
        return {"bytes": 2 * case["count"] * _page_bytes(case)}
    if case["op"] == "fork":
        # parents are drawn evenly: on average half a page is copied, and a table row read and written
        return {"bytes": case["count"] * (_page_bytes(case) + 16 * int(lens.mean() / page) + 16)}
    if case["op"] == "grow":
        more = np.maximum(1, case["count"] - _spread(len(lens), 0, case["count"] // 3) * (np.arange(len(lens)) > 0))
        return {"bytes": int(more.sum()) * 4 * WIDTH * case["layers"] + 24 * len(lens)}
    # the share of the pages that is freed has to be refilled from above: of n pages with a share f free, f (1 - f) n move
    pages = int((_prefixes(case) // page).sum() + (_ceil(lens, page) - np.repeat(_prefixes(case) // page, case["seqs"])).sum())
    n = pages + case["spare"]
    gone = pages * case["count"] / len(lens) * (1 - 1 / case["seqs"] if case["count"] < len(lens) else 1)
    f = (gone + case["spare"]) / n
    return {"bytes": 2 * f * (1 - f) * n * _page_bytes(case) + 8 * n + 8 * int(_ceil(lens, page).sum())}


# ---- the definition, in 64 bits --------------------------------------------------

def exact(case, seed):
    """Attention: each sequence's tokens listed one after another and attended by its queries alone.  Upkeep moves values
    and computes none."""
    if case["op"] != "attend":
        return None
    st = prepare(case, seed)
    H, Q, page = case["heads"], case["queries"], case["page"]
    outs, logs = [], []
    for b, length in enumerate(_lens(case)):
        pos = torch.arange(int(length), device="cuda")
        rows = st["kv"][st["table"][b].long()[pos // page], pos % page].double()
        scores = torch.einsum("qhd,ld->qhl", st["q"][b * Q:(b + 1) * Q].double(), rows) / math.sqrt(WIDTH)
        last = int(length) - Q + torch.arange(Q, device="cuda")
        scores = scores.masked_fill((pos[None, :] > last[:, None])[:, None, :], -math.inf)
        lse = torch.logsumexp(scores, -1)
        w = torch.where(lse.isinf()[..., None], 0.0, torch.exp(scores - torch.where(lse.isinf(), 0.0, lse)[..., None]))
        outs.append(torch.einsum("qhl,ld->qhd", w, rows))
        logs.append(lse)
    return torch.cat(outs), torch.cat(logs)
