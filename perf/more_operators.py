"""Cases of the sparse latent attention at both ends of a reinforcement-learning step.

A rollout extends sequences in a paged cache and attends, from each chunk of new
tokens, the pools that the indexer chose; the training step then sends gradients
back through the same attention over the same choice.  Two kinds of operator, in
the absorbed latent form (64 heads, 512-wide latent rows that are keys and values):

* "grad":  the backward pass of the attention over listed tokens, which recomputes
  the probabilities from the saved log-sums: gradients of the queries and of the
  latent rows;
* "paged": the forward pass for a chunk of new tokens (one, a few drafted ones, or a
  piece of a prompt) over a paged cache.

`run` computes each in plain torch operations, or, where `own` is true, with the
framework's calls.  Lengths follow from the case alone; the seed sets the values,
the choice of pools and where the pages lie.
"""
import math

import numpy as np
import torch

own = False

HEADS = 64
WIDTH = 512            # latent width
SCALE = WIDTH ** -0.5


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # a short answer on its own: every token is visible, latency counts
        {"name": "grad_small", "op": "grad", "form": "pools", "rows": 61, "docs": 1, "keys": 0, "pool": 4, "topk": 2048,
         "tail": True, "lse": False},
        # packed answers of uneven lengths, pools of eight, a small budget
        {"name": "grad_packed", "op": "grad", "form": "pools", "rows": 3001, "docs": 7, "keys": 0, "pool": 8, "topk": 512,
         "tail": True, "lse": False},
        # lists from another selector: odd width, holes, repeated tokens, rows without any; the log-sums have gradients too
        {"name": "grad_lists", "op": "grad", "form": "lists", "rows": 1111, "docs": 1, "keys": 5003, "pool": 1, "topk": 333,
         "tail": False, "lse": True},
        # answers trained on behind long prompts: few queries, many keys
        {"name": "grad_answers", "op": "grad", "form": "at", "rows": 2048, "docs": 3, "keys": 30011, "pool": 4, "topk": 2048,
         "tail": True, "lse": False},
        # an ordinary training sequence
        {"name": "grad_8k", "op": "grad", "form": "pools", "rows": 8192, "docs": 1, "keys": 0, "pool": 4, "topk": 2048,
         "tail": True, "lse": False},
        # a long training sequence
        {"name": "grad_32k", "op": "grad", "form": "pools", "rows": 32768, "docs": 1, "keys": 0, "pool": 4, "topk": 2048,
         "tail": True, "lse": False},
        # one sequence decodes a token: latency counts
        {"name": "paged_single", "op": "paged", "seqs": 1, "queries": 1, "context_lo": 9001, "context_hi": 9001, "page": 64,
         "layers": 1, "pool": 4, "topk": 2048, "tail": True},
        # drafted tokens verified five at a time, ragged contexts, some below the budget
        {"name": "paged_drafts", "op": "paged", "seqs": 7, "queries": 5, "context_lo": 33, "context_hi": 7777, "page": 16,
         "layers": 2, "pool": 4, "topk": 1024, "tail": True},
        # a decode step of a rollout batch
        {"name": "paged_decode", "op": "paged", "seqs": 128, "queries": 1, "context_lo": 4000, "context_hi": 24000, "page": 64,
         "layers": 1, "pool": 4, "topk": 2048, "tail": True},
        # pieces of three prompts, pools of eight
        {"name": "paged_chunk", "op": "paged", "seqs": 3, "queries": 333, "context_lo": 2500, "context_hi": 40000, "page": 32,
         "layers": 2, "pool": 8, "topk": 2048, "tail": True},
        # a large piece of a long prompt
        {"name": "paged_prompt", "op": "paged", "seqs": 1, "queries": 8192, "context_lo": 65536, "context_hi": 65536, "page": 128,
         "layers": 1, "pool": 4, "topk": 2048, "tail": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = {"op": rng.choice(["grad", "paged"]), "pool": rng.choice([1, 2, 4, 4, 8, 16]), "tail": rng.random() < 0.8}
        case["topk"] = max(case["pool"], _log(rng, 16, 2048) // case["pool"] * case["pool"])
        if case["op"] == "grad":
            case["form"] = rng.choice(["pools", "pools", "at", "lists"])
            case["rows"], case["lse"] = _log(rng, 1, 16384), rng.random() < 0.3
            case["docs"] = 1 if case["form"] == "lists" else min(case["rows"], _log(rng, 1, 40))
            case["keys"] = 0 if case["form"] == "pools" else case["rows"] + _log(rng, 1, 60000)
            if case["form"] == "lists":
                case["pool"], case["tail"] = 1, False
            # the choice is drawn from a score for each row and pool
            if case["rows"] * max(case["rows"], case["keys"]) // case["pool"] <= 1 << 28:
                return case
        else:
            case["seqs"], case["queries"], case["page"] = _log(rng, 1, 256), _log(rng, 1, 4096), rng.choice([16, 32, 64, 128])
            case["layers"], hi = rng.choice([1, 1, 2, 3]), _log(rng, 20, 100000)
            case["context_hi"] = max(hi, case["queries"])
            case["context_lo"] = max(case["queries"], rng.randint(hi // 4, hi))
            tokens, rows = case["seqs"] * case["context_hi"], case["seqs"] * case["queries"]
            if tokens * case["layers"] <= 4000000 and rows <= 8192 and rows * case["context_hi"] // case["pool"] <= 1 << 28:
                return case


# ---- positions (from the case alone) -----------------------------------------

def _spread(n, lo, hi):
    """n whole numbers over lo..hi, uneven."""
    return lo + np.floor((hi - lo + 1) * ((np.arange(n) + 1) * 0.6180339887498949 % 1.0)).astype(np.int64)


def _split(total, n):
    """n uneven parts of `total`, each at least 1 where there are enough."""
    share = _spread(n, 1000, 3000).astype(np.float64)
    cut = np.floor(np.cumsum(share) / share.sum() * (total - n)).astype(np.int64)
    parts = 1 + np.diff(np.concatenate([[0], cut]))
    parts[-1] += total - parts.sum()
    return parts


def _layout(case):
    """(queries, keys) of each sequence; its queries are its last tokens."""
    if case["op"] == "paged":
        n = case["seqs"]
        # all but the first have a little fewer queries
        queries = np.maximum(1, case["queries"] - _spread(n, 0, case["queries"] // 4) * (np.arange(n) > 0))
        return queries, np.maximum(queries, _spread(n, case["context_lo"], case["context_hi"]))
    queries = _split(case["rows"], case["docs"])
    if case["form"] == "pools":
        return queries, queries
    return queries, queries + (_split(case["keys"] - case["rows"] + case["docs"], case["docs"]) - 1)


def _positions(queries, keys):
    """For each query row its sequence and its position there."""
    seq = np.repeat(np.arange(len(queries)), queries)
    return seq, np.concatenate([np.arange(k - q, k) for q, k in zip(queries, keys)])


def _listed_tokens(case):
    """How many tokens all rows list together."""
    if case["op"] == "grad" and case["form"] == "lists":
        return case["rows"] * case["topk"] * 0.8           # about a fifth are holes
    _, tau = _positions(*_layout(case))
    pool = case["pool"]
    return int((np.minimum((tau + 1) // pool, case["topk"] // pool) * pool + ((tau + 1) % pool if case["tail"] else 0)).sum())


# ---- inputs --------------------------------------------------------------------

def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _normal(shape, gen, size=1.0):
    """bf16 normals, drawn on the GPU."""
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, size, generator=gen)


def _choose(case, queries, keys, gen):
    """Selected pools of each row, ascending, as packed pool numbers with -1 behind them.  Some pools are liked by a whole
    sequence, some by neighbouring queries, recent ones by all: neighbours choose much the same."""
    pool, budget = case["pool"], case["topk"] // case["pool"]
    first = np.concatenate([[0], np.cumsum(keys // pool)])
    out = torch.full((int(queries.sum()), budget), -1, dtype=torch.int32, device="cuda")
    row = 0
    for d, (nq, nk) in enumerate(zip(queries, keys)):
        n_pools = int(nk // pool)
        if n_pools:
            at = torch.arange(n_pools, device="cuda")
            liked = torch.empty(n_pools, device="cuda").normal_(generator=gen)
            step = max(1, min(int(nq), (1 << 25) // n_pools // 16 * 16))
            for lo in range(0, int(nq), step):
                n = min(step, int(nq) - lo)
                tau = int(nk - nq) + lo + torch.arange(n, device="cuda")
                near = torch.empty(-(-n // 16), n_pools, device="cuda").normal_(generator=gen)
                score = torch.empty(n, n_pools, device="cuda").normal_(0.0, 0.5, generator=gen)
                score += near.repeat_interleave(16, 0)[:n] + liked
                score += 4.0 * (at > (tau[:, None] - 128) // pool)
                seen = (tau + 1) // pool
                score.masked_fill_(at >= seen[:, None], -math.inf)
                top, which = score.topk(min(budget, n_pools), dim=1)
                which = torch.where(top.isinf(), n_pools, which).sort(1).values
                out[row + lo:row + lo + n, :which.shape[1]] = torch.where(which < n_pools, which + int(first[d]), -1).int()
        row += int(nq)
    return out, _ints(first)


def _tokens(case, chosen, tau, first_pool):
    """[rows, budget * pool + pool - 1] token positions in the rows' sequences, -1 where there is none."""
    pool = case["pool"]
    local = chosen.long() - first_pool[:, None]
    toks = local[:, :, None] * pool + torch.arange(pool, device="cuda")
    toks = torch.where(chosen[:, :, None] >= 0, toks, -1).flatten(1)
    if not case["tail"]:
        return toks
    back = tau[:, None] - torch.arange(pool - 1, device="cuda")
    return torch.cat([toks, torch.where(torch.arange(pool - 1, device="cuda") < (tau[:, None] + 1) % pool, back, -1)], 1)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    queries, keys = _layout(case)
    n, rows = len(queries), int(queries.sum())
    seq, tau = _positions(queries, keys)
    # sharper than unit scores, as trained queries are
    st = {"op": case["op"], "pool": case["pool"], "topk": case["topk"], "tail": case["tail"],
          "q": _normal((rows, HEADS, WIDTH), gen, 2.0)}
    st["seq"], st["tau"] = torch.from_numpy(seq).cuda(), torch.from_numpy(tau).cuda()
    st["cu_q"], st["pos"] = _ints(np.concatenate([[0], np.cumsum(queries)])), _ints(keys - queries)
    if case["op"] == "grad" and case["form"] == "lists":
        st["form"] = "lists"
        n_keys = int(keys.sum())
        toks = torch.randint(0, n_keys, (rows, case["topk"]), generator=gen, device="cuda", dtype=torch.int32)
        hole = torch.rand(rows, case["topk"], generator=gen, device="cuda") < 0.2
        if rows > 16:                                    # (of a few rows each has tokens)
            hole |= torch.rand(rows, 1, generator=gen, device="cuda") < 0.02
        st["toks"] = torch.where(hole, -1, toks)
    else:
        st["chosen"], st["cu_pools"] = _choose(case, queries, keys, gen)
    if case["op"] == "paged":
        page, layers = case["page"], case["layers"]
        used = -(-keys // page)
        n_pages = int(used.sum()) + 3
        ids = rng.permutation(n_pages)
        col, at = np.arange(int(used.max()))[None, :], np.concatenate([[0], np.cumsum(used)[:-1]])[:, None]
        table = np.where(col < used[:, None], ids[np.minimum(at + col, n_pages - 1)], -1)
        st["table"], st["lens"], st["page"] = _ints(table), _ints(keys), page
        # one layer of a store whose pages hold all layers
        st["kv"] = _normal((n_pages, layers, page, WIDTH), gen)[:, layers - 1]
        return st
    st["form"] = case["form"]
    st["cu_k"] = _ints(np.concatenate([[0], np.cumsum(keys)]))
    st["kv"] = _normal((int(keys.sum()), WIDTH), gen)
    # what the forward pass left, and the gradients that come back to it
    o, lse = [], []
    for lo, hi in _blocks(rows, st):
        o_, lse_ = _attend_rows(st, lo, hi)
        o.append(o_)
        lse.append(lse_)
    st["o"], st["lse"] = torch.cat(o), torch.cat(lse)
    st["d_o"] = _normal((rows, HEADS, WIDTH), gen, 0.05)
    st["d_lse"] = torch.empty(rows, HEADS, device="cuda").normal_(0.0, 0.5, generator=gen) if case["lse"] else None
    return st


# ---- one pass ----------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    rows = st["q"].shape[0]
    if st["op"] == "paged":
        parts = [_attend_rows(st, lo, hi) for lo, hi in _blocks(rows, st)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    d_kv = torch.zeros(st["kv"].shape, device="cuda")
    d_q = torch.cat([_grad_rows(st, lo, hi, d_kv) for lo, hi in _blocks(rows, st)])
    return d_q, d_kv.to(torch.bfloat16)


def _run_own(st):
    import sparse_attention_kpool_compress_gb300 as K
    if st["op"] == "paged":
        return K.kpool_sparse_mla_fwd_pools_paged(
            st["q"], st["kv"], st["table"], st["lens"], st["chosen"], st["pool"], st["topk"], SCALE, st["cu_q"], st["pos"],
            st["cu_pools"], always_select_tail=st["tail"])
    saved = st["o"], st["lse"], st["d_o"]
    if st["form"] == "lists":
        return K.kpool_sparse_mla_bwd(st["q"], st["kv"], st["toks"], *saved, SCALE, d_lse=st["d_lse"])
    if st["form"] == "at":
        return K.kpool_sparse_mla_bwd_pools_at(
            st["q"], st["kv"], st["chosen"], *saved, st["pool"], st["topk"], SCALE, st["cu_q"], st["pos"], st["cu_k"],
            st["cu_pools"], always_select_tail=st["tail"], d_lse=st["d_lse"])
    return K.kpool_sparse_mla_bwd_pools(
        st["q"], st["kv"], st["chosen"], *saved, st["pool"], st["topk"], SCALE, st["cu_k"], st["cu_pools"],
        always_select_tail=st["tail"], d_lse=st["d_lse"])


def _blocks(rows, st):
    """Row ranges whose listed latent rows take about half a GiB in 32 bits."""
    wide = st["toks"].shape[1] if "toks" in st else st["topk"] + st["pool"]
    step = max(1, (1 << 29) // (wide * WIDTH * 4))
    return [(lo, min(rows, lo + step)) for lo in range(0, rows, step)]


def _where(st, lo, hi):
    """Where the tokens of rows lo..hi lie in the flat latent rows (0 for none), which there are, and the flat rows."""
    if "toks" in st:
        toks = st["toks"][lo:hi].long()
        return toks.clamp(min=0), toks >= 0, st["kv"]
    seq, tau = st["seq"][lo:hi], st["tau"][lo:hi]
    toks = _tokens(st, st["chosen"][lo:hi], tau, st["cu_pools"].long()[seq])
    at = toks.clamp(min=0)
    if st["op"] == "paged":
        page, kv = st["page"], st["kv"]
        ids = st["table"].long()[seq[:, None], at // page]
        apart = kv.stride(0) // WIDTH
        flat = kv.as_strided(((kv.shape[0] - 1) * apart + page, WIDTH), (WIDTH, 1))
        return ids * apart + at % page, toks >= 0, flat
    return at + st["cu_k"].long()[seq][:, None], toks >= 0, st["kv"]


def _attend_rows(st, lo, hi):
    at, valid, flat = _where(st, lo, hi)
    keys = flat[at].float()                                               # [rows, tokens, 512]
    s = torch.matmul(st["q"][lo:hi].float() * SCALE, keys.transpose(1, 2))
    s.masked_fill_(~valid[:, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, keys) / torch.where(total > 0, total, 1.0)
    return o.to(torch.bfloat16), (top + total.log())[..., 0]


def _grad_rows(st, lo, hi, d_kv):
    """Gradients of the queries lo..hi; those of the latent rows are added to d_kv."""
    at, valid, flat = _where(st, lo, hi)
    keys = flat[at].float()
    q, d_o = st["q"][lo:hi].float() * SCALE, st["d_o"][lo:hi].float()
    p = torch.matmul(q, keys.transpose(1, 2))
    p.masked_fill_(~valid[:, None, :], -math.inf)
    lse = st["lse"][lo:hi, :, None]
    p.sub_(torch.where(lse.isinf(), 0.0, lse)).exp_()
    back = (d_o * st["o"][lo:hi].float()).sum(-1)
    if st["d_lse"] is not None:
        back = back - st["d_lse"][lo:hi]
    ds = torch.matmul(d_o, keys.transpose(1, 2)).sub_(back[..., None]).mul_(p)
    d_q = torch.matmul(ds, keys) * SCALE
    d_keys = torch.matmul(p.transpose(1, 2), d_o).baddbmm_(ds.transpose(1, 2), q)
    d_kv.index_add_(0, at[valid], d_keys[valid])
    return d_q.to(torch.bfloat16)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    queries, keys = _layout(case)
    rows, listed_tokens = int(queries.sum()), _listed_tokens(case)
    # latent rows that some query lists, each once; the choice itself
    read = min(int(keys.sum()), listed_tokens)
    choice = 4 * (rows * case["topk"] // case["pool"])
    if case["op"] == "paged":
        return {"bytes": rows * HEADS * (4 * WIDTH + 4) + read * 2 * WIDTH + choice + 4 * read // case["page"],
                "flops": 4 * HEADS * WIDTH * listed_tokens}
    # q, o and d_o in, d_q out; the log-sums; latent rows in, gradients of all of them out
    return {"bytes": rows * HEADS * (8 * WIDTH + 4 + (4 if case["lse"] else 0)) + (read + int(keys.sum())) * 2 * WIDTH + choice,
            "flops": 10 * HEADS * WIDTH * listed_tokens}


# ---- the definition, in 64 bits --------------------------------------------------

def _row_lists(case, st):
    """Each row's latent rows [rows, tokens] in one flat array, by the definition: a row's pools and its tail as a truth value
    for every token that there is, or the listed tokens one by one."""
    if "toks" in st:
        return [r[r >= 0].long() for r in st["toks"]]
    pool, out = case["pool"], []
    cu_pools, chosen = st["cu_pools"].cpu().numpy(), st["chosen"].cpu().numpy()
    queries, keys = _layout(case)
    starts = np.concatenate([[0], np.cumsum(keys)])
    table = st["table"].cpu().numpy().astype(np.int64) if case["op"] == "paged" else None
    for r, (d, tau) in enumerate(zip(*_positions(queries, keys))):
        mine = chosen[r][chosen[r] >= 0] - cu_pools[d]
        seen = np.zeros(tau + 1, bool)
        for s in range(pool):
            seen[mine * pool + s] = True
        if case["tail"]:
            seen[(tau + 1) // pool * pool:] = True
        toks = np.flatnonzero(seen)
        if table is None:
            out.append(toks + starts[d])
        else:
            out.append(table[d][toks // st["page"]] * st["page"] + toks % st["page"])
    return out


def exact(case, seed):
    # (the 64-bit products of more would take longer than some seconds)
    if _listed_tokens(case) > 18000000:
        return None
    st = prepare(case, seed)
    kv = st["kv"].reshape(-1, WIDTH).double()
    lists = _row_lists(case, st)
    outs, logs = [], []
    d_kv = torch.zeros_like(kv)
    for r, toks in enumerate(lists):
        toks = torch.as_tensor(toks, device="cuda")
        keys, q = kv[toks], st["q"][r].double()
        scores = q @ keys.T / math.sqrt(WIDTH)
        if case["op"] == "paged":
            lse = torch.logsumexp(scores, 1)
            outs.append(torch.exp(scores - lse[:, None]) @ keys)
            logs.append(lse)
            continue
        d_o, o = st["d_o"][r].double(), st["o"][r].double()
        p = torch.exp(scores - st["lse"][r].double()[:, None])
        d_s = d_o @ keys.T - (d_o * o).sum(1, keepdim=True)
        if st["d_lse"] is not None:
            d_s = d_s + st["d_lse"][r].double()[:, None]
        d_s = p * d_s / math.sqrt(WIDTH)
        outs.append(d_s @ keys)
        d_kv.index_add_(0, toks, d_s.T @ q + p.T @ d_o)
    return (torch.stack(outs), torch.stack(logs)) if case["op"] == "paged" else (torch.stack(outs), d_kv)
