"""The serving operators' cases: packed prompts, draft trees over a cache, and the pages of a cache.

Each case names an operator and its sizes.  ``run`` makes one pass: the framework's calls where
``own`` is true, else the same mathematics in elementary torch operations (32-bit arithmetic,
one rounding at the end).  ``exact`` is the definition in 64 bits, one sequence at a time.

Operators:
  varlen   attention over packed prompts of different lengths (``gqa_attn_fwd_varlen``)
  tree     attention of a tree of drafted tokens over a cache (``gqa_attn_fwd_tree``)
  fork     sequences that share their parent's pages, with the last page copied (``gqa_cache_fork``)
  compact  the accepted nodes of a tree made contiguous, the rest dropped (``gqa_cache_compact``)
  resize   sequences grown, shrunk and freed: pages taken and returned (``gqa_cache_resize``)
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # three short prompts of a small model, one of them empty: launch latency counts
        dict(name="varlen small", op="varlen", B=4, max_q=130, max_k=130, low=0.0, Hq=8, Hk=2, d=64, causal=True),
        # the prompts that arrive in one scheduling step: lengths from a few tokens to long
        dict(name="varlen mixed", op="varlen", B=16, max_q=4096, max_k=4096, low=0.002, Hq=32, Hk=8, d=128, causal=True),
        # a full batch of prompts, 64 of up to 2048 tokens (the prefill benchmark's shape, ragged)
        dict(name="varlen batch", op="varlen", B=64, max_q=2048, max_k=2048, low=0.5, Hq=32, Hk=8, d=128, causal=True),
        # one request of a small model, eight drafted tokens, a dense cache
        dict(name="tree small", op="tree", B=1, T=8, cap=512, low=0.5, Hq=8, Hk=2, d=64, page=0),
        # a serving batch with 31 drafted tokens each over pages of 64 keys
        dict(name="tree batch", op="tree", B=32, T=31, cap=8192, low=0.1, Hq=32, Hk=8, d=128, page=64),
        # long contexts: 64 sequences of up to 16384 keys, pages of 16, 16 drafted tokens
        dict(name="tree long", op="tree", B=64, T=16, cap=16384, low=0.3, Hq=32, Hk=8, d=128, page=16),
        # two parents, six samples each of a small cache
        dict(name="fork small", op="fork", parents=2, copies=3, cap=200, layers=2, Hk=2, d=64, page=16),
        # parallel sampling: 16 prompts, 15 samples each, 8 layers
        dict(name="fork samples", op="fork", parents=16, copies=15, cap=1024, layers=8, Hk=8, d=128, page=64),
        # one verification step of two requests
        dict(name="compact small", op="compact", B=2, T=8, cap=100, layers=2, Hk=2, d=64, page=16),
        # one verification step of 128 requests with trees of 64 nodes, 8 layers
        dict(name="compact batch", op="compact", B=128, T=64, cap=512, layers=8, Hk=8, d=128, page=16),
        # a few sequences grow by a token, one ends, one starts
        dict(name="resize small", op="resize", S=8, cap=256, page=16),
        # 256 slots of up to 32768 keys in pages of 16: a scheduling step of a large server
        dict(name="resize server", op="resize", S=256, cap=32768, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["varlen", "varlen", "tree", "tree", "fork", "compact", "resize"])
    Hk = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "varlen":
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        B = _log_int(rng, 1, 64)
        max_q = _log_int(rng, 1, 4096)
        while B * max_q * max_q * max(Hq, 8) > 64 * 2048 * 2048 * 32 or B * max_q > 131072:
            max_q = max(1, max_q // 2)
        max_k = max_q
        causal = rng.random() < 0.75
        if rng.random() < 0.3:  # queries at the end of longer contexts
            max_k = max_q + _log_int(rng, 1, 4096)
            while B * max_q * max_k * max(Hq, 8) > 64 * 2048 * 2048 * 32 or B * max_k > 131072:
                max_k = max(max_q, max_k // 2)
        return dict(op=op, B=B, max_q=max_q, max_k=max_k, low=rng.choice([0.0, 0.1, 0.7]), Hq=Hq, Hk=Hk, d=d, causal=causal)
    if op == "tree":
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, 96)
        cap = max(_log_int(rng, 64, 16384), 2 * T)
        while B * cap * Hk * d > 64 * 16384 * 8 * 128 // 2 or B * cap * T * Hq > 64 * 16384 * 16 * 32:
            B = max(1, B // 2)
        return dict(op=op, B=B, T=T, cap=cap, low=rng.choice([0.0, 0.3, 0.9]), Hq=Hq, Hk=Hk, d=d, page=rng.choice([0, 16, 32, 64, 128, 256]))
    if op == "fork":
        return dict(op=op, parents=_log_int(rng, 1, 16), copies=_log_int(rng, 1, 15), cap=_log_int(rng, 20, 1024), layers=_log_int(rng, 1, 8), Hk=Hk, d=d, page=min(page, 64))
    if op == "compact":
        return dict(op=op, B=_log_int(rng, 1, 128), T=_log_int(rng, 1, 64), cap=_log_int(rng, 32, 512), layers=_log_int(rng, 1, 8), Hk=Hk, d=d, page=min(page, 64))
    return dict(op=op, S=_log_int(rng, 2, 256), cap=_log_int(rng, 64, 32768), page=rng.choice([16, 32, 64]))


# ---------------------------------------------------------------- what a program has in hand

def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).bfloat16()


def _pool(gen, *shape):
    """A large bf16 tensor, filled a slice at a time (a whole one in 32 bits would be twice as large)."""
    t = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    flat = t.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=gen, device="cuda", dtype=torch.float32)
    return t


def _lengths(rs, B, low, high):
    """One length of each range: the longest is there, the others uniform between low * high and high."""
    x = rs.randint(int(low * high), high + 1, B)
    x[rs.randint(B)] = high
    if low == 0.0 and B > 2:
        x[(int(np.argmax(x)) + 1) % B] = 0
    return x.astype(np.int64)


def _tree(rs, T):
    """Ancestors of each node of a random tree (itself among them) as truth values [T, T]; parents come first."""
    see = np.zeros((T, T), dtype=bool)
    for i in range(T):
        p = rs.randint(max(-1, i - 6), i)  # children of recent nodes: the trees are some levels deep
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def _bits(see):
    """Truth values [..., T] as 32-bit words [..., ceil(T / 32)], bit j % 32 of word j // 32."""
    T = see.shape[-1]
    W = (T + 31) // 32
    full = np.zeros(see.shape[:-1] + (W * 32,), dtype=np.uint64)
    full[..., :T] = see
    words = (full.reshape(see.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def _table(rs, lens, page, M, spare):
    """A block table whose pages are handed out in a random order, and the pages' reference counts."""
    need = -(-lens // page)
    P = int(need.sum()) + spare
    perm = rs.permutation(P)
    table = np.full((len(lens), M), -1, dtype=np.int64)
    refs = np.zeros(P, dtype=np.int64)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(len(lens)):
        table[b, :need[b]] = perm[at[b]:at[b + 1]]
        refs[table[b, :need[b]]] = 1
    return table, refs


def _host(case, seed):
    """The lengths, trees and tables of a case: everything of it that is not a tensor of K, V or Q.

    The sizes are the case's own, in an order that the seed gives, so that every seed has the same number of tokens and pages."""
    size, rs = np.random.RandomState(7), np.random.RandomState(seed % (1 << 31))
    op = case["op"]
    h = {}
    if op == "varlen":
        B = case["B"]
        lq = _lengths(size, B, case["low"], case["max_q"])
        # with a longer context the keys before the queries are added to each sequence's own
        extra = case["max_k"] - case["max_q"]
        lk = lq + (size.randint(0, extra + 1, B) if extra else 0)
        order = rs.permutation(B)
        h.update(lq=lq[order], lk=lk[order])
    elif op == "tree":
        B, T = case["B"], case["T"]
        lens = np.maximum(_lengths(size, B, case["low"], case["cap"]), 1)
        n = np.minimum(np.maximum(T - size.randint(0, 3, B) * (T // 8), 1), lens)
        order = rs.permutation(B)
        lens, n = lens[order], n[order]
        h.update(lens=lens, n=n, see=np.stack([_tree(rs, T) for _ in range(B)]))
        if case["page"]:
            h["table"], h["refs"] = _table(rs, lens, case["page"], -(-case["cap"] // case["page"]), 5)
    elif op == "fork":
        n, c, page = case["parents"], case["copies"], case["page"]
        lens = np.maximum(_lengths(size, n, 0.3, case["cap"]), 1)[rs.permutation(n)]
        M = -(-case["cap"] // page) + 1
        table, refs = _table(rs, lens, page, M, n * c + 3)
        h.update(lens=np.concatenate([lens, np.zeros(n * c, dtype=np.int64)]), refs=refs,
                 table=np.concatenate([table, np.full((n * c, M), -1, dtype=np.int64)]),
                 parents=np.repeat(np.arange(n), c), children=n + np.arange(n * c))
    elif op == "compact":
        B, T, page = case["B"], case["T"], case["page"]
        base = _lengths(size, B, 0.2, case["cap"])
        n = np.maximum(T - size.randint(0, 3, B) * (T // 8), 1)
        order = rs.permutation(B)
        base, n = base[order], n[order]
        M = -(-(case["cap"] + T) // page)
        table, refs = _table(rs, base, page, M, int((-(-(base + n) // page) - -(-base // page)).sum()) + 3)
        keep = np.zeros((B, T), dtype=np.int64)
        m = np.zeros(B, dtype=np.int64)
        for b in range(B):  # a path from a root down: the accepted tokens
            path = np.flatnonzero(_tree(rs, int(n[b]))[rs.randint(int(n[b]))])
            m[b] = len(path)
            keep[b, :m[b]] = path
        h.update(base=base, n=n, table=table, refs=refs, keep=keep, m=m)
    else:
        S, page, cap = case["S"], case["page"], case["cap"]
        a = size.randint(0, cap // 2 + 1, S)
        a[size.rand(S) < 0.1] = 0
        b = np.minimum(a + size.randint(1, 9, S), cap)  # a few tokens more ...
        b[size.rand(S) < 0.15] = 0  # ... some end, some are cut back, some start
        cut = size.rand(S) < 0.1
        b[cut] = a[cut] // 2
        start = a == 0
        b[start] = size.randint(1, cap // 4 + 2, int(start.sum()))
        order = rs.permutation(S)
        a, b = a[order], b[order]
        table, refs = _table(rs, a, page, -(-cap // page), int(np.maximum(-(-b // page) - -(-a // page), 0).sum()) + 7)
        h.update(a=a, b=b, table=table, refs=refs, slots=rs.permutation(S))
    return h


def prepare(case, seed):
    h = _host(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op == "varlen":
        tq, tk = int(h["lq"].sum()), int(h["lk"].sum())
        s["q"] = _randn(gen, tq, case["Hq"], case["d"])
        s["k"] = _randn(gen, tk, case["Hk"], case["d"])
        s["v"] = _randn(gen, tk, case["Hk"], case["d"])
        s["cu_q"] = _ints(np.concatenate([[0], np.cumsum(h["lq"])]))
        s["cu_k"] = _ints(np.concatenate([[0], np.cumsum(h["lk"])]))
        s["max_q"], s["max_k"] = int(h["lq"].max()), int(h["lk"].max())
    elif op == "tree":
        B, T = case["B"], case["T"]
        s["q"] = _randn(gen, B, T, case["Hq"], case["d"])
        s["mask"], s["lens"], s["n"] = _ints(_bits(h["see"])), _ints(h["lens"]), _ints(h["n"])
        if case["page"]:
            shape = (len(h["refs"]), case["page"], case["Hk"], case["d"])
            s["table"] = _ints(h["table"])
        else:
            shape = (B, case["cap"], case["Hk"], case["d"])
            s["table"] = None
        s["k"], s["v"] = _pool(gen, *shape), _pool(gen, *shape)
    else:
        s["table"], s["refs"] = _ints(h["table"]), _ints(h["refs"])
        if op == "resize":
            slots = h["slots"]
            s["lens"], s["slots"] = _ints(h["a"]), _ints(slots)
            s["to"], s["back"] = _ints(h["b"][slots]), _ints(h["a"][slots])
        else:
            shape = (case["layers"], len(h["refs"]), case["page"], case["Hk"], case["d"])
            s["k"], s["v"] = _pool(gen, *shape), _pool(gen, *shape)
            if op == "fork":
                s["lens"], s["parents"], s["children"] = _ints(h["lens"]), _ints(h["parents"]), _ints(h["children"])
                # the samples of the step before, which the pass replaces
                _plain_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
            else:
                s["lens"], s["drafted"], s["n"] = _ints(h["base"]), _ints(h["base"] + h["n"]), _ints(h["n"])
                s["keep"], s["m"] = _ints(h["keep"]), _ints(h["m"])
                s["slots"] = _ints(np.arange(case["B"]))
                s["back"] = _ints(h["base"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if op == "varlen":
        if own:
            import gqa_exact_attention_b200 as G
            out, lse = G.gqa_attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], out_dtype=torch.bfloat16)
        else:
            out, lse = _plain_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], c["causal"])
        return {"out": out, "lse": lse}
    if op == "tree":
        if own:
            import gqa_exact_attention_b200 as G
            out, lse = G.gqa_attn_fwd_tree(s["q"], s["k"], s["v"], s["mask"], s["lens"], block_table=s["table"], tree_lens=s["n"], out_dtype=torch.bfloat16)
        else:
            out, lse = _plain_tree(s["q"], s["k"], s["v"], s["mask"], s["lens"], s["table"], s["n"], c["cap"])
        return {"out": out, "lse": lse}
    if op == "fork":
        if own:
            import gqa_exact_attention_b200 as G
            st = G.gqa_cache_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
        else:
            st = _plain_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
        return {"k": s["k"], "v": s["v"], "table": s["table"], "lens": s["lens"], "refs": s["refs"], "status": st}
    if op == "compact":
        # room for the drafted nodes, the accepted ones kept, and the step undone so that a pass can be made again
        if own:
            import gqa_exact_attention_b200 as G
            a = G.gqa_cache_resize(s["table"], s["lens"], s["refs"], c["page"], s["drafted"], s["slots"])
            b = G.gqa_cache_compact(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["keep"], s["m"], tree_lens=s["n"])
            kept, table = s["lens"].clone(), s["table"].clone()
            e = G.gqa_cache_resize(s["table"], s["lens"], s["refs"], c["page"], s["back"], s["slots"])
        else:
            a = _plain_resize(s["table"], s["lens"], s["refs"], c["page"], s["drafted"], s["slots"])
            b = _plain_compact(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["keep"], s["m"], s["n"])
            kept, table = s["lens"].clone(), s["table"].clone()
            e = _plain_resize(s["table"], s["lens"], s["refs"], c["page"], s["back"], s["slots"])
        return {"k": s["k"], "v": s["v"], "kept": kept, "table": table, "lens": s["lens"], "refs": s["refs"], "status": [a, b, e]}
    if own:
        import gqa_exact_attention_b200 as G
        a = G.gqa_cache_resize(s["table"], s["lens"], s["refs"], c["page"], s["to"], s["slots"])
        table, refs = s["table"].clone(), s["refs"].clone()
        b = G.gqa_cache_resize(s["table"], s["lens"], s["refs"], c["page"], s["back"], s["slots"])
    else:
        a = _plain_resize(s["table"], s["lens"], s["refs"], c["page"], s["to"], s["slots"])
        table, refs = s["table"].clone(), s["refs"].clone()
        b = _plain_resize(s["table"], s["lens"], s["refs"], c["page"], s["back"], s["slots"])
    return {"grown": table, "grown_refs": refs, "table": s["table"], "lens": s["lens"], "refs": s["refs"], "status": [a, b]}


# ---------------------------------------------------------------- plain forms

def _softmax_pv(x, v):
    """Rows of scores x (overwritten; -inf where masked) and values: (output, log of the sum)."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return o, (m + torch.log(l)).squeeze(-1)


def _grouped(q, Hk):
    """[B, S, Hq, d] -> [B, Hk, g * S, d] (rows: head of the group, then position)."""
    B, S, Hq, d = q.shape
    return q.view(B, S, Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, d)


def _plain_varlen(q, k, v, cu_q, cu_k, max_q, max_k, causal):
    Tq, Hq, d = q.shape
    Tk, Hk = k.shape[0], k.shape[1]
    g = Hq // Hk
    B = cu_q.numel() - 1
    iq, ik = torch.arange(max_q, device="cuda"), torch.arange(max_k, device="cuda")
    lq, lk = (cu_q[1:] - cu_q[:-1]).long(), (cu_k[1:] - cu_k[:-1]).long()
    qp = q[(cu_q[:-1, None] + iq).clamp(max=Tq - 1)].float()
    at = (cu_k[:-1, None] + ik).clamp(max=Tk - 1)
    kp, vp = k[at].float().transpose(1, 2), v[at].float().transpose(1, 2)
    x = torch.matmul(_grouped(qp, Hk), kp.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    hide = (ik >= lk[:, None])[:, None, :]
    if causal:
        hide = hide | (ik[None, None, :] > iq[None, :, None] + (lk - lq)[:, None, None])
    x.view(B, Hk, g, max_q, max_k).masked_fill_(hide[:, None, None], -math.inf)
    o, lse = _softmax_pv(x, vp)
    t = torch.arange(Tq, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu_q, t, right=True) - 1  # the last sequence that starts at or before row t
    i = t.long() - cu_q[b].long()
    out = o.view(B, Hq, max_q, d)[b, :, i].to(torch.bfloat16)
    return out, lse.view(B, Hq, max_q)[b, :, i].t().contiguous()


def _plain_tree(q, k, v, mask, lens, table, n, cap):
    B, T, Hq, d = q.shape
    if table is not None:
        P, page, Hk = k.shape[:3]
        pages = table.long().clamp(0, P - 1)
        k = k[pages].view(B, -1, Hk, d)[:, :cap]
        v = v[pages].view(B, -1, Hk, d)[:, :cap]
    Hk = k.shape[2]
    j, i = torch.arange(k.shape[1], device="cuda"), torch.arange(T, device="cuda")
    L, nn = lens.long()[:, None], n.long()[:, None]
    node = j[None] - (L - nn)  # [B, cap]: the tree node of a key, or below 0
    word = mask.long().gather(2, (node.clamp(0, T - 1) // 32)[:, None].expand(-1, T, -1))
    see = ((word >> (node.clamp(0, T - 1) % 32)[:, None]) & 1).bool() | (node < 0)[:, None]
    see = see & (j[None] < L)[:, None] & (i[None] < nn)[:, :, None]
    x = torch.matmul(_grouped(q.float(), Hk), k.float().permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d))
    x.view(B, Hk, Hq // Hk, T, -1).masked_fill_(~see[:, None, None], -math.inf)
    o, lse = _softmax_pv(x, v.float().transpose(1, 2))
    return o.view(B, Hq, T, d).transpose(1, 2).to(torch.bfloat16).contiguous(), lse.view(B, Hq, T)


DONE, NO_PAGES, INVALID, SHARED = 0, 1, 2, 3


def _rows_of(x, slots, act, value):
    """x[slots[i]] = value[i] where act[i], with every slot of act different."""
    more = torch.cat([x, x[:1]])
    more[torch.where(act, slots, torch.full_like(slots, len(x)))] = value.to(x.dtype)
    x.copy_(more[:-1])


def _release(rows, refs, first, end, act):
    """The pages of entries [first, end) of the table rows are given up; returns the rows without them."""
    j = torch.arange(rows.shape[1], device="cuda")
    gone = act[:, None] & (j >= first[:, None]) & (j < end[:, None])
    known = gone & (rows >= 0) & (rows < len(refs))
    refs.index_add_(0, rows.clamp(0, len(refs) - 1).flatten(), -known.flatten().int())
    return rows.masked_fill(gone, -1)


def _take(rows, refs, first, need, act):
    """need[i] free pages, the lowest first, to entries first[i].. of row i, in order; which rows got theirs."""
    need = torch.where(act, need, torch.zeros_like(need))
    upto = need.cumsum(0)
    got = act & ((upto <= (refs == 0).sum()) | (need == 0))
    free = torch.argsort((refs != 0).int(), stable=True)
    j = torch.arange(rows.shape[1], device="cuda")
    new = got[:, None] & (j >= first[:, None]) & (j < (first + need)[:, None])
    page = free[((upto - need - first)[:, None] + j).clamp(0, len(refs) - 1)]
    refs.index_add_(0, page.flatten(), new.flatten().int())
    return torch.where(new, page.to(rows.dtype), rows), got


def _again(x):
    """Whether an earlier element has the same value."""
    return (x[:, None] == x[None, :]).tril(-1).any(1)


def _plain_resize(table, lens, refs, page, new_lens, slots):
    S, M = table.shape
    slot, new = slots.long(), new_lens.long()
    valid = (slot >= 0) & (slot < S) & (new >= 0) & (new <= M * page) & ~_again(slot)
    slot = slot.clamp(0, S - 1)
    old = lens[slot].long().clamp(0, M * page)
    stay = torch.minimum(old, new)  # the page that stays in part must not be another sequence's too
    last = table[slot, (stay // page).clamp(max=M - 1)].long()
    shared = (stay % page != 0) & (new != old) & (last >= 0) & (last < len(refs)) & (refs[last.clamp(0, len(refs) - 1)] > 1)
    act = valid & ~shared
    had, want = (old + page - 1) // page, (new + page - 1) // page
    rows = _release(table[slot], refs, want, had, act)
    rows, got = _take(rows, refs, had, (want - had).clamp(min=0), act)
    _rows_of(table, slot, got, rows)
    _rows_of(lens, slot, got, new)
    st = torch.where(got, DONE, NO_PAGES)
    return torch.where(valid, torch.where(shared, SHARED, st), INVALID).int()


def _copy_rows(pools, src, dst, act):
    """Row dst of every layer becomes row src, where act; all reads come before the writes."""
    src, dst, act = src.flatten(), dst.flatten(), act.flatten()
    one = torch.argmax(act.int())  # rows that do not move repeat one that does (none does: row 0 stays itself)
    some = act.any()
    src = torch.where(act, src, torch.where(some, src[one], 0))
    dst = torch.where(act, dst, torch.where(some, dst[one], 0))
    for x in pools:
        rows = x.view(x.shape[0], -1, x.shape[3] * x.shape[4])
        rows[:, dst] = rows[:, src]


def _plain_fork(k, v, table, lens, refs, parents, children):
    S, M = table.shape
    page = k.shape[2]
    par, kid = parents.long(), children.long()
    same = par == kid
    valid = (par >= 0) & (par < S) & (kid >= 0) & (kid < S) & ~_again(kid) & (same | ~(kid[:, None] == par[None]).any(1))
    act = valid & ~same
    par, kid = par.clamp(0, S - 1), kid.clamp(0, S - 1)
    L, held = lens[par].long().clamp(0, M * page), lens[kid].long().clamp(0, M * page)
    whole, tail = L // page, L % page
    rows = _release(table[kid], refs, torch.zeros_like(held), (held + page - 1) // page, act)
    j = torch.arange(M, device="cuda")
    ours = act[:, None] & (j < whole[:, None])
    theirs = table[par]
    known = ours & (theirs >= 0) & (theirs < len(refs))
    refs.index_add_(0, theirs.clamp(0, len(refs) - 1).flatten().long(), known.flatten().int())
    rows, got = _take(torch.where(ours, theirs, rows), refs, whole, (tail > 0).long(), act)
    # without a page for its last rows a child ends up empty, and the shared pages go back
    rows = _release(rows, refs, torch.zeros_like(whole), whole, act & ~got)
    _rows_of(table, kid, act, rows)
    _rows_of(lens, kid, act, torch.where(got, L, 0))
    r = torch.arange(page, device="cuda")
    at = whole.clamp(max=M - 1)[:, None]
    src = theirs.long().gather(1, at) * page + r
    dst = rows.long().gather(1, at) * page + r
    _copy_rows((k, v), src, dst, got[:, None] & (r < tail[:, None]))
    return torch.where(valid, torch.where(got | same, DONE, NO_PAGES), INVALID).int()


def _plain_compact(k, v, table, lens, refs, keep, keep_lens, tree_lens):
    S, M = table.shape
    page, T, P = k.shape[2], keep.shape[1], len(refs)
    L = lens.long().clamp(0, M * page)
    n = torch.minimum(tree_lens.long().clamp(0, T), L)
    m, kp = keep_lens.long(), keep.long()
    base = L - n
    i = torch.arange(T, device="cuda")
    live = i < m[:, None]
    before = torch.cat([torch.full_like(kp[:, :1], -1), kp[:, :-1]], 1)
    bad = (m < 0) | (m > n) | (live & ((kp <= before) | (kp >= n[:, None]))).any(1)
    end = base + m
    j = torch.arange(M, device="cuda")
    stay = (j >= (base // page)[:, None]) & (j < ((end + page - 1) // page)[:, None])
    known = (table >= 0) & (table < P)
    shared = (stay & known & (refs[table.long().clamp(0, P - 1)] > 1)).any(1)
    act = ~bad & ~shared
    at = lambda pos: table.long().gather(1, (pos // page).clamp(0, M - 1)) * page + pos % page  # noqa: E731
    src, dst = at(base[:, None] + kp.clamp(0, T - 1)), at(base[:, None] + i)
    _copy_rows((k, v), src, dst, act[:, None] & live & (kp > i))
    table.copy_(_release(table, refs, (end + page - 1) // page, (L + page - 1) // page, act))
    lens.copy_(torch.where(act, end.int(), lens))
    return torch.where(bad, INVALID, torch.where(shared, SHARED, DONE)).int()


# ---------------------------------------------------------------- work and the definition in 64 bits

def work(case):
    h = _host(case, 1)  # another seed has the same lengths in another order
    op = case["op"]
    if op == "varlen":
        lq, lk = h["lq"].astype(float), h["lk"].astype(float)
        pairs = lq * lk - (lq * (lq - 1) / 2 if case["causal"] else 0)
        b = 2.0 * (2 * lq.sum() * case["Hq"] + 2 * lk.sum() * case["Hk"]) * case["d"] + 4 * lq.sum() * case["Hq"] + 8 * (case["B"] + 1)
        return {"bytes": b, "flops": 4.0 * pairs.sum() * case["Hq"] * case["d"]}
    if op == "tree":
        lens, n, T = h["lens"].astype(float), h["n"].astype(float), case["T"]
        pairs = n * (lens - n) + sum(float(h["see"][b][:int(n[b]), :int(n[b])].sum()) for b in range(case["B"])) / case["B"]
        b = 4.0 * lens.sum() * case["Hk"] * case["d"] + 4.0 * case["B"] * T * case["Hq"] * case["d"] + 4.0 * case["B"] * T * case["Hq"]
        b += 4.0 * h["see"].shape[0] * T * ((T + 31) // 32) + 8 * case["B"]
        if case["page"]:
            b += 4.0 * np.sum(-(-h["lens"] // case["page"]))
        return {"bytes": b, "flops": 4.0 * pairs.sum() * case["Hq"] * case["d"]}
    if op == "resize":
        page = case["page"]
        held, want = -(-h["a"] // page), -(-h["b"] // page)
        moved = np.abs(held - want).sum()
        # two calls: the entries that change with their counts, the counts once to find the free pages, lengths and answers;
        # and the copies of the table and of the counts between them
        return {"bytes": 2.0 * (12 * moved + 4 * len(h["refs"]) + 20 * case["S"]) + 8.0 * (h["table"].size + len(h["refs"])), "flops": 0}
    row = 4.0 * case["layers"] * case["Hk"] * case["d"]  # K and V of one token, all layers
    page = case["page"]
    if op == "fork":
        L = h["lens"][:case["parents"]]
        tail, whole = L % page, L // page
        c = case["copies"]
        return {"bytes": row * tail.sum() * (1 + c) + (24.0 * whole.sum() + 40 * case["parents"]) * c + 4.0 * len(h["refs"]), "flops": 0}
    moved = sum(int((h["keep"][b, :h["m"][b]] > np.arange(h["m"][b])).sum()) for b in range(case["B"]))
    pages = (-(-(h["base"] + h["n"]) // page) - -(-h["base"] // page)).sum()
    return {"bytes": 2 * row * moved + 24.0 * pages + 8.0 * len(h["refs"]) + 4.0 * h["keep"].size + 60 * case["B"] + 8.0 * h["table"].size, "flops": 0}


def _exact_rows(q, k, v, see):
    """One sequence, one kv head: q [S, g, d], k and v [L, d], see [S, L]; out [S, g, d] and lse [g, S] in 64 bits."""
    x = torch.einsum("sgd,ld->gsl", q.double(), k.double()) / math.sqrt(q.shape[2])
    x = x.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(x, -1) if x.shape[2] else torch.full(x.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("gsl,ld->sgd", w, v.double()), lse


def exact(case, seed):
    if case["op"] not in ("varlen", "tree"):
        return None  # rows that are moved and whole numbers: nothing is rounded
    s = prepare(case, seed)
    h = _host(case, seed)
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    g = Hq // Hk
    if case["op"] == "varlen":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full((Hq, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
        aq = ak = 0
        for a, b in zip(h["lq"].tolist(), h["lk"].tolist()):
            for hk in range(Hk if a else 0):
                see = torch.ones((a, b), dtype=torch.bool, device="cuda")
                if case["causal"]:
                    see = see.tril(b - a)
                o, x = _exact_rows(s["q"][aq:aq + a, hk * g:hk * g + g], s["k"][ak:ak + b, hk], s["v"][ak:ak + b, hk], see)
                out[aq:aq + a, hk * g:hk * g + g] = o
                lse[hk * g:hk * g + g, aq:aq + a] = x
            aq, ak = aq + a, ak + b
        return {"out": out, "lse": lse}
    B, T, page = case["B"], case["T"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = int(h["lens"][b]), int(h["n"][b])
        k, v = s["k"], s["v"]
        if page:
            at = torch.as_tensor(h["table"][b, :-(-L // page)]).cuda()
            k, v = k[at].reshape(-1, Hk, d)[:L], v[at].reshape(-1, Hk, d)[:L]
        else:
            k, v = k[b, :L], v[b, :L]
        see = torch.ones((n, L), dtype=torch.bool, device="cuda")
        see[:, L - n:] = torch.as_tensor(h["see"][b][:n, :n]).cuda()
        for hk in range(Hk):
            o, x = _exact_rows(s["q"][b, :n, hk * g:hk * g + g], k[:, hk], v[:, hk], see)
            out[b, :n, hk * g:hk * g + g] = o
            lse[b, hk * g:hk * g + g, :n] = x
    return {"out": out, "lse": lse}
