"""Cases of the paged KV cache operators: page assignment with its slot map, the
cache write, attention of drafted token trees over the cache, and the move of an
accepted path to the sequence's tail.

``run`` computes a case in plain torch (``own`` false) or through the library's
entry points (``own`` true) on the same inputs.  Head dimension 128 throughout.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
D = 128
E4M3_MAX = 448.0
# static bounds of standard-normal activations with the usual margin (q, k, v)
BOUNDS = (7.5, 7.0, 7.25)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _pages(name, rows, lo, hi, new_lo, new_hi, page, pad, lens):
    return {"op": "pages", "name": name, "rows": rows, "lo": lo, "hi": hi, "new_lo": new_lo,
            "new_hi": new_hi, "page": page, "pad": pad, "lens": lens}


def _write(name, tokens, heads, page, fp8, pad, fused, head_major, lens):
    return {"op": "write", "name": name, "tokens": tokens, "heads": heads, "page": page,
            "fp8": fp8, "pad": pad, "fused": fused, "head_major": head_major, "lens": lens}


def _tree(name, rows, lo, hi, nodes_lo, nodes_hi, q_heads, kv_heads, page, fp8, tree, head_major,
          lens):
    return {"op": "tree", "name": name, "rows": rows, "lo": lo, "hi": hi, "nodes_lo": nodes_lo,
            "nodes_hi": nodes_hi, "q_heads": q_heads, "kv_heads": kv_heads, "page": page,
            "fp8": fp8, "tree": tree, "head_major": head_major, "lens": lens}


def _keep(name, rows, lo, hi, nodes_lo, nodes_hi, depth, heads, page, fp8, lens):
    return {"op": "keep", "name": name, "rows": rows, "lo": lo, "hi": hi, "nodes_lo": nodes_lo,
            "nodes_hi": nodes_hi, "depth": depth, "heads": heads, "page": page, "fp8": fp8,
            "lens": lens}


def listed():
    return [
        # one decoding step of a small server: a token for each of 64 requests
        _pages("pages, decode 64", 64, 0, 8192, 1, 1, 16, 0, 1),
        # prompts of up to 1024 tokens admitted for 1500 requests and let go again
        _pages("pages, admit 1500", 1500, 0, 0, 1, 1024, 32, 777, 2),
        # the cache write of a decoding step for a layer kept in bf16
        _write("write, decode 64", 64, 8, 16, False, 0, False, True, 3),
        # the write of a long prompt, straight from a fused QKV projection in a
        # padded step buffer
        _write("write, prompt 8075", 8075, 16, 64, True, 117, True, False, 4),
        # one user, one token: latency over a context of 8192
        _tree("attend, one token", 1, 8192, 8192, 1, 1, 16, 2, 64, True, False, True, 6),
        # a server's decoding step: 64 requests of mixed lengths
        _tree("attend, decode 64", 64, 33, 16384, 1, 1, 32, 8, 64, True, False, False, 7),
        # verification of drafted trees of up to 64 nodes
        _tree("attend, trees of 64", 8, 1000, 8192, 33, 64, 32, 8, 16, True, True, True, 8),
        # the same for a layer kept in bf16, small trees, five query heads to a KV head
        _tree("attend, bf16 trees", 16, 100, 5000, 1, 25, 40, 8, 32, False, True, False, 9),
        # drafted chains of 4 over short contexts, a KV head for every query head, bf16
        _tree("attend, short chains", 128, 5, 300, 2, 4, 16, 16, 16, False, False, False, 10),
        # two very long contexts (whole repositories or videos) with trees of 8
        _tree("attend, long", 2, 100000, 131072, 8, 8, 64, 8, 128, True, True, True, 11),
        # after verification: the accepted nodes of each request's tree move down
        _keep("keep, 4 trees", 4, 500, 2000, 9, 25, 5, 16, 32, False, 13),
        _keep("keep, 96 trees", 96, 80, 600, 20, 64, 8, 8, 16, True, 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    caps = {}
    for c in listed():
        w = work(c)
        for key in ("bytes", "flops"):
            caps[c["op"], key] = max(caps.get((c["op"], key), 0), w[key])
    while True:
        op = rng.choice(["pages", "write", "tree", "tree", "tree", "keep"])
        page = rng.choice([16, 32, 64, 128])
        lens = rng.randrange(1 << 20)
        if op == "pages":
            c = _pages("", _log_int(rng, 1, 1500), 0, rng.choice([0, _log_int(rng, 1, 20000)]), 1,
                       _log_int(rng, 1, 1024), page, rng.choice([0, rng.randrange(1, 999)]), lens)
        elif op == "write":
            c = _write("", _log_int(rng, 1, 8192), rng.choice([1, 2, 5, 8, 16, 40]), page,
                       rng.random() < 0.6, rng.choice([0, rng.randrange(1, 300)]),
                       rng.random() < 0.5, rng.random() < 0.5, lens)
        elif op == "tree":
            kv = rng.choice([1, 2, 4, 8, 16])
            nodes = _log_int(rng, 1, 64)
            lo = _log_int(rng, nodes, 131072)
            c = _tree("", _log_int(rng, 1, 128), lo, _log_int(rng, lo, 131072),
                      rng.randint(1, nodes), nodes, kv * rng.choice([1, 2, 4, 5, 8]), kv, page,
                      rng.random() < 0.6, rng.random() < 0.6, rng.random() < 0.5, lens)
        else:
            nodes = _log_int(rng, 4, 64)
            lo = nodes + _log_int(rng, 1, 300)
            c = _keep("", _log_int(rng, 1, 96), lo, lo + _log_int(rng, 1, 300),
                      rng.randint(1, nodes), nodes, rng.randint(1, 12), rng.choice([1, 4, 8]),
                      page, rng.random() < 0.6, lens)
        del c["name"]
        w = work(c)
        # the plain form's padded gather is bounded too: rows * longest context
        padded = c.get("rows", 1) * c.get("hi", 1) * c.get("kv_heads", 1)
        if all(w[key] <= caps[op, key] for key in ("bytes", "flops")) and \
                (op != "tree" or padded <= 64 * 16384 * 8):
            return c


def _lens(case):
    """Lengths of a case, the same for every seed: (sequence lengths with the
    new tokens, new tokens) per row."""
    r = np.random.Generator(np.random.PCG64(case["lens"]))
    n = case["rows"]
    if case["op"] == "pages":
        old = r.integers(case["lo"], case["hi"] + 1, n)
        new = r.integers(case["new_lo"], case["new_hi"] + 1, n)
        return old + new, new
    nodes = r.integers(case["nodes_lo"], case["nodes_hi"] + 1, n)
    seq = np.maximum(r.integers(case["lo"], case["hi"] + 1, n), nodes)
    return seq, nodes


def _kept(case, nodes):
    """Accepted nodes per row, the same for every seed."""
    r = np.random.Generator(np.random.PCG64(case["lens"] + 1))
    return np.minimum(r.integers(1, case["depth"] + 1, case["rows"]), nodes)


def work(case):
    op = case["op"]
    if op == "write":
        values = 2 * case["tokens"] * case["heads"] * D
        return {"bytes": values * (2 + (1 if case["fp8"] else 2)) + 8 * (case["tokens"] +
                                                                       case["pad"]), "flops": 0}
    seq, new = _lens(case)
    if op == "pages":
        p = case["page"]
        want, owned = -(-seq // p), -(-(seq - new) // p)
        grow = int((want - owned).sum())
        # pages that the new tokens lie in are read from the table; each moved
        # page id is read and written on the way out and on the way back
        held = int((owned - (seq - new) // p).sum())
        slots = int(new.sum()) + case["pad"]
        return {"bytes": 12 * slots + 4 * held + 16 * grow + 40 * case["rows"], "flops": 0}
    if op == "keep":
        moved = int(_kept(case, new).sum())
        return {"bytes": 4 * moved * case["heads"] * D * (1 if case["fp8"] else 2), "flops": 0}
    kv = 2 * int(seq.sum()) * case["kv_heads"] * D * (1 if case["fp8"] else 2)
    qo = 4 * int(new.sum()) * case["q_heads"] * D
    pairs = int((new * (seq - new)).sum())
    # a chain sees n (n + 1) / 2 pairs of its own nodes; a tree at least one per node
    own_pairs = int((new * (new + 1) // 2).sum()) if not case["tree"] else int(new.sum())
    return {"bytes": kv + qo + 4 * int(seq.sum()) // case["page"],
            "flops": 4 * D * case["q_heads"] * (pairs + own_pairs)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(gen, pages, page, heads, fp8, head_major, bound):
    """A cache [pages, page, heads, 128] full of standard-normal activations
    (E4M3 codes under the bound's scale, or bf16), tokens or heads outermost."""
    shape = (pages, heads, page, D) if head_major else (pages, page, heads, D)
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    if fp8:
        x = _e4m3(x * (E4M3_MAX / bound))
    return x.transpose(1, 2) if head_major else x


def _tables(gen, seq, page, spare):
    """Block tables of these sequences over randomly placed pages, and the
    number of pages of a pool with ``spare`` unused ones."""
    need = -(-seq // page)
    width = max(1, int(need.max()))
    total = int(need.sum())
    perm = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None]
    need_d = torch.as_tensor(need, device=DEV)[:, None]
    start = torch.as_tensor(np.cumsum(need) - need, device=DEV)[:, None]
    at = torch.where(col < need_d, start + col, 0)
    return torch.where(col < need_d, perm[at], -1).to(torch.int32).contiguous(), total + spare


def _scales():
    qs = torch.tensor([E4M3_MAX / b for b in BOUNDS], dtype=torch.float32, device=DEV)
    ds = torch.tensor([b / E4M3_MAX for b in BOUNDS], dtype=torch.float32, device=DEV)
    return qs, ds


def _tree_bits(rng, nodes):
    """Ancestor masks of random trees, [sum(nodes), 1] int64: node 0 is the
    root, every other node's parent is an earlier node (recent ones likelier)."""
    words = np.zeros((int(nodes.sum()), 1), dtype=np.uint64)
    at = 0
    for n in nodes:
        for i in range(int(n)):
            bits = np.uint64(1) << np.uint64(i)
            if i:
                bits |= words[at + max(0, i - 1 - int(rng.integers(0, 4))), 0]
            words[at + i, 0] = bits
        at += int(n)
    return torch.from_numpy(words.view(np.int64)).to(DEV)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def _cu(n):
    return _i32(np.concatenate([[0], np.cumsum(n)]))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, page = case["op"], case.get("page")
    s = {"op": op, "page": page}
    if op == "pages":
        seq, new = _lens(case)
        old = seq - new
        tables, num = _tables(gen, old, page, int((-(-seq // page)).sum()) + 100)
        width = int((-(-seq // page)).max())
        wide = torch.full((case["rows"], width), -1, dtype=torch.int32, device=DEV)
        wide[:, :min(width, tables.shape[1])] = tables[:, :width]
        owned = -(-old // page)
        used = int(owned.sum())
        held = torch.zeros(num, dtype=torch.bool, device=DEV)
        held[wide[wide >= 0].long()] = True
        left = torch.nonzero(~held).flatten().to(torch.int32)
        left = left[torch.randperm(left.numel(), generator=gen, device=DEV)]
        free = torch.full((num,), -1, dtype=torch.int32, device=DEV)
        free[:left.numel()] = left
        s |= {"seq": _i32(seq), "old": _i32(old), "new": _i32(new), "none": _i32(new * 0),
              "tables": wide, "owned": _i32(owned), "free": free,
              "pool": _i32([num - used, 0]), "tokens": int(new.sum()) + case["pad"]}
    elif op == "write":
        n, heads = case["tokens"], case["heads"]
        rows = n + case["pad"]
        if case["fused"]:     # slices of a [T, 3, H, 128] projection
            qkv = torch.empty(rows, 3, heads, D, dtype=torch.bfloat16, device=DEV)
            qkv.normal_(generator=gen)
            s["k"], s["v"] = qkv[:, 1], qkv[:, 2]
        else:
            s["k"] = torch.empty(rows, heads, D, dtype=torch.bfloat16, device=DEV)
            s["v"] = torch.empty_like(s["k"])
            s["k"].normal_(generator=gen)
            s["v"].normal_(generator=gen)
        # one sequence's new tokens in pages from anywhere in the pool (a
        # decoding step: single slots), the padding's slots -1
        pages = -(-n // page) + 3 if n > 256 else n + 3
        perm = torch.randperm(pages, generator=gen, device=DEV)
        t = torch.arange(n, device=DEV)
        slots = perm[t // page] * page + t % page if n > 256 else perm[:n] * page + t % page
        s["slots"] = torch.cat([slots, torch.full((case["pad"],), -1, device=DEV)]).to(torch.int64)
        s["n"] = n
        for i, name in ((1, "k_cache"), (2, "v_cache")):
            s[name] = _cache(gen, pages, page, heads, case["fp8"], case["head_major"], BOUNDS[i])
        s["scale"] = _scales()[0] if case["fp8"] else None
    else:
        seq, nodes = _lens(case)
        heads = case["kv_heads"] if op == "tree" else case["heads"]
        s["tables"], num = _tables(gen, seq, page, 5)
        hm = case.get("head_major", False)
        s["k_cache"] = _cache(gen, num, page, heads, case["fp8"], hm, BOUNDS[1])
        s["v_cache"] = _cache(gen, num, page, heads, case["fp8"], hm, BOUNDS[2])
        s |= {"seq": _i32(seq), "cu": _cu(nodes), "max_nodes": int(nodes.max()),
              "max_seq": int(seq.max())}
        if op == "tree":
            s["q"] = torch.empty(int(nodes.sum()), case["q_heads"], D, dtype=torch.bfloat16,
                                 device=DEV).normal_(generator=gen)
            s["mask"] = _tree_bits(np.random.Generator(np.random.PCG64(seed)), nodes) \
                if case["tree"] else None
            s["descale"] = _scales()[1] if case["fp8"] else None
        else:
            r = np.random.Generator(np.random.PCG64(seed))
            keep = _kept(case, nodes)
            paths = np.zeros((case["rows"], case["depth"]), dtype=np.int32)
            for b in range(case["rows"]):
                # an accepted path starts at the root
                paths[b, 1:keep[b]] = np.sort(r.choice(np.arange(1, nodes[b]), keep[b] - 1,
                                                       replace=False))
            s |= {"paths": _i32(paths), "keep": _i32(keep)}
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"pages": _run_pages, "write": _run_write, "tree": _run_tree, "keep": _run_keep}[s["op"]](s)


def _values(cache):
    """A cache as the numbers it stands for."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _run_pages(s):
    """A step's pages and slots, then the step taken back (a rejected draft, or
    the requests' end): the pool is as before."""
    args = (s["tables"], s["owned"], s["free"], s["pool"], s["page"])
    if own:
        import quantization_amax_reduce_b200 as qar
        cu, slots, positions = qar.kv_assign_pages(s["seq"], s["new"], *args, s["tokens"])
        qar.kv_assign_pages(s["old"], s["none"], *args, 0)
    else:
        cu, slots, positions = _plain_pages(s["seq"], s["new"], *args, s["tokens"])
        _plain_pages(s["old"], s["none"], *args, 0)
    return [cu, slots, positions, s["tables"], s["owned"], s["free"], s["pool"]]


def _plain_pages(seq, new, tables, owned, free, pool, page, tokens):
    dev, width = seq.device, tables.shape[1]
    want = (seq + page - 1) // page
    grow, drop = (want - owned).clamp(min=0), (owned - want).clamp(min=0)
    g0, d0 = grow.cumsum(0) - grow, drop.cumsum(0) - drop
    wanted, dropped, count = grow.sum(), drop.sum(), pool[0]
    col = torch.arange(width, device=dev)[None]
    # the dropped pages, by rank
    gone = (col >= want[:, None]) & (col < owned[:, None])
    rank = torch.where(gone, d0[:, None] + col - want[:, None], free.numel())
    by_rank = torch.full((free.numel() + 1,), -1, dtype=torch.int32, device=dev)
    by_rank.scatter_(0, rank.flatten(), torch.where(gone, tables, -1).flatten())
    # the wanted ones: dropped pages first, then the free list from its end
    fresh = (col >= owned[:, None]) & (col < want[:, None])
    k = torch.where(fresh, g0[:, None] + col - owned[:, None], 0)
    got = torch.where(k < dropped, by_rank[k.clamp(max=free.numel())],
                      free[(count - 1 - (k - dropped)).clamp(0, free.numel() - 1)])
    tables.copy_(torch.where(fresh, got, tables))
    # what was dropped and not wanted goes back
    i = torch.arange(free.numel(), device=dev)
    back = count + dropped - 1 - i
    put = (i >= count) & (back >= wanted) & (back < dropped)
    free.copy_(torch.where(put, by_rank[back.clamp(0, free.numel())], free))
    pool[0] = count + dropped - wanted
    owned.copy_(want)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
    t = torch.arange(tokens, device=dev)
    row = torch.searchsorted(cu[1:], t.to(torch.int32), right=True)
    inside = row < new.numel()
    row = row.clamp(max=new.numel() - 1)
    pos = torch.where(inside, (seq - new)[row] + t - cu[row], 0)
    slot = tables[row, pos // page].long() * page + pos % page
    return cu, torch.where(inside, slot, -1), pos.to(torch.int32)


def _run_write(s):
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    if own:
        import quantization_amax_reduce_b200 as qar
        qar.kv_write(s["k"], s["v"], s["slots"], k_cache, v_cache, s["scale"])
    else:
        at = s["slots"][:s["n"]]
        page, off = at // s["page"], at % s["page"]
        for i, x, cache in ((1, s["k"], k_cache), (2, s["v"], v_cache)):
            x = x[:s["n"]]
            if s["scale"] is not None:
                x = _e4m3(x.float() * s["scale"][i])
            cache[page, off] = x
    return [_values(k_cache), _values(v_cache)]


def _run_tree(s):
    if own:
        import quantization_amax_reduce_b200 as qar
        return qar.kv_tree_fwd(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq"], s["cu"],
                               s["max_nodes"], s["max_seq"], s["descale"], s["mask"])
    q, tables, seq, cu, page = s["q"], s["tables"], s["seq"].long(), s["cu"].long(), s["page"]
    dev, (T, hq, _) = q.device, q.shape
    hkv = s["k_cache"].shape[2]
    g, B, N, L = hq // hkv, seq.numel(), s["max_nodes"], tables.shape[1] * page
    n = cu[1:] - cu[:-1]
    at = tables.clamp(min=0)

    def keys(cache, i):        # [B, Hkv, L, 128] in 32 bits
        x = _values(cache[at]).float().reshape(B, L, hkv, D).transpose(1, 2)
        return x * s["descale"][i] if s["descale"] is not None else x

    i = torch.arange(N, device=dev)
    tok = (cu[:-1, None] + i).clamp(max=T - 1)                          # [B, N]
    qn = q[tok].float().view(B, N, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * g, D)
    score = qn @ keys(s["k_cache"], 1).transpose(2, 3) * (1 / math.sqrt(D))
    # which keys a node sees: the context, and its nodes by the mask's bits
    j = torch.arange(L, device=dev) - (seq - n)[:, None]                # [B, L], node of a key
    if s["mask"] is not None:
        word = s["mask"][tok][:, :, 0]                                  # [B, N]
        seen = (word[:, :, None] >> j[:, None].clamp(0, 63)) & 1 == 1
    else:
        seen = j[:, None] <= i[:, None]
    seen = ((j < 0)[:, None] | (seen & (j < n[:, None])[:, None])).repeat_interleave(g, 1)[:, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp()
    out = (p @ keys(s["v_cache"], 2)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.view(B, hkv, N, g, D).permute(0, 2, 1, 3, 4).reshape(B, N, hq, D)
    row = torch.searchsorted(cu[1:], torch.arange(T, device=dev), right=True)
    return out[row, torch.arange(T, device=dev) - cu[row]].to(torch.bfloat16)


def _run_keep(s):
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    if own:
        import quantization_amax_reduce_b200 as qar
        qar.kv_keep_path(k_cache, v_cache, s["tables"], s["seq"], s["cu"], s["paths"], s["keep"])
    else:
        page, n = s["page"], s["cu"][1:] - s["cu"][:-1]
        i = torch.arange(s["paths"].shape[1], device=n.device)
        start = (s["seq"] - n)[:, None]
        # entries past the path copy a node that stays where it is
        still = torch.minimum(i, n[:, None] - 1)
        live = i < s["keep"][:, None]
        src = start + torch.where(live, s["paths"], still)
        dst = start + torch.where(live, i, still)
        sp, so = s["tables"].gather(1, (src // page).long()), src % page
        dp, do = s["tables"].gather(1, (dst // page).long()), dst % page
        for cache in (k_cache, v_cache):
            cache[dp, do] = cache[sp, so]
    return [_values(k_cache), _values(v_cache)]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What ``run`` returns on a new state, row by row from the definition in
    64 bits; nothing for page tables, which are whole numbers."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "write":
        out = []
        for i, x, cache in ((1, s["k"], s["k_cache"]), (2, s["v"], s["v_cache"])):
            c = _values(cache).double().clone(memory_format=torch.contiguous_format)
            flat = c.view(-1, *c.shape[2:])
            x = x.double()
            if s["scale"] is not None:
                x = (x * s["scale"][i].double()).clamp(-E4M3_MAX, E4M3_MAX)
            flat[s["slots"][:s["n"]]] = x[:s["n"]]
            out.append(c)
        return out
    seq, cu = s["seq"].tolist(), s["cu"].tolist()
    if case["op"] == "keep":
        out = []
        paths, keep = s["paths"].tolist(), s["keep"].tolist()
        for cache in (s["k_cache"], s["v_cache"]):
            c = _values(cache).double().clone(memory_format=torch.contiguous_format)
            flat = c.view(-1, *c.shape[2:])
            for b in range(len(seq)):
                first = seq[b] - (cu[b + 1] - cu[b])
                pos = torch.arange(seq[b], device=DEV)
                slot = s["tables"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]
                moved = flat[slot[[first + m for m in paths[b][:keep[b]]]]]
                flat[slot[first:first + keep[b]]] = moved
            out.append(c)
        return out
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    hq, hkv = s["q"].shape[1], s["k_cache"].shape[2]
    ds = s["descale"].double().tolist() if s["descale"] is not None else [1.0] * 3
    for b, length in enumerate(seq):
        a, z = cu[b], cu[b + 1]
        n, pages = z - a, s["tables"][b, :-(-length // s["page"])].long()
        sees = torch.ones(n, length, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            sees[:, length - n:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        else:
            words = s["mask"][a:z, 0].cpu().numpy().view(np.uint8).reshape(n, 8)
            bits = np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)
            sees[:, length - n:] = torch.from_numpy(bits).to(DEV)
        for h in range(hkv):
            k = _values(s["k_cache"][pages, :, h]).double().reshape(-1, D)[:length] * ds[1]
            v = _values(s["v_cache"][pages, :, h]).double().reshape(-1, D)[:length] * ds[2]
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.einsum("ngd,ld->ngl", s["q"][a:z, heads].double(), k) / math.sqrt(D)
            x = torch.where(sees[:, None], x, -math.inf)
            w = torch.softmax(x, -1).nan_to_num(0.0)
            out[a:z, heads] = torch.einsum("ngl,ld->ngd", w, v)
    return out
