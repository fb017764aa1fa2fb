"""Cases for measuring the paged-cache operators around models with normed
heads, sliding windows with sinks, and drafted tokens: append with norms,
attention with sinks, attention of a tree of drafted tokens, keeping a tree's
accepted path, and forking sequences with copy on write.

``run`` computes them in plain torch operations (``own`` false) or through the
package's entry points (``own`` true).  Attention and append are one layer's
call of a serving step, keep and fork one call for the whole cache.  Shapes
are those of this repository's workloads: 8 KV heads x 128 (64 query heads, 80
layers), 32 or 40 heads x 128 without grouping, 4 layers of 4 x 128 (tiny).

A case's fields: ``op``; ``heads``, ``kv_heads``, ``head_dim``; ``page``
(tokens in a page); ``io`` and ``cache`` (types); ``lens`` (tokens of each
sequence in the cache, the new ones included; 0 is an unused slot of a padded
batch); ``new`` (new tokens of each sequence, "" for one each); ``tree`` (the
number that the drafted tokens' tree is made from, 0: no tree).
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
LAYERS, LAYER = 2, 1  # append and attention run on one layer of a pool of two
EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# ceilings for drawn cases, below the largest listed case of each operator
APPEND_BYTES = 400_000_000
SINK_BYTES = 700_000_000
PROMPT_FLOPS = 300_000_000_000
TREE_BYTES = 700_000_000
TREE_FLOPS = 250_000_000_000
POOL_BYTES = 1_300_000_000  # of keep's and fork's caches


def _ints(text):
    return [int(x) for x in text.split()] if text else []


def _text(values):
    return " ".join(str(int(v)) for v in values)


def _spread(seed, n, lo, hi):
    """n lengths between lo and hi, spread over their logarithm."""
    r = random.Random(seed)
    return [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(n)]


def _case(name, op, heads, kv_heads, head_dim, page, io, cache, lens, new="", **more):
    c = dict(name=name, op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
             io=io, cache=cache, lens=lens, new=new, tree=0)
    c.update(more)
    return c


def listed():
    return [
        # one decode step of eight streams of a model with normed heads: all latency
        _case("norm-step", "append", 64, 8, 128, 16, "bf16", "f16",
              _text(_spread(1, 8, 1000, 16000)), rotary=128, interleaved=False),
        # a whole context of an ungrouped model, rotation of half of each head
        _case("norm-context", "append", 40, 40, 128, 64, "bf16", "bf16", "9000 1 77",
              "7000 1 77", rotary=64, interleaved=True),
        # one stream deep in its context, a chunk's worth of window: latency
        _case("sinks-one", "sinks", 64, 8, 128, 16, "f16", "f16", "16000", window=1024, sinks=4),
        # a padded batch, pages that do not fit the tiles, some shorter than the window
        _case("sinks-batch", "sinks", 64, 8, 128, 20, "bf16", "f16",
              _text(_spread(3, 44, 2000, 16000) + [0, 1, 0, 4099]), window=4096, sinks=16),
        # prompts behind restored contexts and a fresh one
        _case("sinks-prompt", "sinks_prompt", 64, 8, 128, 16, "bf16", "f16", "17500 9011 4001 1",
              "1500 1011 4001 1", window=2048, sinks=4),
        # a tree of 26 drafted tokens of one stream over a restored context: latency
        _case("tree-one", "tree", 64, 8, 128, 16, "f16", "f16", "16026", "26", tree=11),
        # short drafts of an ungrouped model, contexts spread
        _case("tree-draft", "tree", 32, 32, 128, 32, "bf16", "bf16",
              _text(_spread(4, 12, 900, 9000)), _text([5, 8, 3, 8, 1, 6, 8, 7, 2, 8, 8, 4]),
              tree=12),
        # larger trees of a batch with an unused slot
        _case("tree-batch", "tree", 64, 8, 128, 16, "bf16", "f16",
              _text(_spread(5, 15, 1500, 16000) + [0]), _text([60, 33, 17, 60] * 4), tree=13),
        # one stream's accepted path, the tiny cache
        _case("keep-one", "keep", 4, 4, 128, 16, "f16", "f16", "1526", "26", kept="5", layers=4,
              tree=14),
        # a batch's accepted paths through the 70B-shaped cache
        _case("keep-batch", "keep", 64, 8, 128, 16, "bf16", "f16",
              _text(_spread(6, 47, 64, 200) + [0]), _text([60, 33, 17, 60] * 12),
              kept=_text([1 + (7 * i) % 8 for i in range(47)] + [0]), layers=80, tree=15),
        # four continuations of one stream's chunk
        _case("fork-one", "fork", 64, 8, 128, 16, "f16", "f16", "1511", forks="4", layers=4),
        # sixteen streams' continuations, large pages: most of it is copy on write
        _case("fork-batch", "fork", 64, 8, 128, 64, "bf16", "bf16",
              _text(_spread(7, 15, 64, 512) + [128]), forks=_text([4, 3, 5, 4] * 4), layers=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "sinks", "sinks", "sinks_prompt", "tree", "tree", "tree",
                     "keep", "fork"])
    head_dim = rng.choice([64, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
    while kv_heads * group > 96:
        group = max(1, group // 2)
    heads = kv_heads * group
    page = rng.choice([1, 8, 10, 16, 16, 20, 32, 48, 64, 128, _log(rng, 1, 300)])
    io, cache = rng.choice([("f16", "f16"), ("bf16", "bf16"), ("bf16", "f16")])
    row = 4 * kv_heads * head_dim  # bytes of one token's K and V
    c = dict(op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, io=io,
             cache=cache, tree=0)
    if op == "append":
        seqs = _log(rng, 1, 64)
        longest = min(9000, max(1, APPEND_BYTES // (2 * (2 * heads * head_dim + row)) // seqs))
        form = rng.choice(["single", "prompt", "drafts"])
        if form == "single":
            new = [1] * seqs
        elif form == "drafts":
            new = [_log(rng, 1, min(longest, 64)) for _ in range(seqs)]
            c["tree"] = rng.randrange(1, 1 << 30)
        else:
            new = [_log(rng, 1, longest) for _ in range(seqs)]
        lens = [n + rng.choice([0, rng.randrange(0, 4000)]) for n in new]
        c.update(lens=_text(lens), new="" if form == "single" else _text(new),
                 rotary=rng.choice([head_dim, head_dim // 2, 32]),
                 interleaved=rng.random() < 0.5)
        return c
    if op in ("sinks", "sinks_prompt"):
        c.update(window=_log(rng, 16, 8000), sinks=rng.choice([1, 4, 4, 16, _log(rng, 1, 300)]))
    if op == "sinks":
        seqs = _log(rng, 1, 64)
        seen = c["window"] + c["sinks"]
        while seqs > 1 and seqs * min(seen, 16000) * row > SINK_BYTES:
            seqs = (seqs + 1) // 2
        lens = [_log(rng, 1, 32000 if seqs < 8 else 8000) for _ in range(seqs)]
        if seqs > 2 and rng.random() < 0.3:
            lens[rng.randrange(seqs)] = 0
        c.update(lens=_text(lens), new="")
        return c
    if op == "sinks_prompt":
        seqs = _log(rng, 1, 8)
        new = [_log(rng, 1, 2500) for _ in range(seqs)]
        lens = [n + rng.choice([0, _log(rng, 1, 16000)]) for n in new]
        while 4 * heads * head_dim * _pairs(new, lens, c["window"], c["sinks"]) > PROMPT_FLOPS:
            new = [max(1, n // 2) for n in new]
            lens = [max(n, m // 2) for n, m in zip(new, lens)]
        c.update(lens=_text(lens), new=_text(new))
        return c
    if op == "tree":
        seqs = _log(rng, 1, 32)
        most = rng.choice([4, 8, 16, 32, 64, 150])
        new = [_log(rng, 1, most) for _ in range(seqs)]
        lens = [n + _log(rng, 1, 16000) for n in new]
        while (sum(lens) * row > TREE_BYTES
               or 4 * heads * head_dim * sum(a * b for a, b in zip(new, lens)) > TREE_FLOPS):
            lens = [n + max(1, (m - n) // 2) for n, m in zip(new, lens)]
        if seqs > 2 and rng.random() < 0.3:
            lens[rng.randrange(seqs)] = 0
        c.update(lens=_text(lens), new=_text(new), tree=rng.randrange(1, 1 << 30))
        return c
    c["layers"] = layers = _log(rng, 1, 64)
    slots = POOL_BYTES // (row * layers)  # tokens that the cache may hold
    if op == "keep":
        seqs = _log(rng, 1, 48)
        new = [_log(rng, 2, 64) for _ in range(seqs)]
        lens = [n + _log(rng, 1, 400) for n in new]
        while sum(lens) + (seqs + 7) * page > slots and seqs > 1:
            seqs = (seqs + 1) // 2
            new, lens = new[:seqs], lens[:seqs]
        kept = [rng.randrange(0, n // 2 + 1) for n in new]
        c.update(lens=_text(lens), new=_text(new), kept=_text(kept), tree=rng.randrange(1, 1 << 30))
        return c
    seqs = _log(rng, 1, 32)
    lens = [_log(rng, 1, 1000) for _ in range(seqs)]
    forks = [rng.randrange(0, 6) for _ in range(seqs)]
    while seqs > 1 and sum(lens) + (seqs + sum(forks) + 7) * page > slots:
        seqs = (seqs + 1) // 2
        lens, forks = lens[:seqs], forks[:seqs]
    c.update(lens=_text(lens), new="", forks=_text([forks[0] + 1] + forks[1:]))
    return c


# ------------------------------------------------------------------- trees
def _parents(case):
    """For each sequence its drafted tokens' parents (-1: the cached context).
    Token 0 is the last accepted one; the others hang on an earlier token, the
    one before them often, as a drafter's best guesses do."""
    rng = random.Random(case["tree"])
    trees = []
    for n in _ints(case["new"]):
        t = [-1]
        for i in range(1, n):
            t.append(i - 1 if rng.random() < 0.4 else rng.randrange(max(0, i - 9), i))
        trees.append(t)
    return trees


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


# ------------------------------------------------------------------ work
def _visible(pos, window, sinks):
    """Keys that a token at position pos sees."""
    lo = max(pos + 1 - window, 0) if window else 0
    return max(pos + 1 - lo, 0) + max(min(sinks, lo), 0)


def _pairs(new, lens, window, sinks):
    """(new token, visible key) pairs of a batch."""
    return sum(_visible(m - n + i, window, sinks) for n, m in zip(new, lens) for i in range(n))


def _counts(case):
    lens = _ints(case["lens"])
    new = _ints(case["new"]) or [1] * len(lens)
    return lens, new


def _fork_copies(case):
    """Tokens that copy on write copies."""
    return sum(f * (m % case["page"]) for m, f in zip(_ints(case["lens"]), _ints(case["forks"])))


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    lens, new = _counts(case)
    if case["op"] == "keep":
        moved = 0
        for n, m, k in zip(new, lens, _ints(case["kept"])):
            moved += sum(1 for i, s in enumerate(_path(n, k)) if i != s) if m else 0
        return {"bytes": 2 * case["layers"] * 2 * moved * hk * d * 2, "flops": 0}
    if case["op"] == "fork":
        copied = 2 * case["layers"] * 2 * _fork_copies(case) * hk * d * 2
        pages = sum((f + 1) * ((m + case["page"] - 1) // case["page"])
                    for m, f in zip(lens, _ints(case["forks"])))
        return {"bytes": copied + 8 * pages, "flops": 0}
    n_tok = sum(n for n, m in zip(new, lens) if m)
    if case["op"] == "append":
        moved = 2 * n_tok * (h + 2 * hk) * d * 2
        return {"bytes": moved + n_tok * case["rotary"] * 4,
                "flops": n_tok * (h + hk) * (3 * case["rotary"] + 4 * d)}
    if case["op"] == "tree":
        seen = sum(lens)
        pairs = sum(n * (m - n) + sum(_depths(t)) + n
                    for n, m, t in zip(new, lens, _parents(case)) if m)
    else:
        window, sinks = case["window"], case["sinks"]
        seen = sum(min(m, max(m - n, 0) - max(m - n - window + 1, 0) + n
                       + max(min(sinks, m - n - window + 1), 0)) for n, m in zip(new, lens))
        pairs = _pairs(new, lens, window, sinks)
    return {"bytes": seen * 2 * hk * d * 2 + 2 * n_tok * h * d * 2 + n_tok * h * 4,
            "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------- prepare
def _values(gen, rows, channels, dtype):
    """Keys or values as the codec's workloads have them: per channel a mean
    and a spread of its own, every hundredth channel eight times as wide."""
    mu = torch.randn(channels, generator=gen, device=DEVICE)
    s = torch.exp(0.5 * torch.randn(channels, generator=gen, device=DEVICE))
    wide = torch.randperm(channels, generator=gen, device=DEVICE)[: max(1, channels // 100)]
    s[wide] *= 8
    x = torch.randn((rows, channels), generator=gen, device=DEVICE)
    return (x * s + mu).to(dtype)


def _path(n, kept):
    """The accepted path: drafted token 0, some that follow it at once, then
    later ones.  None is a place that the path itself moves tokens to, so a
    second pass on the same cache finds the same tokens."""
    a = (kept + 1) // 2
    rest = kept - a
    return list(range(a)) + [kept + (j * (n - kept)) // rest for j in range(rest)]


def _table(rng, need, spare=7, width=0):
    """A page table of scattered pages (unused entries -1) and the pool's size."""
    n_pages = sum(need) + spare
    ids = list(range(n_pages))
    rng.shuffle(ids)
    width = max(need + [width, 1])
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return table, n_pages


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, h, hk, d, page = (case["op"], case["heads"], case["kv_heads"], case["head_dim"],
                          case["page"])
    io, cache = TYPES[case["io"]], TYPES[case["cache"]]
    c = hk * d
    lens, new = _counts(case)
    need = [(m + page - 1) // page for m in lens]
    spare, width = 7, 0
    if op == "fork":
        forks = _ints(case["forks"])
        spare, width = sum(forks) + 7, max(need) + 1
    table, n_pages = _table(rng, need, spare, width)
    layers = case.get("layers", LAYERS)
    st = {"case": case, "lens_host": lens, "new_host": new, "n_pages": n_pages}
    pool = torch.zeros((layers, 2, n_pages * page, c), dtype=cache, device=DEVICE)
    st["pool"] = pool
    if op in ("keep", "fork"):
        for layer in range(layers):
            for kv in range(2):
                pool[layer, kv] = _values(gen, pool.shape[2], c, cache)
    else:
        for kv in range(2):
            pool[LAYER, kv] = _values(gen, n_pages * page, c, cache)
    if op == "fork":
        # the rows behind the streams' are their continuations', empty at first
        table += [[-1] * width for _ in range(sum(forks))]
        st["src_host"] = [b for b, f in enumerate(forks) for _ in range(f)]
        st["dst_host"] = [len(lens) + i for i in range(sum(forks))]
        refs = [0] * n_pages
        for row, n in zip(table, need):
            for page_id in row[:n]:
                refs[page_id] += 1
        st["refs"] = _int32(refs)
        st["src"], st["dst"] = _int32(st["src_host"]), _int32(st["dst_host"])
        st["lens"] = _int32(lens + [0] * sum(forks))
        # each continuation gets room for one more token
        st["new_lens_host"] = lens + [lens[b] + 1 for b in st["src_host"]]
        st["new_lens"] = _int32(st["new_lens_host"])
    else:
        st["lens"] = _int32(lens)
    st["table"] = _int32(table)
    n_tok = sum(new)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    st["start_host"] = start
    if case["new"]:
        st["q_start"] = _int32(start)
    if case["tree"]:
        trees = _parents(case)
        st["parent"] = _int32([p for t in trees for p in t])
        st["depth_host"] = [x for t in trees for x in _depths(t)]
        st["depth"] = torch.tensor(st["depth_host"], device=DEVICE)
    if op == "keep":
        kept = _ints(case["kept"])
        st["path_host"] = [_path(n, k) for n, k in zip(new, kept)]
        wide = max(kept + [1])
        st["path"] = _int32([p + [0] * (wide - len(p)) for p in st["path_host"]])
        st["kept"] = _int32(kept)
        st["new_lens"] = torch.zeros_like(st["lens"])
    elif op == "append":
        # q, k and v are slices of one projection's rows, as a model has them
        qkv = torch.empty((n_tok, (h + 2 * hk) * d), dtype=io, device=DEVICE)
        qkv[:, :h * d] = torch.randn((n_tok, h * d), generator=gen, device=DEVICE).to(io)
        qkv[:, h * d:(h + hk) * d] = _values(gen, n_tok, c, io)
        qkv[:, (h + hk) * d:] = _values(gen, n_tok, c, io)
        st["q"] = qkv[:, :h * d].unflatten(1, (h, d))
        st["k"] = qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
        st["v"] = qkv[:, (h + hk) * d:].unflatten(1, (hk, d))
        st["q_out"] = torch.zeros((n_tok, h, d), dtype=io, device=DEVICE)
        for name in ("q_weight", "k_weight"):
            st[name] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=DEVICE)
        r = case["rotary"]
        inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEVICE) / r)
        ang = torch.arange(max(lens), dtype=torch.float64, device=DEVICE)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    elif op != "fork":
        st["q"] = torch.randn((n_tok, h, d), generator=gen, device=DEVICE).to(io)
        st["out"] = torch.zeros((n_tok, h, d), dtype=io, device=DEVICE)
        st["lse"] = torch.zeros((n_tok, h), dtype=torch.float32, device=DEVICE)
        if op == "tree":
            # the tree's shape is the drafter's, the same every step: which
            # drafted tokens each one sees is laid out once
            st["see"] = [torch.tensor(_ancestors(t), device=DEVICE) for t in trees]
    if own:
        import kv_cache_compression_decode_amd as kvc

        st["desc"] = kvc.make_paged_desc(layers, h, hk, d, page, n_pages, cache_dtype=cache,
                                         io_dtype=io)
        if op == "fork":
            st["ledger"] = kvc.PageLedger(st["desc"], st["table"], st["lens"], st["refs"])
            return st
        st["batch"] = kvc.PagedBatch(st["table"], st["lens"], q_start=st.get("q_start"),
                                     max_len=max(lens))
        if op == "keep":
            st["status"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)
            return st
        if case["tree"]:
            st["draft"] = kvc.Tree(st["parent"], max(new))
        st["wsp"] = kvc.PagedWorkspace(st["desc"], st["batch"], n_tok, tree=st.get("draft"))
        if case["tree"]:
            kvc.tree_async(st["desc"], st["batch"], st["draft"], st["wsp"])
        if op == "append":
            st["rope"] = kvc.Rope(st["cos_sin"], interleaved=case["interleaved"])
            st["norm"] = kvc.HeadNorm(st["q_weight"], st["k_weight"], EPS)
    return st


# -------------------------------------------------------------------- run
def _run_own(st):
    import kv_cache_compression_decode_amd as kvc

    case = st["case"]
    op = case["op"]
    if op == "append":
        kvc.append_async(st["desc"], st["batch"], LAYER, st["pool"], st["k"], st["v"], st["wsp"],
                         rope=st["rope"], q=st["q"], q_out=st["q_out"], norm=st["norm"],
                         tree=st.get("draft"))
        return st["pool"], st["q_out"]
    if op == "keep":
        kvc.keep_async(st["desc"], st["batch"], st["pool"], st["path"], st["kept"],
                       st["new_lens"], st["start_host"][-1], st["status"])
        return st["pool"], st["new_lens"]
    if op == "fork":
        kvc.fork_async(st["ledger"], st["src"], st["dst"])
        kvc.resize_async(st["ledger"], st["pool"], st["new_lens"])
        return st["pool"], st["table"], st["lens"], st["refs"]
    if op == "tree":
        kvc.attend_tree_async(st["desc"], st["batch"], st["draft"], LAYER, st["pool"], st["q"],
                              st["out"], st["wsp"], lse=st["lse"])
        return st["out"], st["lse"]
    attend = kvc.attend_async if op == "sinks" else kvc.attend_prompt_async
    attend(st["desc"], st["batch"], LAYER, st["pool"], st["q"], st["out"], st["wsp"],
           window=case["window"], lse=st["lse"], sinks=case["sinks"])
    return st["out"], st["lse"]


def _slots(table_row, pos, page):
    """Token slots of the pool for positions pos of one sequence."""
    return table_row[pos // page].long() * page + pos % page


def _norm(x, weight):
    """x [tokens, heads, dim] float."""
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _rotate(x, cos, sin, rotary, interleaved):
    """x [tokens, heads, dim] float, cos and sin [tokens, rotary / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    rot, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :rotary // 2], rot[..., rotary // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _append_plain(st):
    case, lens, new = st["case"], st["lens_host"], st["new_host"]
    page, r, inter = case["page"], case["rotary"], case["interleaved"]
    pool, q_out = st["pool"], st["q_out"]
    counts = torch.tensor(new, device=DEVICE)
    total = sum(new)
    seq = torch.repeat_interleave(torch.arange(len(new), device=DEVICE), counts, output_size=total)
    first = torch.tensor([m - n - s for m, n, s in zip(lens, new, st["start_host"])],
                         device=DEVICE)
    row = torch.arange(total, device=DEVICE)
    pos = first[seq] + row
    slot = st["table"][seq, pos // page].long() * page + pos % page
    if "depth" in st:  # drafted tokens stand at their depth's position
        pos = torch.tensor([m - n for m, n in zip(lens, new)], device=DEVICE)[seq] + st["depth"]
    cs = st["cos_sin"][pos]
    cos, sin = cs[:, :r // 2], cs[:, r // 2:]
    q_out.copy_(_rotate(_norm(st["q"].float(), st["q_weight"]), cos, sin, r, inter))
    k = _rotate(_norm(st["k"].float(), st["k_weight"]), cos, sin, r, inter)
    pool[LAYER, 0, slot] = k.flatten(1).to(pool.dtype)
    pool[LAYER, 1, slot] = st["v"].float().flatten(1).to(pool.dtype)
    return pool, q_out


def _attend_rows(q, k, v, hidden, scale):
    """q [n, heads, d], k and v [m, kv_heads, d], hidden [n, m] or None: out
    and log-sum-exp."""
    n, h, d = q.shape
    m, hk, _ = k.shape
    g = h // hk
    rows = q.view(n, hk, g, d).permute(1, 0, 2, 3).reshape(hk, n * g, d)
    s = torch.bmm(rows, k.permute(1, 2, 0).contiguous()) * scale
    if hidden is not None:
        s.view(hk, n, g, m).masked_fill_(hidden[None, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, v.permute(1, 0, 2).contiguous()) / total
    lse = top + total.log()
    return (out.view(hk, n, g, d).permute(1, 0, 2, 3).reshape(n, h, d),
            lse.view(hk, n, g).permute(1, 0, 2).reshape(n, h))


def _attend_plain(st):
    case = st["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    out, lse, pool = st["out"], st["lse"], st["pool"]
    for b, (m, n) in enumerate(zip(st["lens_host"], st["new_host"])):
        a = st["start_host"][b]
        if m == 0:
            out[a:a + n] = 0
            lse[a:a + n] = float("-inf")
            continue
        for i0 in range(0, n, 1024):  # the scores of 1,024 tokens at a time
            i1 = min(n, i0 + 1024)
            # the first rows' window and what follows it; the sinks before it
            end = m - n + i1
            lo = max(0, m - n + i0 + 1 - window) if window else 0
            pos = torch.arange(lo, end, device=DEVICE)
            if min(sinks, lo):
                pos = torch.cat([torch.arange(min(sinks, lo), device=DEVICE), pos])
            slot = _slots(st["table"][b], pos, page)
            k = pool[LAYER, 0, slot].float().view(-1, hk, d)
            v = pool[LAYER, 1, slot].float().view(-1, hk, d)
            hidden = None
            if case["op"] == "tree":
                hidden = torch.zeros((n, m), dtype=torch.bool, device=DEVICE)
                hidden[:, m - n:] = ~st["see"][b]
                hidden = hidden[i0:i1, :end]
            elif n > 1:
                t = torch.arange(m - n + i0, end, device=DEVICE)[:, None]
                hidden = pos[None] > t
                if window:
                    hidden = hidden | ((pos[None] <= t - window) & (pos[None] >= sinks))
            q = st["q"][a + i0:a + i1].float()
            o, e = _attend_rows(q, k, v, hidden, d ** -0.5)
            out[a + i0:a + i1] = o.to(out.dtype)
            lse[a + i0:a + i1] = e
    return out, lse


def _keep_plain(st):
    case, page = st["case"], st["case"]["page"]
    src, dst = [], []
    for b, path in enumerate(st["path_host"]):
        base = st["lens_host"][b] - st["new_host"][b]
        src += [(b, base + s) for s in path]
        dst += [(b, base + i) for i in range(len(path))]
    if src:
        b, s, t = torch.tensor([(b, s, t) for (b, s), (_, t) in zip(src, dst)], device=DEVICE).T
        table = st["table"]
        s = table[b, s // page].long() * page + s % page
        t = table[b, t // page].long() * page + t % page
        st["pool"].index_copy_(2, t, st["pool"][:, :, s])
    n = torch.tensor(st["new_host"], dtype=torch.int32, device=DEVICE)
    new_lens = torch.where(st["lens"] > 0, st["lens"] - n + st["kept"], st["lens"])
    st["new_lens"].copy_(new_lens)
    return st["pool"], st["new_lens"]


def _fork_plain(st):
    page, table, lens, refs = st["case"]["page"], st["table"], st["lens"], st["refs"]
    src, dst, pool = st["src"].long(), st["dst"].long(), st["pool"]
    entry = torch.arange(table.shape[1], device=DEVICE)
    # what the continuations of the last step held is given back
    for rows, sign in ((dst, -1), (src, 1)):
        held = entry[None] < ((lens[rows] + page - 1) // page)[:, None]
        ids = torch.where(held, table[rows], 0).flatten().long()
        refs.index_add_(0, ids, (sign * held.flatten()).int())
        if sign > 0:
            table[dst] = torch.where(held, table[rows], table[dst])
    lens[dst] = lens[src]
    # room for the next token: a new page each, into which the shared page's
    # tokens are copied where it is only partly filled
    n = dst.numel()
    new = torch.sort(refs != 0, stable=True).indices[:n]  # the lowest free pages
    last = lens[dst].long() // page
    part = lens[dst].long() % page
    old = torch.where(part > 0, table[dst, last], -1).long()
    table[dst, last] = new.int()
    refs[new] = 1
    refs.index_add_(0, old.clamp(min=0), -(old >= 0).int())
    lens.copy_(st["new_lens"])
    for i, b in enumerate(st["src_host"]):
        r = st["lens_host"][b] % page
        if r:
            t = torch.arange(r, device=DEVICE)
            pool.index_copy_(2, new[i] * page + t, pool[:, :, old[i] * page + t])
    return pool, table, lens, refs


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "append":
        return _append_plain(state)
    if op == "keep":
        return _keep_plain(state)
    if op == "fork":
        return _fork_plain(state)
    return _attend_plain(state)


# ------------------------------------------------------------------ exact
def _ancestors(parents):
    """see[i][t]: token i of the tree sees token t (itself and what it hangs on)."""
    see = []
    for i, p in enumerate(parents):
        row = list(see[p]) if p >= 0 else [False] * len(parents)
        row[i] = True
        see.append(row)
    return see


def _exact_fork(st):
    page, table = st["case"]["page"], st["table"].tolist()
    refs, lens = st["refs"].tolist(), st["lens"].tolist()
    pool = st["pool"].clone()
    for s, t in zip(st["src_host"], st["dst_host"]):
        for e in range((lens[s] + page - 1) // page):
            table[t][e] = table[s][e]
            refs[table[s][e]] += 1
        lens[t] = lens[s]
    for b, n in enumerate(st["new_lens_host"]):
        e = lens[b] // page
        if n > lens[b] and (lens[b] % page == 0 or refs[table[b][e]] > 1):
            new = refs.index(0)
            refs[new] = 1
            if lens[b] % page:
                old = table[b][e]
                refs[old] -= 1
                pool[:, :, new * page:new * page + lens[b] % page] = \
                    pool[:, :, old * page:old * page + lens[b] % page]
            table[b][e] = new
        lens[b] = n
    return pool, _int32(table), _int32(lens), _int32(refs)


def exact(case, seed):
    """The operators' definitions in 64 bits, token by token or head by head."""
    st = prepare(case, seed)
    op, h, hk, d, page = (case["op"], case["heads"], case["kv_heads"], case["head_dim"],
                          case["page"])
    if op == "fork":
        return _exact_fork(st)
    lens, new, table = st["lens_host"], st["new_host"], st["table"].tolist()
    if op == "keep":
        pool = st["pool"].clone()
        after = list(lens)
        for b, path in enumerate(st["path_host"]):
            if lens[b] == 0:
                continue
            base = lens[b] - new[b]
            for i, s in enumerate(path):
                s, t = base + s, base + i
                pool[:, :, table[b][t // page] * page + t % page] = \
                    st["pool"][:, :, table[b][s // page] * page + s % page]
            after[b] = base + len(path)
        return pool, _int32(after)
    if op == "append":
        r = case["rotary"]
        pool = st["pool"].double()
        pos, slots, rows = [], [], []
        for b, (m, n) in enumerate(zip(lens, new)):
            for i in range(n):
                t, row = m - n + i, st["start_host"][b] + i
                rows.append(row)
                pos.append(m - n + st["depth_host"][row] if case["tree"] else t)
                slots.append(table[b][t // page] * page + t % page)
        pos = torch.tensor(pos, dtype=torch.float64, device=DEVICE)
        slots = torch.tensor(slots, device=DEVICE)
        rows = torch.tensor(rows, device=DEVICE)
        # each pair is a complex number, turned by position * 10000^(-2i/r)
        freq = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device=DEVICE) / r)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                           pos[:, None] * freq[None])[:, None]
        even = torch.arange(r // 2, device=DEVICE)
        if case["interleaved"]:
            ia, ib = 2 * even, 2 * even + 1
        else:
            ia, ib = even, even + r // 2

        def turned(x, weight):
            x = x.double()
            x = x / torch.sqrt((x.square().sum(-1, keepdim=True) / d + EPS)) * weight.double()
            z = torch.complex(x[..., ia], x[..., ib]) * turn
            y = x.clone()
            y[..., ia], y[..., ib] = z.real, z.imag
            return y

        pool[LAYER, 0, slots] = turned(st["k"][rows], st["k_weight"]).flatten(1)
        pool[LAYER, 1, slots] = st["v"][rows].double().flatten(1)
        q_out = torch.zeros((sum(new), h, d), dtype=torch.float64, device=DEVICE)
        q_out[rows] = turned(st["q"][rows], st["q_weight"])
        return pool, q_out
    window, sinks, g = case.get("window", 0), case.get("sinks", 0), h // hk
    trees = _parents(case) if op == "tree" else None
    out = torch.zeros((sum(new), h, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((sum(new), h), float("-inf"), dtype=torch.float64, device=DEVICE)
    for b, (m, n) in enumerate(zip(lens, new)):
        if m == 0:
            continue
        a = st["start_host"][b]
        slots = torch.tensor([table[b][t // page] * page + t % page for t in range(m)],
                             device=DEVICE)
        key = torch.arange(m, device=DEVICE)
        for head in range(hk):
            cols = slice(head * d, (head + 1) * d)
            k = st["pool"][LAYER, 0, :, cols][slots].double()
            v = st["pool"][LAYER, 1, :, cols][slots].double()
            kt = k.t().contiguous()
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                t = torch.arange(m - n + i0, m - n + i1, device=DEVICE)[:, None]
                if op == "tree":
                    seen = (key < m - n).repeat(i1 - i0, 1)
                    seen[:, m - n:] = torch.tensor(_ancestors(trees[b])[i0:i1], device=DEVICE)
                else:
                    near = key[None] > t - window if window else True
                    seen = (key[None] <= t) & (near | (key[None] < sinks))
                for j in range(head * g, (head + 1) * g):
                    s = st["q"][a + i0:a + i1, j].double() @ kt / math.sqrt(d)
                    s = torch.where(seen, s, torch.full_like(s, float("-inf")))
                    e = torch.logsumexp(s, -1)
                    lse[a + i0:a + i1, j] = e
                    out[a + i0:a + i1, j] = torch.exp(s - e[:, None]) @ v
    return out, lse
