"""The operators of a drafting and long-running serving loop as measured work: new rows
normed, rotated by position and appended to a KV cache; the attention of a tree of drafted
tokens; attention through a sliding window with a few first tokens that stay visible; the
rows of an accepted path moved together in the cache; and the next tokens sampled from
logits with temperature, top-k, top-p and min-p.

`run` computes them in plain torch operations, or, with `own` set, through the library's
entries (qwen35_cache_append_rope, qwen35_tree_attention, qwen35_window_attention,
qwen35_cache_keep, qwen35_sample). Head layouts, rotary dims and the vocabulary are those of
the configurations in the package's `synth` module ("4b": 16 query heads over 4 kv-heads of
256, 248320 tokens; "tiny": 4 over 1 of 64; "tiny_alt": 3 over 3 of 128), contexts and pages
those of the benchmark.

A case's fields: `op` (rope: rows normed, rotated and appended, and for quantised caches read
back; tree; window; keep; sample), `heads`/`kv_heads`/`dim`/`rotary`, `fmt` (bf16, or turbo8:
rotated E4M3 codes with a bf16 scale per 16 elements), `seqs` sequences holding between `lo`
and `hi` tokens before the call, each with between `rows_lo` and `rows_hi` rows (tree and keep:
drafted nodes), `page` tokens per pool block (0: contiguous rows), `window` and `first` tokens
seen, `vocab` logits a row and `mode` of their filters.
"""

import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 16  # elements that share a Turbo8 scale
EPS, THETA = 1e-6, 1e7


def _cache_case(name, op, heads, kv_heads, dim, rotary, fmt, seqs, lo, hi, rows_lo, rows_hi, page, window=0, first=0):
    return dict(name=name, op=op, heads=heads, kv_heads=kv_heads, dim=dim, rotary=rotary, fmt=fmt, seqs=seqs, lo=lo,
                hi=hi, rows_lo=rows_lo, rows_hi=rows_hi, page=page, window=window, first=first)


def _sample_case(name, rows, vocab, mode):
    return dict(name=name, op="sample", seqs=rows, vocab=vocab, mode=mode)


def listed():
    return [
        # one decode step's new rows of a small batch: pure latency
        _cache_case("rope_decode_8", "rope", 16, 4, 256, 64, "bf16", 8, 300, 100000, 1, 1, 16),
        # ragged prompts into a quantised cache, some after rows that are there already
        _cache_case("rope_prompts_turbo8", "rope", 16, 4, 256, 64, "turbo8", 5, 0, 9000, 700, 4097, 64),
        # a few drafted tokens after a short context: the smallest tree
        _cache_case("tree_small", "tree", 16, 4, 256, 64, "bf16", 1, 1000, 1000, 8, 8, 0),
        # a full tree of drafts at the benchmark's context, paged
        _cache_case("tree_64_at_8k", "tree", 16, 4, 256, 64, "bf16", 1, 8191, 8191, 64, 64, 16),
        # a serving batch of trees over quantised caches of unequal lengths
        _cache_case("tree_batch_turbo8", "tree", 16, 4, 256, 64, "turbo8", 16, 1000, 16383, 12, 33, 64),
        # one sequence decoding through a short window
        _cache_case("window_decode_1", "window", 16, 4, 256, 64, "bf16", 1, 8191, 8191, 1, 1, 0, 512, 4),
        # a serving batch decoding through a long window
        _cache_case("window_batch", "window", 16, 4, 256, 64, "bf16", 32, 1023, 16383, 1, 1, 64, 4096, 4),
        # pieces of prompts through a window, quantised
        _cache_case("window_chunks_turbo8", "window", 16, 4, 256, 64, "turbo8", 4, 500, 8000, 100, 257, 32, 1024, 16),
        # accepted paths of a serving batch's trees
        _cache_case("keep_paths", "keep", 16, 4, 256, 64, "bf16", 32, 200, 700, 20, 64, 16),
        # the same of small quantised caches, contiguous
        _cache_case("keep_paths_turbo8", "keep", 3, 3, 128, 32, "turbo8", 8, 50, 400, 30, 64, 0),
        # one sequence's next token
        _sample_case("sample_1", 1, 248320, "all"),
        # a serving batch's next tokens, every row with settings of its own
        _sample_case("sample_64", 64, 248320, "mixed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "window", "window", "keep", "sample"])
    if op == "sample":
        vocab = _log_int(rng, 500, 248320)
        case = _sample_case(None, _log_int(rng, 1, 64), vocab, rng.choice(["all", "mixed", "none"]))
        del case["name"]
        return case
    heads, kv_heads, dim, rotary = rng.choice([(16, 4, 256, 64), (16, 4, 256, 64), (4, 1, 64, 16), (3, 3, 128, 32),
                                               (32, 4, 128, 128), (16, 1, 128, 64), (8, 1, 64, 32)])
    fmt = rng.choice(["bf16", "turbo8"])
    page = rng.choice([0, 16, 32, 64])
    seqs = _log_int(rng, 1, 24)
    window = first = 0
    if op == "rope":
        rows_hi = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(2, 9000 // seqs))
        lo = rng.randrange(0, 500)
        hi = lo + _log_int(rng, 1, 100000 // seqs)
    elif op == "keep":
        rows_hi = rng.randrange(8, 65)
        lo = rng.randrange(1, 300)
        hi = lo + rng.randrange(0, 400)
    else:
        rows_hi = rng.randrange(2, 65) if op == "tree" else rng.choice([1, 1, 1, 3, 40, 130])
        rows_hi = min(rows_hi, max(1, 640 // seqs))
        hi = _log_int(rng, 40, min(30000, 120000 // seqs))
        lo = max(1, hi // rng.choice([1, 2, 7, 30]))
        if op == "window":
            window, first = _log_int(rng, 16, 4096), rng.choice([0, 1, 4, 4, 64])
    rows_lo = max(8 if op == "keep" else 1, rows_hi // rng.choice([1, 2, 3]))
    case = _cache_case(None, op, heads, kv_heads, dim, rotary, fmt, seqs, lo, hi, rows_lo, rows_hi, page, window, first)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, evenly on a log scale, in a fixed mixed order."""
    if n == 1:
        return [hi]
    v = [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (n - 1)))) - 1
         for i in range(n)]
    while math.gcd(step, n) != 1:
        step += 1
    return [v[(i * step) % n] for i in range(n)]


def _layout(case):
    """(tokens before, rows) per sequence and the capacity they share."""
    n, unit = case["seqs"], max(case["page"], 16)
    pos = _spread(case["lo"], case["hi"], n, 5)
    rows = _spread(case["rows_lo"], case["rows_hi"], n, 7)
    cap = (max(p + r for p, r in zip(pos, rows)) + unit - 1) // unit * unit
    return pos, rows, cap


def _paths(case):
    """Accepted nodes of each sequence's tree: the root, then one a level, rising (as many as fit twice)."""
    rng = random.Random(case["seqs"] * 1000 + case["rows_hi"])
    _, rows, _ = _layout(case)
    paths = []
    for r in rows:
        n = rng.randrange(1, min(9, r // 2 + 1))
        paths.append([0] + sorted(rng.sample(range(n, r), n - 1)))
    return paths


def _hadamard(dim):
    h = torch.ones(1, 1, device=DEV)
    while h.shape[0] < dim:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(dim)


def _quantise(x, had):
    """Rows [..., dim] in bf16 -> (E4M3 codes as bytes [..., dim], bf16 scales [..., dim / 16]) of the
    rotated row: scale = bf16(max / 448) per group, code = e4m3(value / scale)."""
    r = (x.float() @ had).to(torch.bfloat16).float()
    g = r.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 448.0).to(torch.bfloat16)
    q = torch.where(scale[..., None] > 0, g / scale[..., None].float(), torch.zeros_like(g))
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), scale


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _starts(counts):
    start = [0]
    for c in counts:
        start.append(start[-1] + c)
    return _ints(start)


def _prepare_sample(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    n, vocab, mode = case["seqs"], case["vocab"], case["mode"]
    x = torch.randn(n, vocab, generator=gen, device=DEV) * 2.5
    # a few tokens stand out, as a model's choices do
    few = torch.randint(0, vocab, (n, min(vocab, 24)), generator=gen, device=DEV)
    x.scatter_add_(1, few, 9.0 + 2.0 * torch.randn(few.shape, generator=gen, device=DEV))
    u = torch.rand(4, n, generator=gen, device=DEV)
    s = {"case": case, "logits": x.to(torch.bfloat16), "u": u[0].contiguous()}
    s["temperature"] = (0.5 + u[1]).contiguous()
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if mode == "all":
        s["top_k"] = torch.full((n,), 50, dtype=torch.int32, device=DEV)
        s["top_p"] = torch.full((n,), 0.95, device=DEV)
        s["min_p"] = torch.full((n,), 0.02, device=DEV)
    if mode == "mixed":
        i = torch.arange(n, device=DEV)
        s["temperature"] = torch.where(i % 8 == 7, 0.0, s["temperature"])  # some rows are greedy
        s["top_k"] = torch.where(i % 2 == 0, 1 + (u[2] * 200).int(), 0).int()
        s["top_p"] = torch.where(i % 3 == 0, 0.5 + 0.5 * u[3], 1.0).float()
        s["min_p"] = torch.where(i % 5 == 0, 0.1 * u[3], 0.0).float()
    return s


def prepare(case, seed):
    if case["op"] == "sample":
        return _prepare_sample(case, seed)
    gen = torch.Generator(DEV).manual_seed(seed)
    op, hkv, dim, h = case["op"], case["kv_heads"], case["dim"], case["heads"]
    pos, rows, cap = _layout(case)
    n = case["seqs"]
    s = {"case": case, "cap": cap, "had": _hadamard(dim), "pos": _ints(pos)}
    if op == "keep":
        paths = _paths(case)
        rows = [len(p) for p in paths]
        s["path"] = _ints([x for p in paths for x in p])
    s["row_start"] = _starts(rows) if max(rows) > 1 or op == "keep" else None
    s["n_rows"], s["most"] = sum(rows), max(rows)
    total = n * cap
    if case["page"]:
        nb = total // case["page"] + 3
        s["table"] = torch.randperm(nb, generator=gen, device=DEV)[:total // case["page"]].to(torch.int32).view(n, -1)
        s["num_blocks"] = nb
        total = nb * case["page"]
    else:
        s["table"], s["num_blocks"] = None, 0
    turbo8 = case["fmt"] == "turbo8"
    groups = hkv * dim // GROUP
    stride = (groups + 7) // 8 * 8
    for name in ("k", "v"):
        pool = torch.empty(total, hkv, dim, dtype=torch.uint8 if turbo8 else torch.bfloat16, device=DEV)
        if turbo8:
            s[name + "_scales"] = torch.zeros(total, stride, dtype=torch.bfloat16, device=DEV)
        for a in range(0, total, 65536):
            e = min(total, a + 65536)
            x = torch.randn(e - a, hkv, dim, generator=gen, device=DEV).to(torch.bfloat16)
            if turbo8:
                pool[a:e], scales = _quantise(x, s["had"])
                s[name + "_scales"][a:e, :groups] = scales.flatten(1)
            else:
                pool[a:e] = x
        s[name] = pool

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)

    if op in ("tree", "window"):
        s["q"], s["gate"] = normal(s["n_rows"], h, dim), normal(s["n_rows"], h, dim)
    if op == "tree":  # nodes in the order of their levels, a few children each; now and then a second root
        rng = random.Random(seed)
        parent = []
        for r in rows:
            p = [-1] * r
            for i in range(1, r):
                p[i] = -1 if rng.random() < 0.04 else rng.randrange(max(0, (i - 1) // 4), min(i, (i - 1) // 2 + 1))
            parent += p
        s["parent"] = _ints(parent)
    if op == "rope":
        # projections as they come: each head's query beside its gate, values well away from norm 1
        s["qg"] = (3.0 * torch.randn(s["n_rows"], h, 2, dim, generator=gen, device=DEV)).to(torch.bfloat16)
        s["k_new"] = (2.0 * torch.randn(s["n_rows"], hkv, dim, generator=gen, device=DEV)).to(torch.bfloat16)
        s["v_new"] = normal(s["n_rows"], hkv, dim)
        s["q_norm"], s["k_norm"] = ((1 + 0.1 * torch.randn(dim, generator=gen, device=DEV)).to(torch.bfloat16)
                                    for _ in range(2))
    return s


def _physical(s, seq, t):
    """Row of the cache arrays that holds token t of sequence seq (broadcast)."""
    page = s["case"]["page"]
    if page:
        return s["table"].long()[seq, t // page] * page + t % page
    return seq * s["cap"] + t


# ---------------------------------------------------------------- the plain forms


def _rows(s):
    """Per row of the call: its sequence, which of its rows it is, the sequence's tokens before."""
    i = torch.arange(s["n_rows"], device=DEV)
    if s["row_start"] is None:
        return i, torch.zeros_like(i), s["pos"].long()
    start = s["row_start"].long()
    seq = torch.searchsorted(start, i, right=True) - 1
    return seq, i - start[seq], s["pos"].long()[seq]


def _values(s, name, at):
    """The cache's rows at physical rows `at` in 32 bits (Turbo8: still rotated)."""
    x = s[name][at]
    if s["case"]["fmt"] != "turbo8":
        return x.float()
    hkv = s["case"]["kv_heads"]
    sc = s[name + "_scales"][at][..., :hkv * s["case"]["dim"] // GROUP].float().unflatten(-1, (hkv, -1))
    return x.view(torch.float8_e4m3fn).float() * sc.repeat_interleave(GROUP, -1)


def _rotated(x, weight, pos, rotary):
    """bf16(RMSNorm(x) weight), then the first `rotary` dims rotated by position in halves, rounded to
    bf16. In 64 bits: a value next to a border between two bf16 numbers goes to the right side. The
    angle itself is the 32-bit product of position and frequency, as the layers take it."""
    y = x.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.double()
    y = y.to(torch.bfloat16).double()
    half = rotary // 2
    freq = (THETA ** (-2.0 * torch.arange(half, device=DEV, dtype=torch.float64) / rotary)).float()
    angle = (pos.float()[:, None] * freq).double()[:, None]
    c, sn = torch.cos(angle), torch.sin(angle)
    a, b = y[..., :half], y[..., half:rotary]
    return torch.cat([a * c - b * sn, b * c + a * sn, y[..., rotary:]], -1).to(torch.bfloat16)


def _rope(s):
    c = s["case"]
    seq, i, before = _rows(s)
    pos = before + i
    at = _physical(s, seq, pos)
    q = _rotated(s["qg"][:, :, 0], s["q_norm"], pos, c["rotary"])
    new = {"k": _rotated(s["k_new"], s["k_norm"], pos, c["rotary"]), "v": s["v_new"]}
    if c["fmt"] != "turbo8":
        s["k"][at], s["v"][at] = new["k"], new["v"]
        return q, s["k"], s["v"]
    groups = c["kv_heads"] * c["dim"] // GROUP
    s["k"][at], k_scales = _quantise(new["k"], s["had"])
    s["v"][at], v_scales = _quantise(new["v"], s["had"])
    s["k_scales"][at, :groups], s["v_scales"][at, :groups] = k_scales.flatten(1), v_scales.flatten(1)
    return q, *((_values(s, name, at) @ s["had"]).to(torch.bfloat16) for name in ("k", "v"))


def _attention(s, t, seen):
    """softmax(q K^T / sqrt(dim)) V over each sequence's tokens t [seqs, tokens], those that are
    seen [seqs, rows, tokens], times sigmoid(gate)."""
    c = s["case"]
    n, most, hkv, dim = c["seqs"], s["most"], c["kv_heads"], c["dim"]
    seq, i, _ = _rows(s)
    at = _physical(s, torch.arange(n, device=DEV)[:, None], t)
    k, v = (_values(s, name, at).transpose(1, 2) for name in ("k", "v"))  # [seqs, kv_heads, tokens, dim]
    q = torch.zeros(n, most, c["heads"], dim, device=DEV)
    q[seq, i] = s["q"].float()
    if c["fmt"] == "turbo8":
        q = q @ s["had"]
    q = q.unflatten(2, (hkv, -1)).transpose(1, 2)  # [seqs, kv_heads, rows, group, dim]
    group = q.shape[3]
    x = (q.flatten(2, 3) @ k.transpose(2, 3) / math.sqrt(dim)).unflatten(2, (most, group))
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = ((x / x.sum(-1, keepdim=True)).flatten(2, 3) @ v).unflatten(2, (most, group))
    if c["fmt"] == "turbo8":
        o = o @ s["had"]
    o = o.transpose(1, 2).flatten(2, 3)[seq, i]
    return (o / (1 + torch.exp(-s["gate"].float()))).to(torch.bfloat16)


def _tree(s):
    """A node sees the tokens before the tree, its ancestors and itself."""
    n, most = s["case"]["seqs"], s["most"]
    seq, i, _ = _rows(s)
    up = torch.zeros(n, most, most, dtype=torch.float64, device=DEV)
    up[seq, i, i] = 1.0
    has = s["parent"] >= 0
    up[seq[has], i[has], s["parent"].long()[has]] = 1.0
    line = torch.linalg.matrix_power(up, most) > 0  # node, ancestor or itself
    line = line | torch.eye(most, dtype=torch.bool, device=DEV)  # rows of padding see themselves
    before = s["pos"].long()
    t = torch.arange(s["case"]["hi"] + most, device=DEV)[None].expand(n, -1)
    node = t - before[:, None]
    inside = (node >= 0) & (node < most)
    seen = line.gather(2, torch.where(inside, node, 0)[:, None].expand(-1, most, -1)) & inside[:, None]
    return _attention(s, torch.where(t < s["cap"], t, 0), seen | (node < 0)[:, None])


def _window(s):
    """A row at position p sees the tokens (p - window, p] and the first few."""
    c = s["case"]
    first, window, most = c["first"], c["window"], s["most"]
    before = s["pos"].long()
    start = (before - window + 1).clamp(min=0)
    t = torch.cat([torch.arange(first, device=DEV)[None].expand(c["seqs"], -1),
                   start[:, None] + torch.arange(window + most, device=DEV)], 1)
    p = (before[:, None] + torch.arange(most, device=DEV))[:, :, None]
    seen = (t[:, None] <= p) & ((t[:, None] > p - window) | (t[:, None] < first))
    seen[:, :, :first] &= (t[:, None, :first] < start[:, None, None])  # not counted twice
    return _attention(s, torch.where(t < s["cap"], t, 0), seen)


def _keep(s):
    """Row path[i] of each sequence's new rows to place i."""
    seq, i, before = _rows(s)
    src, dst = _physical(s, seq, before + s["path"].long()), _physical(s, seq, before + i)
    s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    if s["case"]["fmt"] == "turbo8":
        s["k_scales"][dst], s["v_scales"][dst] = s["k_scales"][src], s["v_scales"][src]
    return _kept(s)


def _kept(s):
    """The cache (Turbo8: the E4M3 numbers and the scales they are times)."""
    if s["case"]["fmt"] != "turbo8":
        return s["k"], s["v"]
    return tuple(s[name].view(torch.float8_e4m3fn) for name in ("k", "v")) + (s["k_scales"], s["v_scales"])


def _sample(s):
    """Tokens in falling order, the lower index of equal ones first; the first top_k, of those as long as what
    comes before has less than top_p of the sum, and at least min_p of the largest; of what is left
    the first whose running sum passes u times the whole. In 64 bits: sums lie next to borders."""
    x = s["logits"].double()
    n, vocab = x.shape
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)
    rank = torch.arange(vocab, device=DEV)[None]
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t))
    w = torch.where(greedy & (rank > 0), 0.0, w)
    top = torch.ones(n, vocab, dtype=torch.bool, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        top = (rank < k) | (k <= 0)
    w = torch.where(top, w, 0.0)
    if s["top_p"] is not None:
        before = torch.cumsum(w, -1) - w
        w = torch.where((before < s["top_p"].double()[:, None] * w.sum(-1, keepdim=True)) | (rank == 0), w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0.0)
    total = w.sum(-1, keepdim=True)
    at = (torch.cumsum(w, -1) <= s["u"].double()[:, None] * total).sum(-1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(-1, keepdim=True) - 1)
    return order.gather(1, at)[:, 0].to(torch.int32), (w.gather(1, at) / total)[:, 0].float()


# ---------------------------------------------------------------- the library's entries


def _handles(s):
    """What a program keeps beside its tensors: the library's structs, scratch and outputs."""
    if "handles" in s:
        return s["handles"]
    from full_attention_decode_gb300 import binding as B
    from full_attention_decode_gb300 import synth
    c = s["case"]
    B.qwen35_init()
    n_rows = s.get("n_rows", 0)
    if c["op"] == "sample":
        s["handles"] = dict(B=B, token=torch.empty(c["seqs"], dtype=torch.int32, device=DEV),
                            prob=torch.empty(c["seqs"], device=DEV))
        return s["handles"]
    cfg = B.make_config(synth.config("4b") | {"num_heads": c["heads"], "num_kv_heads": c["kv_heads"],
                                              "head_dim": c["dim"], "rotary_dim": c["rotary"], "rms_eps": EPS,
                                              "rope_theta": THETA})
    turbo8, paged = c["fmt"] == "turbo8", s["table"] is not None
    kv = B.qwen35_kv_cache(s["k"].data_ptr(), s["v"].data_ptr(), s["cap"],
                           B.QWEN35_KV_TURBO8 if turbo8 else B.QWEN35_KV_BF16,
                           s["k_scales"].data_ptr() if turbo8 else None, s["v_scales"].data_ptr() if turbo8 else None,
                           s["table"].data_ptr() if paged else None, c["page"], 0)
    rows = B.DeviceRows(s["pos"], s["row_start"], n_rows, s["num_blocks"])
    need = B.qwen35_rows_scratch_bytes(cfg, n_rows)
    x = torch.empty(n_rows, c["kv_heads"], c["dim"], dtype=torch.bfloat16, device=DEV)
    s["handles"] = dict(B=B, cfg=cfg, kv=kv, rows=rows, scratch=B.new_scratch(need), k=x, v=torch.empty_like(x),
                        out=torch.empty(n_rows, c["heads"], c["dim"], dtype=torch.bfloat16, device=DEV))
    return s["handles"]


def _ok(status):
    if status != 0:
        raise RuntimeError(f"the library refused the call: {status}")


def _run_own(s):
    h, op = _handles(s), s["case"]["op"]
    B = h["B"]
    if op == "sample":
        _ok(B.qwen35_sample(s["logits"], s["u"], h["token"], temperature=s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"], prob=h["prob"]))
        return h["token"], h["prob"]
    c, kv, rows, out, scratch = s["case"], h["kv"], h["rows"], h["out"], h["scratch"]
    if op == "rope":
        _ok(B.qwen35_cache_append_rope(h["cfg"], kv, rows, s["qg"], s["k_new"], s["v_new"], out, scratch,
                                       q_norm=s["q_norm"], k_norm=s["k_norm"], q_stride=2 * c["dim"]))
        if c["fmt"] != "turbo8":
            return out, s["k"], s["v"]
        _ok(B.qwen35_cache_read(h["cfg"], kv, rows, h["k"], h["v"], scratch))
        return out, h["k"], h["v"]
    if op == "tree":
        _ok(B.qwen35_tree_attention(h["cfg"], kv, rows, s["parent"], s["q"], out, scratch, gate=s["gate"]))
        return out
    if op == "window":
        _ok(B.qwen35_window_attention(h["cfg"], kv, rows, c["window"], c["first"], s["q"], out, scratch,
                                      gate=s["gate"]))
        return out
    _ok(B.qwen35_cache_keep(h["cfg"], kv, rows, s["path"], scratch))
    return _kept(s)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _rope(state)
    if op == "tree":
        return _tree(state)
    if op == "window":
        return _window(state)
    if op == "keep":
        return _keep(state)
    return _sample(state)


def work(case):
    if case["op"] == "sample":
        n = case["seqs"]
        return {"bytes": n * case["vocab"] * 2 + n * 28, "flops": 3 * n * case["vocab"]}
    pos, rows, _ = _layout(case)
    h, hkv, dim, op = case["heads"], case["kv_heads"], case["dim"], case["op"]
    turbo8 = case["fmt"] == "turbo8"
    n = sum(rows)
    kept = 2 * hkv * (dim + dim // GROUP * 2 if turbo8 else 2 * dim)  # a token's K and V in the cache
    plain = 2 * hkv * dim * 2  # and as bf16 rows
    rotate = 2 * dim * int(math.log2(dim)) if turbo8 else 0  # a head's row into the rotated basis, or back
    if op == "rope":
        return {"bytes": n * (2 * h * dim * 2 + plain + kept * (2 if turbo8 else 1) + (plain if turbo8 else 0)),
                "flops": n * ((h + hkv) * (4 * dim + 3 * case["rotary"]) + 4 * hkv * rotate)}
    if op == "keep":
        moved = sum(i != x for p in _paths(case) for i, x in enumerate(p))
        return {"bytes": moved * 2 * kept, "flops": 0}
    io = n * h * dim * 2 * 3  # q, gate, out
    if op == "tree":
        read = sum(p + r for p, r in zip(pos, rows))
        dots = sum(r * p + 4 * r for p, r in zip(pos, rows))
    else:
        first, window = case["first"], case["window"]
        read = sum(p + r if p < window + first else window + r - 1 + first for p, r in zip(pos, rows))
        dots = sum(min(p + i + 1, window + first) for p, r in zip(pos, rows) for i in range(r))
    return {"bytes": read * kept + io, "flops": 4 * dots * h * dim + 2 * n * h * rotate}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_sample(case, seed):
    s = prepare(case, seed)
    logits = s["logits"].double().cpu()
    tokens, probs = [], []
    for r in range(case["seqs"]):
        x = logits[r]
        t = float(s["temperature"][r])
        best = int((x == x.max()).nonzero()[0])
        if t <= 0:
            tokens.append(best)
            probs.append(1.0)
            continue
        order = sorted(range(len(x)), key=(-x).tolist().__getitem__)
        w = torch.exp((x[order] - x[best]) / t)
        k = int(s["top_k"][r]) if s["top_k"] is not None else 0
        w = w[:k] if k > 0 else w
        if s["top_p"] is not None:
            limit, c = float(s["top_p"][r]) * float(w.sum()), torch.cumsum(w, 0)
            w = w[:1 + int((c[:-1] < limit).sum())]
        if s["min_p"] is not None:
            w = w[w >= float(s["min_p"][r])]
        c = torch.cumsum(w, 0)
        j = min(int((c <= float(s["u"][r]) * float(w.sum())).sum()), len(w) - 1)
        tokens.append(order[j])
        probs.append(float(w[j] / w.sum()))
    return torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.tensor(probs, dtype=torch.float64, device=DEV)


def exact(case, seed):
    """Sequence by sequence in float64: the rotation as butterflies, the cache turned back
    to unrotated rows before the attention, a tree's ancestors followed one by one."""
    if case["op"] == "sample":
        return _exact_sample(case, seed)
    s = prepare(case, seed)
    c, dim, hkv, op = case, case["dim"], case["kv_heads"], case["op"]
    turbo8 = case["fmt"] == "turbo8"

    def rotate(x):
        x, w = x.double(), 1
        while w < dim:
            y = x.unflatten(-1, (-1, 2, w))
            x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).flatten(-3)
            w *= 2
        return x / math.sqrt(dim)

    def physical(b, t):
        if not c["page"]:
            return b * s["cap"] + t
        return s["table"][b].long()[torch.div(t, c["page"], rounding_mode="floor")] * c["page"] + t % c["page"]

    def held(name, at):  # rows of the cache as the unrotated values they stand for
        if not turbo8:
            return s[name][at].double()
        x = s[name][at].view(torch.float8_e4m3fn).double()
        sc = s[name + "_scales"][at][:, :hkv * dim // GROUP].double().view(len(x), hkv, dim // GROUP, 1)
        return rotate((x.view(len(x), hkv, dim // GROUP, GROUP) * sc).view(len(x), hkv, dim))

    def turned(x, weight, p):  # head rows [rows, heads, dim] at positions p, one frequency after another
        y = x.double()
        y = (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.double()).to(torch.bfloat16).double()
        out = y.clone()
        for i in range(c["rotary"] // 2):
            f = torch.tensor(THETA ** (-2.0 * i / c["rotary"]), dtype=torch.float32, device=DEV)
            a = (p.to(torch.float32) * f).double()[:, None]
            j = i + c["rotary"] // 2
            out[:, :, i] = y[:, :, i] * torch.cos(a) - y[:, :, j] * torch.sin(a)
            out[:, :, j] = y[:, :, j] * torch.cos(a) + y[:, :, i] * torch.sin(a)
        return out

    pos, rows, _ = _layout(case)
    if op == "keep":
        for b, path in enumerate(_paths(case)):
            src = physical(b, pos[b] + torch.tensor(path, device=DEV))
            dst = physical(b, pos[b] + torch.arange(len(path), device=DEV))
            for name in ("k", "v") + (("k_scales", "v_scales") if turbo8 else ()):
                s[name][dst] = s[name][src].clone()
        if not turbo8:
            return s["k"].double(), s["v"].double()
        return tuple(s[name].view(torch.float8_e4m3fn).double() for name in ("k", "v")) + tuple(
            s[name].double() for name in ("k_scales", "v_scales"))
    if op == "rope":
        out = []
        for b, (p0, r) in enumerate(zip(pos, rows)):
            mine = slice(sum(rows[:b]), sum(rows[:b + 1]))
            p = p0 + torch.arange(r, device=DEV)
            at = physical(b, p)
            q, k = turned(s["qg"][mine, :, 0], s["q_norm"], p), turned(s["k_new"][mine], s["k_norm"], p)
            for name, x in (("k", k), ("v", s["v_new"][mine].double())):
                if turbo8:
                    y = rotate(x.to(torch.bfloat16)).to(torch.bfloat16).double().view(r, hkv, dim // GROUP, GROUP)
                    sc = (y.abs().amax(-1) / 448).to(torch.bfloat16)
                    z = torch.where(sc[..., None] > 0, y / sc[..., None].double(), 0.0).clamp(-448, 448)
                    s[name][at] = z.float().to(torch.float8_e4m3fn).view(torch.uint8).view(r, hkv, dim)
                    s[name + "_scales"][at, :sc[0].numel()] = sc.view(r, -1)
                else:
                    s[name][at] = x.to(torch.bfloat16)
            out.append((q, held("k", at), held("v", at)) if turbo8 else (q,))
        if not turbo8:
            return torch.cat([o[0] for o in out]), s["k"].double(), s["v"].double()
        return tuple(torch.cat([o[i] for o in out]) for i in range(3))
    out = []
    for b, (p0, r) in enumerate(zip(pos, rows)):
        first = sum(rows[:b])
        t = torch.arange(p0 + r, device=DEV)
        at = physical(b, t)
        k, v = held("k", at), held("v", at)
        parent = s["parent"][first:first + r].tolist() if op == "tree" else None
        for i in range(r):
            q = s["q"][first + i].double().view(hkv, -1, dim)
            p = p0 + i
            if op == "tree":
                see = list(range(p0))
                j = i
                while j >= 0:
                    see.append(p0 + j)
                    j = parent[j]
            else:
                low = max(0, p - c["window"] + 1)
                see = list(range(min(c["first"], low))) + list(range(low, p + 1))
            see = torch.tensor(see, device=DEV)
            x = torch.einsum("ghd,tgd->ght", q, k[see]) / math.sqrt(dim)
            o = torch.einsum("ght,tgd->ghd", torch.softmax(x, -1), v[see]).flatten(0, 1)
            out.append(o * torch.sigmoid(s["gate"][first + i].double()))
    return torch.stack(out)
