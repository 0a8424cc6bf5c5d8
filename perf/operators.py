"""The cached-attention operators as measured work: rows written to a KV cache and read
back, blocks of a long cache chosen by their key bounds, and the attention of new
tokens over the whole cache or over the chosen blocks.

`run` computes them in plain torch operations, or, with `own` set, through the
library's entries (qwen35_cache_append, qwen35_cache_read, qwen35_select_blocks,
qwen35_decode_attention). Sizes are those of the configurations in the package's
`synth` module ("4b": 16 query heads over 4 kv-heads of 256; "tiny": 4 over 1 of 64;
"tiny_alt": 3 over 3 of 128) and of the benchmark's contexts (512 to 131072 tokens,
16-token pages, 8 sequences of 1024 to 65536 tokens), with a few other groupings of
heads among the drawn ones.

A case's fields: `op` (append: bf16 rows into the cache; roundtrip: rows in and back out;
read: rows out; attend: attention over every token; sparse: selection, then attention
over the selected blocks), `heads`/`kv_heads`/`dim`, `fmt` (bf16 or turbo8: rotated E4M3
codes with a bf16 scale per 16 elements), `seqs` sequences holding between `lo` and
`hi` tokens before the call, each adding between `rows_lo` and `rows_hi` rows, `page`
tokens per pool block (0: contiguous rows), `block` tokens per selection block and
`select` blocks chosen.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 16  # elements that share a Turbo8 scale


def _case(name, op, heads, kv_heads, dim, fmt, seqs, lo, hi, rows_lo, rows_hi, page, block=64, select=0):
    return dict(name=name, op=op, heads=heads, kv_heads=kv_heads, dim=dim, fmt=fmt, seqs=seqs, lo=lo, hi=hi,
                rows_lo=rows_lo, rows_hi=rows_hi, page=page, block=block, select=select)


def listed():
    return [
        # one decode step's new rows of a small batch: pure latency
        _case("append_decode_8", "append", 16, 4, 256, "bf16", 8, 300, 1000, 1, 1, 16, 16),
        # three prompts of ragged length, one cut off in mid-block by rows cached before
        _case("roundtrip_prompts", "roundtrip", 16, 4, 256, "turbo8", 3, 0, 777, 411, 1500, 64, 64),
        # a long document's rows in one call
        _case("roundtrip_32k", "roundtrip", 16, 4, 256, "turbo8", 1, 0, 0, 32768, 32768, 16, 16),
        # prefixes taken out of a contiguous quantised cache (to move or convert it)
        _case("read_prefixes", "read", 3, 3, 128, "turbo8", 8, 0, 600, 1000, 4097, 0, 32),
        # the smallest decode attention: one sequence, 512 tokens
        _case("attend_512", "attend", 16, 4, 256, "bf16", 1, 511, 511, 1, 1, 0),
        # the benchmark's context, paged
        _case("attend_8k_paged", "attend", 16, 4, 256, "bf16", 1, 8191, 8191, 1, 1, 16),
        # one long context in the quantised format
        _case("attend_128k_turbo8", "attend", 16, 4, 256, "turbo8", 1, 131071, 131071, 1, 1, 0),
        # a serving batch of unequal lengths
        _case("attend_batch_ragged", "attend", 16, 4, 256, "bf16", 32, 1023, 16383, 1, 1, 64),
        # drafted tokens being verified, one query head per kv-head
        _case("attend_draft", "attend", 3, 3, 128, "turbo8", 12, 500, 3000, 1, 5, 32),
        # a long context read at 32 of 1024 blocks
        _case("sparse_64k", "sparse", 16, 4, 256, "bf16", 1, 65535, 65535, 1, 1, 64, 64, 32),
        # a serving batch of long contexts in the quantised format
        _case("sparse_batch_turbo8", "sparse", 16, 4, 256, "turbo8", 16, 16383, 65535, 1, 1, 64, 32, 64),
        # drafted tokens on a small model
        _case("sparse_draft", "sparse", 4, 1, 64, "bf16", 5, 1200, 8000, 2, 4, 16, 16, 48),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _drawn(*fields):
    case = _case(None, *fields)
    del case["name"]
    return case


def draw(rng):
    op = rng.choice(["append", "roundtrip", "read", "attend", "attend", "sparse", "sparse"])
    heads, kv_heads, dim = rng.choice([(16, 4, 256), (16, 4, 256), (4, 1, 64), (3, 3, 128), (32, 4, 128), (16, 1, 128),
                                       (8, 1, 64)])
    fmt = "bf16" if op == "append" else rng.choice(["bf16", "turbo8"])  # quantised rows: written and read back
    block = rng.choice([16, 32, 64])
    page = rng.choice([0, 64, 128]) if op == "sparse" else rng.choice([0, 16, 32, 64])
    if op in ("append", "roundtrip", "read"):
        seqs = _log_int(rng, 1, 24)
        most = max(2, 16384 // seqs)
        rows_hi = 1 if op == "append" and rng.random() < 0.5 else _log_int(rng, 1, most)
        rows_lo = max(1, rows_hi // rng.choice([1, 2, 3]))
        lo = rng.randrange(0, 500)
        block = min(block, page) if page else block
        return _drawn(op, heads, kv_heads, dim, fmt, seqs, lo, lo + rng.randrange(0, 700), rows_lo, rows_hi, page, block)
    seqs = _log_int(rng, 1, 24)
    rows_hi = rng.choice([1, 1, 1, 2, 4, 6]) if seqs <= 12 else 1
    hi = _log_int(rng, 40, min(65000, 300000 // (seqs * rows_hi)))
    lo = max(1, hi // rng.choice([1, 2, 7, 30]))
    return _drawn(op, heads, kv_heads, dim, fmt, seqs, lo, hi, 1, rows_hi, page, block,
                  rng.choice([4, 16, 33, 64]) if op == "sparse" else 0)


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
    """(tokens before, rows added) per sequence and the capacity they share."""
    n, unit = case["seqs"], max(case["page"], case["block"], 16)
    pos = _spread(case["lo"], case["hi"], n, 5)
    rows = _spread(case["rows_lo"], case["rows_hi"], n, 7)
    cap = (max(p + r for p, r in zip(pos, rows)) + unit - 1) // unit * unit
    return pos, rows, cap


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


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    hkv, dim, h = case["kv_heads"], case["dim"], case["heads"]
    pos, rows, cap = _layout(case)
    n, n_rows = case["seqs"], sum(rows)
    s = {"case": case, "cap": cap, "had": _hadamard(dim)}
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    s["row_start"] = torch.tensor(start, dtype=torch.int32, device=DEV) if max(rows) > 1 else None
    s["n_rows"] = n_rows
    total = n * cap
    if case["page"]:
        nb = total // case["page"] + 3
        s["table"] = torch.randperm(nb, generator=gen, device=DEV)[:total // case["page"]].to(torch.int32).view(n, -1)
        s["num_blocks"] = nb
        total = nb * case["page"]
    else:
        s["table"], s["num_blocks"] = None, 0
    # keys lean towards a centre of their block, as neighbouring tokens' keys do
    block = case["block"]
    centre = torch.randn(total // block + 1, 1, hkv, dim, generator=gen, device=DEV)
    turbo8 = case["fmt"] == "turbo8"
    groups = hkv * dim // GROUP
    stride = (groups + 7) // 8 * 8
    writes = case["op"] in ("append", "roundtrip")
    keep_bounds = case["op"] in ("append", "roundtrip", "sparse")
    if keep_bounds:
        held = torch.zeros(total, dtype=torch.bool, device=DEV)
        for b in range(n):
            t = torch.arange(pos[b] + (0 if writes else rows[b]), device=DEV)
            held[_physical(s, torch.tensor([[b]], device=DEV), t[None])] = True
        bounds = torch.zeros(total // block, hkv, 2, dim, dtype=torch.bfloat16, device=DEV)
    for name in ("k", "v"):
        if turbo8:
            pool = torch.empty(total, hkv, dim, dtype=torch.uint8, device=DEV)
            s[name + "_scales"] = torch.zeros(total, stride, dtype=torch.bfloat16, device=DEV)
        else:
            pool = torch.empty(total, hkv, dim, dtype=torch.bfloat16, device=DEV)
        for a in range(0, total, 65536):
            e = min(total, a + 65536)
            x = torch.randn(e - a, hkv, dim, generator=gen, device=DEV)
            if name == "k":
                x = 0.8 * x + 0.6 * centre[a // block:(e - 1) // block + 1].expand(-1, block, -1, -1).flatten(0, 1)[:e - a]
                x = x.to(torch.bfloat16)
                if keep_bounds:
                    y = x.float().unflatten(0, (-1, block))
                    m = held[a:e].view(-1, block, 1, 1)
                    any_held = m.any(1)
                    lo = torch.where(m, y, math.inf).amin(1)
                    hi = torch.where(m, y, -math.inf).amax(1)
                    bounds[a // block:e // block, :, 0] = torch.where(any_held, lo, 0.0).to(torch.bfloat16)
                    bounds[a // block:e // block, :, 1] = torch.where(any_held, hi, 0.0).to(torch.bfloat16)
            x = x.to(torch.bfloat16)
            if turbo8:
                codes, scales = _quantise(x, s["had"])
                pool[a:e] = codes
                s[name + "_scales"][a:e, :groups] = scales.flatten(1)
            else:
                pool[a:e] = x
        s[name] = pool
    s["bounds"] = bounds if keep_bounds else None
    s["q"] = torch.randn(n_rows, h, dim, generator=gen, device=DEV).to(torch.bfloat16)
    s["gate"] = torch.randn(n_rows, h, dim, generator=gen, device=DEV).to(torch.bfloat16)
    if writes:
        s["k_new"] = torch.randn(n_rows, hkv, dim, generator=gen, device=DEV).to(torch.bfloat16)
        s["v_new"] = torch.randn(n_rows, hkv, dim, generator=gen, device=DEV).to(torch.bfloat16)
    return s


def _physical(s, seq, t):
    """Row of the cache arrays that holds token t of sequence seq (broadcast)."""
    page = s["case"]["page"]
    if page:
        return s["table"].long()[seq, t // page] * page + t % page
    return seq * s["cap"] + t


# ---------------------------------------------------------------- the plain forms


def _rows(s):
    """Per row of the call: its sequence and its token's position."""
    i = torch.arange(s["n_rows"], device=DEV)
    if s["row_start"] is None:
        return i, s["pos"].long()
    start = s["row_start"].long()
    seq = torch.searchsorted(start, i, right=True) - 1
    return seq, s["pos"].long()[seq] + i - start[seq]


def _numbers(x):
    """Cache elements in 32 bits: bf16 values, or the E4M3 numbers that bytes are."""
    return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).float()


def _values(s, name, at):
    """The cache's rows at physical rows `at` in 32 bits (Turbo8: still rotated)."""
    x = _numbers(s[name][at])
    if s["case"]["fmt"] == "turbo8":
        groups = s["case"]["kv_heads"] * s["case"]["dim"] // GROUP
        sc = s[name + "_scales"][at][..., :groups].float().unflatten(-1, (s["case"]["kv_heads"], -1))
        x = x * sc.repeat_interleave(GROUP, -1)
    return x


def _append(s):
    seq, t = _rows(s)
    at = _physical(s, seq, t)
    for name in ("k", "v"):
        x = s[name + "_new"]
        if s["case"]["fmt"] == "turbo8":
            codes, scales = _quantise(x, s["had"])
            s[name][at] = codes
            s[name + "_scales"][at, :scales[0].numel()] = scales.flatten(1)
        else:
            s[name][at] = x
    # the bounds: a block's first row starts them anew, every other row widens them
    block, b = s["case"]["block"], s["bounds"]
    fresh = at[t % block == 0] // block
    b[fresh, :, 0], b[fresh, :, 1] = math.inf, -math.inf
    x = s["k_new"].flatten(1)
    where = (at // block)[:, None].expand_as(x)
    lo, hi = b[:, :, 0].flatten(1), b[:, :, 1].flatten(1)
    lo.scatter_reduce_(0, where, x, "amin")
    hi.scatter_reduce_(0, where, x, "amax")
    b[:, :, 0], b[:, :, 1] = lo.view_as(b[:, :, 0]), hi.view_as(b[:, :, 1])


def _read(s):
    at = _physical(s, *_rows(s))
    back = []
    for name in ("k", "v"):
        x = _values(s, name, at)
        back.append((x @ s["had"] if s["case"]["fmt"] == "turbo8" else x).to(torch.bfloat16))
    return back


def _attend(s, blocks=None):
    c = s["case"]
    seq, p = _rows(s)
    if blocks is None:  # every token: [rows, 1, tokens]
        t = torch.arange(c["hi"] + c["rows_hi"], device=DEV)[None, None]
        seen = t <= p[:, None, None]
    else:  # the selected blocks' tokens: [rows, kv_heads, tokens]
        t = (blocks.long()[..., None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten(2)
        seen = (t <= p[:, None, None]) & (blocks >= 0).repeat_interleave(c["block"], 2)
    at = _physical(s, seq[:, None, None], torch.where(seen, t, 0))
    if blocks is None:
        k, v = (_values(s, n, at[:, 0]).transpose(1, 2) for n in ("k", "v"))
    else:
        g = torch.arange(c["kv_heads"], device=DEV)[None, :, None]
        k, v = (_picked(s, n, at, g) for n in ("k", "v"))
    q = s["q"].float()
    if c["fmt"] == "turbo8":
        q = q @ s["had"]
    q = q.unflatten(1, (c["kv_heads"], -1))
    x = q @ k.transpose(2, 3) / math.sqrt(c["dim"])
    x = x.masked_fill(~seen[:, :, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x / x.sum(-1, keepdim=True)) @ v
    if c["fmt"] == "turbo8":
        o = o @ s["had"]
    return (o.flatten(1, 2) / (1 + torch.exp(-s["gate"].float()))).to(torch.bfloat16)


def _picked(s, name, at, g):
    """One head's row of each physical row: [rows, kv_heads, tokens, dim], as _values."""
    x = _numbers(s[name][at, g])
    if s["case"]["fmt"] == "turbo8":
        groups = s["case"]["kv_heads"] * s["case"]["dim"] // GROUP
        sc = s[name + "_scales"][:, :groups].unflatten(-1, (s["case"]["kv_heads"], -1))[at, g].float()
        x = x * sc.repeat_interleave(GROUP, -1)
    return x


def _select(s):
    """The blocks of the largest upper bounds, ties to the lower index, in order; the first
    and the last block always. In 64 bits: two blocks' scores may be next to each other."""
    c = s["case"]
    block = c["block"]
    seq, p = _rows(s)
    j = torch.arange((c["hi"] + c["rows_hi"] + block - 1) // block, device=DEV)
    count = p[:, None] // block + 1
    here = j < count
    b = s["bounds"][_physical(s, seq[:, None], torch.where(here, j, 0) * block) // block].double()
    q = s["q"].double().unflatten(1, (c["kv_heads"], -1))
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    x = torch.einsum("rgd,rjgd->rgj", up, b[:, :, :, 1]) + torch.einsum("rgd,rjgd->rgj", down, b[:, :, :, 0])
    x = x.masked_fill(((j < 1) | (j == count - 1))[:, None], math.inf)
    x = x.masked_fill(~here[:, None], -math.inf)
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :c["select"]]
    if best.shape[-1] < c["select"]:
        best = torch.nn.functional.pad(best, (0, c["select"] - best.shape[-1]), value=1 << 30)
    best = torch.where(best < count[:, :, None], best, 1 << 30).sort(-1).values
    return torch.where(best < 1 << 30, best, -1).to(torch.int32)


# ---------------------------------------------------------------- the library's entries


def _handles(s):
    """What a program keeps beside its tensors: the library's structs, scratch and outputs."""
    if "handles" in s:
        return s["handles"]
    from full_attention_decode_gb300 import binding as B
    from full_attention_decode_gb300 import synth
    c, n_rows = s["case"], s["n_rows"]
    B.qwen35_init()
    cfg = B.make_config(synth.config("4b") | {"num_heads": c["heads"], "num_kv_heads": c["kv_heads"],
                                              "head_dim": c["dim"]})
    turbo8, paged = c["fmt"] == "turbo8", s["table"] is not None
    kv = B.qwen35_kv_cache(s["k"].data_ptr(), s["v"].data_ptr(), s["cap"],
                           B.QWEN35_KV_TURBO8 if turbo8 else B.QWEN35_KV_BF16,
                           s["k_scales"].data_ptr() if turbo8 else None, s["v_scales"].data_ptr() if turbo8 else None,
                           s["table"].data_ptr() if paged else None, c["page"], 0)
    rows = B.DeviceRows(s["pos"], s["row_start"], n_rows, s["num_blocks"])
    bounds = B.DeviceKeyBounds(s["bounds"], c["block"]) if s["bounds"] is not None else None
    need = B.qwen35_cache_scratch_bytes(cfg, s["cap"], c["block"], n_rows)
    scratch = B.new_scratch(need)
    x = torch.empty(n_rows, c["kv_heads"], c["dim"], dtype=torch.bfloat16, device=DEV)
    s["handles"] = dict(B=B, cfg=cfg, kv=kv, rows=rows, bounds=bounds, scratch=scratch, k=x, v=torch.empty_like(x),
                        out=torch.empty_like(s["q"]),
                        blocks=torch.empty(n_rows, c["kv_heads"], max(1, c["select"]), dtype=torch.int32, device=DEV))
    return s["handles"]


def _ok(status):
    if status != 0:
        raise RuntimeError(f"the library refused the call: {status}")


def _run_own(s):
    h = _handles(s)
    B, op = h["B"], s["case"]["op"]
    if op in ("append", "roundtrip"):
        _ok(B.qwen35_cache_append(h["cfg"], h["kv"], h["rows"], h["bounds"], s["k_new"], s["v_new"], h["scratch"]))
    if op in ("read", "roundtrip"):
        _ok(B.qwen35_cache_read(h["cfg"], h["kv"], h["rows"], h["k"], h["v"], h["scratch"]))
        return (h["k"], h["v"]) if op == "read" else (h["k"], h["v"], s["bounds"])
    if op == "append":
        return s["k"], s["v"], s["bounds"]
    if op == "sparse":
        _ok(B.qwen35_select_blocks(h["cfg"], h["kv"], h["rows"], h["bounds"], s["q"], h["blocks"], h["scratch"],
                                   n_first=1, n_last=1))
        _ok(B.qwen35_decode_attention(h["cfg"], h["kv"], h["rows"], s["q"], h["out"], h["scratch"], gate=s["gate"],
                                      blocks=h["blocks"], block=s["case"]["block"]))
        return h["blocks"], h["out"]
    _ok(B.qwen35_decode_attention(h["cfg"], h["kv"], h["rows"], s["q"], h["out"], h["scratch"], gate=s["gate"]))
    return h["out"]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("append", "roundtrip"):
        _append(state)
    if op in ("read", "roundtrip"):
        back = _read(state)
        return tuple(back) if op == "read" else (*back, state["bounds"])
    if op == "append":
        return state["k"], state["v"], state["bounds"]
    if op == "sparse":
        blocks = _select(state)
        return blocks, _attend(state, blocks)
    return _attend(state)


def work(case):
    pos, rows, _ = _layout(case)
    h, hkv, dim = case["heads"], case["kv_heads"], case["dim"]
    n = sum(rows)
    kept = 2 * hkv * (dim + dim // GROUP * 2 if case["fmt"] == "turbo8" else 2 * dim)  # a token's K and V in the cache
    plain = 2 * hkv * dim * 2  # and as bf16 rows
    touched = sum((p + r - 1) // case["block"] - p // case["block"] + 1 for p, r in zip(pos, rows))
    bound = 2 * hkv * dim * 2
    rotate = 2 * 2 * hkv * dim * int(math.log2(dim)) if case["fmt"] == "turbo8" else 0
    if case["op"] == "append":
        return {"bytes": n * (plain + kept) + touched * bound, "flops": n * rotate}
    if case["op"] == "roundtrip":
        return {"bytes": n * 2 * (plain + kept) + touched * bound, "flops": 2 * n * rotate}
    if case["op"] == "read":
        return {"bytes": n * (plain + kept), "flops": n * rotate}
    io = n * h * dim * 2 * 3  # q, gate, out
    if case["op"] == "attend":
        read = sum(p + r for p, r in zip(pos, rows))
        dots = sum(r * p + r * (r + 1) // 2 for p, r in zip(pos, rows))
        return {"bytes": read * kept + io, "flops": 4 * dots * h * dim}
    block, most = case["block"], case["select"] * case["block"]
    ends = [(p + i + 1, r) for p, r in zip(pos, rows) for i in range(r)]
    scored = sum((p + r - 1) // block + 1 for p, r in zip(pos, rows))
    read = sum(min(p + r, r * most) for p, r in zip(pos, rows))
    dots = sum(min(e, most) for e, _ in ends)
    return {"bytes": scored * bound + read * kept + io + n * hkv * case["select"] * 4,
            "flops": 4 * dots * h * dim + 4 * hkv * dim * sum((e - 1) // block + 1 for e, _ in ends)}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    """Sequence by sequence in float64: the rotation as butterflies, the cache turned back
    to unrotated rows before the attention."""
    s = prepare(case, seed)
    c, dim, hkv = case, case["dim"], case["kv_heads"]
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
        sc = s[name + "_scales"][at][:, :hkv * dim // GROUP].double().view(len(at), hkv, dim // GROUP, 1)
        return rotate((x.view(len(at), hkv, dim // GROUP, GROUP) * sc).view(len(at), hkv, dim))

    pos, rows, _ = _layout(case)
    out, chosen, first = [], [], 0
    bounds = s["bounds"].clone() if s["bounds"] is not None else None
    for b, (p0, r) in enumerate(zip(pos, rows)):
        mine = slice(first, first + r)
        first += r
        t_new = torch.arange(p0, p0 + r, device=DEV)
        at = physical(b, t_new)
        if c["op"] in ("append", "roundtrip"):
            for name in ("k", "v"):
                x = s[name + "_new"][mine]
                if turbo8:
                    y = rotate(x).to(torch.bfloat16).double().view(r, hkv, dim // GROUP, GROUP)
                    sc = (y.abs().amax(-1) / 448).to(torch.bfloat16)
                    q = torch.where(sc[..., None] > 0, y / sc[..., None].double(), 0.0).clamp(-448, 448)
                    s[name][at] = q.float().to(torch.float8_e4m3fn).view(torch.uint8).view(r, hkv, dim)
                    s[name + "_scales"][at, :sc[0].numel()] = sc.view(r, -1)
                else:
                    s[name][at] = x
            for j in range(p0 // c["block"], (p0 + r - 1) // c["block"] + 1):
                in_block = s["k_new"][mine][torch.div(t_new, c["block"], rounding_mode="floor") == j].double()
                at_j = physical(b, torch.tensor(j * c["block"], device=DEV)) // c["block"]
                lo, hi = in_block.amin(0), in_block.amax(0)
                if j * c["block"] < p0:
                    lo = torch.minimum(lo, bounds[at_j, :, 0].double())
                    hi = torch.maximum(hi, bounds[at_j, :, 1].double())
                bounds[at_j, :, 0], bounds[at_j, :, 1] = lo.to(torch.bfloat16), hi.to(torch.bfloat16)
        if c["op"] in ("read", "roundtrip"):
            out.append((held("k", at), held("v", at)))
            continue
        if c["op"] == "append":
            continue
        t = torch.arange(p0 + r, device=DEV)
        k, v = held("k", physical(b, t)), held("v", physical(b, t))
        for i in range(r):
            q = s["q"][mine][i].double().view(hkv, -1, dim)
            n = p0 + i + 1
            see = torch.ones(hkv, n, dtype=torch.bool, device=DEV)
            if c["op"] == "sparse":
                nb = (n - 1) // c["block"] + 1
                bb = bounds[physical(b, torch.arange(nb, device=DEV) * c["block"]) // c["block"]].double()
                score = torch.maximum(q[None] * bb[:, :, 0, None], q[None] * bb[:, :, 1, None]).sum((2, 3)).T
                score[:, 0] = score[:, -1] = math.inf
                order = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :c["select"]]
                inside = torch.zeros(hkv, nb, dtype=torch.bool, device=DEV).scatter_(1, order, True)
                see = inside.repeat_interleave(c["block"], 1)[:, :n]
                pick = torch.full((hkv, c["select"]), -1, dtype=torch.int32, device=DEV)
                pick[:, :order.shape[1]] = order.sort(-1).values.to(torch.int32)
                chosen.append(pick)
            x = torch.einsum("ghd,tgd->ght", q, k[:n]) / math.sqrt(dim)
            x = torch.softmax(x.masked_fill(~see[:, None], -math.inf), -1)
            o = torch.einsum("ght,tgd->ghd", x, v[:n]).flatten(0, 1)
            out.append(o * torch.sigmoid(s["gate"][mine][i].double()))
    if c["op"] == "append":
        return s["k"].double(), s["v"].double(), bounds.double()
    if c["op"] in ("read", "roundtrip"):
        back = tuple(torch.cat([o[i] for o in out]) for i in (0, 1))
        return back if c["op"] == "read" else back + (bounds.double(),)
    if c["op"] == "sparse":
        return torch.stack(chosen), torch.stack(out)
    return torch.stack(out)
