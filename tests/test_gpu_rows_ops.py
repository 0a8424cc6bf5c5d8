"""The operators of a drafting loop on the GPU against plain float64 implementations.

Tolerances, derived before the first run (a rounding to bf16 is off by at most 2^-8 of the value, to f16 by
2^-11, to fp32 by 2^-24):
 - rows moved, codes and scales of rotated rows against qwen35_cache_append of the same rows, tokens sampled: equal;
 - a rotated value y = a cos - b sin: its rounding, 2^-8 |y|; the rounding of the normed a and b, 2^-8 (|a| + |b|),
   where there is a norm; and the fp32 arithmetic, far below 2^-18 (|a| + |b|);
 - attention over a bf16 cache: the output's rounding, 2^-8 |y|, and 2^-14 of the largest value: the weights
   are good to 2^-16, scores and sums are fp32;
 - over a Turbo8 cache the rotated q, the keys and so the scores are off by 2^-11 each: 2^-10 sum |q_d k_d| / sqrt D <=
   2^-10 |q| |k| / sqrt D = d; weights and values lose 2^-11 each: an error of the rotated output of
   norm at most (2 d + 2^-10) max |v|, which the rotation back keeps. Roundings are of either sign, so the whole output's
   2-norm is also held to 2^-8 + 2^-9 of the reference's (one bf16 rounding, and half of that for all others).
"""

import numpy as np
import pytest
import torch

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth
from oracle import qwen35_oracle as O

from test_gpu_cache_ops import BF16, HEADS, TURBO8, Setup, bf16, f64
from test_gpu_cache_ranges import put

pytestmark = pytest.mark.gpu

NAN = float("nan")


def status(s):
    torch.cuda.synchronize()
    return B.qwen35_read_device_status(s.scratch)


def setup(heads, fmt, lens, rows, **kw):
    s = Setup(heads, fmt, lens, rows, **kw)
    s.scratch = B.new_scratch(B.qwen35_rows_scratch_bytes(s.cfg, s.n_rows))
    return s


# ---------------------------------------------------------------- attention


def visible_tree(parent, pos, i):
    see = list(range(pos))
    while i >= 0:
        see.append(pos + i)
        i = parent[i]
    return see


def visible_window(p, window, first):
    low = max(0, p - window + 1)
    return list(range(min(first, low))) + list(range(low, p + 1))


def expect(s, see, gate=None):
    """{row: (float64 output [H][D], tolerance)} with see(b, i, p) -> tokens."""
    out = {}
    for b, (m, r) in enumerate(zip(s.lens, s.rows)):
        for i in range(r):
            row, p = s.start[b] + i, m - r + i
            t = see(b, i, p)
            if t is None:
                continue
            at = s.at(b, np.asarray(t))
            k, v = (s.stands[n][at] for n in "kv")
            q = f64(s.q[row]).reshape(s.Hkv, -1, s.D)
            x = np.einsum("ghd,tgd->ght", q, k) / np.sqrt(s.D)
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            o = np.einsum("ght,tgd->ghd", w, v).reshape(s.H, s.D)
            if s.fmt == TURBO8:
                d = 2.0 ** -10 * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max() / np.sqrt(s.D)
                tol = (2 * d + 2.0 ** -10) * np.linalg.norm(v, axis=-1).max()
            else:
                tol = 2.0 ** -14 * np.abs(v).max()
            z = 1.0
            if gate is not None:
                z = 1 / (1 + np.exp(-f64(gate[row]).reshape(s.H, -1)[:, :s.D]))
            out[row] = (o * z, tol)
    return out


def check(s, out, want):
    got = f64(out)
    for r in range(s.n_rows):
        if r not in want:
            assert np.isnan(got[r]).all(), f"row {r} is not left as it was"
            continue
        ref, tol = want[r]
        err = np.abs(got[r] - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + tol).all(), (r, float(np.nanmax(err)), tol, np.isnan(got[r]).sum())
    if want:
        a, b = (np.stack([x[r] for r in sorted(want)]) for x in (got, {r: w[0] for r, w in want.items()}))
        assert np.linalg.norm(a - b) <= (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(b)


def blank(s):
    return torch.full((s.n_rows, s.H, s.D), NAN, dtype=torch.bfloat16, device="cuda")


def tree_of(kind, n, rng):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1 if i % 5 == 0 else int(rng.integers(0, i)) for i in range(n)]
    return [-1] + [int(rng.integers(max(0, (i - 1) // 4), i)) for i in range(1, n)]


def run_tree(s, parents, gate=None, **kw):
    flat = np.full(s.n_rows, 7777, dtype=np.int32)
    for b, p in enumerate(parents):
        flat[s.start[b]:s.start[b] + len(p)] = p
    out = blank(s)
    rc = B.qwen35_tree_attention(s.cfg, s.kv, s.r, torch.from_numpy(flat).cuda(), s.q.cuda(), out, s.scratch, gate=gate,
                                 **kw)
    assert rc == 0
    return out


@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("fmt,page", [(BF16, 0), (BF16, 16), (TURBO8, 0), (TURBO8, 64)])
def test_trees(heads, fmt, page):
    rng = np.random.default_rng(1)
    nodes = [1, 7, 0, 33, 16, 64, 5]
    before = [0, 1, 40, 63, 200, 130, 517]
    s = setup(heads, fmt, [n + b for n, b in zip(nodes, before)], nodes, page=page, lead=2, tail=3)
    kinds = ["chain", "star", "chain", "random", "forest", "random", "chain"]
    parents = [tree_of(k, n, rng) if n else [] for k, n in zip(kinds, nodes)]
    out = run_tree(s, parents)
    check(s, out, expect(s, lambda b, i, p: visible_tree(parents[b], before[b], i)))
    assert status(s) == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("n", [31, 32, 33, 65, 127, 128])
@pytest.mark.parametrize("kind", ["chain", "random"])
def test_large_trees_with_gates(fmt, n, kind):
    rng = np.random.default_rng(n)
    s = setup("4b", fmt, [300 + n, n], [n, n], page=16)
    parents = [tree_of(kind, n, rng) for _ in range(2)]
    gate = bf16(rng.standard_normal((s.n_rows, s.H, 2 * s.D))).cuda()
    out = run_tree(s, parents, gate=gate, gate_stride=2 * s.D)
    check(s, out, expect(s, lambda b, i, p: visible_tree(parents[b], [300, 0][b], i), gate))
    assert status(s) == 0


@pytest.mark.parametrize("heads,fmt", [("4b", BF16), ("4b", TURBO8), ("tiny_alt", TURBO8), ("tiny", BF16)])
def test_a_long_context_is_split_and_joined(heads, fmt):
    rng = np.random.default_rng(5)
    s = setup(heads, fmt, [9001 + 40, 700 + 3], [40, 3], page=32)
    parents = [tree_of("random", 40, rng), tree_of("star", 3, rng)]
    want = expect(s, lambda b, i, p: visible_tree(parents[b], [9001, 700][b], i))
    first = run_tree(s, parents)
    check(s, first, want)
    for _ in range(3):
        assert torch.equal(run_tree(s, parents).view(torch.int16), first.view(torch.int16))
    assert status(s) == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_nodes_that_a_row_does_not_see_leave_no_trace(fmt, bad):
    """Key and value of a node that holds no number: only the nodes below it are spoiled."""
    s = setup("4b", fmt, [100 + 20], [20], page=16)
    parent = [-1, 0, 0, 1, 1, 2, 3, 3, 4, 5, 5, 6, 8, 9, -1, 14, 14, 15, 17, 18]
    at = s.at(0, np.asarray([100 + 3, 100 + 15]))
    under = [i for i in range(20) if any(t - 100 in (3, 15) for t in visible_tree(parent, 100, i))]
    if fmt == TURBO8:
        for n in "kv":
            s.t[n + "s"][torch.from_numpy(at).cuda()] = bf16([bad]).view(torch.int16).item()
            s.stands[n][at] = np.nan
    else:
        for n in "kv":
            s.t[n][torch.from_numpy(at).cuda()] = bad
            s.stands[n][at] = bad
    out = run_tree(s, [parent])
    want = expect(s, lambda b, i, p: None if i in under else visible_tree(parent, 100, i))
    got = f64(out)
    for i in under:
        assert not np.isfinite(got[i]).all()
        out[i] = NAN
    check(s, out, want)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_values_that_are_infinite_reach_the_rows_that_see_them(fmt):
    """One element of one node's value is infinite: the node's descendants get that dimension (Turbo8: its
    group's scale is infinite, so they get no number), the others nothing."""
    s = setup("tiny_alt", fmt, [64 + 6], [6])
    parent, at = [-1, 0, 0, 1, 2, 3], int(s.at(0, 65))
    if fmt == BF16:
        s.t["v"][at, 1, 77] = float("inf")
        s.stands["v"][at, 1, 77] = np.inf
    else:
        s.t["vs"][at, (128 + 77) // 16] = bf16([float("inf")]).view(torch.int16).item()
    got = f64(run_tree(s, [parent]))
    for i in range(6):
        below = 1 in [t - 64 for t in visible_tree(parent, 64, i)]
        assert np.isfinite(got[i][[0, 2]]).all()
        if fmt == BF16:
            assert np.isfinite(np.delete(got[i][1], 77)).all()
            assert not np.isfinite(got[i][1, 77]) if below else np.isfinite(got[i][1, 77])
        else:
            assert not np.isfinite(got[i][1]).all() if below else np.isfinite(got[i][1]).all()


def test_bad_nodes_are_skipped_and_reported():
    s = setup("tiny", BF16, [50 + 9, 30 + 4, 20 + 3], [9, 4, 3])
    parents = [[-1, 0, 5, 2, 1, -2, 5, 7, 0], [-1, 0, 1, 2], [0, 0, 99]]
    out = run_tree(s, parents)
    ok = {0: [0, 1, 4, 8], 1: [0, 1, 2, 3], 2: []}
    check(s, out, expect(s, lambda b, i, p: visible_tree(parents[b], [50, 30, 20][b], i) if i in ok[b] else None))
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE


def test_nodes_behind_the_most_are_skipped_and_reported():
    s = setup("tiny", BF16, [10 + 131], [131])
    parent = [-1] + [0] * 130
    out = run_tree(s, [parent])
    check(s, out, expect(s, lambda b, i, p: visible_tree(parent, 10, i) if i < 128 else None))
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE


@pytest.mark.parametrize("pos", [-1, 2 ** 31 - 1, 190])
def test_trees_at_positions_outside_the_cache(pos):
    s = setup("tiny", BF16, [40 + 5, 60 + 2], [5, 2], page=16)
    assert s.cap == 64
    s.pos[0] = pos
    parents = [tree_of("star", 5, None), [-1, 0]]
    out = run_tree(s, parents)
    check(s, out, expect(s, lambda b, i, p: visible_tree(parents[b], 60, i) if b else None))
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_blocks_outside_the_pool_are_left_out_and_reported(fmt):
    s = setup("4b", fmt, [80 + 4], [4], page=16)
    s.table[0, 2] = s.nb
    s.table[0, 4] = -5
    parent = [-1, 0, 0, 1]
    gone = set(range(32, 48)) | set(range(64, 80))
    out = run_tree(s, [parent])
    check(s, out, expect(s, lambda b, i, p: [t for t in visible_tree(parent, 80, i) if t not in gone]))
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE


def test_a_row_without_a_token_gets_zeros():
    s = setup("4b", BF16, [3, 70], [1, 2], page=16)
    s.table[0, 0] = s.nb
    out = run_tree(s, [[-1], [-1, 0]])
    assert (out[0] == 0).all()
    assert torch.isfinite(out[1:].float()).all()
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE


def run_window(s, window, first, gate=None, **kw):
    out = blank(s)
    rc = B.qwen35_window_attention(s.cfg, s.kv, s.r, window, first, s.q.cuda(), out, s.scratch, gate=gate, **kw)
    assert rc == 0
    return out


@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("fmt,page", [(BF16, 0), (BF16, 64), (TURBO8, 0), (TURBO8, 16)])
@pytest.mark.parametrize("window,first", [(1, 0), (64, 4), (200, 70)])
def test_windows(heads, fmt, page, window, first):
    lens = [1, 2, 65, 64, 700, 331, 9]
    s = setup(heads, fmt, lens, None, page=page)
    out = run_window(s, window, first)
    check(s, out, expect(s, lambda b, i, p: visible_window(p, window, first)))
    assert status(s) == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (7, 0), (63, 5), (65, 64), (128, 0), (10 ** 6, 3), (2 ** 32 - 1, 0),
                                          (100, 2 ** 32 - 1), (8, 300)])
def test_windows_of_several_rows(fmt, window, first):
    s = setup("4b", fmt, [300, 130, 40, 77], [130, 130, 3, 0], page=16, lead=1, tail=2)
    gate = bf16(s.rng.standard_normal((s.n_rows, s.H, s.D))).cuda()
    out = run_window(s, window, first, gate=gate)
    check(s, out, expect(s, lambda b, i, p: visible_window(p, window, first), gate))
    assert status(s) == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_pages_outside_the_window_are_not_read(fmt):
    """Their entries name no block, or blocks without a number."""
    s = setup("4b", fmt, [640, 641], None, page=16)
    window, first = 100, 20
    for b, p in enumerate((639, 640)):
        seen = {t // 16 for t in visible_window(p, window, first)}
        for j in range(640 // 16 + 1):
            if j not in seen:
                s.table[b, j] = -1
    want = expect(s, lambda b, i, p: visible_window(p, window, first))
    out = run_window(s, window, first)
    check(s, out, want)
    assert status(s) == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_tokens_that_left_the_window_leave_no_trace(fmt, bad):
    """Rows of one call: the first ones see a token without a number, the later ones no longer."""
    s = setup("4b", fmt, [300], [60])
    at = int(s.at(0, 180))  # seen up to position 180 + 79
    for n in "kv":
        if fmt == TURBO8:
            s.t[n + "s"][at] = bf16([bad]).view(torch.int16).item()
        else:
            s.t[n][at] = bad
        s.stands[n][at] = np.nan
    out = run_window(s, 80, 2)
    got = f64(out)
    assert all(not np.isfinite(got[i]).all() for i in range(20))
    out[:20] = NAN
    check(s, out, expect(s, lambda b, i, p: visible_window(p, 80, 2) if i >= 20 else None))


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_a_long_window_of_a_long_context(fmt):
    s = setup("4b", fmt, [20000, 12345, 4000, 700, 6000], None, page=64)
    out = run_window(s, 5000, 4)
    check(s, out, expect(s, lambda b, i, p: visible_window(p, 5000, 4)))
    assert status(s) == 0


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 40])
def test_values_and_scores_of_any_size(scale):
    """V scaled by a power of two scales the output. Not bit for bit: V's exponent goes into the weight's, and a weight
    (x - m) + E with |E| = 40 is rounded at 2^-24 of up to 64, 2^-18 of it, which may take it over a border of f16: half a
    step, 2^-11, on either side, an error of the rotated output of norm up to 2^-10 max |v|; and both outputs are
    rounded, 2^-8 each."""
    s = setup("4b", TURBO8, [200 + 3], [3])
    plain = f64(run_tree(s, [[-1, 0, 0]])) * scale
    s.t["vs"] = (s.t["vs"].view(torch.bfloat16).float() * scale).to(torch.bfloat16).view(torch.int16)
    s.kv.v_scales = s.t["vs"].data_ptr()
    got = f64(run_tree(s, [[-1, 0, 0]]))
    most = scale * np.linalg.norm(s.stands["v"][s.at(0, np.arange(203))], axis=-1).max()
    assert (np.abs(got - plain) <= 2 * 2.0 ** -8 * np.abs(plain) + (2.0 ** -10 + 2.0 ** -18) * most).all()
    assert np.linalg.norm(got - plain) <= 2.0 ** -9 * np.linalg.norm(plain)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_large_scores(fmt):
    """One key far ahead of the others, at several places; equal outputs to its value."""
    s = setup("4b", fmt, [500], None, spread=4.0)
    s.q = s.q * 16
    out = run_window(s, 400, 1)
    want = expect(s, lambda b, i, p: visible_window(p, 400, 1))
    if fmt == BF16:
        check(s, out, want)
    assert torch.isfinite(out.float()).all()


def test_chains_are_decode_attention():
    s = setup("4b", BF16, [900, 77], [6, 2], page=16)
    out = run_tree(s, [[-1, 0, 1, 2, 3, 4], [-1, 0]])
    other = blank(s)
    scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(s.cfg, s.cap, 0, s.n_rows))
    assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, s.q.cuda(), other, scratch) == 0
    a, b = f64(out), f64(other)
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2.0 ** -13 * 5).all()


# ---------------------------------------------------------------- rotated rows


def rotated(cfg, x, w, pos):
    """float64: the normed (not rounded) pairs' parts a, b and the rotated value, dim by dim."""
    y = f64(x)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + cfg.rms_eps) * f64(w)
    R = cfg.rotary_dim
    out, size = y.copy(), np.abs(y)
    if R:
        i = np.arange(R // 2)
        freq = (float(cfg.rope_theta) ** (-2.0 * i / R)).astype(np.float32)
        a = (np.asarray(pos, dtype=np.float32)[:, None, None] * freq).astype(np.float32).astype(np.float64)
        lo, hi = y[..., :R // 2], y[..., R // 2:R]
        out[..., :R // 2] = lo * np.cos(a) - hi * np.sin(a)
        out[..., R // 2:R] = hi * np.cos(a) + lo * np.sin(a)
        size[..., :R // 2] = size[..., R // 2:R] = np.abs(lo) + np.abs(hi)
    return out, size


def rope_setup(heads, fmt, lens, rows, R, page=0, **kw):
    s = setup(heads, fmt, lens, rows, page=page, **kw)
    s.cfg.rotary_dim, s.cfg.rope_theta, s.cfg.rms_eps = R, 1e7, 1e-6
    rng = s.rng
    s.qg = bf16(2 * rng.standard_normal((s.n_rows, s.H, 2 * s.D))).cuda()
    s.k_new = bf16(3 * rng.standard_normal((s.n_rows, s.Hkv, s.D))).cuda()
    s.v_new = bf16(rng.standard_normal((s.n_rows, s.Hkv, s.D))).cuda()
    s.wq, s.wk = (bf16(1 + 0.1 * rng.standard_normal(s.D)).cuda() for _ in range(2))
    s.q_out = blank(s)
    s.k_out = torch.full_like(s.k_new, NAN)
    return s


def cache_state(s):
    return {n: t.clone() for n, t in s.t.items()}


@pytest.mark.parametrize("heads,R", [("4b", 64), ("tiny", 16), ("tiny_alt", 32), ("wide", 128), ("eight", 2), ("odd", 6),
                                     ("twelve", 250), ("4b", 0), ("4b", 256)])
@pytest.mark.parametrize("fmt,page", [(BF16, 0), (BF16, 16), (TURBO8, 0), (TURBO8, 64)])
@pytest.mark.parametrize("norm", [True, False])
def test_rotated_rows(heads, R, fmt, page, norm):
    lens, rows = [1, 90, 64, 700, 30], [1, 17, 0, 40, 3]
    s = rope_setup(heads, fmt, lens, rows, R, page=page, lead=2, tail=1)
    before = cache_state(s)
    kw = dict(q_norm=s.wq, k_norm=s.wk) if norm else {}
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, s.qg, s.k_new, s.v_new, s.q_out, s.scratch, q_stride=2 * s.D,
                                      k_out=s.k_out, **kw) == 0
    assert status(s) == 0
    rows_pos = list(s.each_row())
    idx, pos = [r for r, _, _ in rows_pos], [p for _, _, p in rows_pos]
    for got, x, w in ((s.q_out, s.qg[..., :s.D], s.wq), (s.k_out, s.k_new, s.wk)):
        ref, size = rotated(s.cfg, x[idx], w if norm else None, pos)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 if norm else 0) * size + 2.0 ** -18 * size
        assert (np.abs(f64(got[idx]) - ref) <= tol).all()
        rest = [r for r in range(s.n_rows) if r not in idx]
        assert torch.isnan(got[rest].float()).all()
    # the cache: what qwen35_cache_append makes of the rotated keys, and nothing else
    after = cache_state(s)
    for n in s.t:
        s.t[n].copy_(before[n])
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, s.k_out, s.v_new, s.scratch) == 0
    for n in s.t:
        assert torch.equal(s.t[n].view(torch.uint8), after[n].view(torch.uint8)), n


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_positions_of_a_tree_and_far_ones(fmt):
    s = rope_setup("4b", fmt, [100, 50], [10, 4], 64, page=16)
    where = [0, 5, 131071, 7, 1 << 20, 105615, 105616, 99999999, 3, 2 ** 31 - 1, 0, 1, 1, 2]
    rp = torch.tensor(where, dtype=torch.int32, device="cuda")
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, s.qg, s.k_new, s.v_new, s.q_out, s.scratch, q_norm=s.wq,
                                      k_norm=s.wk, q_stride=2 * s.D, rope_pos=rp, k_out=s.k_out) == 0
    for got, x, w in ((s.q_out, s.qg[..., :s.D], s.wq), (s.k_out, s.k_new, s.wk)):
        ref, size = rotated(s.cfg, x, w, where)
        assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -18) * size).all()


@pytest.mark.parametrize("heads,fmt,page", [("4b", BF16, 64), ("4b", TURBO8, 0), ("tiny", TURBO8, 32)])
def test_in_place_and_with_bounds(heads, fmt, page):
    lens, rows = [90, 33], [50, 33]
    s = rope_setup(heads, fmt, lens, rows, 16, page=page, block=16)
    q = s.qg[..., :s.D].contiguous()
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, q, s.k_new, s.v_new, s.q_out, s.scratch, q_norm=s.wq,
                                      k_norm=s.wk, k_out=s.k_out) == 0
    one, k1, q1 = cache_state(s), s.k_out.clone(), s.q_out.clone()
    s.lo_hi.zero_()
    k_in = s.k_new.clone()
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, q, k_in, s.v_new, q, s.scratch, q_norm=s.wq, k_norm=s.wk,
                                      k_out=k_in, bounds=s.bounds) == 0
    assert torch.equal(q, q1) and torch.equal(k_in, k1)
    for n in s.t:
        assert torch.equal(s.t[n].view(torch.uint8), one[n].view(torch.uint8)), n
    got = s.lo_hi.clone()
    s.lo_hi.zero_()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k1, s.v_new, s.scratch) == 0
    assert torch.equal(got, s.lo_hi)


def test_keys_alone_and_rows_outside():
    s = rope_setup("tiny", BF16, [20, 30, 10], [2, 3, 1], 16, page=16)
    s.pos[1] = s.cap - 1  # its second row is outside
    s.table[2, 0] = s.nb
    before = cache_state(s)
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, None, s.k_new, s.v_new, None, s.scratch, k_norm=s.wk,
                                      k_out=s.k_out) == 0
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE
    assert torch.isfinite(s.k_out[[0, 1, 2]].float()).all() and torch.isnan(s.k_out[[3, 4, 5]].float()).all()
    changed = (s.t["k"].view(torch.int16) != before["k"].view(torch.int16)).any(-1).any(-1).sum()
    assert changed == 3


def test_rows_turned_and_turned_back():
    """Rows turned by p, then by -p, are themselves within two roundings."""
    s = rope_setup("4b", BF16, [40], [40], 64)
    rp = torch.arange(40, dtype=torch.int32, device="cuda")
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, None, s.k_new, s.v_new, None, s.scratch, k_out=s.k_out,
                                      rope_pos=rp) == 0
    back = torch.empty_like(s.k_out)
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, None, s.k_out, s.v_new, None, s.scratch, k_out=back,
                                      rope_pos=-rp) == 0
    a, b = f64(back), f64(s.k_new)
    size = np.abs(b).copy()
    size[..., :32] = size[..., 32:64] = np.abs(b[..., :32]) + np.abs(b[..., 32:64])
    assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + 2 * 2.0 ** -8 * size).all()


# ---------------------------------------------------------------- kept rows


def run_keep(s, paths, bounds=None):
    flat = [x for p in paths for x in p]
    start = np.concatenate([[0], np.cumsum([len(p) for p in paths])]).astype(np.int32)
    rows = B.DeviceRows(s.pos, torch.from_numpy(start).cuda(), max(1, len(flat)), s.nb)
    path = torch.tensor(flat or [0], dtype=torch.int32, device="cuda")
    return B.qwen35_cache_keep(s.cfg, s.kv, rows, path, s.scratch, bounds=bounds)


@pytest.mark.parametrize("heads", ["4b", "tiny", "tiny_alt", "wide"])
@pytest.mark.parametrize("fmt,page", [(BF16, 0), (BF16, 16), (TURBO8, 0), (TURBO8, 8)])
def test_kept_rows(heads, fmt, page):
    n = [20, 128, 64, 1, 9, 128]
    s = setup(heads, fmt, [b + x for b, x in zip([5, 70, 0, 33, 16, 8], n)], n, page=page, block=16 if page != 8 else 16)
    rng = np.random.default_rng(3)
    paths = [[0, 2, 9, 19], sorted(rng.choice(128, 40, replace=False).tolist()), [], [0], [8], list(range(128))]
    want = cache_state(s)
    for b, path in enumerate(paths):
        p0 = int(s.pos[b])
        src = torch.from_numpy(s.at(b, p0 + np.asarray(path, dtype=np.int64))).cuda()
        dst = torch.from_numpy(s.at(b, p0 + np.arange(len(path)))).cuda()
        for t in want:
            want[t][dst] = want[t][src].clone()
    assert run_keep(s, paths) == 0
    assert status(s) == 0
    for t in want:
        assert torch.equal(s.t[t].view(torch.uint8), want[t].view(torch.uint8)), t


@pytest.mark.parametrize("path", [[3, 2], [1, 1], [-1, 2], [0, 5, 4000], list(range(129))])
def test_bad_paths_move_nothing(path):
    s = setup("tiny", BF16, [40 + 130, 40 + 130], [130, 130], page=16)
    before = cache_state(s)
    assert run_keep(s, [path, [0, 4]]) == 0
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE
    dst, src = int(s.at(1, 41)), int(s.at(1, 44))
    before["k"][dst], before["v"][dst] = before["k"][src].clone(), before["v"][src].clone()
    for t in before:
        assert torch.equal(s.t[t].view(torch.uint8), before[t].view(torch.uint8))


def test_paths_in_blocks_outside_the_pool():
    s = setup("tiny", BF16, [16 + 20], [20], page=16)
    s.table[0, 2] = s.nb + 4
    before = cache_state(s)
    assert run_keep(s, [[0, 17]]) == 0
    assert status(s) == B.QWEN35_ERR_DEVICE_RANGE
    assert torch.equal(s.t["k"].view(torch.uint8), before["k"].view(torch.uint8))


def test_bounds_hold_the_kept_keys():
    s = setup("4b", BF16, [25 + 60], [60], page=32, block=16)
    s.set_bounds()
    path = [0, 8, 20, 21, 39, 59]
    assert run_keep(s, [path], bounds=s.bounds) == 0
    lo_hi = f64(s.lo_hi)
    for i in range(len(path)):
        at = int(s.at(0, 25 + i))
        key = f64(s.t["k"][at])
        lo, hi = lo_hi[at // 16, :, 0], lo_hi[at // 16, :, 1]
        assert (lo <= key).all() and (key <= hi).all()


# ---------------------------------------------------------------- sampling


def plain_sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """float64, one row [vocab] of logits: (token, probability)."""
    ids = np.nonzero(~np.isnan(x))[0]
    if len(ids) == 0:
        return -1, 0.0
    x = x[ids]
    order = np.lexsort((ids, -x))
    x, ids = x[order], ids[order]
    if not t > 0:
        return int(ids[0]), 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == x[0], 1.0, np.exp((x - x[0]) / t))
    if k > 0:
        w = w[:k]
    if p < 1:
        c = np.cumsum(w)
        w = w[:1 + int((c[:-1] < max(p, 0.0) * c[-1]).sum())]
    w = w[w >= min(m, 1.0)] if m > 0 else w
    c = np.cumsum(w)
    u = 0.0 if not u > 0 else u
    j = min(int((c <= u * c[-1]).sum()), int((w > 0).sum()) - 1)
    return int(ids[j]), w[j] / c[-1]


def dev(x, dtype=torch.float32):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def run_sample(x, u, t=None, k=None, p=None, m=None):
    n = x.shape[0]
    token = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((n,), NAN, device="cuda")
    u = dev(u)
    rc = B.qwen35_sample(x, u, token, temperature=dev(t), top_k=dev(k, torch.int32), top_p=dev(p), min_p=dev(m), prob=prob)
    assert rc == 0
    return token.cpu().numpy(), prob.cpu().numpy()


def check_sample(x, u, t=None, k=None, p=None, m=None):
    token, prob = run_sample(x, u, t, k, p, m)
    f32 = lambda v, r, d: d if v is None else float(np.float32(v[r]))  # noqa: E731
    host = f64(x)
    for r in range(x.shape[0]):
        want, q = plain_sample(host[r], float(np.float32(u[r])), f32(t, r, 1.0), 0 if k is None else int(k[r]),
                               f32(p, r, 1.0), f32(m, r, 0.0))
        assert token[r] == want, (r, token[r], want)
        # fp32 roundings of weight, sum and quotient, and the weight's own 2^-44 of the largest
        assert abs(prob[r] - q) <= 2.0 ** -21 * q + 2.0 ** -43, (r, prob[r], q)


def logits(n, vocab, seed=0, spread=2.5):
    rng = np.random.default_rng(seed)
    x = spread * rng.standard_normal((n, vocab))
    for r in range(n):
        x[r, rng.integers(0, vocab, 12)] += 8
    return bf16(x).cuda()


@pytest.fixture(autouse=True)
def _init():
    from harness import init
    init()


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 64, 65, 500, 4097, 65537, 248320])
@pytest.mark.parametrize("mode", ["none", "all", "mixed"])
def test_samples(vocab, mode):
    n = 24 if vocab < 60000 else 9
    rng = np.random.default_rng(vocab)
    x = logits(n, vocab, vocab)
    u, t = rng.random(n), 0.3 + 1.5 * rng.random(n)
    if mode == "none":
        return check_sample(x, u, t)
    k = rng.integers(1, 100, n) * (1 if mode == "all" else rng.integers(0, 2, n))
    p = 0.3 + 0.69 * rng.random(n) if mode == "all" else np.where(rng.random(n) < 0.5, rng.random(n), 1.0)
    m = 0.2 * rng.random(n) * (1 if mode == "all" else rng.integers(0, 2, n))
    check_sample(x, u, t, k, p, m)


def test_settings_at_their_ends():
    inf = float("inf")
    rows = [dict(u=0.0), dict(u=1.0), dict(u=-3.0), dict(u=NAN), dict(u=7.0), dict(u=1 - 2.0 ** -24), dict(t=0.0), dict(t=-1.0),
            dict(t=NAN), dict(t=1e-30), dict(t=1e30), dict(t=inf), dict(k=1), dict(k=-4), dict(k=2 ** 31 - 1), dict(k=1000),
            dict(p=0.0), dict(p=-1.0), dict(p=1e-9), dict(p=NAN), dict(p=2.0), dict(m=1.0), dict(m=5.0), dict(m=NAN),
            dict(m=-1.0), dict(k=3, p=0.0, m=1.0), dict(t=0.0, k=5, u=0.9), dict(k=5, t=100.0, u=0.999)]
    d = dict(u=0.6, t=0.9, k=0, p=1.0, m=0.0)
    rows = [d | r for r in rows]
    x = logits(1, 1000, 3).expand(len(rows), -1).contiguous()
    check_sample(x, *([r[n] for r in rows] for n in "utkpm"))


@pytest.mark.parametrize("values", [[0.0], [1.0, -0.0, 0.0], [2.0, 2.0, -3.0], [-1e38, -1e38, -3e38], [5.0, -float("inf")],
                                    [-float("inf")], [float("inf"), 3.0], [NAN, 1.0, 0.5], [NAN], [3.4e38, -3.4e38]])
def test_few_values(values):
    """Ties in the thousands: the lower indexes first, whatever the cuts."""
    rng = np.random.default_rng(0)
    n, vocab = 16, 3001
    x = bf16(rng.choice(values, (n, vocab))).cuda()
    u = np.arange(n) / n
    with np.errstate(over="ignore"):
        check_sample(x, u)
        check_sample(x, u, k=1 + np.arange(n) * 150)
        check_sample(x, u, p=np.float32((1 + np.arange(n)) / 16.0))
        check_sample(x, u, t=np.full(n, 2.0), k=np.full(n, 700), p=np.full(n, 0.5), m=np.full(n, 0.3))


def test_the_largest_vocabulary_of_one_value():
    """Counts at their most: every token of a CTA's part equal."""
    vocab = 8 * 65520
    x = torch.ones(3, vocab, dtype=torch.bfloat16, device="cuda")
    token, prob = run_sample(x, [0.0, 0.5, 1.0])
    assert token.tolist() == [0, vocab // 2, vocab - 1]
    assert np.allclose(prob, 1 / vocab, rtol=2.0 ** -22)


@pytest.mark.parametrize("vocab,stride", [(500, 500), (501, 501), (777, 1003), (64, 71), (5, 5)])
def test_rows_at_any_stride(vocab, stride):
    n = 11
    base = torch.full((n, stride), 60000.0, dtype=torch.bfloat16, device="cuda")  # the gaps hold larger values
    x = base[:, :vocab]
    x.copy_(logits(n, vocab, 5))
    rng = np.random.default_rng(1)
    check_sample(x, rng.random(n), k=rng.integers(0, 40, n))


def test_many_rows_and_shares():
    """Tokens come as often as their probabilities say (and every row of 4096 is its own)."""
    n = 4096
    x = bf16([[0.0, 1.0, 2.0, -1.0, 0.5]]).cuda().expand(n, -1).contiguous()
    u = (np.arange(n) + 0.5) / n
    token, _ = run_sample(x, u)
    w = np.exp(f64(x[0]))
    share = np.bincount(token, minlength=5) / n
    assert np.abs(share - w / w.sum()).max() <= 1.5 / n


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("captured", [False, True])
def test_a_drafting_step(fmt, captured):
    """Trees appended, attended, a token sampled for every node, the accepted path kept, the next step on top:
    the cache then holds what appending the accepted tokens alone would have left, and a captured step does the same."""
    H, Hkv, D = HEADS["4b"]
    rows, lens = [7, 7], [100 + 7, 33 + 7]
    s = rope_setup("4b", fmt, lens, rows, 64, page=16)
    parent = [-1, 0, 0, 1, 1, 2, 4]
    depth = torch.tensor([0, 1, 1, 2, 2, 2, 3] * 2, dtype=torch.int32, device="cuda")
    paths = [[0, 1, 4, 6], [0, 2, 5]]
    par = torch.tensor(parent * 2, dtype=torch.int32, device="cuda")
    rope_pos = torch.repeat_interleave(s.pos, 7).int() + depth
    start = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
    keep_rows = B.DeviceRows(s.pos, start, 7, s.nb)
    path = torch.tensor(sum(paths, []), dtype=torch.int32, device="cuda")
    out, head = blank(s), bf16(s.rng.standard_normal((H * D, 300)) / 64).cuda()
    lg = torch.empty(s.n_rows, 300, dtype=torch.bfloat16, device="cuda")
    u = torch.rand(s.n_rows, device="cuda")
    token = torch.empty(s.n_rows, dtype=torch.int32, device="cuda")

    def step():
        assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, s.qg, s.k_new, s.v_new, s.q_out, s.scratch, q_norm=s.wq,
                                          k_norm=s.wk, q_stride=2 * D, rope_pos=rope_pos, k_out=s.k_out) == 0
        assert B.qwen35_tree_attention(s.cfg, s.kv, s.r, par, s.q_out, out, s.scratch, gate=s.qg[..., D:].contiguous()) == 0
        torch.matmul(out.flatten(1), head, out=lg)
        assert B.qwen35_sample(lg, u, token) == 0
        assert B.qwen35_cache_keep(s.cfg, s.kv, keep_rows, path, s.scratch) == 0

    before = cache_state(s)
    step()
    assert status(s) == 0
    results = [t.clone() for t in (s.q_out, out, token)] + list(cache_state(s).values())
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for n in s.t:
            s.t[n].copy_(before[n])
        for t in (s.q_out, out):
            t.fill_(NAN)
        g.replay()
        for a, b in zip([s.q_out, out, token] + list(s.t.values()), results):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert status(s) == 0
    # appending the accepted nodes' rows alone leaves the same rows
    held = cache_state(s)
    for n in s.t:
        s.t[n].copy_(before[n])
    pick = torch.tensor([0, 1, 4, 6, 7, 9, 12], device="cuda")
    r2 = B.DeviceRows(s.pos, start, 7, s.nb)
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, r2, None, s.k_new[pick], s.v_new[pick], None, s.scratch,
                                      k_norm=s.wk) == 0
    for b, p in enumerate(paths):
        at = torch.from_numpy(s.at(b, int(s.pos[b]) + np.arange(len(p)))).cuda()
        for n in s.t:
            assert torch.equal(s.t[n][at].view(torch.uint8), held[n][at].view(torch.uint8))


def test_calls_on_other_streams():
    s = setup("4b", BF16, [500, 90], None, page=16)
    want = run_window(s, 100, 4)
    side = torch.cuda.Stream()
    out = blank(s)
    q = s.q.cuda()
    torch.cuda.synchronize()
    assert B.qwen35_window_attention(s.cfg, s.kv, s.r, 100, 4, q, out, s.scratch, stream=side) == 0
    side.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_offsets_past_32_bits():
    """A contiguous cache of more than 2^32 bytes a tensor: the last sequence's rows lie behind them."""
    s = setup("4b", BF16, [40], None)
    cap, n = 1 << 18, 9  # 9 sequences of 2^18 rows of 2 KB
    k = torch.empty(n * cap, s.Hkv, s.D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    lo = cap * (n - 1) + cap - 40
    k[lo:lo + 40], v[lo:lo + 40] = s.t["k"][:40], s.t["v"][:40]
    kv = B.qwen35_kv_cache(k.data_ptr(), v.data_ptr(), cap, B.QWEN35_KV_BF16)
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pos[-1] = cap - 1
    q = s.q.cuda().expand(n, -1, -1).contiguous()
    out = torch.full_like(q, NAN)
    scratch = B.new_scratch(B.qwen35_rows_scratch_bytes(s.cfg, n))
    assert B.qwen35_window_attention(s.cfg, kv, B.DeviceRows(pos), 40, 0, q, out, scratch) == 0
    ref, tol = expect(s, lambda b, i, p: list(range(40)))[0]
    assert (np.abs(f64(out[-1]) - ref) <= 2.0 ** -8 * np.abs(ref) + tol).all()
    assert torch.isnan(out[:-1].float()).all()


class Banded:
    """A copy of a tensor between two bands of a pattern."""

    def __init__(self, t, band=1 << 16):
        n = t.numel() * t.element_size()
        self.raw = torch.full((n + 2 * band,), 0x5A, dtype=torch.uint8, device="cuda")
        self.t = self.raw[band:band + n].view(t.dtype).view(t.shape)
        self.t.copy_(t)
        self.band = band

    def whole(self):
        return bool((self.raw[:self.band] == 0x5A).all() and (self.raw[-self.band:] == 0x5A).all())


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("rows", [[2, 2, 2], [40, 50, 30]])
@pytest.mark.parametrize("start", [[0, 6, 2, 8], [4, 0, 5, 6], [-5, 1 << 30, -(1 << 30), 1 << 30], [3, 3, 3, 3],
                                   [-(1 << 31), (1 << 31) - 1, 0, 2], [0, 200, 120, 2]])
def test_row_starts_that_run_backwards_touch_nothing_outside(fmt, rows, start):
    s = rope_setup("tiny_alt", fmt, [80, 90, 70], rows, 32)
    bands = {n: Banded(t) for n, t in s.t.items()}
    s.kv.k, s.kv.v = bands["k"].t.data_ptr(), bands["v"].t.data_ptr()
    if fmt == TURBO8:
        s.kv.k_scales, s.kv.v_scales = bands["ks"].t.data_ptr(), bands["vs"].t.data_ptr()
    for n in ("q_out", "k_out", "scratch", "pos"):
        bands[n] = Banded(getattr(s, n))
    out = bands["out"] = Banded(blank(s))
    starts = bands["start"] = Banded(torch.tensor(start, dtype=torch.int64).to(torch.int32).cuda())
    parent = bands["parent"] = Banded(torch.arange(-1, s.n_rows - 1, dtype=torch.int32, device="cuda"))
    path = bands["path"] = Banded(torch.arange(s.n_rows, dtype=torch.int32, device="cuda"))
    r = B.DeviceRows(bands["pos"].t, starts.t, s.n_rows, s.nb)
    scratch, q = bands["scratch"].t, s.q.cuda()
    assert B.qwen35_cache_append_rope(s.cfg, s.kv, r, s.qg, s.k_new, s.v_new, bands["q_out"].t, scratch, q_norm=s.wq,
                                      k_norm=s.wk, q_stride=2 * s.D, k_out=bands["k_out"].t) == 0
    assert B.qwen35_tree_attention(s.cfg, s.kv, r, parent.t, q, out.t, scratch) == 0
    assert B.qwen35_window_attention(s.cfg, s.kv, r, 20, 4, q, out.t, scratch) == 0
    assert B.qwen35_cache_keep(s.cfg, s.kv, r, path.t, scratch) == 0
    torch.cuda.synchronize()
    assert B.qwen35_read_device_status(scratch) in (0, B.QWEN35_ERR_DEVICE_RANGE)
    for n, x in bands.items():
        assert x.whole(), n


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_arrays_at_16_bytes(fmt):
    """Every array moved to 16 bytes behind a larger boundary gives the bits that it gives at one."""
    s = rope_setup("4b", fmt, [300, 40], [9, 5], 64)

    def moved(t):
        n = t.numel() * t.element_size()
        x = torch.empty(n + 512, dtype=torch.uint8, device="cuda")
        x = x[16 + -x.data_ptr() % 256:][:n].view(t.dtype).view(t.shape)
        return x.copy_(t)

    gate = bf16(s.rng.standard_normal((s.n_rows, s.H, s.D))).cuda()
    parent = torch.tensor([-1, 0, 0, 1, 1, 2, 4, 6, 7] + [-1, 0, 1, 0, 3], dtype=torch.int32, device="cuda")

    def run(f):
        for n in s.t:
            s.t[n] = f(s.t[n])
        s.kv.k, s.kv.v = s.t["k"].data_ptr(), s.t["v"].data_ptr()
        if fmt == TURBO8:
            s.kv.k_scales, s.kv.v_scales = s.t["ks"].data_ptr(), s.t["vs"].data_ptr()
        q_out, k_out, a, b, scratch = (f(t) for t in (blank(s), torch.full_like(s.k_new, NAN), blank(s), blank(s), s.scratch))
        assert B.qwen35_cache_append_rope(s.cfg, s.kv, s.r, f(s.qg), f(s.k_new), f(s.v_new), q_out, scratch, q_norm=f(s.wq),
                                          k_norm=f(s.wk), q_stride=2 * s.D, k_out=k_out) == 0
        assert B.qwen35_tree_attention(s.cfg, s.kv, s.r, parent, q_out, a, scratch, gate=f(gate)) == 0
        assert B.qwen35_window_attention(s.cfg, s.kv, s.r, 70, 3, q_out, b, scratch, gate=f(gate)) == 0
        torch.cuda.synchronize()
        assert B.qwen35_read_device_status(scratch) == 0
        return [t.clone().view(torch.uint8) for t in (q_out, k_out, a, b, *s.t.values())]

    for x, y in zip(run(lambda t: t), run(moved)):
        assert torch.equal(x, y)


def counters(s):
    """The scratch before its work space: the status word and the counters."""
    work = (s.n_rows * s.H + 160 * 128) * (s.D * 4 + 16) + s.n_rows * s.Hkv * 4
    return s.scratch[:s.scratch.numel() - work]


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_counters_are_left_as_they_were(fmt):
    """Parts joined inside the launch and by a second one leave the counters as zeros, and the cache operators'
    append works on the same scratch in between."""
    s = setup("4b", fmt, [5000, 70, 900], None)
    want = {w: run_window(s, w, 4) for w in (50, 3000)}
    k, v = (bf16(s.rng.standard_normal((s.n_rows, s.Hkv, s.D))).cuda() for _ in range(2))
    for _ in range(3):
        for w in want:
            assert torch.equal(run_window(s, w, 4).view(torch.int16), want[w].view(torch.int16))
        assert not counters(s).any()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, k, v, s.scratch) == 0
    assert status(s) == 0 and not counters(s).any()


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_two_graphs_side_by_side(fmt):
    """Two captured graphs, each with its own scratch and output, replayed on two streams at once, many times."""
    s = setup("4b", fmt, [3000, 257, 64, 1900], None, page=64)
    trees = setup("4b", fmt, [2000, 300], [20, 7], page=16)
    parent = torch.tensor([-1] + list(range(19)) + [-1, 0, 0, 1, 2, 2, 5], dtype=torch.int32, device="cuda")
    q, tq = s.q.cuda(), trees.q.cuda()
    out, t_out = blank(s), blank(trees)

    def window():
        assert B.qwen35_window_attention(s.cfg, s.kv, s.r, 700, 4, q, out, s.scratch) == 0

    def tree():
        assert B.qwen35_tree_attention(trees.cfg, trees.kv, trees.r, parent, tq, t_out, trees.scratch) == 0

    window(), tree()
    torch.cuda.synchronize()
    want = [out.clone(), t_out.clone()]
    graphs = []
    for f in (window, tree):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    out.fill_(NAN), t_out.fill_(NAN)
    torch.cuda.synchronize()
    for g in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip((out, t_out), want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert status(s) == 0 and status(trees) == 0


@pytest.mark.parametrize("vocab", [300, 4097, 248320])
def test_a_row_of_many_is_the_row_alone(vocab):
    """Few rows are taken by more CTAs each than many: the same tokens and shares, to the bit."""
    x = logits(40, vocab, seed=5)
    u = np.linspace(0, 0.999, 40)
    t, k, p, m = np.full(40, 0.9), np.full(40, 50), np.full(40, 0.95), np.full(40, 0.01)
    many = run_sample(x, u, t, k, p, m)
    for r in (0, 7, 39):
        one = run_sample(x[r:r + 1].clone(), u[r:r + 1], t[:1], k[:1], p[:1], m[:1])
        assert one[0][0] == many[0][r] and one[1][0] == many[1][r]
    eight = run_sample(x[:8].clone(), u[:8], t[:8], k[:8], p[:8], m[:8])
    assert (eight[0] == many[0][:8]).all() and (eight[1] == many[1][:8]).all()


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "4b", "twelve"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("rows", [None, [20]])
def test_more_parts_than_a_column_has_lanes(heads, fmt, rows):
    """A long item lies in many CTAs, whose parts a column's 8 to 32 lanes take in rounds: inside the launch (one
    row) and by a second one, with a gate."""
    s = setup(heads, fmt, [7000], rows, page=16)
    gate = bf16(s.rng.standard_normal((s.n_rows, s.H, s.D))).cuda()
    check(s, run_window(s, 6900, 4, gate=gate), expect(s, lambda b, i, p: visible_window(p, 6900, 4), gate))
    assert status(s) == 0


@pytest.mark.parametrize("vocab", [5, 777, 4097, 248320])
def test_tokens_drawn_from_one_row(vocab):
    """Logits of row stride 0, of one row, in a column of a wider tensor: as their contiguous copies."""
    rng = np.random.default_rng(vocab)
    u = rng.random(12)
    x = logits(1, vocab, 7)[0].expand(12, -1)
    assert x.stride(0) == 0
    check_sample(x, u, k=rng.integers(0, 40, 12))
    a, b = run_sample(x, u), run_sample(x.contiguous(), u)
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()
    one = torch.zeros(1, dtype=torch.bfloat16, device="cuda").expand(3, 1)
    assert run_sample(one, [0.0, 0.5, 1.0])[0].tolist() == [0, 0, 0]


# ---------------------------------------------------------------- what is no number


def under(s, kind, first=4):
    """(call, see): trees of the rows (stars), or windows of 10^6 or 64 tokens."""
    if kind == "tree":
        parents = [[-1] + [0] * (r - 1) for r in s.rows]
        return lambda: run_tree(s, parents), lambda b, i, p: visible_tree(parents[b], p - i, i)
    window = 10 ** 6 if kind == "all" else 64
    return lambda: run_window(s, window, first), lambda b, i, p: visible_window(p, window, first)


@pytest.mark.parametrize("heads", ["4b", "tiny_alt", "wide"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("kind", ["tree", "all", "near"])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_a_query_without_a_number_gives_none(heads, fmt, kind, bad):
    """One element of a head's query is no number: its scores are NaN (or, of an infinity, of both signs), in every part
    of its tokens, and so are its outputs; the others' are as they were."""
    s = setup(heads, fmt, [4000 + 3, 1, 70 + 2], [3, 1, 2], page=16)
    call, see = under(s, kind)
    want = expect(s, see)
    s.q[1, 1, 5] = s.q[3, 0, 0] = bad
    got = f64(call())
    if not np.isnan(bad) and fmt == BF16:  # an infinite score of one sign among tokens: NaN too, but for a row of one token
        bad_rows = [(1, 1)]                # or of scores that are all -inf, which weigh nothing
    else:
        bad_rows = [(1, 1), (3, 0)]
    for r, h in bad_rows:
        assert np.isnan(got[r, h]).all(), (r, h)
    for r, (ref, tol) in want.items():
        for h in range(s.H):
            if (r, h) not in [(1, 1), (3, 0)]:
                assert (np.abs(got[r, h] - ref[h]) <= 2.0 ** -8 * np.abs(ref[h]) + tol).all(), (r, h)


@pytest.mark.parametrize("heads", ["4b", "tiny"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("kind", ["tree", "all", "near"])
@pytest.mark.parametrize("token", [0, 3999, 4000, 4001])
def test_a_key_without_a_number_spoils_the_rows_that_see_it(heads, fmt, kind, token):
    """Every element of one key is NaN. In a part of its own or not, its rows are NaN."""
    s = setup(heads, fmt, [4000 + 3, 1], [3, 1], page=16)
    call, see = under(s, kind, first=0)
    want = expect(s, see)
    at = s.at(0, token)
    if fmt == BF16:
        s.t["k"][at, 0] = NAN
    else:
        s.t["ks"][at, :s.D // 16] = bf16([NAN]).view(torch.int16).item()
    got, g = f64(call()), s.H // s.Hkv
    for r, (ref, tol) in want.items():
        b, i, p = (0, r, 4000 + r) if r < 3 else (1, 0, 0)
        spoiled = b == 0 and token in see(b, i, p)
        if spoiled:
            assert np.isnan(got[r, :g]).all()
        keep = slice(g if spoiled else 0, None)
        assert (np.abs(got[r, keep] - ref[keep]) <= 2.0 ** -8 * np.abs(ref[keep]) + tol).all()


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_a_row_of_one_token_whose_key_is_no_number(fmt):
    s = setup("4b", fmt, [300, 64, 1], None, page=16)
    for b, p in enumerate((299, 63, 0)):
        if fmt == BF16:
            s.t["k"][s.at(b, p)] = NAN
        else:
            s.t["ks"][s.at(b, p)] = bf16([NAN]).view(torch.int16).item()
    assert torch.isnan(run_window(s, 1, 0)).all()


@pytest.mark.parametrize("heads,quiet", [("4b", False), ("tiny", False), ("tiny_alt", False), ("tiny", True)])
@pytest.mark.parametrize("kind", ["tree", "all", "near"])
@pytest.mark.parametrize("tokens", [{0: 1}, {700: -1}, {3998: 1}, {4001: 1}, {5: 1, 70: 1, 3999: 1}, {64: 1, 2000: -1},
                                    {2000: 1, 3996: 1, 4000: -1}, {3000: "nan"}, {10: 1, 4000: "nan"}], ids=str)
def test_infinite_values_are_the_outputs_of_the_rows_that_see_them(heads, kind, tokens, quiet):
    """bf16, wherever the token lies: one infinity, or several of one sign, give it, both signs or a NaN give NaN; the
    other elements are as without. quiet: the tokens' scores lie 400 below the others."""
    s = setup(heads, BF16, [4000 + 3, 50], [3, 1], page=16)
    call, see = under(s, kind)
    dim = s.D // 2 + 5
    if quiet:
        s.q = bf16(np.full(s.q.shape, 2.0))
        for t in tokens:
            s.t["k"][s.at(0, t)] = -400.0 / 2 / np.sqrt(s.D)
            s.stands["k"][s.at(0, t)] = f64(bf16(-400.0 / 2 / np.sqrt(s.D)))
    want = expect(s, see)
    for t, sign in tokens.items():
        s.t["v"][s.at(0, t), 0, dim] = NAN if sign == "nan" else sign * float("inf")
    got, g = f64(call()), s.H // s.Hkv
    for r, (ref, tol) in want.items():
        b, i, p = (0, r, 4000 + r) if r < 3 else (1, 0, 49)
        seen = {sign for t, sign in tokens.items() if b == 0 and t in see(b, i, p)}
        expected = None if not seen else np.nan if len(seen) > 1 or "nan" in seen else seen.pop() * np.inf
        for h in range(s.H):
            ok = np.abs(got[r, h] - ref[h]) <= 2.0 ** -8 * np.abs(ref[h]) + tol
            if h < g and expected is not None:
                assert np.array_equal(got[r, h, dim], expected, equal_nan=True), (r, h, got[r, h, dim], expected)
                ok[dim] = True
            assert ok.all(), (r, h)


@pytest.mark.parametrize("kind", ["tree", "all"])
@pytest.mark.parametrize("sign", [1, -1])
def test_every_value_infinite(kind, sign):
    """Whole caches of one infinity, then with one of the other sign."""
    s = setup("4b", BF16, [1500 + 40], [40], page=16)
    call, _ = under(s, kind)
    s.t["v"][:] = sign * float("inf")
    assert (call() == sign * float("inf")).all()
    s.t["v"][s.at(0, 777)] = -sign * float("inf")
    assert torch.isnan(call()).all()
    assert status(s) == 0


# ---------------------------------------------------------------- Turbo8: large scores
#
# Tolerances, derived before the first run. The rotated q is held to 2^-22 of a value or 2^-25 of its largest, a key's code times
# its scale exactly (down to 2^-25 of 2^E, the power of two of the token's largest scale), as a product with the scale's upper seven
# bits and one with its last, whose product with q's lower part (2^-7 2^-11 of a term) is left out. The small terms are added first, so
# a score is a sum of D / 16 + 4 fp32 steps of 2^-23 each of at most sum |q_d k_d|, and 2 D / 16 more of 2^-6 of that: for D = 256
# 20 2^-23 + 2^-24 + 2^-18 + 2^-22 + 2^-21 < 2^-17, so 2^-17 sum |q_d k_d| / sqrt D = d in all.
# A weight and a value lose 2^-11 each, so a row is off by 2^-8 |y| (its rounding) and (2 d + 2^-10) max |v|; roundings are of either
# sign, so the whole output's 2-norm is held to 2^-8 + 2^-9 of the reference's, as everywhere in this file.


def along_one(s, scores, noise=0.05):
    """Keys and queries along one direction a kv-head, with noise; scores of about `scores` (natural units)."""
    rng = np.random.default_rng(23)
    u = rng.standard_normal((s.Hkv, s.D))
    a = scores / np.sqrt(s.D)  # |u|^2 is about D
    q = np.repeat(u, s.H // s.Hkv, 0)
    s.q = bf16(a * (q + noise * rng.standard_normal((s.n_rows, s.H, s.D))))
    for b, m in enumerate(s.lens):
        put(s, "k", b, u + noise * rng.standard_normal((m, s.Hkv, s.D)))


def check_scores(s, out, see):
    got, refs = f64(out), {}
    for row, b, p in s.each_row():
        at, i = s.at(b, np.asarray(see(b, row - s.start[b], p))), row - s.start[b]
        ref, tol = np.zeros((s.H, s.D)), np.zeros((s.H, 1))
        for h in range(s.H):
            k, v = (s.stands[n][at, h // (s.H // s.Hkv)] for n in "kv")
            q = f64(s.q[row, h])
            x = k @ q / np.sqrt(s.D)
            w = np.exp(x - x.max())
            ref[h] = w / w.sum() @ v
            d = 2.0 ** -17 * (np.abs(O.wht(k)) @ np.abs(O.wht(q))).max() / np.sqrt(s.D)
            tol[h] = (2 * d + 2.0 ** -10) * np.linalg.norm(v, axis=-1).max()
        assert (np.abs(got[row] - ref) <= 2.0 ** -8 * np.abs(ref) + tol).all(), (row, np.abs(got[row] - ref).max(), tol.max())
        refs[row] = ref
    a, b = (np.stack([x[r] for r in sorted(refs)]) for x in (got, refs))
    err = np.linalg.norm(a - b) / np.linalg.norm(b)
    assert err <= 2.0 ** -8 + 2.0 ** -9, err
    return err


@pytest.mark.parametrize("heads", ["4b", "tiny_alt", "tiny", "wide", "twelve"])
@pytest.mark.parametrize("scores", [4.0, 64.0, 1024.0, 4096.0])
@pytest.mark.parametrize("kind", ["tree", "all", "near"])
def test_turbo8_scores_of_any_size(heads, scores, kind):
    s = setup(heads, TURBO8, [500 + 20, 65 + 1, 1300 + 3], [20, 1, 3], page=16)
    along_one(s, scores)
    call, see = under(s, kind)
    check_scores(s, call(), see)
    assert status(s) == 0


@pytest.mark.parametrize("heads", ["4b", "tiny", "tiny_alt"])
@pytest.mark.parametrize("token", [0, 63, 64, 255, 511, 518, 519])
@pytest.mark.parametrize("kind", ["tree", "all"])
def test_turbo8_one_key_far_ahead_of_the_others(heads, token, kind):
    """The output is its value: other weights are below e^-60."""
    s = setup(heads, TURBO8, [519 + 2], [2], page=16)
    u = np.sign(s.rng.standard_normal((s.Hkv, s.D)))
    k = 0.1 * s.rng.standard_normal((521, s.Hkv, s.D))
    k[token] = 8 * u
    put(s, "k", 0, k)
    s.q = bf16(np.broadcast_to(np.repeat(u, s.H // s.Hkv, 0), (s.n_rows, s.H, s.D))).contiguous()
    call, see = under(s, kind)
    got = f64(call())
    for row in range(2):
        if token in see(0, row, 519 + row):
            v = np.repeat(s.stands["v"][s.at(0, token)], s.H // s.Hkv, 0)
            assert (np.abs(got[row] - v) <= 2.0 ** -8 * np.abs(v) + 2.0 ** -10 * np.linalg.norm(v, axis=-1).max()).all()


@pytest.mark.parametrize("heads", ["4b", "tiny_alt", "twelve"])
@pytest.mark.parametrize("scores", [4.0, 64.0, 1024.0, 4096.0])
def test_turbo8_chains_are_decode_attention(heads, scores):
    """Both are within their own bounds of float64 (2^-8 + 2^-9 of the norm each), so within twice that of each other; and the
    tree's error is not above the decode attention's by more than the roundings of the weights and values, 2^-10."""
    s = setup(heads, TURBO8, [900, 77], [6, 2], page=16)
    along_one(s, scores)
    parents = [[-1, 0, 1, 2, 3, 4], [-1, 0]]
    see = lambda b, i, p: list(range(p + 1))  # noqa: E731
    out, other = run_tree(s, parents), blank(s)
    scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(s.cfg, s.cap, 0, s.n_rows))
    assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, s.q.cuda(), other, scratch) == 0
    a, b = check_scores(s, out, see), check_scores(s, other, see)
    assert a <= b + 2.0 ** -10
    x, y = f64(out), f64(other)
    assert np.linalg.norm(x - y) <= 2 * (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(y)


@pytest.mark.parametrize("n_seqs", [1000, 1700, 1800, 2048])
def test_turbo8_rows_of_many_sequences(n_seqs):
    """The most rows that a call may have, of sequences of their own: as a call of few of them."""
    s = setup("twelve", TURBO8, [1 + 5 * i % 90 for i in range(n_seqs)], None, page=16)
    out = run_window(s, 40, 2)
    some = list(range(0, n_seqs, 97)) + [n_seqs - 1]
    few = B.DeviceRows(s.pos[some].contiguous(), None, len(some), s.nb)
    kv = B.qwen35_kv_cache(s.kv.k, s.kv.v, s.cap, s.kv.dtype, s.kv.k_scales, s.kv.v_scales, None, 16, 0)
    table = s.table[some].contiguous()
    kv.block_table = table.data_ptr()
    other = torch.full((len(some), s.H, s.D), NAN, dtype=torch.bfloat16, device="cuda")
    assert B.qwen35_window_attention(s.cfg, kv, few, 40, 2, s.q[some].cuda(), other, s.scratch) == 0
    assert status(s) == 0
    a, b = f64(out)[some], f64(other)
    # the parts' cuts differ: two outputs of the same values, rounded once each
    assert (np.abs(a - b) <= 2 * 2.0 ** -8 * np.abs(b) + 2.0 ** -9 * np.abs(b).max()).all()
    check(s, torch.where(torch.isin(torch.arange(n_seqs, device="cuda"), torch.tensor(some, device="cuda"))[:, None, None], out,
                         blank(s)), expect(s, lambda b, i, p: visible_window(p, 40, 2) if b in some else None))


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_the_most_rows_in_short_runs(fmt):
    """2048 rows of 300 sequences, among them empty ones, with rows of none before and behind."""
    rows = [i % 14 for i in range(300)]
    s = setup("twelve", fmt, [r + 7 * i % 100 + 1 for i, r in enumerate(rows)], rows, page=16, lead=3, tail=2048 - 3 - sum(rows))
    assert s.n_rows == 2048
    out = run_window(s, 50, 3)
    check(s, out, expect(s, lambda b, i, p: visible_window(p, 50, 3)))
    assert status(s) == 0


@pytest.mark.parametrize("vocab", [3, 1000, 20000])
def test_probabilities_are_rounded_once(vocab):
    """A weight is good to 2^-40 of itself and the sum of what is left to 2^-45 a token, at least 1: with the one rounding to
    fp32 2^-24 + 2^-40 + vocab 2^-45 of the probability; 2^-24 + 2^-30 for all vocabularies here."""
    n = 400
    rng = np.random.default_rng(vocab)
    x = bf16(2 * rng.standard_normal((n, vocab))).cuda()
    u, t, k = rng.random(n), (0.5 + rng.random(n)).astype(np.float32), rng.integers(0, vocab, n)
    token, prob = run_sample(x, u, t=t, k=k)
    host = f64(x)
    for r in range(n):
        want, q = plain_sample(host[r], float(np.float32(u[r])), float(t[r]), int(k[r]))
        assert token[r] == want
        assert abs(float(prob[r]) - q) <= (2.0 ** -24 + 2.0 ** -30) * q, (r, prob[r], q)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("n", [151, 152, 153, 455, 456, 457])
def test_single_rows_on_either_side_of_the_join(fmt, n):
    """Few items an SM are joined inside the launch, many by a second one: the outputs of the same rows."""
    s = setup("tiny", fmt, [1 + 37 * i % 400 for i in range(n)], None, page=16)
    out = run_window(s, 150, 2)
    check(s, out, expect(s, lambda b, i, p: visible_window(p, 150, 2)))
    assert status(s) == 0
    for _ in range(2):
        assert torch.equal(run_window(s, 150, 2).view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("value", [float("inf"), NAN])
@pytest.mark.parametrize("last", [False, True])
def test_long_stretches_without_a_number(value, last):
    """700 000 tokens a sequence, one kv-head, ten rows: stretches of 46 000 tokens, all of whose values are no number, or
    whose last one is. No wait runs out, and the outputs are those of the formula."""
    H, Hkv, D = HEADS["tiny"]
    cfg = B.make_config(synth.config("tiny") | dict(num_heads=H, num_kv_heads=Hkv, head_dim=D))
    n, cap = 10, 700_000
    k = torch.zeros(n * cap, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k) if last else torch.full_like(k, value)
    pos = torch.full((n,), cap - 1, dtype=torch.int32, device="cuda")
    if last:
        v.view(n, cap, Hkv, D)[:, cap - 100] = value  # in a tile that is seen whole
    kv = B.qwen35_kv_cache(k.data_ptr(), v.data_ptr(), cap, B.QWEN35_KV_BF16, None, None, None, 0, 0)
    scratch = B.new_scratch(B.qwen35_rows_scratch_bytes(cfg, n))
    q, out = torch.ones(n, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
    assert B.qwen35_window_attention(cfg, kv, B.DeviceRows(pos, None, n, 0), cap, 0, q, out, scratch) == 0
    torch.cuda.synchronize()
    assert B.qwen35_read_device_status(scratch) == 0
    assert torch.isnan(out).all() if np.isnan(value) else (out == value).all()


@pytest.mark.parametrize("heads", ["twelve", "4b", "tiny_alt"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_equal_calls_give_equal_bits(heads, fmt):
    """Blocks of few and of many columns one after another on a CTA, many times: a warp that has columns of one block and none of
    the block before waits for the same products as the others."""
    rows = [i % 14 * 3 % 40 for i in range(100)]
    s = setup(heads, fmt, [r + 7 * i % 100 + 1 for i, r in enumerate(rows)], rows, page=16, lead=3)
    assert s.n_rows <= 2048
    first = run_window(s, 50, 3)
    check(s, first, expect(s, lambda b, i, p: visible_window(p, 50, 3)))
    differ = sum(not torch.equal(run_window(s, 50, 3).view(torch.int16), first.view(torch.int16)) for _ in range(200))
    assert differ == 0 and status(s) == 0


@pytest.mark.parametrize("heads", ["tiny", "4b"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("kind", ["tree", "all"])
def test_infinite_values_of_parts_without_weight(heads, fmt, kind):
    """The first half of the tokens scores 400 below the rest, so parts of it weigh nothing in 32 bits; one of its values is
    infinite all the same: bf16 gives the infinity, Turbo8 no number in its head."""
    s = setup(heads, fmt, [4000 + 3], [3], page=16)
    call, see = under(s, kind)
    s.q = bf16(np.full(s.q.shape, 2.0))
    k = s.rng.standard_normal((4003, s.Hkv, s.D))
    k[:2000] = -400.0 / 2 / np.sqrt(s.D)
    put(s, "k", 0, k)
    want = expect(s, see)
    at, dim = int(s.at(0, 5)), s.D // 2 + 5
    if fmt == BF16:
        s.t["v"][at, 0, dim] = -float("inf")
    else:
        s.t["vs"][at, dim // 16] = bf16([float("inf")]).view(torch.int16).item()
    got, g = f64(call()), s.H // s.Hkv
    for r, (ref, tol) in want.items():
        ok = np.abs(got[r] - ref) <= 2.0 ** -8 * np.abs(ref) + tol
        if fmt == BF16:
            assert (got[r, :g, dim] == -np.inf).all()
            ok[:g, dim] = True
        else:
            assert not np.isfinite(got[r, :g]).any()
            ok[:g] = True
        assert ok.all()
    assert status(s) == 0
