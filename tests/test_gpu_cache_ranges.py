"""The cache operators on values far apart in size, against plain float64 implementations.

Tolerance of the attention over a Turbo8 cache, derived before the first run: the
output's bf16 rounding, 2^-8 of its norm (the rotation back keeps norms); a weight is off
by at most 2^-14 (scores of up to 128 octaves in fp32: D / 16 + 4 roundings of 2^-24 each,
in octaves, times ln 2, in the weight and in the sum), is rounded to f16 before and after
the product with its V scale (2^-11 each), and a group of 16 values far below its own
token's largest loses 2^-25 of that one. All of it is relative to what a token adds, so to
|sum_t w_t |v_t|| (v_t rotated, as the cache holds it), and not to the largest value a
row sees: 2^-10 + 2^-12 of it in all.
"""

import numpy as np
import pytest
import torch

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth
from oracle import qwen35_oracle as O

from harness import init
from test_gpu_cache_ops import BF16, TURBO8, Setup, bf16, check_choice, choose, f64

pytestmark = pytest.mark.gpu


def put(s, name, b, x):
    """Rows x [tokens][Hkv][D] of sequence b into the cache, and what they stand for."""
    x = f64(bf16(x))
    at = torch.from_numpy(np.asarray(s.at(b, np.arange(len(x)))))
    if s.fmt == BF16:
        s.t[name][at.cuda()] = bf16(x).cuda()
        s.stands[name][at] = x
        return
    c, sc = O.turbo8_quantize(O.bf16_round(O.wht(x)))
    s.t[name][at.cuda()] = torch.from_numpy(c).cuda()
    groups = s.Hkv * s.D // 16
    s.t[name + "s"][at.cuda(), :groups] = torch.from_numpy(O.bf16_bits(sc).reshape(-1, groups).view(np.int16)).cuda()
    s.stands[name][at] = O.wht(O.turbo8_dequantize(c, sc))


def along(s, scores):
    """q of every row along one direction a head group, and keys whose scores are `scores` octaves (before
    the cache's rounding), [tokens]."""
    rng = np.random.default_rng(17)
    u = rng.choice([-1.0, 1.0], size=(s.Hkv, s.D))
    q = np.repeat(u, s.H // s.Hkv, 0)  # q.k / sqrt(D) = sqrt(D) a for k = a u
    s.q = bf16(np.broadcast_to(q, (s.n_rows, s.H, s.D))).contiguous()
    return np.asarray(scores)[:, None, None] * np.log(2) / np.sqrt(s.D) * u


def weighted(s, row, b, p):
    """float64 attention of one row and sum_t w_t |v_t| of its rotated values, [H][D] each."""
    g, rows = s.H // s.Hkv, s.at(b, np.arange(p + 1))
    out, size = np.zeros((s.H, s.D)), np.zeros((s.H, s.D))
    for h in range(s.H):
        k, v = s.stands["k"][rows, h // g], s.stands["v"][rows, h // g]
        x = k @ f64(s.q[row, h]) / np.sqrt(s.D)
        w = np.exp(x - x.max())
        w /= w.sum()
        out[h], size[h] = w @ v, w @ np.abs(O.wht(v) if s.fmt == TURBO8 else v)
    return out, size


def check_weighted(s):
    got = f64(s.attend())
    assert s.status() == 0
    for row, b, p in s.each_row():
        ref, size = weighted(s, row, b, p)
        err = np.linalg.norm(got[row] - ref, axis=1)
        bound = 2.0 ** -8 * np.linalg.norm(ref, axis=1) + (2.0 ** -10 + 2.0 ** -12) * np.linalg.norm(size, axis=1)
        assert np.all(err <= bound), (row, b, p, float((err / bound).max()))


# octaves: of the small values, how far the large ones lie above them, how far their scores lie below
SIZES = [(0, 0, 0), (-10, 15, 40), (0, 20, 60), (0, 24, 60), (-10, 30, 60), (0, 40, 30), (0, 100, 0), (-60, 100, 120),
         (80, 20, 40), (112, 4, 3), (-112, 4, 3), (-100, 180, 3)]


@pytest.mark.parametrize("kw", [dict(heads="tiny", lens=[40, 17]), dict(heads="4b", lens=[100], page=16),
                                dict(heads="wide", lens=[70]), dict(heads="twelve", lens=[50, 33], page=8),
                                dict(heads="tiny_alt", lens=[37, 60], rows=[5, 3]),
                                dict(heads="odd", lens=[18, 40], rows=[3, 2], page=32),
                                dict(heads="tiny", lens=[3000])], ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_turbo8_attention_counts_a_token_by_what_it_adds(kw, sizes):
    """Tokens of large values and low scores among ones of small values and high scores: in most tiles, in the
    call's own rows and in other tiles than the small ones."""
    small, ratio, gap = sizes
    s = Setup(fmt=TURBO8, **kw)
    rng = np.random.default_rng(5)
    for b, m in enumerate(s.lens):
        large = rng.random(m) < 0.2
        large[m // 2:m // 2 + 20] = m > 100
        large[-1] = not large[-2]
        put(s, "k", b, along(s, np.where(large, -gap / 2, gap / 2) + rng.uniform(-1, 1, m)))
        put(s, "v", b, rng.standard_normal((m, s.Hkv, s.D)) * np.exp2(small + ratio * large)[:, None, None])
    check_weighted(s)


def test_turbo8_attention_of_a_small_value_beside_a_large_one_of_no_weight():
    """Two tokens: scales 30 octaves apart, the large one's score 60 octaves below."""
    s = Setup("tiny", TURBO8, [2])
    put(s, "k", 0, along(s, [-30, 30]))
    put(s, "v", 0, np.stack([np.full((1, s.D), 2.0 ** 20), np.full((1, s.D), 2.0 ** -10)]))
    check_weighted(s)
    assert np.all(np.abs(f64(s.attend())[0] / 2.0 ** -10 - 1) < 2.0 ** -6)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("q_size,k_size", [(6, 8), (10, 12), (20, 60), (100, -110), (60, -60)])
@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "wide"])
def test_attention_of_very_large_and_very_small_keys(heads, q_size, k_size, fmt):
    """Scores of 2^14 octaves and more, where the largest takes all the weight and an octave more or less of a token's
    V is below the score's last bit; and ones near 0, where all tokens weigh the same."""
    s = Setup(heads, fmt, [60, 17], page=16)
    for b, m in enumerate(s.lens):
        put(s, "k", b, along(s, s.rng.permutation(m) + 1.0) / m * np.exp2(k_size))
        put(s, "v", b, s.rng.standard_normal((m, s.Hkv, s.D)))
    s.q = bf16(f64(s.q) * np.exp2(q_size))
    check_weighted(s)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("q_size,k_size", [(0, 114), (-20, 117), (3, 110), (-100, 110)])
@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "wide"])
def test_attention_of_keys_near_the_largest(heads, q_size, k_size, fmt):
    """Scores that 32 bits hold, though not 2^15 times as large: the largest takes all the weight."""
    test_attention_of_very_large_and_very_small_keys(heads, q_size, k_size, fmt)


# ---------------------------------------------------------------- rows in and out


@pytest.mark.parametrize("cfg_name", ["tiny", "tiny_alt", "4b"])
def test_turbo8_append_of_nan_rows_equals_the_prefill_of_a_layer(cfg_name):
    """Tokens whose input holds a NaN, through the prefill of a layer and through the operator: codes and scales bit
    for bit, all of them 0 for the rows that are NaN."""
    init()
    cfg = synth.config(cfg_name)
    c = B.make_config(cfg)
    T, cap = 19, 32
    Hkv, D = cfg["num_kv_heads"], cfg["head_dim"]
    layer = B.DeviceFaLayer(synth.fa_layer(1, 1, cfg))
    scratch = B.new_scratch(B.qwen35_prefill_scratch_bytes(c, T))
    rows = np.stack([synth.x_in(1, t, cfg) for t in range(T)])
    rows[[3, 11, 12], 5] = 0x7FC0
    x = B.to_device(rows)
    y = torch.empty_like(x)
    zero = np.zeros((cap, Hkv, D), dtype=np.uint16)
    flat = B.DeviceKv(zero, zero)
    t8, mine = (B.DeviceKvTurbo8(zero.astype(np.uint8), np.zeros((cap, Hkv, D // 16), np.uint16), zero.astype(np.uint8),
                                 np.zeros((cap, Hkv, D // 16), np.uint16), cfg) for _ in "ab")
    for kv in (flat, t8):
        assert B.qwen35_prefill_full_attention(c, layer.struct, scratch, kv.struct, x, y, 0, T) == 0
    r = B.DeviceRows(torch.zeros(1, dtype=torch.int32, device="cuda"),
                     torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
    s2 = B.new_scratch(B.qwen35_cache_scratch_bytes(c, cap, 0, T))
    k, v = (a.view(torch.bfloat16)[:T].contiguous() for a in (flat.k, flat.v))
    assert torch.isnan(v.float()).flatten(1).all(1).cpu().nonzero().flatten().tolist() == [3, 11, 12]
    assert B.qwen35_cache_append(c, mine.struct, r, None, k, v, s2) == 0
    torch.cuda.synchronize()
    for a, b in ((mine.k, t8.k), (mine.v, t8.v), (mine.ks, t8.ks), (mine.vs, t8.vs)):
        assert torch.equal(a[:T], b[:T])
    assert not mine.vs[[3, 11, 12]].any() and not mine.v[[3, 11, 12]].any() and mine.v[[2, 4, 10, 13]].any()


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "4b"])
def test_turbo8_append_of_rows_without_finite_values(heads):
    """Rotated, a row with a NaN is NaN throughout (zeros), one with an infinity infinite throughout (infinite scales,
    NaN codes), one with two of them infinite or NaN by element: by the definition whose maximum skips NaN."""
    s = Setup(heads, TURBO8, [40], rows=[40])
    rng = np.random.default_rng(3)
    x = rng.standard_normal((40, s.Hkv, s.D))
    x[3, :, 7], x[5, :, 0], x[6, :, s.D - 1] = np.nan, np.inf, -np.inf
    x[9, :, 2], x[9, :, 3] = np.inf, np.inf
    x[10, :, 1], x[10, :, s.D // 2 + 1] = np.inf, -np.inf
    x[11, :, 4], x[11, :, 20] = np.inf, np.nan
    x = f64(bf16(x))
    k = bf16(x).cuda()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, k, k, s.scratch) == 0
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        h = np.ones((1, 1))
        while len(h) < s.D:
            h = np.block([[h, h], [h, -h]])
        rot = np.stack([(r[:, None, :] * h).sum(-1) for r in x[[3, 5, 6, 9, 10, 11]]])
        amax = np.fmax.reduce(np.abs(rot.reshape(6, s.Hkv, -1, 16)), axis=-1, initial=0.0)
    assert set(amax[0].flat) == {0.0} and set(amax[1].flat) == {np.inf} and set(amax[5].flat) == {0.0}
    at = [int(s.at(0, p)) for p in (3, 5, 6, 9, 10, 11)]
    for name in "kv":
        sc = O.bf16_to_f64(s.t[name + "s"].cpu().numpy().view(np.uint16)[at][:, :s.Hkv * s.D // 16])
        np.testing.assert_array_equal(sc.reshape(amax.shape), amax)
        codes = s.t[name].cpu().numpy()[at].reshape(amax.shape + (16,))
        np.testing.assert_array_equal(codes & 0x7F, np.where(amax[..., None] > 0, 0x7F, np.zeros(16, np.uint8)))


# ---------------------------------------------------------------- selection


@pytest.mark.parametrize("n_select", [1, 3, 5, 6, 7, 40])
@pytest.mark.parametrize("entry", [0, 2, 5])
def test_selection_reports_a_block_outside_the_pool(n_select, entry):
    """The only fault of the call: one entry of the table, of a block that the row sees. Lists shorter than the blocks
    seen (6) and not."""
    s = Setup("tiny_alt", BF16, [20, 90, 30], page=16, block=16)
    s.set_bounds()
    out = torch.zeros(3, s.Hkv, n_select, dtype=torch.int32, device="cuda")
    q = s.q.cuda()
    assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, out, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == 0
    clean = out.clone()
    s.table[1, entry] = s.nb
    assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, out, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    assert torch.equal(out[[0, 2]], clean[[0, 2]])
    if n_select >= 6:
        assert torch.equal(out, clean)


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "4b"])
@pytest.mark.parametrize("e", [-152, -149, -140, -126, -100])
def test_selection_of_scores_at_the_lower_end_of_32_bits(heads, e):
    """Products of about 2^e: 32-bit sums lose them, or half a unit of 2^-149 of each."""
    s = Setup(heads, BF16, [1600], block=16)
    rng = np.random.default_rng(-e)
    s.q = bf16(np.exp2(-76) * rng.uniform(0.5, 1.0, size=s.q.shape) * np.where(rng.random(s.q.shape) < 0.7, 1, -1))
    b = rng.uniform(0.2, 0.8, size=(s.total // 16, s.Hkv, 2, s.D))
    b *= np.where(rng.random(b.shape) < 0.1, 10, 1) * (rng.random((len(b), 1, 1, 1)) < 0.8)
    b[::3, :, :, 1:] = 0  # blocks of one product
    b[:, :, 0] *= -1
    s.lo_hi.copy_(bf16(b * np.exp2(e + 76)).cuda())
    for n in (1, 7, 30, 66):
        check_choice(s, n, 0, 0)


def test_selection_where_many_small_products_weigh_more_than_one():
    """A score of 64 products of 0.45 units of 2^-149, which 32 bits lose one by one, and one of a product of 5."""
    s = Setup("tiny", BF16, [32], block=16)
    s.q = torch.zeros_like(s.q)
    s.q[0, 0] = 2.0 ** -75
    b = torch.zeros(2, 1, 2, s.D, dtype=torch.float64)
    b[1, 0, 1], b[0, 0, 1, 0] = 0.45 * 2.0 ** -74, 5 * 2.0 ** -74
    s.lo_hi[:2] = b.to(torch.bfloat16).cuda()
    check_choice(s, 1, 0, 0)
    s.lo_hi[:2] = b.flip(0).to(torch.bfloat16).cuda()
    check_choice(s, 1, 0, 0)


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "4b"])
@pytest.mark.parametrize("block", [16, 64, 512])
def test_bounds_of_a_dimension_that_has_only_nan(heads, block):
    """NaN for both bounds until a row brings a number, then that number's; a block with such a dimension has no
    score, so it comes last."""
    s = Setup(heads, BF16, [2 * block, 2 * block - 1], rows=[2 * block - 2, block + 5], block=block)
    rng = np.random.default_rng(8)
    x = rng.standard_normal((s.n_rows, s.Hkv, s.D))
    one = s.start[1]
    x[:block, :, 3] = np.nan  # sequence 0, tokens 2 .. block + 1
    x[one:, 0, 9] = np.nan    # sequence 1, tokens block - 6 .. 2 block - 2
    s.lo_hi.zero_()           # of the blocks' earlier tokens
    k = bf16(x).cuda()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k, k, s.scratch) == 0
    torch.cuda.synchronize()
    got, y = f64(s.lo_hi), f64(k)
    e = [int(s.at(b, j * block)) // block for b in (0, 1) for j in (0, 1)]

    def fold(rows, **kw):
        return np.stack([np.fmin.reduce(rows, 0, **kw), np.fmax.reduce(rows, 0, **kw)], 1)

    np.testing.assert_array_equal(got[e[0]], fold(y[:block - 2], initial=0.0))
    np.testing.assert_array_equal(got[e[1]], fold(y[block - 2:one]))  # two rows of NaN, then numbers
    np.testing.assert_array_equal(got[e[2]], fold(y[one:one + 6], initial=0.0))
    np.testing.assert_array_equal(got[e[3]], fold(y[one + 6:]))
    assert np.isnan(got[e[3], 0, :, 9]).all() and not np.isnan(got[e[:3]]).any()
    check_choice(s, 1, 0, 0)
    # one more row of sequence 1's last block brings numbers
    r = B.DeviceRows(torch.tensor([0, 2 * block - 1], dtype=torch.int32, device="cuda"))
    new = bf16(rng.standard_normal((2, s.Hkv, s.D))).cuda()
    assert B.qwen35_cache_append(s.cfg, s.kv, r, s.bounds, new, new, s.scratch) == 0
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(s.lo_hi)[e[3], 0, :, 9], np.repeat(f64(new)[1, 0, 9], 2))


# ---------------------------------------------------------------- malformed row starts


def _guarded(t, room=4096):
    """A copy of t between two filled bands of its allocation, and what says whether the bands are as they were."""
    n = t.numel() * t.element_size()
    band = (room + 255) // 256 * 256
    raw = torch.full((band + (n + 255) // 256 * 256 + band,), 0xA5, dtype=torch.uint8, device="cuda")
    inner = raw[band:band + n].view(t.dtype).view(t.shape)
    inner.copy_(t)
    return inner, lambda: bool((raw[:band] == 0xA5).all()) and bool((raw[band + n:] == 0xA5).all())


STARTS = [[0, 6, 2, 8], [-5, 1 << 30, -(1 << 30), 1 << 30], [8, 0, 8, 0], [0, 0, 0, (1 << 31) - 1],
          [-(1 << 31), -1, 3, (1 << 31) - 1], [5, 4, 3, 2], [-3, 2, 2, 8], [7, 7, 7, 7]]


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("starts", STARTS, ids=str)
def test_row_starts_that_fall_touch_nothing_outside(starts, fmt, page):
    """Every operator with row starts that fall, lie below 0 or behind the rows: all that is written lies in the call's
    arrays, and in the cache at or behind some sequence's position."""
    s = Setup("tiny_alt", fmt, [30, 30, 44], rows=[2, 2, 2], tail=2, page=page)
    lo, hi = s.set_bounds()
    k, v = (bf16(s.rng.standard_normal((s.n_rows, s.Hkv, s.D))) for _ in "kv")
    bands = {}
    for name in list(s.t):
        s.t[name], bands[name] = _guarded(s.t[name])
    s.lo_hi, bands["bounds"] = _guarded(s.lo_hi)
    s.bounds = B.DeviceKeyBounds(s.lo_hi, s.block)
    ptr = [s.t[n].data_ptr() if n in s.t else None for n in ("k", "v", "ks", "vs")]
    s.kv = B.qwen35_kv_cache(ptr[0], ptr[1], s.cap, B.QWEN35_KV_TURBO8 if fmt == TURBO8 else B.QWEN35_KV_BF16, ptr[2],
                             ptr[3], s.table.data_ptr() if page else None, page, 0)
    outs = {}
    for name, shape, kind in (("k_back", k.shape, torch.bfloat16), ("v_back", v.shape, torch.bfloat16),
                              ("out", s.q.shape, torch.bfloat16), ("sparse", s.q.shape, torch.bfloat16),
                              ("blocks", (s.n_rows, s.Hkv, 2), torch.int32)):
        outs[name], bands[name] = _guarded(torch.full(shape, -9, dtype=kind, device="cuda"))
    s.row_start.copy_(torch.tensor(starts, dtype=torch.int64).to(torch.int32))
    before = {n: t.clone() for n, t in s.t.items()}
    bounds_before = s.lo_hi.clone()
    q = s.q.cuda()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, outs["k_back"], outs["v_back"], s.scratch) == 0
    assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, outs["blocks"], s.scratch) == 0
    assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, outs["out"], s.scratch) == 0
    assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, outs["sparse"], s.scratch, blocks=outs["blocks"],
                                     block=s.block) == 0
    torch.cuda.synchronize()
    assert s.status() in (0, B.QWEN35_ERR_DEVICE_RANGE)
    assert [n for n, ok in bands.items() if not ok()] == []
    may = np.zeros(s.total, dtype=bool)
    for b, p in enumerate(s.pos.tolist()):
        may[s.at(b, np.arange(p, s.cap))] = True
    for name, t in s.t.items():
        assert torch.equal(before[name].cpu().view(torch.uint8)[~may], t.cpu().view(torch.uint8)[~may])
    kept = ~may.reshape(-1, s.block).any(1)
    assert torch.equal(bounds_before.cpu().view(torch.int16)[kept], s.lo_hi.cpu().view(torch.int16)[kept])
    # the operators work on as before with row starts as they should be
    s.row_start.copy_(torch.tensor(s.start, dtype=torch.int32))
    B.qwen35_scratch_init(s.scratch)
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    back = [torch.zeros_like(x).cuda() for x in (k, v)]
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *back, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == 0
    if fmt == BF16:
        assert torch.equal(back[0][:6].cpu(), k[:6]) and torch.equal(back[1][:6].cpu(), v[:6])


# ---------------------------------------------------------------- rows in and out, further


@pytest.mark.parametrize("heads", ["tiny", "4b"])
def test_turbo8_codes_of_rows_whose_rotation_is_exact(heads):
    """Whole numbers below 16: the rotation's sums and its power of two are exact in 32 bits, so the codes and scales
    are the oracle's, every one."""
    s = Setup(heads, TURBO8, [700, 45], rows=[650, 45], page=32)
    x = np.random.default_rng(2).integers(-15, 16, size=(s.n_rows, s.Hkv, s.D)).astype(np.float64)
    x *= np.exp2(np.random.default_rng(3).integers(-20, 21, size=(s.n_rows, 1, 1)))
    k = bf16(x)
    np.testing.assert_array_equal(f64(k), x)
    c, sc = O.turbo8_quantize(O.bf16_round(O.wht(x)))
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, k.cuda(), k.flip(0).cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    at = [int(s.at(b, p)) for _, b, p in s.each_row()]
    for name, codes, scales in (("k", c, sc), ("v", c[::-1], sc[::-1])):
        np.testing.assert_array_equal(s.t[name].cpu().numpy()[at], codes)
        got = O.bf16_to_f64(s.t[name + "s"].cpu().numpy().view(np.uint16)[at][:, :s.Hkv * s.D // 16])
        np.testing.assert_array_equal(got.reshape(scales.shape), scales)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("n,per,block", [(24, 2, 64), (60, 1, 256), (40, 1, 1024), (200, 3, 16), (90, 5, 32),
                                         (64, 0, 128)])
def test_bounds_of_many_short_runs(n, per, block, fmt):
    """A few rows of each of many sequences, 0 to 2 per of them, many runs to a block's span of rows: some start a
    block, some cross into the next, some widen one."""
    rows = [(b * 7) % (2 * per + 1) if per else int(b == 40) for b in range(n)]
    lens = [block - 2 + (b * 5) % 7 + rows[b] for b in range(n)]
    s = Setup("tiny", fmt, lens, rows=rows, block=block, lead=1, tail=2)
    s.set_bounds()
    before = f64(s.lo_hi).copy()
    k, v = (bf16(5 * s.rng.standard_normal((s.n_rows, s.Hkv, s.D))) for _ in "kv")
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == 0
    want, x = before.copy(), f64(k)
    for row, b, p in s.each_row():
        e = int(s.at(b, p)) // block
        new = np.stack([x[row], x[row]], 1)
        want[e] = new if p % block == 0 else np.stack([np.fmin(want[e, :, 0], x[row]), np.fmax(want[e, :, 1], x[row])], 1)
    np.testing.assert_array_equal(f64(s.lo_hi), want)


def test_selections_at_once_with_their_own_scratch():
    """Two streams, each with selections whose items several CTAs score, and a third with attention."""
    a = Setup("tiny", BF16, [30000, 9000], page=64, block=16, seed=1)
    b = Setup("odd", BF16, [20000, 8000, 700], block=32, seed=2)
    c = Setup("4b", TURBO8, [2800, 100], page=16, seed=3)
    jobs = []
    for s, n in ((a, 40), (b, 64)):
        s.set_bounds()
        check_choice(s, n)
        out = torch.full((s.n_rows, s.Hkv, n), -9, dtype=torch.int32, device="cuda")
        q = s.q.cuda()
        assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, out, s.scratch) == 0
        jobs.append((s, q, out, torch.zeros_like(out), torch.cuda.Stream()))
    ref, qc, oc, sc = c.attend().clone(), c.q.cuda(), torch.zeros_like(c.q).cuda(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, _, out, st in jobs:
            assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, out, s.scratch, stream=st) == 0
        assert B.qwen35_decode_attention(c.cfg, c.kv, c.r, qc, oc, c.scratch, stream=sc) == 0
    torch.cuda.synchronize()
    for s, _, want, got, _ in jobs:
        assert torch.equal(want, got) and s.status() == 0
    assert torch.equal(ref, oc)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_bounds_of_many_blocks(block, fmt):
    """Long prompts, more blocks and heads than are folded by a CTA each (16 to 64 tokens); one begins inside a block."""
    s = Setup("eight", fmt, [9000, 3011], rows=[9000, 2990], page=128, block=block)
    s.set_bounds()
    want = f64(s.lo_hi).copy()
    k, v = (bf16(s.rng.standard_normal((s.n_rows, s.Hkv, s.D))) for _ in "kv")
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == 0
    x = f64(k)
    for b, (m, r) in enumerate(zip(s.lens, s.rows)):
        for j in range((m - r) // block, (m - 1) // block + 1):
            e, p0 = int(s.at(b, j * block)) // block, max(j * block, m - r)
            rows = x[s.start[b] + p0 - (m - r):s.start[b] + min(m, (j + 1) * block) - (m - r)]
            lo, hi = rows.min(0), rows.max(0)
            if p0 > j * block:
                lo, hi = np.minimum(lo, want[e, :, 0]), np.maximum(hi, want[e, :, 1])
            want[e] = np.stack([lo, hi], 1)
    np.testing.assert_array_equal(f64(s.lo_hi), want)


# ---------------------------------------------------------------- bounds of rows that are in the cache already


@pytest.mark.parametrize("fmt,page", [(BF16, 0), (BF16, 32), (TURBO8, 0), (TURBO8, 32)])
def test_bounds_of_a_cache_that_holds_rows(fmt, page):
    """Rows that came without bounds are read and appended with them: in place for bf16, into a bf16 cache of the same
    layout for Turbo8. The cache stays as it is, the bounds are those of the rows as cached, and selection takes them."""
    s = Setup("tiny_alt", fmt, [300, 77, 200], rows=[300, 77, 200], page=page, block=32)
    s.lo_hi.zero_()
    rows = [torch.zeros(s.n_rows, s.Hkv, s.D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kept = {n: t.clone() for n, t in s.t.items()}
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *rows, s.scratch) == 0
    kv = s.kv
    if fmt == TURBO8:
        other = [torch.zeros(s.total, s.Hkv, s.D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        kv = B.qwen35_kv_cache(other[0].data_ptr(), other[1].data_ptr(), s.cap, B.QWEN35_KV_BF16, None, None,
                               s.table.data_ptr() if page else None, page, 0)
    assert B.qwen35_cache_append(s.cfg, kv, s.r, s.bounds, *rows, s.scratch) == 0
    torch.cuda.synchronize()
    for name, t in s.t.items():
        assert torch.equal(t.view(torch.uint8), kept[name].view(torch.uint8))
    x, got = f64(rows[0]), f64(s.lo_hi)
    for b, m in enumerate(s.lens):
        for j in range((m - 1) // 32 + 1):
            y = x[s.start[b] + 32 * j:s.start[b] + min(m, 32 * j + 32)]
            np.testing.assert_array_equal(got[int(s.at(b, 32 * j)) // 32], np.stack([y.min(0), y.max(0)], 1))
    check_choice(s, 3)
    assert s.status() == 0


# ---------------------------------------------------------------- sizes and replays


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("cap", [1, 7, 17, 37])
def test_a_contiguous_cache_of_any_capacity(cap, fmt):
    """Capacities that end inside a tile of 16 tokens; the last sequence's last row is the cache's last."""
    s = Setup("odd", fmt, [cap, max(1, cap - 3), cap], rows=[min(cap, 3), 1, min(cap, 2)])
    groups, n = s.Hkv * s.D // 16, 3 * cap
    t, stands = {}, {}
    for name, x in s.t.items():
        x = x.view(3, s.cap, *x.shape[1:])[:, :cap]
        t[name], _ = _guarded(x.reshape(n, *x.shape[2:]))
    for name in "kv":
        stands[name] = s.stands[name].reshape(3, s.cap, s.Hkv, s.D)[:, :cap].reshape(n, s.Hkv, s.D)
    s.t, s.stands, s.cap, s.total = t, stands, cap, n
    scales = [t[a].data_ptr() if fmt == TURBO8 else None for a in ("ks", "vs")]
    s.kv = B.qwen35_kv_cache(t["k"].data_ptr(), t["v"].data_ptr(), cap,
                             B.QWEN35_KV_TURBO8 if fmt == TURBO8 else B.QWEN35_KV_BF16, *scales, None, 0, 0)
    check_weighted(s)
    rows = [torch.zeros(s.n_rows, s.Hkv, s.D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *rows, s.scratch) == 0
    torch.cuda.synchronize()
    at = [int(s.at(b, p)) for _, b, p in s.each_row()]
    for name, got in zip("kv", rows):
        err = np.abs(f64(got) - s.stands[name][at])
        norm = np.linalg.norm(s.stands[name][at], axis=-1, keepdims=True)
        assert np.all(err <= 2.0 ** -8 * np.abs(s.stands[name][at]) + 2.0 ** -20 * norm)
    before = {a: x.clone() for a, x in t.items()}
    if fmt == BF16:
        assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, *rows, s.scratch) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(before[a].view(torch.int16), t[a].view(torch.int16)) for a in t)
    assert s.status() == 0


@pytest.mark.parametrize("fmt,page", [(BF16, 64), (TURBO8, 0)])
def test_a_graph_replayed_at_positions_far_apart(fmt, page):
    """Selection and attention captured once and replayed with positions from the first token to the last, in any
    order (one CTA, few parts, all of them): each replay gives the eager call's bits, whatever ran before it."""
    s = Setup("tiny", fmt, [12000, 12000, 12000], page=page, block=16, seed=5)
    s.set_bounds()
    q = s.q.cuda()
    blocks = torch.zeros(3, 1, 20, dtype=torch.int32, device="cuda")
    out, part = torch.zeros_like(q), torch.zeros_like(q)

    def step(scratch):
        assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, blocks, scratch) == 0
        assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, out, scratch) == 0
        assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, part, scratch, blocks=blocks, block=16) == 0

    step(s.scratch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s.scratch)
    for pos in ([0, 15, 16], [11999, 0, 300], [5, 11999, 7000], [319, 320, 321], [11999] * 3, [1, 2, 3], [0, 15, 16]):
        s.pos.copy_(torch.tensor(pos, dtype=torch.int32))
        for t in (blocks, out, part):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (blocks, out, part)]
        for t in (blocks, out, part):
            t.zero_()
        fresh = B.new_scratch(s.scratch.numel())
        step(fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (blocks, out, part)))
        for r, p in enumerate(pos):
            np.testing.assert_array_equal(got[0][r].cpu().numpy(), choose(s, r, r, p, 20, 1, 1))
            ref, size = weighted(s, r, r, p)
            err = np.linalg.norm(f64(got[1][r]) - ref, axis=1)
            assert np.all(err <= 2.0 ** -8 * np.linalg.norm(ref, axis=1) +
                          (2.0 ** -10 + 2.0 ** -12) * np.linalg.norm(size, axis=1))
    assert s.status() == 0


def test_the_most_rows_of_an_append_and_a_read():
    """2^20 rows of one sequence, in both formats; the last row lies at the last position."""
    init()
    cfg = B.make_config(synth.config("tiny"))
    n, D = 1 << 20, 64
    x = torch.randn(n, 1, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    rows = B.DeviceRows(torch.zeros(1, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(cfg, n, 0, n))
    for fmt in (BF16, TURBO8):
        kind = torch.bfloat16 if fmt == BF16 else torch.uint8
        t = [torch.zeros(n, 1, D, dtype=kind, device="cuda") for _ in "kv"]
        sc = [torch.zeros(n, 8, dtype=torch.int16, device="cuda") for _ in "kv"]
        lo_hi = torch.zeros(n // 16, 1, 2, D, dtype=torch.bfloat16, device="cuda")
        kv = B.qwen35_kv_cache(t[0].data_ptr(), t[1].data_ptr(), n, B.QWEN35_KV_BF16 if fmt == BF16 else B.QWEN35_KV_TURBO8,
                               sc[0].data_ptr(), sc[1].data_ptr(), None, 0, 0)
        assert B.qwen35_cache_append(cfg, kv, rows, B.DeviceKeyBounds(lo_hi, 16), x, x.flip(0), scratch) == 0
        back = [torch.zeros_like(x) for _ in "kv"]
        assert B.qwen35_cache_read(cfg, kv, rows, *back, scratch) == 0
        torch.cuda.synchronize()
        y = x.view(n // 16, 16, 1, D)
        assert torch.equal(lo_hi[:, :, 0], y.amin(1)) and torch.equal(lo_hi[:, :, 1], y.amax(1))
        for got, want in zip(back, (x, x.flip(0))):
            if fmt == BF16:
                assert torch.equal(got, want)
            else:  # a rotated value is off by 2^-4 of itself or 2^-10 of its group's largest, and rounded to 8 bits twice
                norm = want.float().norm(dim=-1)
                assert bool(((got.float() - want.float()).norm(dim=-1) <= (2.0 ** -4 + 2.0 ** -6) * norm).all())
    assert B.qwen35_read_device_status(scratch) == 0
