"""The cache operators on the GPU against plain float64 implementations.

Tolerances, derived before the first run:
 - rows of a bf16 cache, Turbo8 codes and scales, key bounds, selected blocks: equal
   (a code is decided on the same fp32 quotient of the same bf16 rows; the rotation's
   fp32 sums against float64 ones may land on the other side of a bf16 rounding
   boundary, so codes are compared with the oracle's quantiser on the rotation read
   back from the layer path, and rows against float64 by the values' half steps);
 - a Turbo8 row read back: one bf16 rounding (half a step, 2^-8 relative) plus the fp32
   butterflies, 8 additions deep, of values up to the row's norm: 2^-20 of it;
 - attention: the output's bf16 rounding, 2^-8 relative, plus what the weights and
   values lose inside: for a bf16 cache the weights enter the products to 2^-16 and
   scores and sums are fp32 (2^-14 of the largest value in all); for a Turbo8 cache
   weights and values enter in 11-bit halves (2^-12 each, 2^-10 in all with the
   scores' part), an error of the rotated output that the rotation back keeps in norm.
"""

import numpy as np
import pytest
import torch

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth
from oracle import qwen35_oracle as O

from harness import init

pytestmark = pytest.mark.gpu

BF16, TURBO8 = "bf16", "turbo8"
HEADS = {"4b": (16, 4, 256), "tiny": (4, 1, 64), "tiny_alt": (3, 3, 128), "wide": (32, 2, 128), "eight": (8, 1, 64),
         "odd": (6, 2, 64), "twelve": (12, 1, 256)}


def bf16(a):
    """float array -> CPU bf16 tensor."""
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


class Setup:
    """A cache of `lens` sequences (tokens it holds, the call's rows included) with the
    tokens behind them, the pool's spare blocks and the gaps between filled with NaN; the
    float64 rows it stands for; and the call's rows: the last rows[b] tokens of each."""

    def __init__(self, heads, fmt, lens, rows=None, page=0, block=16, seed=0, spread=1.0, lead=0, tail=0,
                 share_first=False):
        init()
        self.H, self.Hkv, self.D = HEADS[heads]
        self.fmt, self.page, self.block = fmt, page, block
        self.cfg = B.make_config(synth.config("tiny") | dict(num_heads=self.H, num_kv_heads=self.Hkv, head_dim=self.D))
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.lens, n = list(lens), len(lens)
        self.ragged = rows is not None
        self.rows = list(rows) if self.ragged else [1] * n
        unit = max(page, block, 16)
        self.cap = (max(max(lens), 1) + unit - 1) // unit * unit
        if page:
            per = self.cap // page
            self.nb = n * per + 3
            self.table_np = rng.permutation(self.nb)[:n * per].reshape(n, per).astype(np.int32)
            if share_first:
                self.table_np[:, 0] = self.table_np[0, 0]
            self.table = torch.from_numpy(self.table_np).cuda()
            self.total = self.nb * page
        else:
            self.nb, self.table, self.total = 0, None, n * self.cap
        Hkv, D = self.Hkv, self.D
        self.val = {}
        self.t = {}
        for name in "kv":
            x = bf16(spread * rng.standard_normal((n, self.cap, Hkv, D)))
            if share_first:
                x[:, :page] = x[:1, :page]
            for b, m in enumerate(self.lens):
                x[b, m:] = float("nan")
            self.val[name] = x  # as given
            flat = torch.full((self.total, Hkv, D), float("nan"), dtype=torch.bfloat16)
            for b in range(n):
                flat[self.at(b, np.arange(self.cap))] = x[b]
            if fmt == TURBO8:
                y = f64(flat)
                codes = np.full((self.total, Hkv, D), 0x7F, dtype=np.uint8)
                ss = B.turbo8_sstride(dict(num_kv_heads=Hkv, head_dim=D))
                sc = np.full((self.total, ss), 0x7FC0, dtype=np.uint16)
                held = ~np.isnan(y).any(axis=(1, 2))
                c, s = O.turbo8_quantize(O.bf16_round(O.wht(y[held])))
                codes[held] = c
                sc[held, :Hkv * D // 16] = O.bf16_bits(s).reshape(int(held.sum()), -1)
                self.t[name] = torch.from_numpy(codes).cuda()
                self.t[name + "s"] = torch.from_numpy(sc.view(np.int16)).cuda()
                back = np.full(y.shape, np.nan)
                back[held] = O.wht(O.turbo8_dequantize(c, s))  # float64 rows the cache stands for
                self.stands = getattr(self, "stands", {})
                self.stands[name] = back
            else:
                self.t[name] = flat.cuda()
                self.stands = getattr(self, "stands", {})
                self.stands[name] = f64(flat)
        self.kv = B.qwen35_kv_cache(self.t["k"].data_ptr(), self.t["v"].data_ptr(), self.cap,
                                    B.QWEN35_KV_TURBO8 if fmt == TURBO8 else B.QWEN35_KV_BF16,
                                    self.t["ks"].data_ptr() if fmt == TURBO8 else None,
                                    self.t["vs"].data_ptr() if fmt == TURBO8 else None,
                                    self.table.data_ptr() if page else None, page, 0)
        start = [lead]
        for r in self.rows:
            start.append(start[-1] + r)
        self.start, self.n_rows = start, start[-1] + tail
        pos = [m - r for m, r in zip(self.lens, self.rows)]
        self.pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
        self.row_start = torch.tensor(start, dtype=torch.int32, device="cuda") if self.ragged else None
        self.r = B.DeviceRows(self.pos, self.row_start, self.n_rows, self.nb)
        self.q = bf16(rng.standard_normal((self.n_rows, self.H, D)))
        self.lo_hi = torch.full((self.total // block, Hkv, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.bounds = B.DeviceKeyBounds(self.lo_hi, block)
        self.scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(self.cfg, self.cap, block, self.n_rows))

    def at(self, b, t):
        t = np.asarray(t)
        if self.page:
            return self.table_np[b][t // self.page].astype(np.int64) * self.page + t % self.page
        return b * self.cap + t

    def each_row(self):
        """(row, sequence, position) of every row a sequence has."""
        for b, (m, r) in enumerate(zip(self.lens, self.rows)):
            for i in range(r):
                yield self.start[b] + i, b, m - r + i

    def set_bounds(self):
        """The bounds of every block that holds a token, from the rows as given."""
        x = np.full((self.total, self.Hkv, self.D), np.nan)
        for b, m in enumerate(self.lens):
            x[self.at(b, np.arange(m))] = f64(self.val["k"][b, :m])
        x = x.reshape(-1, self.block, self.Hkv, self.D)
        with np.errstate(all="ignore"):
            import warnings
            with warnings.catch_warnings():
                warnings.simplefilter("ignore")
                lo, hi = np.nanmin(x, axis=1), np.nanmax(x, axis=1)
        self.lo_hi.copy_(bf16(np.stack([lo, hi], axis=2)).cuda())
        return lo, hi

    def status(self):
        return B.qwen35_read_device_status(self.scratch)

    def attend(self, out=None, **kw):
        out = torch.full((self.n_rows, self.H, self.D), float("nan"), dtype=torch.bfloat16, device="cuda") \
            if out is None else out
        assert B.qwen35_decode_attention(self.cfg, self.kv, self.r, self.q.cuda(), out, self.scratch, **kw) == 0
        torch.cuda.synchronize()
        return out

    def reference(self, row, b, p, blocks=None):
        """float64 attention of one row; blocks [Hkv][n]: listed blocks only."""
        g = self.H // self.Hkv
        out = np.zeros((self.H, self.D))
        vmax = np.zeros(self.H)
        q = f64(self.q[row])
        for h in range(self.H):
            t = np.arange(p + 1)
            if blocks is not None:
                t = np.concatenate([np.arange(j * self.block, (j + 1) * self.block) for j in blocks[h // g] if j >= 0]
                                   or [np.zeros(0)]).astype(np.int64)
                t = t[t <= p]
            if len(t) == 0:
                continue
            rows = self.at(b, t)
            k, v = self.stands["k"][rows, h // g], self.stands["v"][rows, h // g]
            x = k @ q[h] / np.sqrt(self.D)
            w = np.exp(x - x.max())
            out[h] = (w / w.sum()) @ v
            vmax[h] = np.abs(O.wht(v) if self.fmt == TURBO8 else v).max()
        return out, vmax

    def check(self, out, blocks=None, gate=None):
        got = f64(out)
        seen = set()
        for row, b, p in self.each_row():
            seen.add(row)
            ref, vmax = self.reference(row, b, p, None if blocks is None else blocks[row])
            if gate is not None:
                ref = ref / (1 + np.exp(-f64(gate[row])))
            err = np.abs(got[row] - ref)
            if self.fmt == BF16:
                bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * vmax[:, None]
                assert np.all(err <= bound), (row, b, p, float((err / (bound + 1e-300)).max()))
            else:
                err = np.linalg.norm(err, axis=1)
                bound = 2.0 ** -8 * np.linalg.norm(ref, axis=1) + 2.0 ** -10 * vmax * np.sqrt(self.D)
                assert np.all(err <= bound), (row, b, p, float((err / bound).max()))
        for row in set(range(self.n_rows)) - seen:
            assert np.isnan(got[row]).all(), row  # left as it was


# ---------------------------------------------------------------- rows in and out


def _new_rows(s, seed=5):
    rng = np.random.default_rng(seed)
    return [bf16(rng.standard_normal((s.n_rows, s.Hkv, s.D)) * rng.uniform(0.01, 30, size=(s.n_rows, 1, 1)))
            for _ in "kv"]


APPENDS = [dict(heads="tiny", fmt=BF16, lens=[1]), dict(heads="tiny", fmt=TURBO8, lens=[1], page=16),
           dict(heads="4b", fmt=TURBO8, lens=[17, 300, 64], page=32, block=32),
           dict(heads="tiny_alt", fmt=TURBO8, lens=[40, 33, 90], rows=[40, 0, 57], page=8 * 4, block=16, tail=3),
           dict(heads="4b", fmt=BF16, lens=[130, 5, 77], rows=[100, 5, 1], page=16, block=16, lead=2, tail=1),
           dict(heads="odd", fmt=BF16, lens=[200, 513], rows=[129, 70], block=64),
           dict(heads="tiny", fmt=TURBO8, lens=[1100, 700], rows=[1100, 3], block=1024)]


@pytest.mark.parametrize("kw", APPENDS)
def test_append_then_read(kw):
    s = Setup(**kw)
    k, v = _new_rows(s)
    before = {n: t.clone() for n, t in s.t.items()}
    lo, hi = s.set_bounds()
    b0 = s.lo_hi.clone()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    back = [torch.full_like(k, float("nan")).cuda() for _ in "kv"]
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *back, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == 0
    written = np.zeros(s.total, dtype=bool)
    rows = list(s.each_row())
    where = np.array([s.at(b, p) for _, b, p in rows], dtype=np.int64)
    idx = [r for r, _, _ in rows]
    written[where] = True
    for name, x, y in (("k", k, back[0]), ("v", v, back[1])):
        old, new = before[name].cpu().view(torch.uint8), s.t[name].cpu().view(torch.uint8)
        assert torch.equal(old[~written], new[~written])  # every other row as it was
        left = sorted(set(range(s.n_rows)) - set(idx))
        assert torch.isnan(y[left]).all()
        if s.fmt == BF16:
            assert torch.equal(s.t[name].cpu()[where], x[idx]) and torch.equal(y.cpu()[idx], x[idx])
            continue
        assert torch.equal(before[name + "s"].cpu()[~written], s.t[name + "s"].cpu()[~written])
        sc = O.bf16_to_f64(s.t[name + "s"].cpu().numpy().view(np.uint16)[where][:, :s.Hkv * s.D // 16])
        codes = s.t[name].cpu().numpy()[where]
        rot = O.wht(f64(x[idx]))
        c, want = O.turbo8_quantize(O.bf16_round(rot))
        same = (codes == c).mean()
        assert same > 0.999 and (sc.reshape(want.shape) == want).mean() > 0.999
        stands = O.turbo8_dequantize(codes, sc.reshape(want.shape))
        # a step of E4M3 is at most 2^-3 of the value, of a group's largest at least 2^-9 of it
        group = np.repeat(np.abs(rot.reshape(want.shape + (16,))).max(-1), 16, axis=-1).reshape(rot.shape)
        assert np.all(np.abs(stands - rot) <= 2.0 ** -4 * 1.02 * np.abs(rot) + 2.0 ** -16 * group)
        plain = O.wht(stands)
        norm = np.linalg.norm(plain, axis=-1, keepdims=True)
        assert np.all(np.abs(f64(y[idx]) - plain) <= 2.0 ** -8 * np.abs(plain) + 2.0 ** -20 * norm)
    # the bounds: blocks with a new row, over all their rows; the others untouched
    x = {int(w): f64(k[r]) for w, r in zip(where, idx)}
    start = {int(s.at(b, p)) // s.block: p - p % s.block for _, b, p in rows}
    touched = np.zeros(s.total // s.block, dtype=bool)
    got = f64(s.lo_hi)
    for b, m in enumerate(s.lens):
        p0 = m - s.rows[b]
        for j in sorted({p // s.block for p in range(p0, m)}):
            e = int(s.at(b, j * s.block)) // s.block
            touched[e] = True
            new = np.stack([x[int(s.at(b, p))] for p in range(max(p0, j * s.block), min(m, (j + 1) * s.block))])
            l, h = new.min(0), new.max(0)
            if j * s.block < p0:
                l, h = np.minimum(l, f64(b0)[e, :, 0]), np.maximum(h, f64(b0)[e, :, 1])
            np.testing.assert_array_equal(got[e, :, 0], l)
            np.testing.assert_array_equal(got[e, :, 1], h)
    assert start.keys() == set(np.flatnonzero(touched).tolist())
    assert torch.equal(b0.cpu().view(torch.int16)[~touched], s.lo_hi.cpu().view(torch.int16)[~touched])


@pytest.mark.parametrize("cfg_name", ["tiny", "tiny_alt", "4b"])
def test_turbo8_append_equals_the_prefill_of_a_layer(cfg_name):
    """The same rows into a cache by the prefill of a layer and by the operator: codes and
    scales bit for bit. The layer's bf16 cache holds the rows before they are quantised."""
    init()
    cfg = synth.config(cfg_name)
    c = B.make_config(cfg)
    T, cap = 37, 48
    Hkv, D = cfg["num_kv_heads"], cfg["head_dim"]
    layer = B.DeviceFaLayer(synth.fa_layer(1, 1, cfg))
    scratch = B.new_scratch(B.qwen35_prefill_scratch_bytes(c, T))
    x = B.to_device(np.stack([synth.x_in(1, t, cfg) for t in range(T)]))
    y = torch.empty_like(x)
    zero = np.zeros((cap, Hkv, D), dtype=np.uint16)
    flat = B.DeviceKv(zero, zero)
    if cfg["num_heads"] // Hkv in (1, 2, 4, 8):
        t8 = B.DeviceKvTurbo8(zero.astype(np.uint8), np.zeros((cap, Hkv, D // 16), np.uint16), zero.astype(np.uint8),
                              np.zeros((cap, Hkv, D // 16), np.uint16), cfg)
        for kv in (flat, t8):
            assert B.qwen35_prefill_full_attention(c, layer.struct, scratch, kv.struct, x, y, 0, T) == 0
        mine = B.DeviceKvTurbo8(zero.astype(np.uint8), np.zeros((cap, Hkv, D // 16), np.uint16), zero.astype(np.uint8),
                                np.zeros((cap, Hkv, D // 16), np.uint16), cfg)
        rows = B.DeviceRows(torch.zeros(1, dtype=torch.int32, device="cuda"),
                            torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)
        s2 = B.new_scratch(B.qwen35_cache_scratch_bytes(c, cap, 0, T))
        assert B.qwen35_cache_append(c, mine.struct, rows, None, flat.k[:T].contiguous(), flat.v[:T].contiguous(), s2) == 0
        torch.cuda.synchronize()
        for a, b in ((mine.k, t8.k), (mine.v, t8.v), (mine.ks, t8.ks), (mine.vs, t8.vs)):
            assert torch.equal(a[:T], b[:T])


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "4b"])
def test_rows_aligned_to_16_bytes_only(heads):
    s = Setup(heads, TURBO8, [40, 33], rows=[40, 5])
    k, v = [x.cuda() for x in _new_rows(s)]
    off = []
    for x in (k, v, torch.zeros_like(k), torch.zeros_like(k)):
        room = torch.zeros(x.numel() + 8, dtype=torch.bfloat16, device="cuda")
        assert (room.data_ptr() + 16) % 32 == 16
        y = room[8:].view_as(x)
        y.copy_(x)
        off.append(y)
    back = [torch.zeros_like(k) for _ in "kv"]
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, k, v, s.scratch) == 0
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *back, s.scratch) == 0
    torch.cuda.synchronize()
    kept = {n: t.clone() for n, t in s.t.items()}
    for t in s.t.values():
        t.zero_()
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, off[0], off[1], s.scratch) == 0
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, off[2], off[3], s.scratch) == 0
    torch.cuda.synchronize()
    at = [int(s.at(b, p)) for _, b, p in s.each_row()]
    groups = s.Hkv * s.D // 16  # (a row of scales is padded behind them)
    assert all(torch.equal(kept[n][at, :groups], s.t[n][at, :groups]) for n in ("ks", "vs"))
    assert all(torch.equal(kept[n][at], s.t[n][at]) for n in "kv")
    assert torch.equal(back[0], off[2]) and torch.equal(back[1], off[3])


@pytest.mark.parametrize("e", [-132, -126, -110, -60, 60, 110, 118])
def test_turbo8_append_at_the_ends_of_the_range(e):
    """Rows near the smallest and the largest bf16 values: the oracle's codes and scales."""
    s = Setup("tiny", TURBO8, [64], rows=[64])
    rng = np.random.default_rng(abs(e))
    x = np.zeros((64, 1, s.D))
    x[np.arange(64), 0, rng.integers(0, s.D, 64)] = np.exp2(e) * rng.integers(128, 256, 64) / 128  # rotated: +-x / 8
    k = bf16(x)
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, None, k.cuda(), k.cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        c, sc = O.turbo8_quantize(O.bf16_round(O.wht(f64(k))))
    at = [int(s.at(0, p)) for p in range(64)]
    got = O.bf16_to_f64(s.t["ks"].cpu().numpy().view(np.uint16)[at][:, :s.D // 16]).reshape(sc.shape)
    np.testing.assert_array_equal(got, sc)
    np.testing.assert_array_equal(s.t["k"].cpu().numpy()[at].reshape(c.shape), c)


def test_append_skips_nan_in_bounds_and_keeps_special_rows():
    s = Setup("tiny", BF16, [20, 16], rows=[20, 16], block=16)
    k, v = _new_rows(s)
    k[3, 0, 5] = float("nan")
    k[4, 0, 6] = float("inf")
    k[5, 0, 7] = -float("inf")
    k[20:, 0, 9] = float("nan")  # a dimension without a number
    v[2] = float("nan")
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    got = f64(s.lo_hi)
    x = f64(k)
    np.testing.assert_array_equal(got[0, 0, 0], np.nanmin(x[:16, 0], axis=0))
    np.testing.assert_array_equal(got[0, 0, 1], np.nanmax(x[:16, 0], axis=0))
    e = s.cap // s.block  # sequence 1's first block
    ok = np.arange(s.D) != 9
    np.testing.assert_array_equal(got[e, 0, 0][ok], x[20:, 0].min(0)[ok])
    flat = s.t["k"].cpu()
    assert torch.equal(flat[:20].view(torch.int16), k[:20].view(torch.int16))


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_rows_out_of_range_are_skipped_and_reported(fmt):
    """A position outside the cache, a block outside the pool: the status word says so, the
    other rows are written, nothing else is touched."""
    s = Setup("tiny", fmt, [20, 20, 20, 20], page=16)
    s.pos.copy_(torch.tensor([19, -1, s.cap, 3], dtype=torch.int32))
    s.table[3, 0] = s.nb
    k, v = _new_rows(s)
    before = {n: t.clone() for n, t in s.t.items()}
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    changed = (before["k"].cpu().view(torch.uint8) != s.t["k"].cpu().view(torch.uint8)).flatten(1).any(1)
    assert torch.nonzero(changed).flatten().tolist() == [int(s.at(0, 19))]
    back = [torch.full_like(k, 7.0).cuda() for _ in "kv"]
    B.qwen35_scratch_init(s.scratch)
    assert s.status() == 0
    assert B.qwen35_cache_read(s.cfg, s.kv, s.r, *back, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    assert (back[0][1:] == 7).all() and not (back[0][0] == 7).any()
    out = torch.full((4, s.H, s.D), 7.0, dtype=torch.bfloat16, device="cuda")
    B.qwen35_scratch_init(s.scratch)
    s.attend(out)
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    assert (out[1:3] == 7).all() and not (out[0] == 7).any()
    blocks = torch.full((4, s.Hkv, 1), 7, dtype=torch.int32, device="cuda")
    B.qwen35_scratch_init(s.scratch)
    assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, s.q.cuda(), blocks, s.scratch) == 0
    torch.cuda.synchronize()
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    assert (blocks[1:3] == 7).all() and not (blocks[0] == 7).any()


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("page", [8, 32])
def test_attention_leaves_a_block_outside_the_pool_out(fmt, page):
    s = Setup("tiny", fmt, [100, 60], rows=[3, 2], page=page, block=16)
    s.table[0, 1] = s.nb + 5
    s.table[1, 0] = -1
    out = s.attend()
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    got = f64(out)
    for row, b, p in s.each_row():
        t = np.arange(p + 1)
        t = t[t // page != (1 if b == 0 else 0)]
        rows = s.at(b, t)
        k, v, q = s.stands["k"][rows, 0], s.stands["v"][rows, 0], f64(s.q[row])
        x = q @ k.T / np.sqrt(s.D)
        w = np.exp(x - x.max(-1, keepdims=True))
        ref = (w / w.sum(-1, keepdims=True)) @ v
        err, vmax = np.linalg.norm(got[row] - ref, axis=1), np.abs(O.wht(v) if fmt == TURBO8 else v).max()
        assert np.all(err <= 2.0 ** -8 * np.linalg.norm(ref, axis=1) + 2.0 ** -10 * vmax * np.sqrt(s.D))


def test_a_row_start_that_runs_backwards_touches_nothing_outside():
    s = Setup("tiny", BF16, [30, 30, 30], rows=[2, 2, 2], tail=2)
    s.row_start.copy_(torch.tensor([0, 6, 2, 8], dtype=torch.int32))
    k, v = _new_rows(s)
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    s.attend()
    s.row_start.copy_(torch.tensor([-5, 1 << 30, -(1 << 30), 1 << 30], dtype=torch.int32))
    assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k.cuda(), v.cuda(), s.scratch) == 0
    s.attend()
    assert s.status() in (0, B.QWEN35_ERR_DEVICE_RANGE)


# ---------------------------------------------------------------- attention


ATTENDS = [dict(heads="tiny", fmt=BF16, lens=[1]), dict(heads="tiny", fmt=TURBO8, lens=[1]),
           dict(heads="tiny", fmt=BF16, lens=[15, 16, 17, 31, 32, 33, 64, 65], page=16),
           dict(heads="tiny", fmt=TURBO8, lens=[15, 16, 17, 31, 32, 33, 64, 65], page=16),
           dict(heads="4b", fmt=BF16, lens=[1, 257, 1000]), dict(heads="4b", fmt=TURBO8, lens=[1, 257, 1000], page=64),
           dict(heads="4b", fmt=BF16, lens=[2000], page=8), dict(heads="4b", fmt=TURBO8, lens=[2000], page=8),
           dict(heads="tiny_alt", fmt=BF16, lens=[7, 700], rows=[5, 3], page=32, lead=1, tail=2),
           dict(heads="tiny_alt", fmt=TURBO8, lens=[7, 700, 40], rows=[5, 3, 0], page=32, tail=2),
           dict(heads="wide", fmt=BF16, lens=[300, 33]), dict(heads="wide", fmt=TURBO8, lens=[300, 33]),
           dict(heads="eight", fmt=BF16, lens=[129, 64, 511], page=128),
           dict(heads="eight", fmt=TURBO8, lens=[129, 64, 511], page=128),
           dict(heads="odd", fmt=BF16, lens=[90, 200], spread=6.0), dict(heads="odd", fmt=TURBO8, lens=[90, 200]),
           dict(heads="twelve", fmt=BF16, lens=[140, 19]), dict(heads="twelve", fmt=TURBO8, lens=[140, 19]),
           dict(heads="tiny", fmt=BF16, lens=list(range(1, 90)), page=16),
           # several rows of a sequence: across a tile's end, from the first token on, more than fit an item
           dict(heads="tiny_alt", fmt=BF16, lens=[17, 16, 33, 18, 9, 140], rows=[5, 16, 8, 3, 9, 20], page=16),
           dict(heads="tiny_alt", fmt=TURBO8, lens=[17, 16, 33, 18, 9, 140], rows=[5, 16, 8, 3, 9, 20], page=8),
           dict(heads="odd", fmt=BF16, lens=[65, 34, 2, 50], rows=[3, 4, 2, 1], page=16, lead=3),
           dict(heads="odd", fmt=TURBO8, lens=[65, 34, 2, 50], rows=[3, 4, 2, 1], lead=3),
           dict(heads="4b", fmt=TURBO8, lens=[600, 49], rows=[7, 2]), dict(heads="wide", fmt=BF16, lens=[77], rows=[4]),
           dict(heads="tiny", fmt=TURBO8, lens=[40] * 40, page=16, share_first=True)]


@pytest.mark.parametrize("kw", ATTENDS)
def test_attention_over_every_token(kw):
    s = Setup(**kw)
    s.check(s.attend())
    assert s.status() == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("heads,lens", [("tiny", [6000]), ("tiny", [9001, 3]), ("wide", [7000]), ("odd", [5000, 2500]),
                                        ("twelve", [4500]), ("eight", [4000])])
def test_attention_joined_from_many_parts(heads, lens, fmt):
    """Few long sequences: up to every CTA of the GPU has a part of an item, more than a thread takes at a time."""
    s = Setup(heads, fmt, lens, page=32)
    s.check(s.attend())


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_attention_gate_and_its_stride(fmt):
    s = Setup("4b", fmt, [70, 300])
    gate = bf16(3 * s.rng.standard_normal((2, s.H, s.D)))
    s.check(s.attend(gate=gate.cuda()), gate=gate)
    packed = torch.stack([s.q, gate], dim=2).cuda()  # [rows][H][2][D]: q_proj's rows [Q_h | gate_h]
    a = s.attend(gate=gate.cuda())
    b = s.attend(gate=packed.data_ptr() + 2 * s.D, gate_stride=2 * s.D)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_attention_large_scores_and_one_heavy_token(fmt):
    """Scores of several hundred: one token takes all the weight, wherever it lies."""
    s = Setup("tiny", fmt, [333, 333, 333, 333], page=16, spread=4.0)
    s.q = 25 * s.q
    s.check(s.attend())


def test_attention_of_zero_and_equal_rows():
    s = Setup("tiny", BF16, [50, 1])
    s.q = torch.zeros_like(s.q)  # every token weighs the same
    s.check(s.attend())
    z = Setup("tiny", TURBO8, [50, 1], spread=0.0)
    assert (z.attend() == 0).all()


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_a_nan_in_a_key_spoils_only_rows_that_see_it(fmt):
    s = Setup("tiny", fmt, [40, 40], rows=[4, 4])
    at = s.at(0, 38)  # positions 36..39 are the call's rows: the first two do not see it
    if fmt == BF16:
        s.t["k"][at, 0, 3] = float("nan")
        s.t["v"][at, 0, 3] = float("inf")
    else:
        s.t["k"][at, 0, 3] = 0x7F
    got = f64(s.attend())
    assert np.isfinite(got[[0, 1, 4, 5, 6, 7]]).all() and np.isnan(got[[2, 3]]).any(axis=(1, 2)).all()


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
@pytest.mark.parametrize("rows", [False, True])
def test_attention_of_many_rows(fmt, rows):
    """More rows than threads of a CTA, of lengths 1 to 40, sequences without a row among them."""
    n = 700
    kw = dict(rows=[(b * 5) % 4 for b in range(n)]) if rows else {}
    s = Setup("tiny", fmt, [4 + (b * 7) % 37 for b in range(n)], page=8, **kw)
    s.check(s.attend())
    assert s.status() == 0


def test_attention_of_the_most_rows():
    s = Setup("tiny", BF16, [2 + b % 3 for b in range(2048)])
    s.check(s.attend())
    t = Setup("tiny", BF16, [2 + b % 3 for b in range(4096)], rows=[b % 2 for b in range(4096)])
    t.check(t.attend())
    assert s.status() == 0 and t.status() == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_rows_that_run_out_of_the_cache(fmt):
    """The last two of four rows lie behind the capacity: reported, left as they were, the others right."""
    s = Setup("tiny_alt", fmt, [48, 20], rows=[4, 3])
    assert s.cap == 48
    s.pos[0] = 46
    out = f64(s.attend())
    assert s.status() == B.QWEN35_ERR_DEVICE_RANGE
    assert np.isnan(out[[2, 3]]).all()
    for row, p in ((0, 46), (1, 47)):
        ref, vmax = s.reference(row, 0, p)
        assert np.linalg.norm(out[row] - ref) <= 2.0 ** -7 * np.linalg.norm(ref) + 2.0 ** -10 * vmax.max() * np.sqrt(ref.size)
    assert np.isfinite(out[[4, 5, 6]]).all()


def test_turbo8_values_of_very_different_sizes():
    """V rows from 2^-40 to 2^40 of one another, each format's step relative to its own group."""
    s = Setup("tiny", TURBO8, [200, 37], page=16, seed=3)
    rng = np.random.default_rng(1)
    scale = np.exp2(rng.integers(-40, 41, size=(s.total, 1)))
    sc = O.bf16_to_f64(s.t["vs"].cpu().numpy().view(np.uint16)) * scale
    s.t["vs"].copy_(torch.from_numpy(O.bf16_bits(sc).view(np.int16)))
    s.stands["v"] = s.stands["v"] * scale[:, :, None]
    s.check(s.attend())
    small = Setup("tiny", TURBO8, [100], seed=4)  # all of them tiny, and all of them large
    base = small.t["vs"].clone()
    stands = small.stands["v"].copy()
    for e in (-50, 50):
        sc = O.bf16_to_f64(base.cpu().numpy().view(np.uint16)) * 2.0 ** e
        small.t["vs"].copy_(torch.from_numpy(O.bf16_bits(sc).view(np.int16)))
        small.stands["v"] = stands * 2.0 ** e
        small.check(small.attend())


@pytest.mark.parametrize("heads", ["tiny", "tiny_alt", "odd", "eight"])
@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_what_later_rows_of_a_call_hold_is_not_seen(fmt, heads):
    """Rows 0 .. 6 of one sequence; the tokens of rows 3 and 5 hold infinities and NaN in K and V."""
    s = Setup(heads, fmt, [35, 20], rows=[7, 2])
    clean = f64(s.attend()).copy()
    for pos, name in ((31, "v"), (33, "k"), (33, "v")):
        at = s.at(0, pos)
        if fmt == BF16:
            s.t[name][at, :, 3] = float("inf")
            s.t[name][at, :, 4] = float("nan")
        else:
            s.t[name][at, :, 3] = 0x7F
            s.t[name + "s"][at, 1] = 0x7F80
    got = f64(s.attend())
    keep = [0, 1, 2, 7, 8]
    np.testing.assert_array_equal(got[keep], clean[keep])
    assert all(np.isnan(got[r]).any() or np.isinf(got[r]).any() for r in (3, 4, 5, 6))


def _lists(s, n, seed=3, holes=True):
    rng = np.random.default_rng(seed)
    out = np.full((s.n_rows, s.Hkv, n), -1, dtype=np.int32)
    for row, b, p in s.each_row():
        for g in range(s.Hkv):
            seen = p // s.block + 1
            pick = rng.permutation(seen)[:n]
            out[row, g, :len(pick)] = np.sort(pick) if not holes else pick
    return out


SPARSE = [dict(heads="tiny", fmt=BF16, lens=[100, 17, 1], block=16, page=16),
          dict(heads="tiny", fmt=TURBO8, lens=[100, 17, 1], block=16),
          dict(heads="4b", fmt=BF16, lens=[900, 640], block=64, page=128),
          dict(heads="4b", fmt=TURBO8, lens=[900, 640], block=64, page=64),
          dict(heads="tiny_alt", fmt=TURBO8, lens=[300, 200], rows=[3, 2], block=32, page=32, tail=1),
          dict(heads="wide", fmt=BF16, lens=[1500], block=128), dict(heads="eight", fmt=TURBO8, lens=[777], block=16)]


@pytest.mark.parametrize("n", [1, 5, 16])
@pytest.mark.parametrize("kw", SPARSE)
def test_attention_over_listed_blocks(kw, n):
    s = Setup(**kw)
    n = min(n, s.cap // s.block)
    lists = _lists(s, n)
    s.check(s.attend(blocks=torch.from_numpy(lists).cuda(), block=s.block), blocks=lists)
    assert s.status() == 0


@pytest.mark.parametrize("fmt", [BF16, TURBO8])
def test_listed_blocks_in_any_form(fmt):
    """Empty lists give zeros; entries behind the row or negative count as none; one
    listed twice counts twice; a row past the first block need not list its own."""
    s = Setup("tiny", fmt, [100, 100, 100, 100, 100], block=16)
    n = s.cap // 16
    assert n == 7
    lists = np.full((5, 1, n), -1, dtype=np.int32)
    lists[1, 0] = [-1, 3, -7, 3, 0, -1, -1]
    lists[2, 0] = [7, 1 << 30, (1 << 31) - 1, -(1 << 31), 6, 1 << 28, 2]
    lists[3, 0] = [0, 0, 0, 0, 0, 0, 0]
    lists[4, 0] = [7, 8, 9, 10, 11, 12, 13]
    clean = [[[j for j in row[0] if 0 <= j <= 6]] for row in lists]
    out = s.attend(blocks=torch.from_numpy(lists).cuda(), block=16)
    s.check(out, blocks=clean)
    assert (out[0] == 0).all() and (out[4] == 0).all()
    assert s.status() == 0


@pytest.mark.parametrize("kw", [dict(heads="4b", fmt=BF16, lens=[3000, 100], page=16),
                                dict(heads="tiny", fmt=TURBO8, lens=[3000, 100], page=16)])
def test_every_block_listed_equals_every_token(kw):
    s = Setup(**kw)
    n = s.cap // 16
    lists = np.full((2, s.Hkv, n), -1, dtype=np.int32)
    for r, m in enumerate(s.lens):
        lists[r, :, :(m + 15) // 16] = np.arange((m + 15) // 16)
    a, b = s.attend(), s.attend(blocks=torch.from_numpy(lists).cuda(), block=16)
    s.check(b)
    assert np.allclose(f64(a), f64(b), rtol=2.0 ** -7, atol=1e-3)


# ---------------------------------------------------------------- selection


def choose(s, row, b, p, n, first, last):
    """The definition in float64: [Hkv][n]."""
    g, seen = s.H // s.Hkv, p // s.block + 1
    q = f64(s.q[row]).reshape(s.Hkv, g, s.D)
    bounds = f64(s.lo_hi)[s.at(b, np.arange(seen) * s.block) // s.block]
    with np.errstate(all="ignore"):  # the bound of q.k: hi where q is not negative, lo where it is
        score = np.where(q[:, :, None] < 0, q[:, :, None] * bounds[:, :, 0].transpose(1, 0, 2)[:, None],
                         q[:, :, None] * bounds[:, :, 1].transpose(1, 0, 2)[:, None]).sum((1, 3))
    score = np.where(np.isnan(score), -np.inf, score)
    j = np.arange(seen)
    rank = np.where((j < first) | (j >= seen - last), 1, 0)
    out = np.full((s.Hkv, n), -1, dtype=np.int64)
    for h in range(s.Hkv):
        order = sorted(range(seen), key=lambda i: (-rank[i], 0 if rank[i] else -score[h, i], i))[:n]
        out[h, :len(order)] = sorted(order)
    return out


def select(s, n, first=1, last=1):
    out = torch.full((s.n_rows, s.Hkv, n), -9, dtype=torch.int32, device="cuda")
    assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, s.q.cuda(), out, s.scratch, first, last) == 0
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check_choice(s, n, first=1, last=1):
    got = select(s, n, first, last)
    seen = set()
    for row, b, p in s.each_row():
        seen.add(row)
        np.testing.assert_array_equal(got[row], choose(s, row, b, p, n, first, last), err_msg=str((row, b, p)))
    assert (got[sorted(set(range(s.n_rows)) - seen)] == -9).all()
    assert s.status() == 0


@pytest.mark.parametrize("first,last", [(1, 1), (0, 0), (0, 3), (40, 2), (2, 1 << 31)])
@pytest.mark.parametrize("kw,n", [(dict(heads="tiny", fmt=BF16, lens=[1, 16, 17, 500, 4000], page=16), 7),
                                  (dict(heads="4b", fmt=TURBO8, lens=[1500, 90], block=32, page=64), 16),
                                  (dict(heads="tiny_alt", fmt=BF16, lens=[700, 650], rows=[6, 2], tail=2, lead=1), 5),
                                  (dict(heads="wide", fmt=BF16, lens=[2100], block=16), 131),
                                  (dict(heads="tiny", fmt=BF16, lens=[70000, 300000], block=16), 33),
                                  (dict(heads="eight", fmt=TURBO8, lens=[9000, 10], block=16, page=32), 33)])
def test_selection(kw, n, first, last):
    s = Setup(**kw)
    s.set_bounds()
    check_choice(s, n, first, last)


def test_lists_longer_than_the_cache_has_blocks():
    s = Setup("tiny", TURBO8, [40, 1, 17], block=16)
    s.set_bounds()
    check_choice(s, 50)
    lists = select(s, 50)
    s.check(s.attend(blocks=torch.from_numpy(lists).cuda(), block=16), blocks=lists)


@pytest.mark.parametrize("lens", [[400], [40000]])
def test_selection_of_equal_scores_takes_the_lowest(lens):
    s = Setup("tiny", BF16, lens, block=16)
    s.lo_hi.copy_(s.lo_hi[:1].nan_to_num(1.0).expand_as(s.lo_hi).clone())
    check_choice(s, 9)  # equal bounds
    s.set_bounds()
    s.q = torch.zeros_like(s.q)
    check_choice(s, 12)  # equal products: 0


def test_selection_tells_scores_apart_that_32_bits_cannot():
    """Scores 2^40 + j: all equal in 32 bits."""
    s = Setup("tiny", BF16, [3200], block=16)
    n = 200
    s.q = torch.zeros_like(s.q)
    s.q[0, 0, 0], s.q[0, 0, 1], s.q[0, 1, 2] = 2.0 ** 20, 1.0, -1.0
    b = torch.zeros(s.total // 16, 1, 2, s.D)
    j = torch.randperm(n, generator=torch.Generator().manual_seed(2)).float()
    b[:n, 0, 1, 0] = 2.0 ** 20
    b[:n, 0, 1, 1] = j           # up to 199: bf16 keeps 8 bits
    b[:n, 0, 0, 2] = -(j % 3)
    s.lo_hi.copy_(b.to(torch.bfloat16).cuda())
    check_choice(s, 20)
    check_choice(s, 21, 0, 0)


@pytest.mark.parametrize("gap", [2.0 ** -10, 2.0 ** -30, 2.0 ** -60, 0.0])
def test_selection_tells_close_scores_apart(gap):
    """Blocks whose scores differ by `gap` of a score of 2^8 or so (0: equal), in falling order of index."""
    s = Setup("tiny", BF16, [1600], block=16)
    s.set_bounds()
    rows = s.lo_hi[:100].clone()
    rows[20:40] = rows[20]
    rows[:, :, :, 60:] = 0
    s.q[0, :, 60:] = 0
    s.q[0, 1, 61] = 1.0
    for i in range(20):  # one more product, too small for 32 bits beside the others
        rows[20 + i, 0, 1, 61] = gap * 2.0 ** 8 * i
    s.lo_hi[:100] = rows
    for n in (5, 17, 30, 60):
        check_choice(s, n, 0, 0)


@pytest.mark.parametrize("blocks", [700, 2049, 20000])
@pytest.mark.parametrize("kind", ["octaves", "outliers", "neighbours", "two values"])
def test_selection_of_scores_of_every_spread(kind, blocks):
    """Scores whose K-th largest needs one step of its search or all of them: one product each, exact in 32 bits."""
    s = Setup("tiny", BF16, [16 * blocks], block=16)
    s.q = torch.zeros_like(s.q)
    s.q[0, 0, 0] = 1.0
    g = torch.Generator().manual_seed(blocks)
    x = torch.randperm(blocks, generator=g).double()
    if kind == "octaves":
        x = torch.where(x % 2 == 0, 1.0, -1.0) * 2.0 ** (x % 201 - 100)
    elif kind == "outliers":
        x = torch.where(x == 0, 2.0 ** 100, torch.where(x == 1, -2.0 ** 100, 1 + (x % 100) / 128))
    elif kind == "neighbours":
        x = (x % 30000 + 0x3000).to(torch.int16).view(torch.bfloat16).double()
    else:
        x = torch.where(x < blocks // 3, 1.0, -1.0)
    n = s.total // 16
    b = torch.zeros(n, 1, 2, s.D, dtype=torch.float64)
    b[:blocks, 0, :, 0] = x[:, None]
    s.lo_hi.copy_(b.to(torch.bfloat16).cuda())
    for k in (1, 2, 50, blocks // 3, blocks // 3 + 1, blocks - 1):
        check_choice(s, k, 0, 0)
    check_choice(s, 50, 3, 2)


def test_selection_with_infinities_and_nans():
    s = Setup("tiny", BF16, [1000], block=16)
    s.set_bounds()
    s.lo_hi[3, 0, 1, 5] = float("inf")
    s.lo_hi[7, 0, 0, 6] = float("nan")
    s.lo_hi[11, 0, 0, 7] = -float("inf")
    check_choice(s, 10)
    check_choice(s, 62)
    s.q[0, 2, 9] = float("nan")
    check_choice(s, 10)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("use_graph", [False, True])
@pytest.mark.parametrize("fmt,page", [(BF16, 0), (TURBO8, 32)])
def test_a_serving_loop(fmt, page, use_graph):
    """Prompts appended, then steps of append, selection and attention (one graph, replayed
    with the positions advanced on the device), each step against the definition on the cache
    as it then is."""
    s = Setup("tiny", fmt, [250, 190, 222], page=page, block=16, seed=4)
    rng = np.random.default_rng(9)
    n_seqs, steps, n = 3, 7, 6
    have = [120, 3, 97]
    keys = [bf16(rng.standard_normal((sum(have), 1, s.D))) for _ in "kv"]
    start = torch.tensor(np.concatenate([[0], np.cumsum(have)]), dtype=torch.int32, device="cuda")
    prompt = B.DeviceRows(torch.zeros(3, dtype=torch.int32, device="cuda"), start, sum(have), s.nb)
    scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(s.cfg, s.cap, 16, sum(have)))
    assert B.qwen35_cache_append(s.cfg, s.kv, prompt, s.bounds, keys[0].cuda(), keys[1].cuda(), scratch) == 0
    hist = [[[x[start[b]:start[b + 1]]] for b in range(3)] for x in [k for k in keys]]
    s.pos.copy_(torch.tensor(have, dtype=torch.int32))
    k, v, q, out = (torch.zeros(n_seqs, h, s.D, dtype=torch.bfloat16, device="cuda") for h in (1, 1, s.H, s.H))
    blocks = torch.zeros(n_seqs, 1, n, dtype=torch.int32, device="cuda")

    def step():
        assert B.qwen35_cache_append(s.cfg, s.kv, s.r, s.bounds, k, v, scratch) == 0
        assert B.qwen35_select_blocks(s.cfg, s.kv, s.r, s.bounds, q, blocks, scratch) == 0
        assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, out, scratch, blocks=blocks, block=16) == 0
        s.pos.add_(1)

    graph = None
    if use_graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for i in range(steps):
        new = [bf16(rng.standard_normal((n_seqs, h, s.D))) for h in (1, 1, s.H)]
        for dst, src in zip((k, v, q), new):
            dst.copy_(src)
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        for x, h in zip(new[:2], hist):
            for b in range(3):
                h[b].append(x[b:b + 1])
        s.lens, s.q = [m + i + 1 for m in have], new[2]
        for name, h in zip("kv", hist):
            for b in range(3):
                rows = f64(torch.cat(h[b]))
                at = s.at(b, np.arange(s.lens[b]))
                if fmt == TURBO8:
                    codes = s.t[name].cpu().numpy()[at]
                    sc = O.bf16_to_f64(s.t[name + "s"].cpu().numpy().view(np.uint16)[at][:, :s.D // 16])
                    rows = O.wht(O.turbo8_dequantize(codes, sc.reshape(len(at), 1, -1)))
                s.stands[name][at] = rows
        got = blocks.cpu().numpy()
        want = np.stack([choose(s, b, b, s.lens[b] - 1, n, 1, 1) for b in range(3)])
        np.testing.assert_array_equal(got, want)
        s.check(out, blocks=got)
    assert B.qwen35_read_device_status(scratch) == 0


def test_two_calls_at_once_with_their_own_scratch():
    a = Setup("4b", BF16, [3000, 2500], page=16, seed=1)
    b = Setup("4b", TURBO8, [2800, 100], page=16, seed=2)
    ref = a.attend(), b.attend()
    qa, qb = a.q.cuda(), b.q.cuda()
    outs = [torch.zeros_like(ref[0]), torch.zeros_like(ref[1])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, o, st in ((a, qa, outs[0], streams[0]), (b, qb, outs[1], streams[1])):
            assert B.qwen35_decode_attention(s.cfg, s.kv, s.r, q, o, s.scratch, stream=st) == 0
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])


def test_the_same_call_gives_the_same_bits():
    s = Setup("4b", BF16, [5000, 70, 900], page=16)
    a = s.attend().clone()
    for _ in range(5):
        assert torch.equal(s.attend(), a)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: the last token's rows lie behind them."""
    init()
    H, Hkv, D = 16, 4, 256
    cfg = B.make_config(synth.config("4b"))
    cap = 1 << 20  # 2 KiB a row and array: 2 sequences pass 2^32 bytes
    k = torch.zeros(2 * cap, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() * 2 >= 1 << 32
    kv = B.qwen35_kv_cache(k.data_ptr(), v.data_ptr(), cap, B.QWEN35_KV_BF16, None, None, None, 0, 0)
    pos = torch.tensor([5, cap - 1], dtype=torch.int32, device="cuda")
    rows = B.DeviceRows(pos)
    lo_hi = torch.zeros(2 * cap // 1024, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    bounds = B.DeviceKeyBounds(lo_hi, 1024)
    scratch = B.new_scratch(B.qwen35_cache_scratch_bytes(cfg, cap, 1024, 2))
    new = [torch.randn(2, Hkv, D, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(torch.bfloat16)
           for i in (1, 2)]
    assert B.qwen35_cache_append(cfg, kv, rows, bounds, *new, scratch) == 0
    torch.cuda.synchronize()
    assert torch.equal(k[-1], new[0][1]) and torch.equal(v[-1], new[1][1])
    assert torch.equal(k[5], new[0][0]) and int((k != 0).flatten(1).any(1).sum()) == 2
    back = [torch.zeros_like(x) for x in new]
    assert B.qwen35_cache_read(cfg, kv, rows, *back, scratch) == 0
    # the last token's key points along q: it takes the weight of a million zero keys' each
    q = (40 * new[0][1].float().repeat_interleave(4, 0)).to(torch.bfloat16)[None].repeat(2, 1, 1)
    blocks = torch.zeros(2, Hkv, 4, dtype=torch.int32, device="cuda")
    out, part = torch.zeros_like(q), torch.zeros_like(q)
    assert B.qwen35_select_blocks(cfg, kv, rows, bounds, q, blocks, scratch) == 0
    assert B.qwen35_decode_attention(cfg, kv, rows, q, out, scratch) == 0
    assert B.qwen35_decode_attention(cfg, kv, rows, q, part, scratch, blocks=blocks, block=1024) == 0
    torch.cuda.synchronize()
    assert torch.equal(back[0], new[0]) and torch.equal(back[1], new[1])
    assert blocks[1].cpu().tolist() == [[0, 1, 2, 1023]] * 4
    want = new[1][1].repeat_interleave(4, 0)
    assert torch.allclose(out[1].float(), want.float(), rtol=2.0 ** -7) and torch.equal(out[1], part[1])
    assert B.qwen35_read_device_status(scratch) == 0
