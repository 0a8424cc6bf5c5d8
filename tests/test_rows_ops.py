"""The operators of a drafting loop on the host: the C ABI's refusals, each before anything is
enqueued (fake, never dereferenced addresses, so only where no CUDA device is present), and the
scratch sizes."""

import pytest
import torch

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth

from test_cache_ops import BAD, OK_BUT_NO_DEVICE, PAGED, T8, UNSUPPORTED, _cfg, _Fake, _kv, _rows, no_device

X, Y, Z, W = _Fake(0xB000000), _Fake(0xC000000), _Fake(0xD000000), _Fake(0xE000000)


def _calls(cfg, kv, rows, scratch=None):
    s = scratch or _Fake(0x9000000, 1 << 40)
    return [B.qwen35_cache_append_rope(cfg, kv, rows, X, Y, Z, W, s, stream=0),
            B.qwen35_cache_keep(cfg, kv, rows, X, s, stream=0),
            B.qwen35_tree_attention(cfg, kv, rows, X, Y, Z, s, stream=0),
            B.qwen35_window_attention(cfg, kv, rows, 10, 4, Y, Z, s, stream=0)]


@no_device
@pytest.mark.parametrize("kv,rows", [({}, {}), (T8, {}), (PAGED, dict(num_blocks=40)), (T8 | PAGED, dict(num_blocks=1)),
                                     ({}, dict(n_rows=9, row_start=0x7100000))])
def test_well_formed_calls_pass_every_check(kv, rows):
    assert _calls(_cfg(), _kv(**kv), _rows(**rows)) == [OK_BUT_NO_DEVICE] * 4


@no_device
@pytest.mark.parametrize("kv", [dict(k=None), dict(v=0x6000008), dict(capacity=0), dict(dtype=2), dict(PAGED, block_tokens=4),
                                dict(PAGED, capacity=264), dict(capacity=0x80000010)])
def test_bad_caches(kv):
    assert _calls(_cfg(), _kv(**kv), _rows(num_blocks=40)) == [BAD] * 4


@no_device
@pytest.mark.parametrize("rows", [dict(n_seqs=0, n_rows=0), dict(pos=None), dict(n_rows=4)])
def test_bad_rows(rows):
    assert _calls(_cfg(), _kv(), _rows(**rows)) == [BAD] * 4


@no_device
def test_limits():
    many = _rows(n_seqs=3, n_rows=2049, row_start=0x7100000)
    assert _calls(_cfg(), _kv(), many) == [OK_BUT_NO_DEVICE] * 2 + [UNSUPPORTED] * 2
    long = _kv(capacity=1 << 31)
    wide = _rows(n_seqs=3, n_rows=17, row_start=0x7100000)
    assert _calls(_cfg(), long, wide)[2:] == [UNSUPPORTED, OK_BUT_NO_DEVICE]
    s = _Fake(0x9000000, 1 << 40)
    assert B.qwen35_window_attention(_cfg(), long, wide, (1 << 32) - 1, 0, Y, Z, s, stream=0) == UNSUPPORTED


@no_device
@pytest.mark.parametrize("cfg,status", [(dict(num_heads=0), BAD), (dict(head_dim=96), UNSUPPORTED),
                                        (dict(num_heads=17), UNSUPPORTED), (dict(num_heads=9, num_kv_heads=9), UNSUPPORTED)])
def test_bad_dims(cfg, status):
    c = _cfg(**cfg)
    assert _calls(c, _kv(), _rows()) == [status] * 4
    assert B.qwen35_rows_scratch_bytes(c, 3) == 0


@no_device
def test_scratch():
    c = _cfg()
    need = B.qwen35_rows_scratch_bytes(c, 3)
    assert _calls(c, _kv(), _rows(), _Fake(0x9000000, need)) == [OK_BUT_NO_DEVICE] * 4
    assert _calls(c, _kv(), _rows(), _Fake(0x9000000, need - 1)) == [OK_BUT_NO_DEVICE] * 2 + [BAD] * 2
    assert _calls(c, _kv(), _rows(), _Fake(0x9000000, 255)) == [BAD] * 4
    assert _calls(c, _kv(), _rows(), _Fake(0x9000008, 1 << 40)) == [BAD] * 4


def test_scratch_sizes():
    c = B.make_config(synth.config("4b"))
    sizes = [B.qwen35_rows_scratch_bytes(c, n) for n in (1, 8, 64, 2048)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert B.qwen35_rows_scratch_bytes(c, 1 << 20) == sizes[-1]
    assert B.qwen35_rows_scratch_bytes(c, 0) == 0 == B.qwen35_rows_scratch_bytes(c, (1 << 20) + 1)


@no_device
@pytest.mark.parametrize("cfg,status", [(dict(rotary_dim=66), UNSUPPORTED), (dict(rotary_dim=15), UNSUPPORTED),
                                        (dict(rope_theta=0.0), BAD), (dict(rope_theta=float("nan")), BAD),
                                        (dict(rms_eps=-1.0), BAD), (dict(rotary_dim=0), OK_BUT_NO_DEVICE)])
def test_rotation(cfg, status):
    assert _calls(_cfg(**cfg), _kv(), _rows()) == [status] + [OK_BUT_NO_DEVICE] * 3


@no_device
def test_rotated_append():
    s, odd, b = _Fake(0x9000000, 1 << 20), _Fake(0xB000008), B.DeviceKeyBounds(_Fake(0xA000000), 16)

    def call(q=X, k=Y, v=Z, out=W, **kw):
        return B.qwen35_cache_append_rope(_cfg(), _kv(), _rows(), q, k, v, out, s, stream=0, **kw)

    assert call() == call(q=None, out=None) == call(q_stride=128) == call(q=X, out=X) == OK_BUT_NO_DEVICE
    assert call(bounds=b, k_out=Y) == call(k_out=_Fake(0xF000000)) == OK_BUT_NO_DEVICE
    for bad in (dict(q=odd), dict(k=None), dict(k=odd), dict(v=None), dict(out=None), dict(q_stride=60), dict(q_stride=56),
                dict(q_norm=odd), dict(k_norm=odd), dict(k_out=odd), dict(rope_pos=_Fake(0xB000002)), dict(bounds=b),
                dict(out=X, q_stride=128), dict(bounds=B.DeviceKeyBounds(_Fake(0xA000000), 24), k_out=Y)):
        assert call(**bad) == BAD, bad


@no_device
def test_attention_arguments():
    s, odd = _Fake(0x9000000, 1 << 40), _Fake(0xB000008)
    for q, out, gate, stride in ((odd, Y, None, 0), (X, odd, None, 0), (None, Y, None, 0), (X, Y, odd, 0), (X, Y, Z, 63),
                                 (X, Y, Z, 68)):
        assert B.qwen35_tree_attention(_cfg(), _kv(), _rows(), W, q, out, s, gate=gate, gate_stride=stride, stream=0) == BAD
        assert B.qwen35_window_attention(_cfg(), _kv(), _rows(), 5, 0, q, out, s, gate=gate, gate_stride=stride,
                                         stream=0) == BAD
    assert B.qwen35_tree_attention(_cfg(), _kv(), _rows(), None, X, Y, s, stream=0) == BAD
    assert B.qwen35_tree_attention(_cfg(), _kv(), _rows(), _Fake(0xB000002), X, Y, s, stream=0) == BAD
    assert B.qwen35_window_attention(_cfg(), _kv(), _rows(), 0, 4, X, Y, s, stream=0) == BAD
    assert B.qwen35_cache_keep(_cfg(), _kv(), _rows(), None, s, stream=0) == BAD
    assert B.qwen35_cache_keep(_cfg(), _kv(), _rows(), _Fake(0xB000002), s, stream=0) == BAD


class _Logits(_Fake):
    def stride(self, _):
        return self.n


@no_device
def test_sample_arguments():
    def call(ptr=0xB000000, n=3, vocab=500, stride=500, u=Y, token=Z, **kw):
        return B.qwen35_sample(_Logits(ptr, stride, (n, vocab)), u, token, stream=0, **kw)

    assert call() == call(stride=513) == call(vocab=1, stride=1) == OK_BUT_NO_DEVICE
    assert call(temperature=X, top_k=X, top_p=X, min_p=X, prob=X) == OK_BUT_NO_DEVICE
    assert call(vocab=524160, n=65536) == OK_BUT_NO_DEVICE
    odd = _Fake(0xB000002)
    for bad in (dict(ptr=0xB000008), dict(ptr=None), dict(n=0), dict(vocab=0), dict(u=None), dict(token=None),
                dict(u=odd), dict(token=odd), dict(temperature=odd), dict(top_k=odd), dict(top_p=odd), dict(min_p=odd),
                dict(prob=odd)):
        assert call(**bad) == BAD, bad
    assert B.lib().qwen35_sample(0xB000000, 3, 500, 499, 0xC000000, None, None, None, None, 0xD000000, None, 0) == BAD
    assert call(vocab=524161) == UNSUPPORTED
    assert call(n=65537) == UNSUPPORTED


def _called_with(monkeypatch, logits):
    """(n_rows, vocab, row_stride) that the binding hands to the C entry, which is not called."""
    got = []

    class _Lib:
        @staticmethod
        def qwen35_sample(ptr, n_rows, vocab, row_stride, *_):
            got.append((n_rows, vocab, row_stride))
            return 0

    monkeypatch.setattr(B, "lib", lambda: _Lib)
    assert B.qwen35_sample(logits, Y, Z, stream=0) == 0
    return got[0]


def test_sample_takes_logits_as_they_lie(monkeypatch):
    """Every element that the C entry reads, row r's at r * row_stride + [0, vocab), is one of the tensor's rows."""
    base = torch.arange(6000, dtype=torch.float32)
    for x in (base[:1000], base[:1000].expand(4, -1), base[:1].expand(3, 1), base[:6000].view(6, 1000), base.view(6, 1000)[::2],
              base.view(6, 1000)[:, 8:900], base.view(6, 1000)[2:3], base.view(1000, 6)[:, :1], base[:1000].view(1, 1000).expand(5, -1),
              base[16:].as_strided((5, 1000), (1008, 1)), base.view(1000, 6)[:4, :1], base[:6].view(6, 1).expand(6, 1)):
        n, vocab, stride = _called_with(monkeypatch, x)
        rows = x.view(1, -1) if x.dim() == 1 else x
        assert (n, vocab) == tuple(rows.shape)
        for r in range(n):
            i = x.storage_offset() + r * stride
            assert torch.equal(base[i:i + vocab], rows[r])


@pytest.mark.parametrize("x", [torch.zeros(1000, 4).t(), torch.zeros(2000)[::2], torch.zeros(4, 2000)[:, ::2],
                               torch.zeros(1).expand(4, 1000), torch.zeros(2, 3, 1000), torch.zeros(())])
def test_sample_refuses_logits_that_no_stride_describes(x):
    with pytest.raises(ValueError):
        B.qwen35_sample(x, Y, Z, stream=0)


@no_device
def test_sample_strides():
    """0: one row for all; rows that overlap otherwise are refused."""
    def call(n, stride):
        return B.lib().qwen35_sample(0xB000000, n, 500, stride, 0xC000000, None, None, None, None, 0xD000000, None, 0)

    assert call(3, 0) == call(1, 0) == call(3, 500) == call(3, 501) == OK_BUT_NO_DEVICE
    assert call(3, 1) == call(3, 499) == call(1, 499) == BAD
    x = torch.zeros(1000).as_strided((3, 500), (250, 1))
    assert B.qwen35_sample(x, Y, Z, stream=0) == BAD


@pytest.mark.parametrize("name", ["u", "token", "temperature", "top_k", "top_p", "min_p", "prob"])
def test_sample_refuses_settings_that_do_not_lie_side_by_side(monkeypatch, name):
    """One value expanded to all rows, every other value of a tensor, too few values: the C entry reads n_rows side by side."""
    class _Lib:
        qwen35_sample = staticmethod(lambda *_: 0)

    monkeypatch.setattr(B, "lib", lambda: _Lib)

    def call(t):
        a = dict(u=torch.zeros(4), token=torch.zeros(4, dtype=torch.int32))
        a[name] = t
        return B.qwen35_sample(torch.zeros(4, 100), a.pop("u"), a.pop("token"), stream=0, **a)

    one = torch.zeros(1, dtype=torch.int32 if name in ("token", "top_k") else torch.float32)
    for bad in (one.expand(4), one, one.expand(8)[:4], torch.zeros(8)[::2], torch.zeros(4, 3)[:, 0], torch.zeros(3)):
        with pytest.raises(ValueError):
            call(bad)
    assert call(torch.zeros(4)) == call(torch.zeros(9)[2:7]) == call(torch.zeros(4, 1)) == 0
    assert B.qwen35_sample(torch.zeros(100), one.float(), one.int(), stream=0) == 0


@no_device
@pytest.mark.parametrize("bad", [torch.zeros(1, 3, dtype=torch.int32).expand(3, -1), torch.zeros(18, dtype=torch.int32)[::2],
                                 torch.zeros(8, dtype=torch.int32)])
def test_a_value_a_row_lies_side_by_side(bad):
    """Parents, paths and positions of nine rows: one tree expanded to three sequences, every other value, too few."""
    s, rows = _Fake(0x9000000, 1 << 40), _rows(n_rows=9, row_start=0x7100000)
    for call in (lambda t: B.qwen35_tree_attention(_cfg(), _kv(), rows, t, Y, Z, s, stream=0),
                 lambda t: B.qwen35_cache_keep(_cfg(), _kv(), rows, t, s, stream=0),
                 lambda t: B.qwen35_cache_append_rope(_cfg(), _kv(), rows, X, Y, Z, W, s, rope_pos=t, stream=0)):
        with pytest.raises(ValueError):
            call(bad)
        assert call(torch.zeros(3, 3, dtype=torch.int32)) == call(W) == OK_BUT_NO_DEVICE
