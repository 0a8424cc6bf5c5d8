"""The cache operators on the host: the C ABI's refusals, each before anything is
enqueued (fake, never dereferenced addresses, so only where no CUDA device is
present), and the scratch sizes."""

import pytest
import torch

from full_attention_decode_gb300 import binding as B
from full_attention_decode_gb300 import synth

OK_BUT_NO_DEVICE = B.QWEN35_ERR_CUDA  # past every check, then no device
BAD, UNSUPPORTED = B.QWEN35_ERR_INVALID_ARGUMENT, B.QWEN35_ERR_UNSUPPORTED

no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: run without a GPU")


class _Fake:
    def __init__(self, ptr, n=0, shape=()):
        self.ptr, self.n, self.shape = ptr, n, shape

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.n


def _cfg(**kw):
    return B.make_config(synth.config("tiny") | kw)


def _kv(**kw):
    a = dict(k=0x5000000, v=0x6000000, capacity=256, dtype=B.QWEN35_KV_BF16, k_scales=None, v_scales=None,
             block_table=None, block_tokens=0, reserved=0)
    a.update(kw)
    return B.qwen35_kv_cache(*a.values())


def _rows(n_seqs=3, n_rows=3, row_start=None, pos=0x7000000, num_blocks=0):
    r = B.DeviceRows(_Fake(pos, n_seqs), _Fake(row_start, n_seqs + 1) if row_start else None, n_rows, num_blocks)
    return r


def _calls(cfg, kv, rows, bounds=None, scratch=None, **kw):
    """Every operator's status for the same cache and rows."""
    scr = scratch or _Fake(0x9000000, 1 << 30)
    bounds = bounds or B.DeviceKeyBounds(_Fake(0xA000000), 16)
    x, y = _Fake(0xB000000), _Fake(0xC000000)
    sel = _Fake(0xD000000, shape=(3, 1, 4))
    return [B.qwen35_cache_append(cfg, kv, rows, bounds, x, y, scr, stream=0),
            B.qwen35_cache_read(cfg, kv, rows, x, y, scr, stream=0),
            B.qwen35_select_blocks(cfg, kv, rows, bounds, x, sel, scr, stream=0),
            B.qwen35_decode_attention(cfg, kv, rows, x, y, scr, blocks=sel, block=16, stream=0)]


T8 = dict(dtype=B.QWEN35_KV_TURBO8, k_scales=0xE000000, v_scales=0xF000000)
PAGED = dict(block_table=0x11000000, block_tokens=16)


@no_device
@pytest.mark.parametrize("kv,rows", [({}, {}), (T8, {}), (PAGED, dict(num_blocks=40)),
                                     (T8 | PAGED, dict(num_blocks=1)), ({}, dict(n_rows=9, row_start=0x7100000))])
def test_well_formed_calls_pass_every_check(kv, rows):
    assert _calls(_cfg(), _kv(**kv), _rows(**rows)) == [OK_BUT_NO_DEVICE] * 4


@no_device
@pytest.mark.parametrize("kv", [dict(k=None), dict(v=0x6000008), dict(capacity=0), dict(dtype=2),
                                dict(dtype=B.QWEN35_KV_TURBO8), T8 | dict(v_scales=0xF000004),
                                dict(block_table=0x11000002, block_tokens=16), dict(PAGED, block_tokens=4),
                                dict(PAGED, block_tokens=24), dict(PAGED, block_tokens=512),
                                dict(PAGED, capacity=264), dict(capacity=0x80000010)])
def test_bad_caches(kv):
    assert _calls(_cfg(), _kv(**kv), _rows(num_blocks=40)) == [BAD] * 4


@no_device
def test_a_paged_cache_needs_the_size_of_its_pool():
    assert _calls(_cfg(), _kv(**PAGED), _rows(num_blocks=0)) == [BAD] * 4


@no_device
@pytest.mark.parametrize("rows", [dict(n_seqs=0, n_rows=0), dict(pos=None), dict(pos=0x7000002), dict(n_rows=4),
                                  dict(n_rows=0, row_start=0x7100000), dict(n_rows=4, row_start=0x7100002)])
def test_bad_rows(rows):
    r = _rows(**rows)
    assert _calls(_cfg(), _kv(), r) == [BAD] * 4


@no_device
def test_row_limits():
    many = _rows(n_seqs=3, n_rows=2049, row_start=0x7100000)
    assert _calls(_cfg(), _kv(), many) == [OK_BUT_NO_DEVICE] * 2 + [UNSUPPORTED] * 2
    many = _rows(n_seqs=3, n_rows=(1 << 20) + 1, row_start=0x7100000)
    assert _calls(_cfg(), _kv(), many) == [UNSUPPORTED] * 4
    assert _calls(_cfg(), _kv(), _rows(n_seqs=4097, n_rows=4097)) == [UNSUPPORTED] * 4


@no_device
@pytest.mark.parametrize("cfg,status", [(dict(num_heads=0), BAD), (dict(num_kv_heads=0), BAD),
                                        (dict(num_heads=3, num_kv_heads=2), BAD), (dict(head_dim=96), UNSUPPORTED),
                                        (dict(head_dim=32), UNSUPPORTED), (dict(num_heads=17), UNSUPPORTED),
                                        (dict(num_heads=9, num_kv_heads=9), UNSUPPORTED)])
def test_bad_dims(cfg, status):
    c = _cfg(**cfg)
    assert _calls(c, _kv(), _rows()) == [status] * 4
    assert B.qwen35_cache_scratch_bytes(c, 256, 16, 3) == 0


@no_device
@pytest.mark.parametrize("block", [0, 8, 24, 2048])
def test_bad_selection_blocks(block):
    b = B.DeviceKeyBounds(_Fake(0xA000000), block)
    x, scr = _Fake(0xB000000), _Fake(0x9000000, 1 << 30)
    assert _calls(_cfg(), _kv(capacity=4096), _rows(), bounds=b)[::2] == [BAD] * 2
    assert B.qwen35_decode_attention(_cfg(), _kv(capacity=4096), _rows(), x, x, scr,
                                     blocks=_Fake(0xD000000, shape=(3, 1, 1)), block=block, stream=0) == BAD


@no_device
def test_selection_blocks_divide_capacity_and_pages():
    b = B.DeviceKeyBounds(_Fake(0xA000000), 64)
    assert _calls(_cfg(), _kv(capacity=96), _rows(), bounds=b)[::2] == [BAD] * 2
    assert _calls(_cfg(), _kv(**PAGED), _rows(num_blocks=9), bounds=b)[::2] == [BAD] * 2
    assert _calls(_cfg(), _kv(), _rows(), bounds=B.DeviceKeyBounds(_Fake(0xA000008), 16))[::2] == [BAD] * 2


@no_device
def test_selection_and_attention_arguments():
    cfg, kv, rows, scr = _cfg(), _kv(), _rows(), _Fake(0x9000000, 1 << 30)
    b, x, y = B.DeviceKeyBounds(_Fake(0xA000000), 16), _Fake(0xB000000), _Fake(0xC000000)

    def select(n, **kw):
        a = dict(q=x, blocks=_Fake(0xD000000, shape=(3, 1, n)), scratch=scr) | kw
        return B.qwen35_select_blocks(cfg, kv, rows, b, a["q"], a["blocks"], a["scratch"], stream=0)

    assert select(16) == OK_BUT_NO_DEVICE and select(17) == OK_BUT_NO_DEVICE  # more than the 256 / 16 blocks there are
    assert select(0) == BAD and select(65536) == OK_BUT_NO_DEVICE and select(65537) == UNSUPPORTED
    assert select(4, q=_Fake(0xB000002)) == BAD and select(4, blocks=_Fake(0xD000002, shape=(3, 1, 4))) == BAD
    need = B.qwen35_cache_scratch_bytes(cfg, 1 << 20, 16, 3)  # the scores of 65536 blocks
    kv.capacity = 1 << 20
    assert select(4, scratch=_Fake(0x9000000, need)) == OK_BUT_NO_DEVICE
    assert select(4, scratch=_Fake(0x9000000, need - 256)) == BAD
    kv.capacity = 256

    def attend(**kw):
        return B.qwen35_decode_attention(cfg, kv, rows, kw.pop("q", x), kw.pop("out", y), kw.pop("scratch", scr),
                                         stream=0, **kw)

    assert attend() == OK_BUT_NO_DEVICE
    assert attend(gate=x) == OK_BUT_NO_DEVICE and attend(gate=x, gate_stride=128) == OK_BUT_NO_DEVICE
    assert attend(gate=x, gate_stride=60) == BAD and attend(gate=x, gate_stride=68) == BAD
    assert attend(gate=_Fake(0xB000008)) == BAD
    assert attend(q=_Fake(0xB000008)) == BAD and attend(out=_Fake(None)) == BAD
    assert attend(blocks=_Fake(0xD000000, shape=(3, 1, 17)), block=16) == OK_BUT_NO_DEVICE
    assert attend(blocks=_Fake(0xD000000, shape=(3, 1, 65537)), block=16) == UNSUPPORTED
    assert attend(blocks=_Fake(0xD000000, shape=(3, 1, 0)), block=16) == BAD
    assert attend(blocks=_Fake(0xD000002, shape=(3, 1, 4)), block=16) == BAD
    need = B.qwen35_cache_scratch_bytes(cfg, 256, 0, 3)
    assert attend(scratch=_Fake(0x9000000, need)) == OK_BUT_NO_DEVICE
    assert attend(scratch=_Fake(0x9000008, need)) == BAD and attend(scratch=_Fake(0x9000000, need - 1)) == BAD


@no_device
def test_attention_tile_limit():
    """16-token tiles of all rows and kv-heads: below 2^31."""
    cfg, scr, x = _cfg(num_heads=8, num_kv_heads=8), _Fake(0x9000000, 1 << 40), _Fake(0xB000000)
    for rows, status in ((2, OK_BUT_NO_DEVICE), (3, UNSUPPORTED)):
        r = _rows(n_seqs=rows, n_rows=rows)
        assert B.qwen35_decode_attention(cfg, _kv(capacity=(1 << 31) - 16), r, x, x, scr, stream=0) == status
        few = _Fake(0xD000000, shape=(rows, 8, 100))
        assert B.qwen35_decode_attention(cfg, _kv(capacity=(1 << 31) - 16), r, x, x, scr, blocks=few, block=16,
                                         stream=0) == OK_BUT_NO_DEVICE


@no_device
def test_append_and_read_pointers():
    cfg, kv, rows, scr, x = _cfg(), _kv(), _rows(), _Fake(0x9000000, 256), _Fake(0xB000000)
    assert B.qwen35_cache_append(cfg, kv, rows, None, x, x, scr, stream=0) == OK_BUT_NO_DEVICE
    for f in (lambda k, v: B.qwen35_cache_append(cfg, kv, rows, None, k, v, scr, stream=0),
              lambda k, v: B.qwen35_cache_read(cfg, kv, rows, k, v, scr, stream=0)):
        assert f(_Fake(0xB000008), x) == BAD and f(x, _Fake(None)) == BAD


def test_scratch_sizes():
    c = _cfg()
    small, large = B.qwen35_cache_scratch_bytes(c, 256, 16, 1), B.qwen35_cache_scratch_bytes(c, 1 << 17, 16, 64)
    assert 256 < small < large
    assert B.qwen35_cache_scratch_bytes(c, 1 << 17, 0, 64) < large  # no selection
    assert B.qwen35_cache_scratch_bytes(c, 4096, 24, 64) == 0
    assert B.qwen35_cache_scratch_bytes(c, 4096, 16, 0) == 0 and B.qwen35_cache_scratch_bytes(c, 0, 16, 1) == 0


def test_rows_with_a_row_start_need_their_count():
    with pytest.raises(ValueError):
        B.DeviceRows(torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))


def test_struct_layouts_match_the_c_compiler(tmp_path):
    import ctypes as C
    import subprocess

    from test_abi import HEADER
    structs = {"qwen35_cache_rows": B.qwen35_cache_rows, "qwen35_key_bounds": B.qwen35_key_bounds}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for s, cls in structs.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for s, cls in structs.items():
        assert int(got[s]) == C.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{s}.{f}"]) == getattr(cls, f).offset, (s, f)
