"""The 4-bit paged cache on the CPU: the plain implementation's own pins, and what the entry points
refuse before they touch a device."""
import ctypes

import numpy as np
import pytest

import random_access_kv_fq_b200 as fq
from random_access_kv_fq_b200 import _lib
from tests import kv4_ref as ref

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@pytest.mark.parametrize("d,group", SHAPES)
def test_a_unit_holds_every_code_step_and_zero_once(d, group):
    seen = np.zeros((ref.unit_bytes(d, group), 2), dtype=int)
    for t in range(16):
        for i in range(d):
            for at in (ref.key_code_at, ref.value_code_at):
                b, high = at(t, i, d)
                seen[b, high] += 1
        for g in range(d // group):
            for at in (ref.key_scale_at, ref.value_scale_at):
                for b in at(t, g, d, group):
                    seen[b:b + 2] += 1
    assert (seen == 1).all()
    assert fq.fq_kv4_unit_bytes(d, group) == ref.unit_bytes(d, group)


@pytest.mark.parametrize("d,group", SHAPES)
def test_reference_write_and_read_agree_and_round_to_the_nearest_code(d, group):
    rng = np.random.default_rng(d + group)
    cache = rng.integers(0, 256, (3, 2, 2, ref.unit_bytes(d, group)), dtype=np.uint8)
    k, v = rng.standard_normal((2, 9, 2, d)).astype(np.float16)
    slots = rng.permutation(96)[:9]
    before = cache.copy()
    ref.write(cache, k, v, slots, group)
    for x, got in zip((k, v), ref.read(cache, slots, d, group)):
        c, s, z = ref.quantise(x, group)
        np.testing.assert_array_equal(got, ref.values(c, s, z, group))
        # half a step, and what the range's end loses to the rounding of s (15 of its half steps)
        step = np.repeat(s.astype(np.float64), group, -1)
        assert (np.abs(got - x) <= step * (0.5 + 15 * 2.0 ** -11 + 1e-6)).all()
    others = np.setdiff1d(np.arange(96), slots)
    for a, b in zip(ref.read(cache, others, d, group), ref.read(before, others, d, group)):
        np.testing.assert_array_equal(a, b)


def test_reference_page_step_by_hand():
    tables = np.array([[4, -1, -1], [7, 1, -1], [2, -1, -1]])
    free = np.array([0, 3, 5, -9, -9, -9, -9, -9])
    # request 0 grows from 15 to 33 tokens (two pages), 1 ends (two pages back), 2 adds one to 16
    out = ref.page_step([15, 17, 16], [18, -1, 1], tables, free, 3, 16, 20)
    assert free.tolist() == [0, 3, 5, 7, 1, -9, -9, -9]
    assert tables.tolist() == [[4, 1, 7], [7, 1, -1], [2, 5, -1]]
    lens, cu, slots, refused, count = out
    assert lens.tolist() == [33, 0, 17] and cu.tolist() == [0, 18, 18, 19] and refused == 0 and count == 2
    assert slots.tolist() == [4 * 16 + 15] + list(range(16, 32)) + [7 * 16] + [5 * 16] + [-1]


BASE = 4096  # a fake aligned device address: every call below is refused before it is used


def _write_args(**kw):
    a = dict(k=BASE, v=BASE, type=0, n=4, hkv=2, d=64, kt=128, kh=64, vt=128, vh=64, slots=BASE, cache=BASE,
             n_blocks=8, page=16, group=32, kv=None, vv=None, stream=None)
    a.update(kw)
    return list(a.values())


def _attn_args(**kw):
    a = dict(q=BASE, type=0, n_q=3, hq=8, d=64, qt=512, qh=64, cu=None, B=3, max_q=1, cache=BASE, n_blocks=8, hkv=2,
             page=16, group=32, tables=BASE, mb=4096, lens=BASE, window=0, scale=ctypes.c_float(0.1), out=BASE, ws=BASE,
             ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


def _page_args(**kw):
    a = dict(lens=BASE, new=BASE, B=3, tables=BASE, mb=4, page=16, free=BASE, nb=8, count=BASE, lens_out=BASE,
             count_out=BASE, cu=BASE, slots=BASE, n_slots=5, refused=BASE, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("edit,status", [
    (dict(d=96), 2), (dict(d=0), 2), (dict(group=16), 2), (dict(group=128), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=2048), 2), (dict(n_blocks=1 << 27), 2), (dict(n=1 << 31), 2), (dict(n=-1), 1), (dict(hkv=0), 1),
    (dict(type=3), 1), (dict(n_blocks=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(cache=None), 1), (dict(k=BASE + 1), 3), (dict(type=1, v=BASE + 2), 3), (dict(slots=BASE + 2), 3),
    (dict(cache=BASE + 8), 3), (dict(kv=BASE + 8), 3), (dict(vv=BASE + 2), 3), (dict(n=0, k=None, v=None, slots=None), 0)])
def test_write_refuses(edit, status):
    assert _lib.lib().fq_kv4_write(*_write_args(**edit)) == status


@pytest.mark.parametrize("edit,status", [
    (dict(d=80), 2), (dict(group=48), 2), (dict(page=24), 2), (dict(mb=1 << 27), 2), (dict(n_blocks=1 << 28), 2),
    (dict(B=8193, n_q=8193), 2), (dict(cu=BASE, n_q=1 << 28), 2), (dict(cu=BASE, max_q=1 << 28), 2), (dict(hq=7), 1), (dict(hq=0), 1), (dict(hkv=0), 1),
    (dict(B=-1, n_q=-1), 1), (dict(n_q=4), 1), (dict(max_q=2), 1), (dict(cu=BASE, max_q=-1), 1), (dict(window=-1), 1),
    (dict(type=1), 1), (dict(scale=ctypes.c_float(float("nan"))), 1), (dict(scale=ctypes.c_float(float("inf"))), 1),
    (dict(mb=-1), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(cache=None), 1),
    (dict(tables=None), 1), (dict(q=BASE + 1), 3), (dict(out=BASE + 8), 3), (dict(cache=BASE + 4), 3),
    (dict(cu=BASE + 2), 3), (dict(tables=BASE + 1), 3), (dict(lens=BASE + 2), 3), (dict(ws=None), 4),
    (dict(ws_bytes=0), 4), (dict(ws=BASE + 8), 3), (dict(B=0, n_q=0, q=None, out=None, ws=None), 0),
    (dict(cu=BASE, n_q=0, q=None), 0), (dict(cu=BASE, max_q=0), 0)])
def test_attention_refuses(edit, status):
    assert _lib.lib().fq_kv4_attn(*_attn_args(**edit)) == status


@pytest.mark.parametrize("edit,status", [
    (dict(B=-1), 1), (dict(B=8193), 2), (dict(mb=0), 1), (dict(page=4), 2), (dict(page=17), 2), (dict(mb=1 << 27), 2),
    (dict(nb=-1), 1), (dict(nb=1 << 27), 2), (dict(n_slots=-1), 1), (dict(n_slots=(1 << 30) + 1), 2), (dict(lens=None), 1),
    (dict(new=None), 1), (dict(tables=None), 1), (dict(free=None), 1), (dict(count=None), 1), (dict(lens_out=None), 1),
    (dict(count_out=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(refused=None), 1), (dict(slots=BASE + 2), 3),
    (dict(tables=BASE + 1), 3), (dict(count=BASE + 3), 3)])
def test_page_step_refuses(edit, status):
    assert _lib.lib().fq_page_step(*_page_args(**edit)) == status


def test_sizes():
    assert fq.fq_kv4_unit_bytes(96, 32) == 0 and fq.fq_kv4_unit_bytes(64, 128) == 0 and fq.fq_kv4_unit_bytes(128, 0) == 0
    ws = fq.fq_kv4_attn_workspace_bytes
    assert ws(64, 8, 1, 64, 1, 2048, 16) > 0 and ws(1, 32, 8, 128, 1, 2048, 16) > 0
    assert ws(8, 32, 8, 128, 64, 16, 16) > ws(64, 32, 8, 128, 1, 16, 16) > 0
    assert ws(1, 32, 8, 128, 1, 16, 16) == 0  # nothing is split
    for bad in ((4, 8, 1, 80, 1, 4, 16), (4, 7, 2, 64, 1, 4, 16), (4, 8, 0, 64, 1, 4, 16), (4, 8, 1, 64, -1, 4, 16), (4, 8, 1, 64, 1, 4, 20)):
        assert ws(*bad) == 0


def test_binding_refuses_what_is_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(2, 2, 1, ref.unit_bytes(64, 32), dtype=torch.uint8)
    with pytest.raises(ValueError):
        fq.fq_kv4_write(x, x, i, cache, 32)
    with pytest.raises(ValueError):
        fq.fq_kv4_attn(x, cache, i[:, None], i, 32)
    with pytest.raises(ValueError):
        fq.fq_page_step(i, i, i[:, None], i, i[:1], 16, 4)
