"""The 4-bit paged cache on the GPU where its inputs are at their limits: values that are not numbers,
weights far below the largest, counts and windows outside what a batch holds.  Bounds as in test_gpu_kv4."""
import numpy as np
import pytest
import torch

import random_access_kv_fq_b200 as fq
from tests import kv4_ref as ref
from tests.test_gpu_kv4 import SHAPES, Cache, _check_attn, _cpu, _dev, _q

pytestmark = pytest.mark.gpu


def _scale_bytes(d, group):
    """First bytes of every step and zero of a unit."""
    return sorted(b for at in (ref.key_scale_at, ref.value_scale_at) for t in range(16) for g in range(d // group)
                  for b in at(t, g, d, group))


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_a_nan_makes_its_group_nan_and_leaves_the_others_alone(d, group, dtype):
    rng = np.random.default_rng(d + group)
    n, hkv = 12, 2
    x = rng.standard_normal((2, n, hkv, d)).astype(np.float32)
    x[0, 1, 0, 3] = x[0, 2, 1, d - 1] = x[1, 3, 0, group - 1] = np.nan   # one coordinate
    x[0, 4], x[1, 4, 1, :group] = np.nan, np.nan                           # whole groups
    x[0, 5, 0, 9], x[1, 6, 1, 2], x[0, 7, 1] = np.inf, -np.inf, -np.inf
    x[1, 8, 0, :2] = np.inf, np.nan
    k, v = (torch.from_numpy(a).to(dtype) for a in x)
    cache = rng.integers(0, 256, (1, hkv, 1, ref.unit_bytes(d, group)), dtype=np.uint8)
    slots = rng.permutation(16)[:n].astype(np.int32)
    got = _dev(cache)
    values = fq.fq_kv4_write(k.cuda(), v.cuda(), _dev(slots), got, group, values=True)
    got = _cpu(got)
    with np.errstate(invalid="ignore"):
        ref.write(cache, k.float().numpy(), v.float().numpy(), slots, group)
    at = _scale_bytes(d, group)
    codes = np.setdiff1d(np.arange(cache.shape[-1]), np.concatenate([at, np.array(at) + 1]))
    np.testing.assert_array_equal(got[..., codes], cache[..., codes])
    halves = lambda c: np.ascontiguousarray(c[..., 16 * d:]).view(np.float16)  # noqa: E731
    np.testing.assert_array_equal(halves(got), halves(cache))                  # a NaN equals a NaN
    for a, b in zip((k, v), values):
        with np.errstate(invalid="ignore", over="ignore"):
            want = torch.from_numpy(ref.values(*ref.quantise(a.float().numpy(), group), group).astype(np.float32)).to(dtype)
        torch.testing.assert_close(b.cpu(), want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("hq", [4, 66])  # rows of a kv head: few, and more than 64
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_key_that_is_not_a_number_reaches_only_the_rows_that_see_it(hq, dtype):
    rng = np.random.default_rng(hq)
    c = Cache(rng, [35, 20], 1, 64, 32, 16)
    want, A, S = ref.attend(_cpu(_q(np.random.default_rng(1), 4, hq, 64, dtype).double()), c.host, c.tables, c.lens, 32, [0, 2, 4])
    q, pool = _q(np.random.default_rng(1), 4, hq, 64, dtype), _dev(c.host)
    key = torch.full((1, 1, 64), float("nan"), dtype=dtype, device="cuda")
    slot = int(c.tables[0, 34 // 16]) * 16 + 34 % 16  # the last token of sequence 0: its first query token does not see it
    fq.fq_kv4_write(key, torch.ones_like(key), _dev(np.array([slot], dtype=np.int32)), pool, 32)
    out = fq.fq_kv4_attn(q, pool, _dev(c.tables), _dev(c.lens), 32, cu_q=_dev(np.array([0, 2, 4], dtype=np.int32)), max_q=2)
    assert torch.isnan(out[1]).all()
    for i in (0, 2, 3):
        _check_attn(out[i], want[i], A[i], S[i], 64, dtype, rows=2 * hq)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("B,hq,hkv", [(296, 8, 8), (148, 66, 1)])  # a warp, and a block of the other kernel, to an item
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_small_weights_beside_a_large_one_are_not_lost(B, hq, hkv, dtype):
    """One token of weight 1 and 131,071 of 2^-25.5: together they move the result by 2^-8.5.  Weights are
    fp16 numbers of at least 2^7 for the largest: each is off by at most 2^-25 or 2^-32 of the largest.  Sums
    of weights and of weighted values take n / 16 additions of 2^-24 each."""
    d, group, page, n = 64, 64, 64, 1 << 17
    k, v = np.zeros((2, 2 * page, hkv, d), dtype=np.float32)
    v[:] = np.linspace(0.5, 1.5, d)
    k[page + 5, :, 0] = 25.5 * np.log(2)  # the large one, of value 0, in page 1; every token of page 0 is alike
    v[page + 5] = 0
    host = np.zeros((2, hkv, page // 16, ref.unit_bytes(d, group)), dtype=np.uint8)
    ref.write(host, k, v, np.arange(2 * page), group)
    kq, vq = ref.read(host, np.array([0, page + 5]), d, group)
    tables = np.zeros((B, n // page), dtype=np.int32)
    tables[np.arange(B), np.linspace(0, n // page - 1, B).astype(int)] = 1  # anywhere in the context
    q = np.zeros((B, hq, d))
    q[..., 0] = 1
    out = fq.fq_kv4_attn(torch.from_numpy(q).to(dtype).cuda(), _dev(host), _dev(tables), _dev(np.full(B, n, dtype=np.int32)),
                         group, scale=1.0)
    p = (n - 1) * np.exp(kq[0, 0, 0] - kq[1, 0, 0])
    A = p / (1 + p) * vq[0, 0]
    lost = n * 2.0 ** -32 * np.abs(vq[0, 0])
    want = np.broadcast_to(A, out.shape)
    S = kq[1, 0, 0]
    got = _cpu(out.double())
    rel = 2.0 ** -10 + 2 * n / 16 * 2.0 ** -24 + 2.0 ** -14 + (2 * (d + 8) * 2.0 ** -23 + (2.0 ** -10 if dtype == torch.bfloat16 and hq > 64 else 0)) * S
    half_eps = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    assert (np.abs(got - want) <= (half_eps + rel) * want + lost + 2.0 ** -24).all(), (got[0, 0, :4], want[0, 0, :4])


@pytest.mark.parametrize("hq", [4, 66])  # few rows of a kv head, and more than 64
@pytest.mark.parametrize("cu", [[0, 2, 1, 9], [-3, 2, 4, 6], [0, 5, 7, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 8],
                                [8, 8, 0, 2], [9, 10, 6, 8], [3, 8, 8, 8]])
def test_counts_that_fall_or_lie_outside_the_queries(hq, cu):
    """Such sequences have no rows, and of more than max_q query tokens the first are computed, each in its place."""
    rng = np.random.default_rng(hq)
    n_q, max_q, dtype = 8, 2, torch.float16
    c = Cache(rng, [40, 33, 70], 1, 64, 32, 16)
    q = _q(rng, n_q, hq, 64, dtype)
    room = torch.full((n_q + 8, hq, 64), 7.0, dtype=dtype, device="cuda")
    out = room[4:-4]
    fq.fq_kv4_attn(q, _dev(c.host), _dev(c.tables), _dev(c.lens), 32, cu_q=_dev(np.array(cu, dtype=np.int64).astype(np.int32)),
                   max_q=max_q, out=out)
    assert (room[:4] == 7).all() and (room[-4:] == 7).all()
    left = np.ones(n_q, dtype=bool)
    for b in range(3):
        lo, hi = cu[b], cu[b + 1]
        if 0 <= lo < hi <= n_q:
            rows = slice(lo, min(hi, lo + max_q))
            want = ref.attend(_cpu(q[lo:hi].double()), c.host, c.tables[b:b + 1], c.lens[b:b + 1], 32, [0, hi - lo])
            _check_attn(out[rows], *(w[:max_q] for w in want), 64, dtype, rows=max_q * hq)
            left[rows] = False
    assert (out[torch.from_numpy(left).cuda()] == 7).all()


@pytest.mark.parametrize("hq", [4, 66])  # few rows of a kv head, and more than 64
@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 9, 2 ** 31 - 1])
def test_a_window_wider_than_any_sequence_is_none(hq, window):
    """Sequences with more query tokens than tokens: their first rows end before the first token."""
    rng = np.random.default_rng(window % 97)
    qlens = [8, 1, 6, 12]
    c = Cache(rng, [2, 70, 3, 300], 1, 64, 32, 16)
    q, cu = _q(rng, sum(qlens), hq, 64, torch.bfloat16), np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    out = fq.fq_kv4_attn(q, _dev(c.host), _dev(c.tables), _dev(c.lens), 32, cu_q=_dev(cu), max_q=12, window=window)
    want = ref.attend(_cpu(q.double()), c.host, c.tables, c.lens, 32, cu, window)
    _check_attn(out, *want, 64, torch.bfloat16, rows=12 * hq)
    assert not out[:6].any() and (out[6:8] != 0).any()


def test_a_workspace_has_to_have_the_bytes_that_it_counts():
    rng = np.random.default_rng(3)
    c = Cache(rng, [600, 20], 2, 64, 32, 16, max_blocks=400)
    q, args = _q(rng, 2, 8, 64, torch.float16), (_dev(c.host), _dev(c.tables), _dev(c.lens), 32)
    need = fq.fq_kv4_attn_workspace_bytes(2, 8, 2, 64, 1, 400, 16)
    assert need > 0
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    for bad in (ws[:16].expand(need // 16 + 1, 16), torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        assert bad.numel() >= need
        with pytest.raises(ValueError, match="contiguous"):
            fq.fq_kv4_attn(q, *args, workspace=bad)
    with pytest.raises(fq.FQError):
        fq.fq_kv4_attn(q, *args, workspace=ws[:need - 1])
    _check_attn(fq.fq_kv4_attn(q, *args, workspace=ws[:need].view(torch.float16)),
                *ref.attend(_cpu(q.double()), c.host, c.tables, c.lens, 32), 64, torch.float16)


# ------------------------------------------------------------------ all three together

@pytest.mark.parametrize("hq", [2, 6])
def test_a_refused_request_leaves_the_others_of_its_step_alone(hq):
    rng = np.random.default_rng(hq)
    d, group, page, n_blocks, B = 64, 32, 16, 9, 4
    dtype = torch.float16
    pool = torch.full((n_blocks, 1, 1, ref.unit_bytes(d, group)), 0xFF, dtype=torch.uint8, device="cuda")
    tables, free = torch.full((B, 3), -1, dtype=torch.int32, device="cuda"), _dev(rng.permutation(n_blocks).astype(np.int32))
    lens, count = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.tensor([n_blocks], dtype=torch.int32, device="cuda")
    for adds, turned_away in (([5, 20, 33, 1], []), ([2, 40, 9, 1], [1]), ([1, 3, 20, 14], [2])):
        n = sum(adds)
        new = _dev(np.array(adds, dtype=np.int32))
        before = _cpu(lens)
        lens, cu, slots, refused = fq.fq_page_step(lens, new, tables, free, count, page, n)
        k, v, q = (_q(rng, n, h, d, dtype) for h in (1, 1, hq))
        fq.fq_kv4_write(k, v, slots, pool, group)
        out = fq.fq_kv4_attn(q, pool, tables, lens, group, cu_q=cu, max_q=max(adds))
        assert int(refused) == len(turned_away)
        assert _cpu(lens).tolist() == [int(a) + (0 if b in turned_away else m) for b, (a, m) in enumerate(zip(before, adds))]
        want, A, S = ref.attend(_cpu(q.double()), _cpu(pool), _cpu(tables), _cpu(lens), group, _cpu(cu))
        at = _cpu(cu)
        rows = np.concatenate([np.arange(at[b], at[b + 1]) for b in range(B) if b not in turned_away])
        _check_attn(out[torch.from_numpy(rows).cuda()], want[rows], A[rows], S[rows], d, dtype, rows=max(adds) * hq)
