"""The 4-bit paged cache on the GPU against the plain 64-bit restatement.

Bounds.  Writes and page steps are defined to the bit and have to be equal.  Attention: with
A = sum_t p_t |v_t| per coordinate and S = max_t sum_i |q_i k_ti| scale, an output is off by at most
  eps/2 |out|      its own rounding,
  2^-11 A          values and weights are each rounded to fp16 once (half a step, 2^-12, each),
  2 (d + 8) 2^-23 S A   a score is a sum of d products in 32 bits, each addition off by at most
                   2^-23 of the sum of magnitudes; an error x of the scores moves the weights by 2x,
  2^-11 S A        bf16 outputs of more than 64 rows of a kv head: keys are fp16 numbers too, half a
                   step (2^-12) off, which moves a score by at most 2^-12 S and the weights by twice
                   that (fp16 outputs, and fewer rows, take the keys as they are),
  2^-10 A / 16     exponentials, sums of weights and of weighted values in 32 bits, added step by
                   step (2^-23 for each of at most 2^9 additions),
  2^-24 (15 s + |z| where it is tiny)   fp16 values below 2^-14 have a fixed step: 2^-25 each."""
import math

import numpy as np
import pytest
import torch

import random_access_kv_fq_b200 as fq
from tests import kv4_ref as ref

pytestmark = pytest.mark.gpu

HALF_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _cpu(t):
    return t.detach().cpu().numpy()


def _check_attn(out, want, A, S, d, dtype, rows=1):
    got = _cpu(out.double())
    per_score = 2 * (d + 8) * 2.0 ** -23 + (2.0 ** -11 if dtype == torch.bfloat16 and rows > 64 else 0)
    bound = HALF_EPS[dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -14 + per_score * S[..., None]) * A + 2.0 ** -24
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


class Cache:
    """A pool with random pages written through the reference, its unwritten bytes at 0xFF (codes 15,
    steps and zeros NaN)."""

    def __init__(self, rng, lens, hkv, d, group, page, extra=3, dtype=np.float16, max_blocks=None, spread=1.0):
        self.d, self.group, self.page, self.hkv = d, group, page, hkv
        pages = [-(-n // page) for n in lens]
        self.n_blocks = max(1, sum(pages) + extra)
        ids = rng.permutation(self.n_blocks)
        mb = max_blocks or max(1, max(pages, default=1))
        self.tables = np.full((len(lens), mb), -7, dtype=np.int32)
        at = 0
        for b, m in enumerate(pages):
            self.tables[b, :m] = ids[at:at + m]
            at += m
        self.lens = np.array(lens, dtype=np.int32)
        self.host = np.full((self.n_blocks, hkv, page // 16, ref.unit_bytes(d, group)), 0xFF, dtype=np.uint8)
        slots = np.concatenate([self.tables[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
                                for b, n in enumerate(lens)] + [np.zeros(0, dtype=np.int64)])
        scale = np.exp(0.5 * rng.standard_normal((2, 1, hkv, d))) * spread
        self.k, self.v = (rng.standard_normal((2, len(slots), hkv, d)) * scale).astype(dtype)
        self.fill(slots)

    def fill(self, slots):
        # the reference writes a token at a time: many tokens go through the same routine in one piece
        k, v, d, g = self.k, self.v, self.d, self.group
        unit = self.host.reshape(self.n_blocks, self.hkv, -1, self.host.shape[-1])
        blk, u, tok = slots // self.page, slots % self.page // 16, slots % 16
        for x, code_at, scale_at in ((k, ref.key_code_at, ref.key_scale_at), (v, ref.value_code_at, ref.value_scale_at)):
            c, s, z = ref.quantise(x, g)
            at = np.array([[code_at(t, i, d) for i in range(d)] for t in range(16)])
            sc = np.array([[scale_at(t, j, d, g) for j in range(d // g)] for t in range(16)])
            for t in range(16):
                m = tok == t
                by = np.zeros((m.sum(), self.hkv, self.host.shape[-1]), dtype=np.uint8)
                low, high = at[t, :, 1] == 0, at[t, :, 1] == 1
                by[:, :, at[t, low, 0]] = c[m][:, :, low]
                by[:, :, at[t, high, 0]] |= c[m][:, :, high] << 4
                cols = list(at[t, low, 0])
                for j in range(d // g):
                    for w, part in enumerate((s, z)):
                        b = sc[t, j, w]
                        by[:, :, b:b + 2] = part[m][:, :, j, None].copy().view(np.uint8)
                        cols += [b, b + 1]
                rows = unit[blk[m], :, u[m]]
                rows[:, :, cols] = by[:, :, cols]
                unit[blk[m], :, u[m]] = rows


def _attend(c, q, qlens=None, window=0, scale=None, **kw):
    cu = None if qlens is None else np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    dt = q.dtype
    want = ref.attend(_cpu(q.double()), c.host, c.tables, c.lens, c.group, cu, window, scale)
    max_q = 1 if cu is None else int(max(qlens, default=0))
    out = fq.fq_kv4_attn(q, _dev(c.host), _dev(c.tables), _dev(c.lens), c.group, cu_q=None if cu is None else _dev(cu),
                         max_q=max_q, window=window, scale=scale, **kw)
    _check_attn(out, *want, c.d, dt, rows=max_q * q.shape[1] // c.hkv)
    return out


def _q(rng, n, hq, d, dtype, mul=1.0):
    return (torch.from_numpy(rng.standard_normal((n, hq, d))) * mul).to(dtype).cuda()


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hkv,page", [(1, 1, 16), (37, 3, 32), (130, 2, 128)])
def test_write_equals_the_definition(d, group, dtype, n, hkv, page):
    rng = np.random.default_rng(n + d + group)
    x = (rng.standard_normal((2, n, hkv, d)) * np.exp(rng.standard_normal((2, 1, hkv, d)))).astype(np.float32)
    k, v = (torch.from_numpy(a).to(dtype) for a in x)
    n_blocks = -(-n // page) + 2
    cache = rng.integers(0, 256, (n_blocks, hkv, page // 16, ref.unit_bytes(d, group)), dtype=np.uint8)
    slots = rng.permutation(n_blocks * page)[:n].astype(np.int32)
    if n > 5:  # skipped tokens: their rows may hold anything
        slots[[1, 3, 4]] = -1, n_blocks * page, 2 ** 31 - 1
        k[3], v[1] = float("nan"), float("inf")
    got = _dev(cache)
    kv, vv = fq.fq_kv4_write(k.cuda(), v.cuda(), _dev(slots), got, group, values=True)
    f = lambda t: t.float().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        ref.write(cache, f(k), f(v), slots, group)
    np.testing.assert_array_equal(_cpu(got), cache)
    ok = np.ones(n, dtype=bool)
    ok[[i for i in (1, 3) if n > 5]] = False
    for a, b in ((k, kv), (v, vv)):
        c, s, z = ref.quantise(f(a)[ok], group)
        want = torch.from_numpy(ref.values(c, s, z, group).astype(np.float32)).to(dtype)
        assert torch.equal(b.cpu()[torch.from_numpy(ok)], want)
    # without the values output, the same cache
    again = _dev(np.zeros_like(cache))
    fq.fq_kv4_write(k.cuda(), v.cuda(), _dev(slots), again, group)
    first = _dev(np.zeros_like(cache))
    fq.fq_kv4_write(k.cuda(), v.cuda(), _dev(slots), first, group, values=True)
    assert torch.equal(first, again)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_write_of_special_values(dtype):
    d, group = 64, 32
    big = 60000.0 if dtype == torch.float16 else 3e38
    rows = [np.zeros(d), np.full(d, -3.25), np.linspace(-big, big, d), np.full(d, 6e-8), np.linspace(0, 6e-7, d), np.linspace(-1e-4, 3, d),
            np.linspace(60000, 61000, d), -np.linspace(0, 65000, d), np.where(np.arange(d) == 5, big, 0), np.arange(d) % 16]
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(dtype)[:, None]
    cache = np.zeros((1, 1, 1, ref.unit_bytes(d, group)), dtype=np.uint8)
    got, slots = _dev(cache), np.arange(len(rows), dtype=np.int32)
    kv, _ = fq.fq_kv4_write(x.cuda(), x.cuda(), _dev(slots), got, group, values=True)
    ref.write(cache, x.float().numpy(), x.float().numpy(), slots, group)
    np.testing.assert_array_equal(_cpu(got), cache)
    assert torch.equal(kv[0].cpu(), x[0]) and torch.equal(kv[1].cpu(), x[1]) and torch.isfinite(kv).all()
    assert torch.equal(kv[9].cpu(), x[9])  # 0..15 in a group are held exactly


@pytest.mark.parametrize("offset", [0, 1])
def test_write_takes_strided_and_unaligned_inputs(offset):
    rng = np.random.default_rng(5)
    n, hkv, d, group = 21, 2, 128, 64
    fused = torch.from_numpy(rng.standard_normal((n, 6 * hkv * d + 8 * offset + offset))).half().cuda()
    k = fused[:, offset:offset + hkv * d].unflatten(1, (hkv, d))
    v = torch.as_strided(fused, (n, hkv, d), (fused.stride(0), 2 * d, 1), offset + 2 * hkv * d)
    slots = _dev(rng.permutation(64)[:n].astype(np.int32))
    a = torch.zeros(2, hkv, 2, ref.unit_bytes(d, group), dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    fq.fq_kv4_write(k, v, slots, a, group)
    fq.fq_kv4_write(k.contiguous(), v.contiguous(), slots, b, group)
    assert torch.equal(a, b) and a.any()


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,page", [(8, 1, 16), (3, 3, 32), (14, 2, 64), (32, 2, 128)])
def test_one_query_per_sequence(d, group, dtype, hq, hkv, page):
    rng = np.random.default_rng(hq + page + d + group)
    c = Cache(rng, [1, 15, 0, 16, 17, 333, 64, 1029], hkv, d, group, page)
    out = _attend(c, _q(rng, 8, hq, d, dtype), scale=None)
    assert not out[2].any()  # no token: zeros


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (12, 12), (20, 4), (34, 2)])
def test_head_layouts(d, group, hq, hkv):
    rng = np.random.default_rng(hq + hkv)
    c = Cache(rng, [50, 201], hkv, d, group, 16)
    _attend(c, _q(rng, 2, hq, d, torch.float16))
    _attend(c, _q(rng, 5, hq, d, torch.bfloat16), qlens=[3, 2])


@pytest.mark.parametrize("d,group", [(64, 32), (128, 32), (128, 128)])
@pytest.mark.parametrize("window", [0, 1, 7, 16, 100, 5000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_ragged_queries_and_windows(d, group, window, dtype):
    rng = np.random.default_rng(window + d)
    lens, qlens = [1, 40, 0, 130, 3, 700, 16, 90], [1, 17, 0, 3, 5, 6, 16, 0]
    c = Cache(rng, lens, 2, d, group, 16)
    out = _attend(c, _q(rng, sum(qlens), 6, d, dtype), qlens=qlens, window=window)
    row = sum(qlens[:4])  # sequence 4: 5 query tokens, 3 in the cache: its first two see nothing
    assert not out[row:row + 2].any() and out[row + 2:row + 5].any()


@pytest.mark.parametrize("hq,hkv,m", [(8, 8, 70), (4, 1, 65), (7, 1, 33), (32, 2, 20), (2, 1, 300)])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prefill_of_many_query_tokens(hq, hkv, m, d, group, dtype):
    rng = np.random.default_rng(m)
    c = Cache(rng, [m, m + 75], hkv, d, group, 32)
    _attend(c, _q(rng, 2 * m - 3, hq, d, dtype), qlens=[m, m - 3])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window", [0, 900])
def test_chunks_over_long_contexts_that_span_blocks(dtype, window):
    """A few items of many tiles: every block of the grid holds a part of one."""
    rng = np.random.default_rng(21)
    c = Cache(rng, [9001, 4500], 2, 64, 32, 64)
    _attend(c, _q(rng, 12, 20, 64, dtype), qlens=[5, 7], window=window)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_chunks_with_missing_pages_rising_maxima_and_odd_scales(dtype):
    rng = np.random.default_rng(22)
    c = Cache(rng, [700, 333, 0, 130], 1, 128, 32, 16)
    c.tables[0, [0, 7, 8, 20, 43]] = -1
    c.tables[1, ::2] = c.n_blocks
    c.tables[3] = 2 ** 31 - 1
    q = _q(rng, 40, 8, 128, dtype)
    qlens = [10, 20, 3, 7]
    for scale in (None, 0.0, -0.05, 2.0, 1e-30):
        _attend(c, q, qlens=qlens, scale=scale)
    # keys that grow along the context: the maximum moves in every tile
    c.k *= np.linspace(0.1, 9, len(c.k), dtype=np.float32)[:, None, None].astype(c.k.dtype)
    lens, pages = c.lens.tolist(), [-(-int(n) // 16) for n in c.lens]
    c.tables[:] = -1
    ids = rng.permutation(c.n_blocks)
    at = 0
    for b, m in enumerate(pages):
        c.tables[b, :m] = ids[at:at + m]
        at += m
    c.fill(np.concatenate([c.tables[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16 for b, n in enumerate(lens)]))
    _attend(c, q, qlens=qlens, scale=0.3)
    _attend(c, q, qlens=qlens, scale=0.3, window=50)


def test_rows_of_no_sequence_are_left_alone_and_bad_counts_stay_in_bounds():
    rng = np.random.default_rng(8)
    c = Cache(rng, [20, 33, 5], 1, 64, 32, 16)
    q = _q(rng, 9, 4, 64, torch.float16)
    out = torch.full((9, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    cu = np.array([0, 2, 3, 6], dtype=np.int32)
    fq.fq_kv4_attn(q, _dev(c.host), _dev(c.tables), _dev(c.lens), 32, cu_q=_dev(cu), max_q=4, out=out)
    want = ref.attend(_cpu(q.double()), c.host, c.tables, c.lens, 32, cu)
    _check_attn(out[:6], *(w[:6] for w in want), 64, torch.float16)
    assert (out[6:] == 7).all()


def test_lengths_past_the_table_and_pages_outside_the_pool():
    rng = np.random.default_rng(9)
    c = Cache(rng, [70, 64, 48], 2, 64, 64, 16, max_blocks=5)
    c.tables[0, 1], c.tables[1, 3], c.tables[2, 0] = -1, c.n_blocks, 2 ** 31 - 1
    _attend(c, _q(rng, 3, 8, 64, torch.bfloat16))
    _attend(c, _q(rng, 9, 8, 64, torch.bfloat16), qlens=[3, 2, 4], window=20)
    c.tables[2] = -1
    assert not _attend(c, _q(rng, 3, 8, 64, torch.bfloat16))[2].any()
    full = Cache(rng, [80, 64, 80], 2, 64, 64, 16)
    full.lens[:] = 10 ** 9, 2 ** 31 - 1, -5   # clamped to 80, 80 (a page outside the pool: 64 seen) and 0
    _attend(full, _q(rng, 3, 8, 64, torch.float16))


@pytest.mark.parametrize("dtype,mul", [(torch.float16, 40.0), (torch.bfloat16, 1e4), (torch.bfloat16, 1e-30), (torch.float16, 0.0), (torch.float16, 1e-6)])
def test_scores_of_any_size(dtype, mul):
    rng = np.random.default_rng(10)
    c = Cache(rng, [300, 41], 2, 128, 32, 16)
    scale = 1.0 / (math.sqrt(128) * max(1.0, mul / 40))
    _attend(c, _q(rng, 2, 16, 128, dtype, mul), scale=scale)
    _attend(c, _q(rng, 2, 16, 128, dtype, mul), scale=-scale)
    _attend(c, _q(rng, 2, 16, 128, dtype, mul), scale=0.0)


@pytest.mark.parametrize("spread", [1e-3, 300.0])
def test_caches_of_small_and_large_values(spread):
    rng = np.random.default_rng(11)
    c = Cache(rng, [120, 64], 1, 64, 32, 16, spread=spread)
    _attend(c, _q(rng, 2, 8, 64, torch.float16 if spread < 1 else torch.bfloat16), scale=0.1 / spread)


def test_a_long_context_and_one_peaked_token():
    rng = np.random.default_rng(12)
    c = Cache(rng, [70001, 3], 1, 64, 64, 64)
    q = _q(rng, 2, 8, 64, torch.float16)
    _attend(c, q)
    q[0] = torch.from_numpy(c.k[69000, 0]).cuda() * 4  # nearly all the weight on one token
    _attend(c, q)


def test_offsets_past_31_bits():
    """A pool of over 2^31 bytes whose last pages are used."""
    rng = np.random.default_rng(13)
    d, group, page, hkv = 128, 32, 64, 8
    c = Cache(rng, [150, 64], hkv, d, group, page, extra=0)
    n_blocks = (1 << 31) // (hkv * page // 16 * ref.unit_bytes(d, group)) + 50
    pool = torch.full((n_blocks, hkv, page // 16, ref.unit_bytes(d, group)), 0xFF, dtype=torch.uint8, device="cuda")
    assert pool.numel() > (1 << 31)
    pool[n_blocks - c.n_blocks:] = _dev(c.host)
    tables = _dev(np.where(c.tables >= 0, c.tables + n_blocks - c.n_blocks, -1).astype(np.int32))
    q = _q(rng, 2, 16, d, torch.float16)
    out = fq.fq_kv4_attn(q, pool, tables, _dev(c.lens), group)
    _check_attn(out, *ref.attend(_cpu(q.double()), c.host, c.tables, c.lens, group), d, torch.float16)
    # and a write there
    slot = n_blocks * page - 3
    pool[-1].zero_()
    x = _q(rng, 1, hkv, d, torch.float16)
    fq.fq_kv4_write(x, x, _dev(np.array([slot], dtype=np.int32)), pool, group)
    one = np.zeros((1,) + c.host.shape[1:], dtype=np.uint8)
    ref.write(one, _cpu(x.float()), _cpu(x.float()), [page - 3], group)
    np.testing.assert_array_equal(_cpu(pool[-1:]), one)


def test_strided_and_unaligned_queries():
    rng = np.random.default_rng(14)
    c = Cache(rng, [90, 20, 200], 2, 64, 32, 16)
    plain = None
    for off in (0, 1, 8):
        big = torch.zeros(3, 3 * 8 * 64 + 16, dtype=torch.float16, device="cuda")
        q = torch.as_strided(big, (3, 8, 64), (big.stride(0), 128, 1), off)
        q.copy_(_q(np.random.default_rng(1), 3, 8, 64, torch.float16))
        out = _attend(c, q)
        plain = out if plain is None else plain
        assert torch.equal(out, plain)


def test_results_repeat_bit_for_bit_and_many_batches_agree():
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 400, 300).tolist()
    c = Cache(rng, lens, 2, 64, 32, 16)
    q = _q(rng, 300, 8, 64, torch.bfloat16)
    a = _attend(c, q)
    assert torch.equal(a, _attend(c, q))


def test_another_stream_with_no_wait_for_the_default_one():
    rng = np.random.default_rng(16)
    c = Cache(rng, [500, 300], 2, 64, 32, 16)
    q = _q(rng, 2, 8, 64, torch.float16)
    args = q, _dev(c.host), _dev(c.tables), _dev(c.lens), 32
    want = fq.fq_kv4_attn(*args)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):  # two streams at once, each call with the workspace that it allocates
        outs += [fq.fq_kv4_attn(*args, stream=s1), fq.fq_kv4_attn(*args, stream=s2.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("B,max_q", [(8192, 1), (2100, 3), (1500, 9)])
def test_more_sequences_than_a_block_has_threads(B, max_q):
    rng = np.random.default_rng(B)
    qlens = None if max_q == 1 else rng.integers(0, max_q + 1, B).tolist()
    lens = np.where(rng.random(B) < 0.7, 0, rng.integers(0, 40, B))
    lens[[5, B - 1]] = 900, 300
    if qlens is not None:
        qlens[0] = max_q
        lens = np.maximum(lens, qlens) * (rng.random(B) < 0.9)  # a few whose tokens are not there: rows of 0
    c = Cache(rng, lens.tolist(), 1, 64, 64, 32)
    _attend(c, _q(rng, B if qlens is None else sum(qlens), 8, 64, torch.bfloat16), qlens)


@pytest.mark.parametrize("qlens", [None, [3, 1, 0, 4, 2], [11, 4, 0, 1, 2]])
def test_a_workspace_of_any_content_serves_call_after_call_and_graphs_in_turn(qlens):
    rng = np.random.default_rng(18)
    c = Cache(rng, [5000, 37, 0, 2100, 700], 2, 64, 32, 16)
    one = Cache(rng, [9000], 1, 128, 64, 64)  # one kv head: every block has a part of the only item
    qlens1 = None if qlens is None else [max(qlens)]
    need = max(fq.fq_kv4_attn_workspace_bytes(len(x.lens), 8 * x.hkv, x.hkv, x.d, 1 if qlens is None else max(qlens),
                                              x.tables.shape[1], x.page) for x in (c, one))
    assert need > 0
    calls = []
    for x, m in ((c, qlens), (one, qlens1)):
        q = _q(rng, len(x.lens) if m is None else sum(m), 8 * x.hkv, x.d, torch.float16)
        cu = None if m is None else _dev(np.concatenate([[0], np.cumsum(m)]).astype(np.int32))
        lens = _dev(x.lens)
        kw = dict(cu_q=cu, max_q=1 if m is None else max(m))
        calls.append((q, _dev(x.host), _dev(x.tables), lens, x.group, kw, torch.empty_like(q)))
        _attend(x, q, m)
    want = [[fq.fq_kv4_attn(q, pool, t, n - k, g, **kw) for k in (0, 8, 3)] for q, pool, t, n, g, kw, _ in calls]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for fill in (0, 1, 0x7F, 0xFF, None):
        ws.copy_(torch.randint(0, 256, (need,), dtype=torch.uint8)) if fill is None else ws.fill_(fill)
        for i in (0, 1, 1, 0):
            q, pool, t, n, g, kw, out = calls[i]
            assert torch.equal(fq.fq_kv4_attn(q, pool, t, n, g, out=out.fill_(7), workspace=ws, **kw), want[i][0])
    graphs = []
    torch.cuda.synchronize()
    for q, pool, t, n, g, kw, out in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            fq.fq_kv4_attn(q, pool, t, n, g, out=out, workspace=ws, **kw)
    ws.fill_(0xA5)
    for k, i in ((0, 0), (0, 0), (0, 1), (1, 0), (1, 1), (2, 1), (2, 0), (0, 1), (0, 0)):
        q, pool, t, n, g, kw, out = calls[i]
        n.sub_((0, 8, 3)[k])  # a replay reads the lengths that are there then
        out.fill_(7)
        graphs[i].replay()
        assert torch.equal(out, want[i][k])
        n.add_((0, 8, 3)[k])


def test_binding_refuses_wrong_tensors():
    rng = np.random.default_rng(17)
    c = Cache(rng, [20, 20], 2, 64, 32, 16)
    q, pool, t, n = _q(rng, 2, 8, 64, torch.float16), _dev(c.host), _dev(c.tables), _dev(c.lens)
    for bad in (lambda: fq.fq_kv4_attn(q.float(), pool, t, n, 32), lambda: fq.fq_kv4_attn(q, pool, t.long(), n, 32),
                lambda: fq.fq_kv4_attn(q, pool, t, n, 64), lambda: fq.fq_kv4_attn(q, pool, t[:1], n, 32),
                lambda: fq.fq_kv4_attn(q[..., ::2], pool, t, n, 32), lambda: fq.fq_kv4_attn(q, pool[:, :, :, 1:], t, n, 32),
                lambda: fq.fq_kv4_attn(q, pool, t, n.cpu(), 32), lambda: fq.fq_kv4_attn(q[:1], pool, t, n, 32),
                lambda: fq.fq_kv4_attn(q, pool, t, n, 32, cu_q=n), lambda: fq.fq_kv4_attn(q[:, :7], pool, t, n, 32),
                lambda: fq.fq_kv4_attn(q, pool, t.repeat(1, 500), n, 32, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
                lambda: fq.fq_kv4_write(q, q, n, pool, 32), lambda: fq.fq_kv4_write(q[:, :2], q[:, :2], n.long(), pool, 32),
                lambda: fq.fq_kv4_write(q[:, :2], q[:, :2].float(), n, pool, 32),
                lambda: fq.fq_kv4_write(q[:, :2].double(), q[:, :2].double(), n, pool, 32)):
        with pytest.raises((ValueError, TypeError, fq.FQError)):
            bad()


# ------------------------------------------------------------------ page step

def _step(lens, new, tables, free, count, page, n_slots, alias=False):
    t, f = _dev(tables), _dev(free)
    lt, ct = _dev(np.array(lens, dtype=np.int32)), _dev(np.array([count], dtype=np.int32))
    co = ct if alias else torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fq.fq_page_step(lt, _dev(np.array(new, dtype=np.int32)), t, f, ct, page, n_slots,
                          lens_out=lt if alias else None, free_count_out=None if alias else co)
    wt, wf = tables.copy(), free.copy()
    want = ref.page_step(lens, new, wt, wf, count, page, n_slots)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(_cpu(a).ravel(), np.ravel(b))
    assert int(co) == want[4]
    np.testing.assert_array_equal(_cpu(t), wt)
    np.testing.assert_array_equal(_cpu(f), wf)
    return want, wt, wf


def _pool(rng, lens, max_blocks, page, spare):
    held = [-(-min(max(n, 0), max_blocks * page) // page) for n in lens]
    ids = rng.permutation(sum(held) + spare).astype(np.int32)
    tables = np.full((len(lens), max_blocks), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        tables[b, :h] = ids[at:at + h]
        at += h
    free = np.full(len(ids), -9, dtype=np.int32)
    free[:spare] = ids[at:]
    return tables, free


@pytest.mark.parametrize("B", [0, 1, 5, 63, 1024, 1025, 8192])
@pytest.mark.parametrize("page,max_blocks", [(16, 9), (128, 3)])
@pytest.mark.parametrize("alias", [False, True])
def test_page_steps_equal_the_sequential_definition(B, page, max_blocks, alias):
    rng = np.random.default_rng(B + page)
    lens = rng.integers(0, max_blocks * page + 1, B)
    new = np.where(rng.random(B) < 0.2, -rng.integers(1, 9, B), rng.integers(0, 40, B))
    tokens = int(new[new > 0].sum())
    for spare, n_slots in ((3 * B + 5, tokens + 37), (B // 2, tokens + 1), (0, tokens), (3 * B, tokens // 2), (7, 0)):
        tables, free = _pool(rng, lens, max_blocks, page, spare)
        _step(lens, new, tables, free, spare, page, n_slots, alias)


def test_page_step_with_long_prefills_and_odd_lengths():
    rng = np.random.default_rng(3)
    lens = np.array([0, 5000, -4, 10 ** 9, 64, 0, 17], dtype=np.int64)
    new = np.array([30011, 1, 9, 0, -1, 2 ** 31 - 1, 47], dtype=np.int64)
    tables, free = _pool(rng, lens, 2048, 16, 5000)
    want, _, _ = _step(lens, new, tables, free, 5000, 16, 40000)
    assert want[3] >= 1
    # a count past the pool's size, released pages past its end
    tables, free = _pool(rng, [40, 40], 4, 16, 2)
    _step([40, 40], [-1, -1], tables, free, 100, 16, 4)


def test_page_steps_until_the_pool_is_empty():
    rng = np.random.default_rng(4)
    B, page, mb = 6, 16, 8
    tables, free = np.full((B, mb), -1, dtype=np.int32), rng.permutation(20).astype(np.int32)
    lens, count, refused = np.zeros(B, dtype=np.int64), 20, 0
    for step in range(60):
        new = np.where(rng.random(B) < 0.1, -1, rng.integers(0, 20, B))
        want, tables, free = _step(lens, new, tables, free, count, page, 64)
        lens, count = want[0], want[4]
        refused += want[3]
        held = np.concatenate([tables[b, :-(-int(n) // page)] for b, n in enumerate(lens)] + [free[:count]])
        assert sorted(held.tolist()) == list(range(20))  # every page is held once or free
    assert refused > 0


# ------------------------------------------------------------------ all three together

@pytest.mark.parametrize("d,group,dtype", [(64, 32, torch.float16), (128, 128, torch.bfloat16)])
@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop(d, group, dtype, graph):
    """Prefill, decode and end requests in one pool: page step, write and attention of each step as a
    user calls them (or captured once into a CUDA graph and replayed), against dense 64-bit attention."""
    rng = np.random.default_rng(d)
    B, hq, hkv, page, mb, cap = 4, 6, 2, 16, 12, 64
    n_blocks = 30
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    free = _dev(rng.permutation(n_blocks).astype(np.int32))
    count = torch.tensor([n_blocks], dtype=torch.int32, device="cuda")
    lens, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = torch.full((n_blocks, hkv, page // 16, ref.unit_bytes(d, group)), 0xFF, dtype=torch.uint8, device="cuda")
    q = torch.zeros(cap, hq, d, dtype=dtype, device="cuda")
    k, v = torch.zeros(cap, hkv, d, dtype=dtype, device="cuda"), torch.zeros(cap, hkv, d, dtype=dtype, device="cuda")
    out = torch.zeros(cap, hq, d, dtype=dtype, device="cuda")
    values = {}

    def step():
        _, cu, slots, refused = fq.fq_page_step(lens, new, tables, free, count, page, cap, lens_out=lens)
        values["kv"] = fq.fq_kv4_write(k, v, slots, pool, group, values=True)
        fq.fq_kv4_attn(q, pool, tables, lens, group, cu_q=cu, max_q=cap, out=out)
        values["step"] = cu, refused

    if graph:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()  # nothing is added yet
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    past = [[np.zeros((0, hkv, d))] * 2 for _ in range(B)]
    plan = [[9, 0, 20, 1], [1, 30, 1, 1], [1, 1, -1, 1], [1, 1, 7, 1], [-1, 1, 1, 40], [13, 1, 1, 1], [1, -1, -1, 3], [0, 2, 5, 0]]
    for adds in plan:
        new.copy_(torch.tensor(adds, dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape)).to(dtype))
        out.fill_(9)
        if graph:
            g.replay()
        else:
            step()
        torch.cuda.synchronize()
        cu, refused = values["step"]
        assert int(refused) == 0
        kv, vv = (_cpu(x.double()) for x in values["kv"])
        for b, m in enumerate(adds):
            if m < 0:
                past[b] = [np.zeros((0, hkv, d))] * 2
                continue
            lo, hi = int(cu[b]), int(cu[b + 1])
            assert hi - lo == m
            past[b] = [np.concatenate([p, x[lo:hi]]) for p, x in zip(past[b], (kv, vv))]
            n = len(past[b][0])
            assert n == int(lens[b])
            for i in range(m):
                e = n - m + i + 1
                for h in range(hq):
                    kk, vals = past[b][0][:e, h // 3], past[b][1][:e, h // 3]
                    qr = _cpu(q[lo + i, h].double())
                    p = np.exp(kk @ qr / math.sqrt(d) - (kk @ qr / math.sqrt(d)).max())
                    p /= p.sum()
                    S = (np.abs(kk) @ np.abs(qr)).max() / math.sqrt(d)
                    # the dense side has the values rounded to the inputs' type: half a step of each key
                    # moves a score by at most that share of S, of each value the output by that share of A
                    r = HALF_EPS[dtype]
                    A = p @ np.abs(vals)
                    bound = r * np.abs(p @ vals) + (2.0 ** -11 + 2.0 ** -14 + r + 2 * S * (r + (d + 8) * 2.0 ** -23)) * 1.1 * A + 2.0 ** -20
                    assert (np.abs(_cpu(out[lo + i, h].double()) - p @ vals) <= bound).all()
        assert (out[int(cu[B]):] == 9).all()
