"""The cache operators against float64 numpy: attention over paged bf16 and 4-bit caches (window, sinks, ragged
batches, empty rows), rows appended and read, pages copied."""
import ctypes

import numpy as np
import pytest
import torch

from cache_oracle import PAGE, Pool, attention, dequantise, quantise, tolerance
from dual_ar_decode_gb300 import (TfError, cache_page_bytes, kv_cache, op_attention_cache, op_cache_append,
                                  op_cache_copy, op_cache_read)
from dual_ar_decode_gb300.binding import (TF_CACHE_BAD_LENGTH, TF_CACHE_BAD_PAGE, TF_CACHE_BAD_ROWS)

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Batch:
    """A pool on the device, a batch of rows over it and its description."""

    def __init__(self, pool, counts, extra_rows=0, lens=None, max_length=0):
        self.pool = pool
        self.K, self.V = torch.from_numpy(pool.K).to(DEV), torch.from_numpy(pool.V).to(DEV)
        self.table = torch.from_numpy(pool.table).to(DEV)
        self.counts = counts
        starts = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        self.start = torch.from_numpy(starts).to(DEV)
        self.lens = torch.tensor(pool.lens if lens is None else lens, dtype=torch.int32, device=DEV)
        self.rows = int(starts[-1])
        self.n_rows = self.rows + extra_rows
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cache = kv_cache(pool.fmt, pool.Hkv, pool.D, self.K.data_ptr(), self.V.data_ptr(), pool.n_pages,
                              self.table.data_ptr(), pool.stride, len(counts), self.lens.data_ptr(),
                              self.start.data_ptr(), self.n_rows, max(counts), max_length, self.err.data_ptr())


def queries(batch, Hq, dtype, seed, pad=0, size=1.0):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.standard_normal((batch.n_rows, Hq * batch.pool.D + pad)).astype(np.float32) * size)
    return q.to(TYPES[dtype]).to(DEV)


def attend(batch, q, Hq, dtype, window=0, sinks=0, scale=0.0, pad=0, stream=0):
    out = torch.full((batch.n_rows, Hq * batch.pool.D + pad), 7.0, dtype=TYPES[dtype], device=DEV)
    op_attention_cache(batch.cache, q.data_ptr(), out.data_ptr(), dtype, Hq, window, sinks, scale,
                       q.shape[1] if q.shape[1] != Hq * batch.pool.D else 0, out.shape[1] if pad else 0,
                       stream=stream)
    return out


def check(batch, q, out, Hq, dtype, window=0, sinks=0, scale=None, hidden=None, err=0):
    torch.cuda.synchronize()
    assert batch.err.item() == err
    D, pool = batch.pool.D, batch.pool
    got = out.float().cpu().numpy().astype(np.float64)
    qn = q.float().cpu().numpy().astype(np.float64)
    row = 0
    lens = batch.lens.cpu().numpy()
    for b, r in enumerate(batch.counts):
        n = int(lens[b])
        qb = qn[row:row + r, :Hq * D].reshape(r, Hq, D)
        want, *sizes = attention(qb, pool.k[b][:n], pool.v[b][:n], n, window, sinks, scale,
                                      None if hidden is None else hidden[b][:n])
        tol = tolerance(want, *sizes, D, n, dtype, pool.fmt)
        diff = np.abs(got[row:row + r, :Hq * D].reshape(r, Hq, D) - want)
        assert np.all(diff <= tol), (b, n, r, float((diff / tol).max()), float(diff.max()))
        row += r
    assert np.all(got[row:] == 7.0)                      # rows past the last sequence's
    assert np.all(got[:, Hq * D:] == 7.0)                # between rows
    return got


FORMATS = ["bf16", "nvfp4"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hkv,ratio,D", [(2, 4, 128), (1, 8, 128), (3, 1, 64), (2, 2, 64), (1, 3, 128), (1, 7, 64),
                                         (2, 5, 128), (1, 6, 64)])
def test_decode_rows_of_every_head_layout(fmt, dtype, Hkv, ratio, D):
    """One row per sequence: an empty sequence, one position, and lengths at and around page edges."""
    lens = [1, 0, 31, 32, 33, 95, 200, 519]
    batch = Batch(Pool(fmt, Hkv, D, lens, seed=D + ratio), [1] * len(lens), extra_rows=2)
    q = queries(batch, Hkv * ratio, dtype, 3)
    check(batch, q, attend(batch, q, Hkv * ratio, dtype), Hkv * ratio, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (32, 32), (33, 5), (100, 64), (700, 3),
                                          (64, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_sinks(fmt, dtype, window, sinks):
    lens = [1, 17, 40, 64, 133, 300, 611]
    batch = Batch(Pool(fmt, 2, 128, lens, seed=window % 1000 + sinks % 1000), [1] * len(lens))
    q = queries(batch, 8, dtype, window % 100)
    check(batch, q, attend(batch, q, 8, dtype, window, sinks), 8, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,lens,window,sinks,Hkv,ratio,D", [
    ([5, 3, 1, 2], [40, 3, 77, 131], 0, 0, 2, 4, 128),        # drafts; a sequence that is all rows
    ([4, 6, 2], [2, 3, 0], 0, 0, 1, 4, 64),                   # rows at negative positions: zeros
    ([8, 7, 1, 0, 5], [300, 64, 33, 90, 129], 50, 4, 1, 8, 128),
    ([33, 1, 20], [70, 1, 500], 0, 0, 2, 2, 64),
    ([64, 129], [64, 257], 48, 3, 1, 4, 128),                 # prompt chunks
    ([200, 40, 3], [333, 40, 30], 0, 0, 2, 3, 64),
    ([150], [700], 130, 40, 1, 5, 128),
    ([257, 31], [257, 600], 0, 0, 1, 1, 128),
])
def test_several_rows_per_sequence(fmt, dtype, counts, lens, window, sinks, Hkv, ratio, D):
    batch = Batch(Pool(fmt, Hkv, D, lens, seed=sum(counts)), counts, extra_rows=1)
    q = queries(batch, Hkv * ratio, dtype, 5)
    check(batch, q, attend(batch, q, Hkv * ratio, dtype, window, sinks), Hkv * ratio, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 7, 90]])
def test_strides_scale_and_row_start_null(fmt, dtype, counts):
    """Rows further apart than they are long (and not 16-byte aligned), a scale of the caller's, and the form
    without row_start."""
    lens = [65, 20, 130]
    batch = Batch(Pool(fmt, 2, 64, lens, seed=9), counts)
    for pad in (3, 8):
        q = queries(batch, 4, dtype, 2, pad=pad)
        check(batch, q, attend(batch, q, 4, dtype, 0, 0, 0.5, pad=pad + 1), 4, dtype, scale=0.5)
    if max(counts) == 1:
        batch.cache.row_start = None
        check(batch, q, attend(batch, q, 4, dtype), 4, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_long_sequence_among_short_ones(fmt, dtype):
    lens = [6011, 1, 64, 2048]
    batch = Batch(Pool(fmt, 1, 128, lens, seed=1), [1] * 4)
    q = queries(batch, 8, dtype, 8)
    check(batch, q, attend(batch, q, 8, dtype), 8, dtype)
    batch.cache.max_length = 10                              # only sizes the launch
    check(batch, q, attend(batch, q, 8, dtype), 8, dtype)
    check(batch, q, attend(batch, q, 8, dtype, 1500, 70), 8, dtype, 1500, 70)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [50, 60, 70]])
def test_rows_of_very_different_sizes(fmt, counts):
    """Large scores (a softmax that is one key), values of 1e-6 beside values of 1e4, rows of zeros."""
    pool = Pool(fmt, 1, 64, [100, 64, 90], seed=4)
    rng = np.random.default_rng(0)
    for b in range(3):
        x = rng.standard_normal((64, 1, 64)).astype(np.float32)
        x *= np.float32(10.0) ** rng.integers(-6, 5, size=(64, 1, 1)).astype(np.float32)
        x[::5] = 0
        pool.v[b][:64] = pool.put(1, b, 0, x)
        pool.k[b][:64:7] = 0
        for j in range(0, 64, 7):
            pool.put(0, b, j, np.zeros((1, 1, 64), np.float32))
    batch = Batch(pool, counts)
    for size in (1e-3, 1.0, 30.0):
        for dtype in ("f32", "bf16"):
            q = queries(batch, 4, dtype, 5, size=size)
            check(batch, q, attend(batch, q, 4, dtype), 4, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1], [9], [200]])
@pytest.mark.parametrize("what", ["ramp", "jump", "values"])
def test_references_that_have_to_be_replaced(fmt, dtype, counts, what):
    """Scores that grow with the position (every reference is soon too small), one that jumps by 2^200 over the rest,
    and values whose size grows by 2^40 while the scores fall."""
    n = 700
    pool = Pool(fmt, 1, 128, [n], seed=4)
    rng = np.random.default_rng(1)
    d = rng.choice(np.array([-1.0, 1.0], np.float32), 128)
    top = np.linspace(0, 60, n) if what == "ramp" else np.linspace(0, 3, n)      # scores, natural logarithm
    if what == "jump":
        top[[333, 520]] = 140
    if what == "values":
        top = np.linspace(25, 0, n)
        v = rng.standard_normal((n, 1, 128)) * 2.0 ** np.linspace(-20, 20, n)[:, None, None]
        pool.v[0][:] = pool.put(1, 0, 0, v.astype(np.float32))
    k = d * top[:, None].astype(np.float32) * np.float32(128 ** 0.5 / 128) + 0.05 * rng.standard_normal((n, 128))
    pool.k[0][:] = pool.put(0, 0, 0, k.astype(np.float32)[:, None])
    batch = Batch(pool, counts)
    q = torch.from_numpy(np.tile(d, (batch.n_rows, 4)).astype(np.float32)).to(TYPES[dtype]).to(DEV)
    check(batch, q, attend(batch, q, 4, dtype), 4, dtype)
    check(batch, q, attend(batch, q, 4, dtype, 450, 7), 4, dtype, 450, 7)


@pytest.mark.parametrize("fmt", FORMATS)
def test_constant_values_come_back(fmt):
    """softmax weights sum to one: values that are the same everywhere are the result."""
    pool = Pool(fmt, 1, 128, [777], seed=4)
    pool.v[0][:] = pool.put(1, 0, 0, np.full((777, 1, 128), 1.5, np.float32))
    for r in (1, 100):
        batch = Batch(pool, [r])
        q = queries(batch, 4, "f32", 6)
        out = attend(batch, q, 4, "f32")
        assert torch.allclose(out, torch.full_like(out, pool.v[0][0, 0, 0]), rtol=3e-6, atol=0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1], [90, 40]])
def test_nan_in_a_seen_row_shows_and_in_an_unseen_one_does_not(fmt, counts):
    pool = Pool(fmt, 1, 64, [200, 120], seed=3)
    pool.put(0, 0, 20, np.full((1, 1, 64), np.nan, np.float32))
    pool.put(1, 0, 21, np.full((1, 1, 64), np.inf, np.float32))
    batch = Batch(pool, counts)
    q = queries(batch, 4, "bf16", 1)
    for dtype in ("f32", "bf16"):
        qq = q.to(TYPES[dtype])
        out = attend(batch, qq, 4, dtype)
        torch.cuda.synchronize()
        assert not torch.isfinite(out[:counts[0]]).any()
        assert torch.isfinite(out[counts[0]:]).all()
        window = 200 - counts[0] - 30                        # no row sees positions 20 and 21
        check(batch, qq, attend(batch, qq, 4, dtype, window, 9), 4, dtype, window, 9)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [40, 70, 33, 60]])
def test_bad_descriptions_are_flagged_and_touch_nothing(fmt, counts):
    """A page outside the pool hides its positions; a length beyond the table, a falling row_start or too many rows
    skip that sequence."""
    lens = [100, 150, 64, 96]
    pool = Pool(fmt, 2, 64, lens, seed=2)
    pool.table[1, 2] = pool.n_pages
    pool.table[0, 1] = -5
    batch = Batch(pool, counts)
    hidden = [np.zeros(n, bool) for n in lens]
    hidden[1][64:96] = True
    hidden[0][32:64] = True
    for dtype in ("f32", "bf16"):
        q = queries(batch, 8, dtype, 1)
        check(batch, q, attend(batch, q, 8, dtype), 8, dtype, hidden=hidden, err=TF_CACHE_BAD_PAGE)
        batch.err.zero_()
    pool = Pool(fmt, 2, 64, lens, seed=2)
    for what in ("length", "negative", "rows", "falling"):
        batch = Batch(pool, counts)
        starts = batch.start.clone()
        if what == "length":
            batch.lens[1] = 32 * pool.stride + 1
        elif what == "negative":
            batch.lens[1] = -1
        elif what == "rows":
            batch.cache.max_rows = max(counts) - 1
            if max(counts) == 1:
                continue
        else:
            starts[2] = 0
            batch.cache.row_start = starts.data_ptr()
        q = queries(batch, 4, "f32", 1)
        out = attend(batch, q, 4, "f32")
        torch.cuda.synchronize()
        assert batch.err.item() == (TF_CACHE_BAD_ROWS if what in ("rows", "falling") else TF_CACHE_BAD_LENGTH)
        lo, hi = sum(counts[:1]), sum(counts[:2])
        assert (out[lo:hi] == 7.0).all()
        assert torch.isfinite(out).all() and (out[:lo] != 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,D", [(2, 128), (3, 64)])
@pytest.mark.parametrize("pad", [0, 5])
def test_append_then_read(fmt, dtype, Hkv, D, pad):
    """Rows land at their positions, bit for bit as the quantiser's definition says; every other byte of the pool
    stays (a neighbour in the same byte of V's codes among them)."""
    lens, counts = [40, 33, 7, 64, 90, 5], [1, 33, 2, 31, 0, 8]
    pool = Pool(fmt, Hkv, D, lens, seed=11)
    batch = Batch(pool, counts, extra_rows=2)
    rng = np.random.default_rng(1)
    row = Hkv * D
    rows = {}
    for name in "kv":
        x = rng.standard_normal((batch.n_rows, row + pad)).astype(np.float32)
        x *= np.exp(2 * rng.standard_normal((batch.n_rows, 1))).astype(np.float32)
        x[3] = 0
        x[4, 16:32] = 0
        x[5, 20] = 1e4
        x[6] *= 1e-6
        rows[name] = torch.from_numpy(x).to(TYPES[dtype]).to(DEV)
    op_cache_append(batch.cache, rows["k"].data_ptr(), rows["v"].data_ptr(), dtype, stride=row + pad)
    r = 0
    for b, c in enumerate(counts):
        for isv, name in ((0, "k"), (1, "v")):
            first = lens[b] - c
            x = rows[name][r:r + c, :row].float().cpu().numpy().reshape(c, Hkv, D)
            skip = max(0, -first)
            held = pool.put(isv, b, first + skip, x[skip:])
            (pool.v if isv else pool.k)[b][first + skip:] = held
        r += c
    torch.cuda.synchronize()
    assert batch.err.item() == 0
    assert np.array_equal(batch.K.cpu().numpy(), pool.K)
    assert np.array_equal(batch.V.cpu().numpy(), pool.V)
    got = [torch.full((batch.n_rows, row + pad), 7.0, device=DEV) for _ in range(2)]
    op_cache_read(batch.cache, got[0].data_ptr(), got[1].data_ptr(), "f32", stride=row + pad)
    torch.cuda.synchronize()
    r = 0
    for b, c in enumerate(counts):
        for x, held in zip(got, (pool.k[b], pool.v[b])):
            want = np.zeros((c, row))
            first = lens[b] - c
            if c:
                want[max(0, -first):] = held[max(0, first):].reshape(-1, row)
            assert np.array_equal(x[r:r + c, :row].cpu().numpy(), want.astype(np.float32))
        r += c
    for x in got:
        assert (x[r:] == 7.0).all() and (x[:, row:] == 7.0).all()


def test_append_stores_rows_that_are_not_finite_as_nan_rows():
    pool = Pool("nvfp4", 1, 64, [4], seed=0)
    batch = Batch(pool, [3])
    x = torch.ones((3, 64), device=DEV)
    x[0, 3], x[1, 60] = float("inf"), float("nan")
    op_cache_append(batch.cache, x.data_ptr(), x.data_ptr(), "f32")
    got = torch.empty((2, 3, 64), device=DEV)
    op_cache_read(batch.cache, got[0].data_ptr(), got[1].data_ptr(), "f32")
    torch.cuda.synchronize()
    assert torch.isnan(got[:, :2]).all() and (got[:, 2] == 1.0).all()


def test_append_and_read_with_bad_pages_and_lengths():
    pool = Pool("nvfp4", 2, 64, [64, 64, 64], seed=0)
    pool.table[1, 1] = pool.n_pages + 3
    batch = Batch(pool, [40, 40, 40], lens=[64, 64, 65])
    x = torch.ones((120, 128), device=DEV)
    op_cache_append(batch.cache, x.data_ptr(), x.data_ptr(), "f32")
    got = torch.full((2, 120, 128), 7.0, device=DEV)
    op_cache_read(batch.cache, got[0].data_ptr(), got[1].data_ptr(), "f32")
    torch.cuda.synchronize()
    assert batch.err.item() == TF_CACHE_BAD_PAGE | TF_CACHE_BAD_LENGTH
    assert (got[:, :40] == 1.0).all() and (got[:, 40:48] == 1.0).all()
    assert (got[:, 48:80] == 0.0).all() and (got[:, 80:] == 7.0).all()


@pytest.mark.parametrize("n_pools,n,page_bytes", [(1, 1, 16), (3, 5, 4864), (150, 2, 1280), (2, 900, 48),
                                                  (2, 3, 65536)])
def test_copy_pages(n_pools, n, page_bytes):
    """More pools and more copies than one launch takes, one source for several destinations."""
    rng = np.random.default_rng(n)
    n_pages = 2 * n + 3
    pools = torch.from_numpy(rng.integers(0, 256, (n_pools, n_pages, page_bytes), dtype=np.uint8)).to(DEV)
    before = pools.cpu().numpy().copy()
    ids = rng.permutation(n_pages).astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:2 * n]
    src[-1] = src[0]
    op_cache_copy([p.data_ptr() for p in pools], page_bytes, n_pages, src, dst)
    before[:, dst] = before[:, src]
    assert np.array_equal(pools.cpu().numpy(), before)


def test_a_forked_sequence_reads_its_own_pages_after_a_copy():
    """The operators together: a sequence's pages copied for a second one, both continue with rows of their own."""
    for fmt in FORMATS:
        pool = Pool(fmt, 2, 128, [70, 70], seed=8, stride=4, spare=8)
        batch = Batch(pool, [1, 1])
        op_cache_copy([batch.K.data_ptr(), batch.V.data_ptr()], cache_page_bytes(fmt, 2, 128), pool.n_pages,
                      pool.table[0, :3], pool.table[1, :3])
        pool.k[1], pool.v[1] = pool.k[0].copy(), pool.v[0].copy()
        pool.K[pool.table[1, :3]] = pool.K[pool.table[0, :3]]
        pool.V[pool.table[1, :3]] = pool.V[pool.table[0, :3]]
        rng = np.random.default_rng(3)
        for step in range(30):
            n = 70 + step
            if n % PAGE == 0:                                # both take a page of their own
                free = sorted(set(range(pool.n_pages)) - set(pool.table[pool.table >= 0].tolist()))
                pool.table[0, n // PAGE], pool.table[1, n // PAGE] = free[:2]
                batch.table.copy_(torch.from_numpy(pool.table))
            k, v = rng.standard_normal((2, 2, 2, 128)).astype(np.float32)
            for b in range(2):
                pool.k[b] = np.concatenate((pool.k[b], pool.put(0, b, n, k[b:b + 1])))
                pool.v[b] = np.concatenate((pool.v[b], pool.put(1, b, n, v[b:b + 1])))
            batch.lens.fill_(n + 1)
            kd, vd = torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV)
            op_cache_append(batch.cache, kd.data_ptr(), vd.data_ptr(), "f32")
            q = queries(batch, 8, "f32", step)
            check(batch, q, attend(batch, q, 8, "f32", 40, 4), 8, "f32", 40, 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [90, 60, 40]])
def test_captured_calls_read_lengths_when_they_run(fmt, counts):
    """A captured call replays with the lengths and rows that the arrays hold then; two streams at once agree with
    one after the other, bit for bit."""
    pool = Pool(fmt, 2, 128, [300, 200, 97], seed=6)
    batch = Batch(pool, counts)
    q = queries(batch, 8, "bf16", 6)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        op_attention_cache(batch.cache, q.data_ptr(), out.data_ptr(), "bf16", 8, 100, 4,
                           stream=torch.cuda.current_stream().cuda_stream)
    for lens in ([300, 200, 97], [90, 200, 40], [299, 61, 96]):
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        check(batch, q, out, 8, "bf16", 100, 4)
    outs = [torch.zeros_like(q) for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        op_attention_cache(batch.cache, q.data_ptr(), o.data_ptr(), "bf16", 8, 100, 4,
                           stream=streams[i % 3].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 10 ** 6), (33, 33), (64, 31), (500, 1)])
def test_windows_over_prompt_rows(fmt, dtype, window, sinks):
    """Windows narrower than the rows of a call, sinks that reach into them, windows that begin inside a page."""
    lens, counts = [300, 40, 613], [290, 40, 77]
    batch = Batch(Pool(fmt, 1, 64, lens, seed=window), counts)
    q = queries(batch, 4, dtype, 2)
    check(batch, q, attend(batch, q, 4, dtype, window, sinks), 4, dtype, window, sinks)


@pytest.mark.parametrize("fmt", FORMATS)
def test_more_sequences_than_a_cta_sorts(fmt):
    lens = [(i * 37) % 70 for i in range(400)]
    batch = Batch(Pool(fmt, 1, 64, lens, seed=5), [1] * 400)
    for dtype in ("f32", "bf16"):
        q = queries(batch, 2, dtype, 2)
        check(batch, q, attend(batch, q, 2, dtype), 2, dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[1, 1, 1], [60, 50, 40]])
def test_sequences_that_share_pages(fmt, counts):
    """A common past: the block tables name the same pages, one of them twice in a row of the table."""
    pool = Pool(fmt, 2, 64, [100, 100, 96], seed=5)
    pool.table[1, :3] = pool.table[0, :3]
    pool.table[2, :3] = pool.table[0, [0, 0, 1]]
    pos = [np.arange(100), np.concatenate((np.arange(96), np.arange(96, 100))),
           np.concatenate((np.arange(32), np.arange(32), np.arange(32, 64)))]
    k, v = pool.k[0].copy(), pool.v[0].copy()
    own_k, own_v = pool.k[1].copy(), pool.v[1].copy()
    pool.k[2], pool.v[2] = k[pos[2]], v[pos[2]]
    pool.k[1] = np.concatenate((k[:96], own_k[96:]))
    pool.v[1] = np.concatenate((v[:96], own_v[96:]))
    batch = Batch(pool, counts)
    for dtype in ("f32", "bf16"):
        q = queries(batch, 8, dtype, 2)
        check(batch, q, attend(batch, q, 8, dtype), 8, dtype)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pools_beyond_four_gigabytes(fmt):
    """Pages whose byte offset passes 32 bits: attention (both kernels), append, read and copy."""
    Hkv, D = 8, 128
    page = cache_page_bytes(fmt, Hkv, D)
    n_pages = (5 << 30) // page
    small = Pool(fmt, Hkv, D, [70], seed=3, spare=0)
    at = np.array([n_pages - 1, n_pages // 2 + 7, n_pages - 3], np.int32)
    K = torch.empty((n_pages, page), dtype=torch.uint8, device=DEV)
    V = torch.empty_like(K)
    for pool, src in ((K, small.K), (V, small.V)):
        pool[torch.from_numpy(at).long().to(DEV)] = torch.from_numpy(
            src[small.table[0]].reshape(3, page)).to(DEV)
    table = torch.from_numpy(at).to(DEV)
    for r in (1, 65):
        lens = torch.tensor([70], dtype=torch.int32, device=DEV)
        start = torch.tensor([0, r], dtype=torch.int32, device=DEV)
        cache = kv_cache(fmt, Hkv, D, K.data_ptr(), V.data_ptr(), n_pages, table.data_ptr(), 3, 1, lens.data_ptr(),
                         start.data_ptr(), r, r)
        for dtype in ("f32", "bf16"):
            q = torch.randn((r, 32 * D), device=DEV).to(TYPES[dtype])
            out = torch.empty_like(q)
            op_attention_cache(cache, q.data_ptr(), out.data_ptr(), dtype, 32)
            qn = q.float().cpu().numpy().astype(np.float64).reshape(r, 32, D)
            want, *sizes = attention(qn, small.k[0], small.v[0], 70)
            tol = tolerance(want, *sizes, D, 70, dtype, fmt)
            assert np.all(np.abs(out.float().cpu().numpy().reshape(r, 32, D) - want) <= tol)
    got = torch.empty((2, 65, Hkv, D), device=DEV)
    op_cache_read(cache, got[0].data_ptr(), got[1].data_ptr(), "f32")
    assert np.array_equal(got[0].cpu().numpy(), small.k[0][5:].astype(np.float32))
    assert np.array_equal(got[1].cpu().numpy(), small.v[0][5:].astype(np.float32))
    x = torch.randn((65, Hkv * D), device=DEV)
    op_cache_append(cache, x.data_ptr(), x.data_ptr(), "f32")
    op_cache_read(cache, got[0].data_ptr(), got[1].data_ptr(), "f32")
    assert torch.equal(got[0], got[1]) and not torch.equal(got[0], torch.zeros_like(got[0]))
    op_cache_copy([K.data_ptr(), V.data_ptr()], page, n_pages, at[:1], [n_pages - 2])
    assert torch.equal(K[n_pages - 2], K[n_pages - 1]) and torch.equal(V[n_pages - 2], V[n_pages - 1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_decode_step_captured_whole(fmt):
    """append, attention, read and a page copy in one graph, replayed with other rows and lengths; no err word, no
    row_start."""
    pool = Pool(fmt, 2, 64, [70, 33, 64], seed=5, spare=4)
    batch = Batch(pool, [1, 1, 1])
    batch.cache.row_start = None
    batch.cache.err = None
    k, v = torch.zeros((3, 128), device=DEV), torch.zeros((3, 128), device=DEV)
    back = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device=DEV)
    q = queries(batch, 8, "f32", 1)
    out = torch.zeros_like(q)
    free = sorted(set(range(pool.n_pages)) - set(pool.table[pool.table >= 0].tolist()))[0]
    src = int(pool.table[0, 0])
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        s = torch.cuda.current_stream().cuda_stream
        op_cache_append(batch.cache, k.data_ptr(), v.data_ptr(), "f32", s)
        op_attention_cache(batch.cache, q.data_ptr(), out.data_ptr(), "f32", 8, 40, 3, stream=s)
        op_cache_read(batch.cache, back[0].data_ptr(), back[1].data_ptr(), "bf16", s)
        op_cache_copy([batch.K.data_ptr(), batch.V.data_ptr()], cache_page_bytes(fmt, 2, 64), pool.n_pages, [src],
                      [free], s)
    rng = np.random.default_rng(0)
    for lens in ([70, 33, 64], [69, 20, 32], [1, 33, 64]):
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        rows = rng.standard_normal((2, 3, 2, 64)).astype(np.float32)
        k.copy_(torch.from_numpy(rows[0].reshape(3, 128)))
        v.copy_(torch.from_numpy(rows[1].reshape(3, 128)))
        held = [[], []]
        for b, n in enumerate(lens):
            pool.k[b][n - 1:n] = pool.put(0, b, n - 1, rows[0, b:b + 1])
            pool.v[b][n - 1:n] = pool.put(1, b, n - 1, rows[1, b:b + 1])
            held[0].append(pool.k[b][n - 1])
            held[1].append(pool.v[b][n - 1])
        g.replay()
        check(batch, q, out, 8, "f32", 40, 3)
        want = torch.from_numpy(np.stack([np.stack(h) for h in held])).float().to(torch.bfloat16)
        assert torch.equal(back.cpu(), want.reshape(2, 3, 128))
        assert torch.equal(batch.K[free], batch.K[src]) and torch.equal(batch.V[free], batch.V[src])


def test_append_of_negative_zeros_and_ties_stores_what_the_definition_says():
    """-0, values on the borders between two codes, and a block whose scale rounds to 0 beside a large one."""
    pool = Pool("nvfp4", 1, 64, [8], seed=0)
    batch = Batch(pool, [8])
    x = np.zeros((8, 64), np.float32)
    edges = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    x[0, :8], x[0, 8:16] = edges, -edges
    x[1] = -0.0
    x[1, 5] = 1.0
    x[2, 0], x[2, 16] = 1e30, 1e20
    x[3] = np.float32(1e-38)
    x[4, ::2] = np.nextafter(np.repeat(edges, 4), np.float32(9))[:32]
    x[4, 1::2] = np.nextafter(np.repeat(edges, 4), np.float32(0))[:32]
    x[5] = np.random.default_rng(0).integers(-12, 13, 64) / 2.0
    x[6] = np.float32(3e38)
    xd = torch.from_numpy(x).to(DEV)
    op_cache_append(batch.cache, xd.data_ptr(), xd.data_ptr(), "f32")
    pool.put(0, 0, 0, x[:, None])
    pool.put(1, 0, 0, x[:, None])
    assert np.array_equal(batch.K.cpu().numpy(), pool.K)
    assert np.array_equal(batch.V.cpu().numpy(), pool.V)
