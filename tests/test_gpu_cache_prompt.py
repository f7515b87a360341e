"""Attention over a paged cache for batches of many bfloat16 rows (8 KV heads and a few hundred rows, for which the
tensor-core kernel is the faster one), against float64 numpy."""
import numpy as np
import pytest
import torch

from cache_oracle import Pool
from dual_ar_decode_gb300 import op_attention_cache
from dual_ar_decode_gb300.binding import TF_CACHE_BAD_LENGTH, TF_CACHE_BAD_PAGE, TF_CACHE_BAD_ROWS
from test_gpu_cache import DEV, FORMATS, TYPES, Batch, attend, check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


_POOLS = {}


def pool_of(fmt, Hkv, D, lens):
    key = (fmt, Hkv, D, tuple(lens))
    if key not in _POOLS:
        _POOLS[key] = Pool(fmt, Hkv, D, lens, seed=sum(lens))
    return _POOLS[key]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3), (128, 128), (200, 31), (1000, 7)])
@pytest.mark.parametrize("Hkv,ratio,D", [(8, 4, 128), (8, 2, 64)])
def test_windows(fmt, window, sinks, Hkv, ratio, D):
    """Sequences that are all rows, rows behind a long past, a few rows, none, and rows at negative positions."""
    lens, counts = [257, 600, 290, 64, 30], [257, 300, 5, 0, 45]
    batch = Batch(pool_of(fmt, Hkv, D, lens), counts, extra_rows=3)
    q = queries(batch, Hkv * ratio, "bf16", 5)
    check(batch, q, attend(batch, q, Hkv * ratio, "bf16", window, sinks), Hkv * ratio, "bf16", window, sinks)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hkv,ratio,D", [(8, 1, 128), (8, 3, 128), (8, 5, 64), (6, 6, 64), (8, 7, 128), (8, 8, 64)])
def test_head_layouts(fmt, Hkv, ratio, D):
    """Every number of heads per KV head: those that do not divide a tile leave pairs of one row in two CTAs."""
    lens, counts = [400, 333, 300], [400, 290, 203]
    batch = Batch(pool_of(fmt, Hkv, D, lens), counts, extra_rows=1)
    q = queries(batch, Hkv * ratio, "bf16", 6)
    check(batch, q, attend(batch, q, Hkv * ratio, "bf16", 170, 9), Hkv * ratio, "bf16", 170, 9)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("pad", [1, 3, 8, 64])
def test_strides_and_scale(fmt, pad):
    """Rows further apart than they are long: 16-byte aligned (moved as boxes) and not (moved by the threads)."""
    lens, counts = [300, 280], [299, 130]
    batch = Batch(pool_of(fmt, 8, 64, lens), counts, extra_rows=2)
    q = queries(batch, 32, "bf16", 2, pad=pad)
    check(batch, q, attend(batch, q, 32, "bf16", 0, 0, 0.25, pad=pad), 32, "bf16", scale=0.25)
    check(batch, q, attend(batch, q, 32, "bf16", 90, 2, 0.0, pad=pad + 7), 32, "bf16", 90, 2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_begin_inside_the_buffer_at_odd_places(fmt):
    """Queries and outputs that do not begin on 16 bytes."""
    lens, counts = [260, 200], [250, 160]
    batch = Batch(pool_of(fmt, 8, 128, lens), counts)
    n = batch.n_rows * 4096
    flat = torch.randn(n + 8, device=DEV).to(torch.bfloat16)
    for qo, oo in ((1, 0), (0, 1), (8, 8), (3, 5)):
        q = flat[qo:qo + n].view(batch.n_rows, 4096)
        room = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device=DEV)
        op_attention_cache(batch.cache, q.data_ptr(), room.data_ptr() + 2 * oo, "bf16", 32)
        check(batch, q, room[oo:oo + n].view(batch.n_rows, 4096), 32, "bf16")
        assert (room[:oo] == 7.0).all() and (room[oo + n:] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_positions_that_are_not_finite(fmt):
    """Rows that see them show it, the other rows of the same tile do not."""
    lens, counts = [500, 300], [300, 200]
    pool = Pool(fmt, 8, 64, lens, seed=3)
    bad = np.full((1, 8, 64), np.nan, np.float32)
    pool.put(0, 0, 230, bad)                                 # row 30 of sequence 0 sees it first
    pool.put(1, 0, 333, np.full((1, 8, 64), np.inf, np.float32))
    batch = Batch(pool, counts)
    q = queries(batch, 32, "bf16", 1)
    out = attend(batch, q, 32, "bf16")
    torch.cuda.synchronize()
    fine = torch.isfinite(out)
    assert fine[:30].all() and fine[300:].all() and not fine[30:300].any()
    out = attend(batch, q, 32, "bf16", 50, 0)                # ... and rows past the window no longer
    torch.cuda.synchronize()
    fine = torch.isfinite(out)
    assert fine[:30].all() and not fine[30:80].any() and fine[80:133].all()
    assert not fine[133:183].any() and fine[183:].all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_descriptions(fmt):
    lens, counts = [300, 250, 200], [200, 150, 100]
    pool = Pool(fmt, 8, 64, lens, seed=2)
    pool.table[0, 3] = pool.n_pages
    pool.table[1, 0] = -7
    pool.table[1, 5] = 1 << 30
    hidden = [np.zeros(n, bool) for n in lens]
    hidden[0][96:128] = True
    hidden[1][:32] = True
    hidden[1][160:192] = True
    batch = Batch(pool, counts)
    q = queries(batch, 32, "bf16", 1)
    check(batch, q, attend(batch, q, 32, "bf16"), 32, "bf16", hidden=hidden, err=TF_CACHE_BAD_PAGE)
    pool = pool_of(fmt, 8, 64, lens)
    for what in ("length", "rows"):
        batch = Batch(pool, counts)
        if what == "length":
            batch.lens[1] = -1
        else:
            batch.cache.max_rows = 199
        out = attend(batch, q, 32, "bf16")
        torch.cuda.synchronize()
        assert batch.err.item() == (TF_CACHE_BAD_LENGTH if what == "length" else TF_CACHE_BAD_ROWS)
        skipped = slice(200, 350) if what == "length" else slice(0, 200)
        left = torch.ones(450, dtype=torch.bool)
        left[skipped] = False
        assert (out[skipped] == 7.0).all() and (out[left.to(DEV)] != 7.0).any(1).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("what", ["ramp", "jump", "values"])
def test_references_that_have_to_be_replaced(fmt, what):
    """As the test of the same name for few rows, with every tile of keys outgrowing the references of the ones
    before, inside a tile and between tiles."""
    n, r = 700, 260
    pool = Pool(fmt, 8, 128, [n], seed=4)
    rng = np.random.default_rng(1)
    d = rng.choice(np.array([-1.0, 1.0], np.float32), 128)
    top = np.linspace(0, 60, n) if what == "ramp" else np.linspace(0, 3, n)
    if what == "jump":
        top[[333, 470]] = 140
    if what == "values":
        top = np.linspace(25, 0, n)
        v = rng.standard_normal((n, 8, 128)) * 2.0 ** np.linspace(-20, 20, n)[:, None, None]
        pool.v[0][:] = pool.put(1, 0, 0, v.astype(np.float32))
    k = (d * top[:, None].astype(np.float32) * np.float32(128 ** 0.5 / 128))[:, None] + 0.05 * rng.standard_normal((n, 8, 128))
    pool.k[0][:] = pool.put(0, 0, 0, k.astype(np.float32))
    batch = Batch(pool, [r])
    q = torch.from_numpy(np.tile(d, (batch.n_rows, 32)).astype(np.float32)).to(TYPES["bf16"]).to(DEV)
    check(batch, q, attend(batch, q, 32, "bf16"), 32, "bf16")
    check(batch, q, attend(batch, q, 32, "bf16", 450, 7), 32, "bf16", 450, 7)


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_call_after_another_and_side_by_side(fmt):
    """Results repeat bit for bit, on three streams at once and from a graph."""
    lens, counts = [500, 300], [300, 200]
    batch = Batch(pool_of(fmt, 8, 64, lens), counts)
    q = queries(batch, 32, "bf16", 1)
    first = attend(batch, q, 32, "bf16", 100, 5)
    check(batch, q, first, 32, "bf16", 100, 5)
    outs = [torch.zeros_like(q) for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        op_attention_cache(batch.cache, q.data_ptr(), o.data_ptr(), "bf16", 32, 100, 5, stream=streams[i % 3].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op_attention_cache(batch.cache, q.data_ptr(), outs[0].data_ptr(), "bf16", 32, 100, 5,
                           stream=torch.cuda.current_stream().cuda_stream)
    outs[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first)
    batch.lens.copy_(torch.tensor([450, 270], dtype=torch.int32))
    g.replay()
    check(batch, q, outs[0], 32, "bf16", 100, 5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hkv,ratio,D,pad", [(8, 4, 128, 0), (8, 4, 64, 0), (8, 3, 64, 0), (8, 4, 64, 1)])
def test_many_rows_at_negative_positions(fmt, Hkv, ratio, D, pad):
    """Whole tiles of rows before position 0, among others: zeros, whatever the queries hold, and nothing of them is
    left behind for the tiles that follow."""
    lens, counts = [600, 20, 0, 400], [300, 500, 200, 400]
    batch = Batch(pool_of(fmt, Hkv, D, lens), counts)
    q = queries(batch, Hkv * ratio, "bf16", 8, pad=pad)
    q[300:780] = float("nan")                            # the 480 rows of the second sequence, the 200 of the third
    q[800:1000] = float("nan")
    outs = [attend(batch, q, Hkv * ratio, "bf16", pad=pad) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert (outs[0][300:780, :Hkv * ratio * D] == 0).all() and (outs[0][800:1000, :Hkv * ratio * D] == 0).all()
    q[300:780] = 1.0                                     # (the oracle takes finite queries)
    q[800:1000] = 1.0
    check(batch, q, outs[0], Hkv * ratio, "bf16")
