"""The C-ABI library builds, loads and exports every declared entry point.

No compute calls: these run without a GPU.  Host-side validation that needs
no device (bad configurations, NULL handles) is exercised too.
"""
import ctypes
import os
import re

import pytest

import __graft_entry__
from dual_ar_decode_gb300 import binding
from synth import FULL, TINY

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return binding.lib()


def declared_symbols():
    src = open(os.path.join(ROOT, "include", "tf.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(tf_[a-z0-9_]+)\s*\(", src)))


def test_every_declared_symbol_is_exported(L):
    names = declared_symbols()
    assert {"tf_create", "tf_load_weights", "tf_prefill", "tf_decode_frame", "tf_destroy"} <= set(names)
    for n in names:
        assert hasattr(L, n), n
    assert set(names) == set(binding.EXPORTS)


def test_library_is_built_for_sm103a_only():
    from dual_ar_decode_gb300 import build as b
    assert "arch=compute_103a,code=sm_103a" in " ".join(b.NVCC_FLAGS)


def test_destroy_null_and_last_error(L):
    L.tf_destroy(None)
    assert isinstance(L.tf_last_error(None), bytes)


@pytest.mark.parametrize("change,needle", [
    (dict(head_dim=96), b"head_dim"),
    (dict(n_kv_heads=3), b"multiple of n_kv_heads"),
    (dict(n_codebooks=8), b"n_codebooks"),
    (dict(semantic_vocab=10_000), b"semantic_vocab"),
    (dict(max_seq_len=5), b"max_seq_len"),
    (dict(max_batch=0), b"max_batch"),
    (dict(max_batch=33), b"max_batch"),
    (dict(hidden=250), b"hidden"),
    (dict(flags=16), b"flags"),
])
def test_create_rejects_bad_config_before_touching_a_device(L, change, needle):
    cfg = binding.config_from_dims(TINY)
    for k, v in change.items():
        setattr(cfg, k, v)
    h = ctypes.c_void_p()
    st = L.tf_create(ctypes.byref(cfg), 0, ctypes.byref(h))
    assert st == 1 and not h.value
    assert needle in L.tf_last_error(None)


def test_create_without_device_fails_cleanly(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    cfg = binding.config_from_dims(FULL)
    h = ctypes.c_void_p()
    assert L.tf_create(ctypes.byref(cfg), 0, ctypes.byref(h)) == 1
    assert b"device" in L.tf_last_error(None)


def test_op_argument_validation_is_host_side(L):
    s = binding.TfSampling(0, 1.0, 0, 1.0, 1.0, 0)
    assert L.tf_op_select(None, 1, 64, ctypes.byref(s), 0, 0, 0, None, 0, None, None) == 1
    ok = ctypes.c_void_p(16)   # never dereferenced: the arguments are refused first
    bad_p = binding.TfSampling(30, 1.0, 0, 1.5, 1.0, 0)
    assert L.tf_op_select(ok, 1, 64, ctypes.byref(bad_p), 0, 0, 0, None, 0, ok, None) == 1
    assert L.tf_op_select(ok, 1, 64, ctypes.byref(s), 0, 0, 0, None, 3, ok, None) == 1   # window, no ids
    assert L.tf_op_select(ok, 1, 64, ctypes.byref(s), 0, 0, 0, ok, 65, ok, None) == 1    # window > 64
    assert L.tf_op_quantize_fp8(None, 1, 16, None, None, None) == 1
    assert L.tf_test_inject(None, 1) == 1
    assert L.tf_op_gemv(None, 0, None, 1, 16, None, None, 1, None, None) == 1
    assert L.tf_op_gemm_skinny(None, None, 16, 256, 256, None, None) == 1
    assert L.tf_op_gemm_skinny(1, 1, 65, 256, 256, 1, None) == 1   # more than 64 rows
    assert L.tf_op_gemm_skinny(1, 1, 16, 255, 256, 1, None) == 1   # odd N
    assert L.tf_op_gemm_skinny(1, 1, 16, 256, 100, 1, None) == 1   # K not a multiple of 8


# ---------------------------------------------------------------- cache operators: refusals on the host

def cache_args(**change):
    """A description that would pass the host's checks (its pointers are never followed on the CPU)."""
    a = dict(format=binding.TF_KV_NVFP4, n_kv_heads=2, head_dim=128, n_pages=8, K=1 << 20, V=2 << 20,
             block_table=3 << 20, table_stride=4, n_seq=2, lengths=4 << 20, row_start=5 << 20, n_rows=6,
             max_rows=4, max_length=0, err=None)
    a.update(change)
    return binding.TfKvCache(**a)


BAD_CACHES = [dict(format=2), dict(format=-1), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=0),
              dict(n_pages=0), dict(K=None), dict(V=None), dict(K=(1 << 20) + 64), dict(V=(2 << 20) + 16),
              dict(block_table=None), dict(block_table=(3 << 20) + 2), dict(table_stride=0), dict(n_seq=0),
              dict(n_seq=65536), dict(lengths=None), dict(lengths=(4 << 20) + 1), dict(row_start=(5 << 20) + 3),
              dict(n_rows=-1), dict(max_rows=-1), dict(max_length=-1), dict(err=(6 << 20) + 1),
              dict(row_start=None, n_rows=1), dict(row_start=None, max_rows=0),
              dict(n_pages=1 << 26, n_kv_heads=1), dict(table_stride=1 << 30)]


@pytest.mark.parametrize("change", BAD_CACHES)
def test_cache_operators_refuse_bad_descriptions(L, change):
    c = cache_args(**change)
    q = 7 << 20
    assert L.tf_op_attention_cache(c, q, 0, q + 4096, 0, binding.TF_DTYPE_F32, 8, 0, 0, 0.0, None) == 1
    assert L.tf_op_cache_append(c, q, q, 0, binding.TF_DTYPE_F32, None) == 1
    assert L.tf_op_cache_read(c, q, q, 0, binding.TF_DTYPE_F32, None) == 1


def test_cache_operators_refuse_bad_rows(L):
    c = cache_args()
    f32, bf16, q = binding.TF_DTYPE_F32, binding.TF_DTYPE_BF16, 7 << 20
    call = lambda *a: L.tf_op_attention_cache(c, *a, None)  # noqa: E731
    for a in [(None, 0, q, 0, f32, 8, 0, 0, 0.0), (q, 0, None, 0, f32, 8, 0, 0, 0.0),
              (q + 2, 0, q, 0, f32, 8, 0, 0, 0.0), (q, 0, q + 1, 0, bf16, 8, 0, 0, 0.0),
              (q, 0, q, 0, 1, 8, 0, 0, 0.0), (q, 0, q, 0, 7, 8, 0, 0, 0.0), (q, 0, q, 0, f32, 0, 0, 0, 0.0),
              (q, 0, q, 0, f32, 7, 0, 0, 0.0), (q, 0, q, 0, f32, 18, 0, 0, 0.0), (q, 0, q, 0, f32, 8, -1, 0, 0.0),
              (q, 0, q, 0, f32, 8, 4, -1, 0.0), (q, 0, q, 0, f32, 8, 0, 0, -1.0),
              (q, 0, q, 0, f32, 8, 0, 0, float("nan")), (q, 0, q, 0, f32, 8, 0, 0, float("inf")),
              (q, 1023, q, 0, f32, 8, 0, 0, 0.0), (q, 0, q, 1023, f32, 8, 0, 0, 0.0), (q, -1, q, 0, f32, 8, 0, 0, 0.0)]:
        assert call(*a) == 1, a
    for f in (L.tf_op_cache_append, L.tf_op_cache_read):
        for a in [(None, q, 0, f32), (q, None, 0, f32), (q + 1, q, 0, f32), (q, q + 1, 0, bf16), (q, q, 255, f32),
                  (q, q, -4, f32), (q, q, 0, 1), (q, q, 0, 9)]:
            assert f(c, *a, None) == 1, a
    # no rows: nothing to enqueue, whatever the device
    for none in (cache_args(n_rows=0), cache_args(max_rows=0)):
        assert L.tf_op_attention_cache(none, q, 0, q, 0, f32, 8, 0, 0, 0.0, None) == 0
        assert L.tf_op_cache_append(none, q, q, 0, f32, None) == 0


def test_cache_copy_refuses_overlapping_lists(L):
    pools = (ctypes.c_void_p * 2)(1 << 20, 2 << 20)

    def call(src, dst, n_pools=2, page=4864, pages=10, n=None, p=pools):
        a = (ctypes.c_int32 * max(1, len(src)))(*src)
        b = (ctypes.c_int32 * max(1, len(dst)))(*dst)
        return L.tf_op_cache_copy(p, n_pools, page, pages, a, b, len(src) if n is None else n, None)
    assert call([], []) == 0
    for src, dst in [([0], [10]), ([10], [0]), ([-1], [0]), ([0], [-1]), ([0, 1], [2, 2]), ([0, 1], [1, 2]),
                     ([3], [3]), ([0, 2], [2, 3])]:
        assert call(src, dst) == 1, (src, dst)
    assert call([0], [1], n_pools=0) == 1 and call([0], [1], pages=0) == 1 and call([0], [1], n=-1) == 1
    for page in (0, 8, 4860, 1 << 31):
        assert call([0], [1], page=page) == 1
    assert call([0], [1], p=(ctypes.c_void_p * 2)(1 << 20, None)) == 1
    assert call([0], [1], p=(ctypes.c_void_p * 2)(1 << 20, (2 << 20) + 8)) == 1


def test_cache_page_bytes(L):
    assert binding.cache_page_bytes("bf16", 8, 128) == 65536
    assert binding.cache_page_bytes("nvfp4", 8, 128) == 8 * 2432
    assert binding.cache_page_bytes("nvfp4", 1, 64) == 1280
    assert L.tf_op_cache_page_bytes(2, 1, 64) == 0 and L.tf_op_cache_page_bytes(0, 0, 64) == 0
    assert L.tf_op_cache_page_bytes(0, 1, 63) == 0
