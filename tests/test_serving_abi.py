"""The serving operators' C entries: declared, exported, and checked before any HIP call.  CPU only."""
import ctypes
import os

import pytest

import post_weight_quantization_gptq_amd as g

NAMES = ("gptq_rope_table", "gptq_rope", "gptq_kv_write", "gptq_kv_read", "gptq_tree_attention")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g.library_path()):
        from post_weight_quantization_gptq_amd import build_lib
        build_lib.build()
    return g.load_library()


def test_header_declares_and_library_exports(lib):
    declared = g.exported_symbols()
    for name in NAMES:
        assert name in declared and hasattr(lib, name)


def test_null_context_is_refused(lib):
    """Every entry returns GPTQ_ERR_INVALID_ARG for a null context, whatever else it is given."""
    i64 = ctypes.c_int64
    assert lib.gptq_rope_table(None, 4, 8, 1e4, None, None) == 1
    assert lib.gptq_rope(None, None, 0, i64(1), 1, 8, i64(8), i64(8), None, None, 4, 8, 0, 0, None, 0, i64(8), i64(8)) == 1
    assert lib.gptq_kv_write(None, None, None, None, 0, i64(1), i64(0), i64(0), i64(0), i64(0), None) == 1
    assert lib.gptq_kv_read(None, None, None, i64(1), None, None, 0, i64(0), i64(0), i64(0), i64(0)) == 1
    assert lib.gptq_tree_attention(None, None, None, 1, 1, 1, i64(0), i64(0), i64(0), None, 1, None, None, 0, 1.0, None,
                                   i64(0), i64(0), i64(0)) == 1


def test_descriptors_have_the_header_s_size():
    """Six pointers and six 32-bit numbers; two 32-bit numbers and four doubles."""
    assert ctypes.sizeof(g._KV) == 6 * 8 + 6 * 4
    assert ctypes.sizeof(g._RopeScaling) == 2 * 4 + 4 * 8


def test_cache_needs_gpu_tensors():
    torch = pytest.importorskip("torch")
    t = dict(k_codes=torch.zeros((1, 1, 16, 64), dtype=torch.uint8), k_scales=torch.zeros((1, 1, 16)),
             k_zeros=torch.zeros((1, 1, 16), dtype=torch.uint8), v_codes=torch.zeros((1, 1, 64, 16), dtype=torch.uint8),
             v_scales=torch.zeros((1, 1, 16)), v_zeros=torch.zeros((1, 1, 16), dtype=torch.uint8))
    with pytest.raises(ValueError):
        g.KVCache(bits=8, **t)
    with pytest.raises(ValueError):
        g.KVCache(bits=6, **t)
