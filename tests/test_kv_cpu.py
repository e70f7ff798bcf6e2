"""The 4-bit cache without a device: the statement that the GPU tests compare
with, and what the library refuses before it touches one."""
import ctypes

import numpy as np
import pytest

import kv_plain as K


@pytest.fixture(scope="module")
def q():
    return pytest.importorskip("quantized_base_lora_gb300")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_every_code_has_an_address_of_its_own(dim, page):
    for address in (K.key_address, K.value_address):
        seen = {address(s, c, dim) for s in range(page) for c in range(dim)}
        assert len(seen) == page * dim
        assert min(a for a, _ in seen) == 0 and max(a for a, _ in seen) == page * dim // 2 - 1


def test_addresses_by_hand():
    assert K.key_address(0, 0, 128) == (0, True) and K.key_address(0, 1, 128) == (0, False)
    assert K.key_address(0, 8, 128) == (16, True)       # word 1 of block 0, behind word 0 of the four blocks
    assert K.key_address(0, 32, 128) == (4, True)       # word 0 of block 1
    assert K.key_address(3, 127, 128) == (3 * 64 + 63, False)
    assert K.value_address(0, 1, 128) == (64, True)     # unit 1
    assert K.value_address(0, 8, 128) == (0, False)     # the second channel of unit 0
    assert K.value_address(1, 0, 128) == (8, True)      # the next token's unit 0
    assert K.value_address(8, 0, 128) == (512, True)    # the next 8 tokens


def test_quantizer_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [8.0, -8.0, 0.5, -1.5]                   # d = 1: 8 is clipped to 7, halves go away from zero
    code, d = K.quantize(x)
    assert d[0, 0] == 1 and d[0, 1] == 0
    np.testing.assert_array_equal(code[0, :5], [15, 0, 9, 6, 8])
    assert (code[0, 32:] == 8).all()
    big = np.full((1, 32), np.inf, np.float32)
    big[0, 0] = np.nan
    code, d = K.quantize(big)
    assert d[0, 0] == 65504 and code[0, 0] == 8 and (code[0, 1:] == 15).all()


def test_attention_by_hand():
    k = np.zeros((4, 1, 2))
    v = np.arange(8, dtype=np.float64).reshape(4, 1, 2)
    out, _, _ = K.attention(np.ones((1, 1, 2)), k, v, [2], 1.0)
    np.testing.assert_allclose(out[0, 0], v[:3, 0].mean(0))
    out, _, _ = K.attention(np.ones((1, 1, 2)), k, v, [3], 1.0, window=1, sinks=1)
    np.testing.assert_allclose(out[0, 0], (v[0, 0] + v[3, 0]) / 2)
    out, _, _ = K.attention(np.ones((1, 1, 2)), k, v, [-1], 1.0)
    assert (out == 0).all()


def dims(q, **kw):
    d = dict(n_pages=10, page_tokens=64, n_layers=2, n_kv_heads=8, head_dim=128, max_seqs=4, max_pages=8)
    d.update(kw)
    kv = q.ovl_kv()
    for name, value in d.items():
        setattr(kv, name, value)
    return kv


def test_workspace_size(q):
    st, n = q.ovl_kv_workspace_bytes(dims(q))
    assert st == q.OVL_OK and n >= 4 * 8 * 4
    assert q.ovl_kv_workspace_bytes(dims(q, head_dim=256))[1] > n
    assert q.lib.ovl_kv_workspace_bytes(None, ctypes.byref(ctypes.c_size_t())) == q.OVL_E_ARG
    assert q.lib.ovl_kv_workspace_bytes(ctypes.byref(dims(q)), None) == q.OVL_E_ARG


@pytest.mark.parametrize("bad", [dict(head_dim=0), dict(head_dim=80), dict(page_tokens=0), dict(page_tokens=48),
                                 dict(page_tokens=512), dict(n_pages=0), dict(n_layers=0), dict(n_kv_heads=0),
                                 dict(max_seqs=0), dict(max_seqs=65537), dict(max_pages=0), dict(max_pages=1 << 24),
                                 dict(n_layers=60000, n_kv_heads=64)])
def test_dimensions_that_are_refused(q, bad):
    st, n = q.ovl_kv_workspace_bytes(dims(q, **bad))
    assert st == q.OVL_E_SHAPE and n == 0
    assert q.ovl_last_error(None)


def test_missing_pointers_are_refused_without_a_device(q):
    kv = dims(q)
    assert q.ovl_kv_init(kv) == q.OVL_E_ARG
    assert q.ovl_kv_extend(kv, 16, 16, 1) == q.OVL_E_ARG
    assert q.ovl_kv_check(kv) == q.OVL_E_ARG
    assert "null" in q.ovl_last_error(None)
    for f in ("codes", "scales", "table", "length", "refs"):
        setattr(kv, f, 4096)
    kv.workspace, kv.workspace_bytes = 4096, 128
    assert q.ovl_kv_release(kv, 16, 1) == q.OVL_E_OOM
    kv.workspace_bytes = 1 << 40
    kv.codes = 4104
    assert q.ovl_kv_release(kv, 16, 1) == q.OVL_E_SHAPE
    kv.codes = 4096
    assert q.ovl_kv_release(kv, 16, 1025) == q.OVL_E_ARG
    assert q.ovl_kv_append(kv, 2, 16, 16, 1, 1, 16, 16, q.OVL_F32, 1024, 1024) == q.OVL_E_ARG      # layer
    assert q.ovl_kv_append(kv, 0, 16, 16, 1, 1, 16, 16, 7, 1024, 1024) == q.OVL_E_ARG              # dtype
    assert q.ovl_kv_append(kv, 0, 16, 16, 1, 1, 16, 16, q.OVL_F32, 1000, 1024) == q.OVL_E_SHAPE    # stride
    assert q.ovl_kv_attention(kv, 0, 16, 16, 1, 1, 1, 16, q.OVL_BF16, 12, 1536, 1.0, 0, 0, 16, 1536) == q.OVL_E_SHAPE
    assert q.ovl_kv_attention(kv, 0, 16, 16, 1, 1, 1, 16, q.OVL_BF16, 8, 1024, float("inf"), 0, 0, 16,
                              1024) == q.OVL_E_ARG
