"""The torch side of the 4-bit cache without a device: what reaches the library, and on which device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


class Library:
    """Stands in for the library: records each call with the device that is current."""

    def __init__(self, where):
        self.where, self.calls = where, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.where["device"], args))
            return 0
        return call


@pytest.fixture
def stand_in(monkeypatch):
    """A cache of CPU tensors (their device's index is -1) while device 0 is current, and the library's stand-in."""
    pytest.importorskip("quantized_base_lora_gb300")
    from quantized_base_lora_gb300 import kvcache, ovl_kv
    where = {"device": 0}

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, where["device"] = where["device"], self.index

        def __exit__(self, *_):
            where["device"] = self.before

    lib = Library(where)
    monkeypatch.setattr(kvcache, "lib", lib)
    monkeypatch.setattr(kvcache, "_raw_stream", lambda index: 7000 + index)
    monkeypatch.setattr(kvcache, "_current_device", lambda: where["device"], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: where["device"])
    monkeypatch.setattr(torch.cuda, "device", device)
    c = object.__new__(kvcache.KvCache)
    c.kv = ovl_kv()
    c._at, c._index, c._scale = ctypes.addressof(c.kv), -1, 0.125
    c.device, c.n_kv_heads, c.head_dim, c.page_tokens = torch.device("cpu"), 2, 64, 16
    return c, lib, where


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def every_call(c):
    one, off, x = ints(0), ints(0, 1), torch.zeros((1, 2, 64))
    c.extend(one, off)
    c.append(0, one, off, x, x)
    c.read(0, one, off, 1)
    c.attention(0, one, off, x, 1)
    c.attention(0, one, off, x, 1, out=torch.zeros((1, 2, 64)))
    c.fork(one, ints(1))
    c.fork(one, ints(1), ints(1))
    c.compact(one, ints(1), ints(0), off)
    c.release(one)
    c.check()


def test_every_call_runs_on_the_caches_device(stand_in):
    c, lib, where = stand_in
    every_call(c)
    assert [n for n, _, _ in lib.calls] == ["ovl_kv_" + n for n in (
        "extend", "append", "read", "attention", "attention", "fork", "fork", "compact", "release", "check")]
    for name, device, args in lib.calls:
        assert device == -1, name                        # the cache's device was current
        assert args[0] == c._at and args[-1] == 6999     # and the stream is that device's
    assert where["device"] == 0                          # the caller's device is current again


def test_a_cache_on_the_current_device_changes_no_device(stand_in, monkeypatch):
    c, lib, where = stand_in
    where["device"] = -1
    monkeypatch.setattr(torch.cuda, "device", None)
    every_call(c)
    assert all(device == -1 for _, device, _ in lib.calls) and len(lib.calls) == 10


def test_the_device_is_restored_when_a_call_is_refused(stand_in):
    c, lib, where = stand_in
    from quantized_base_lora_gb300 import OvlError
    lib.ovl_kv_release = lambda *a: -1
    with pytest.raises(OvlError):
        c.release(ints(0))
    assert where["device"] == 0


# ---------------------------------------------------------------- which kernel

FEW, SINGLE, PAIRS = range(3)


def route(n_seqs, n_tokens, max_new, heads, kv=8, dim=128, bf16=True, sms=152):
    q = pytest.importorskip("quantized_base_lora_gb300")
    d = q.ovl_kv()
    for name, value in dict(n_pages=9, page_tokens=64, n_layers=1, n_kv_heads=kv, head_dim=dim, max_seqs=9,
                            max_pages=9).items():
        setattr(d, name, value)
    st, r = q.ovl_debug_kv_route(d, n_seqs, n_tokens, max_new, q.OVL_BF16 if bf16 else q.OVL_F32, heads, sms)
    assert st == q.OVL_OK
    return r


def test_which_kernel_serves_a_call():
    assert route(32, 32, 1, 32) == FEW                                   # decode steps
    assert route(2, 4096, 2048, 32) == PAIRS                             # chunks of prompts
    assert route(2, 4096, 2048, 32, bf16=False) == FEW                   # which f32 calls have no other kernel for
    assert route(4, 3108, 777, 24, kv=3, dim=64) == SINGLE
    assert route(2, 4096, 2048, 32, dim=256) == SINGLE


@pytest.mark.parametrize("dim,rows", [(64, 256), (128, 256), (256, 128)])
def test_row_tiles_beyond_the_grid_stay_with_the_kernel_for_few_rows(dim, rows):
    group, most = 8, 65535 * rows // 8
    assert route(1, most, most, 8 * group, dim=dim) != FEW
    assert route(1, most + 1, most + 1, 8 * group, dim=dim) == FEW
    assert route(1, 2 ** 31 - 1, 2 ** 31 - 1, 8 * 1024, dim=dim) == FEW


def test_refusals_of_the_route():
    q = pytest.importorskip("quantized_base_lora_gb300")
    d = q.ovl_kv()
    assert q.ovl_debug_kv_route(d, 1, 1, 1, q.OVL_BF16, 8, 152)[0] == q.OVL_E_SHAPE
    for name, value in dict(n_pages=9, page_tokens=64, n_layers=1, n_kv_heads=8, head_dim=64, max_seqs=9,
                            max_pages=9).items():
        setattr(d, name, value)
    assert q.ovl_debug_kv_route(d, 1, 1, 1, 77, 8, 152)[0] == q.OVL_E_ARG
    assert q.ovl_debug_kv_route(d, 1, 1, 1, q.OVL_BF16, 8, 0)[0] == q.OVL_E_ARG
    assert q.ovl_debug_kv_route(d, 1, 1, 1, q.OVL_BF16, 12, 152)[0] == q.OVL_E_SHAPE
    assert q.lib.ovl_debug_kv_route(ctypes.byref(d), 1, 1, 1, q.OVL_BF16, 8, 152, None) == q.OVL_E_ARG


# ---------------------------------------------------------------- numbers beyond 32 bits

@pytest.mark.parametrize("bad", [-1, 1 << 32, (1 << 32) + 4])
def test_numbers_that_32_bits_would_change_are_refused(stand_in, bad):
    """-1 sinks would be 2^32 - 1 and make every token visible; 2^32 + 4 would be 4."""
    c, lib, _ = stand_in
    one, off, x = ints(0), ints(0, 1), torch.zeros((1, 2, 64))
    for kw in (dict(sinks=bad), dict(window=bad), dict(window=8, sinks=bad)):
        with pytest.raises(ValueError):
            c.attention(0, one, off, x, 1, **kw)
    for call in (lambda: c.attention(bad, one, off, x, 1), lambda: c.attention(0, one, off, x, bad),
                 lambda: c.append(bad, one, off, x, x), lambda: c.read(bad, one, off, 1),
                 lambda: c.read(0, one, off, bad)):
        with pytest.raises(ValueError):
            call()
    assert not lib.calls
    c.attention(0, one, off, x, 1, window=(1 << 32) - 1, sinks=(1 << 32) - 1)
    assert lib.calls[0][2][-5:-3] == ((1 << 32) - 1, (1 << 32) - 1)


def test_query_heads_beyond_32_bit_offsets_are_refused():
    """Offsets of a token's heads are 32-bit in the kernels; judged before anything touches a device."""
    q = pytest.importorskip("quantized_base_lora_gb300")
    d = q.ovl_kv()
    for name, value in dict(n_pages=9, page_tokens=16, n_layers=1, n_kv_heads=65535, head_dim=256, max_seqs=9,
                            max_pages=9, codes=4096, scales=4096, table=4096, length=4096, refs=4096, workspace=4096,
                            workspace_bytes=1 << 40).items():
        setattr(d, name, value)
    heads = 65535 * 1024

    def attend(heads, tokens=1):
        return q.ovl_kv_attention(d, 0, 16, 16, 1, tokens, 1, 16, q.OVL_BF16, heads, heads * 256, 1.0, 0, 0, 16,
                                  heads * 256)

    assert attend(heads, tokens=0) == q.OVL_E_SHAPE and "2^32" in q.ovl_last_error(None)
    assert attend(65535 * 256, tokens=0) == q.OVL_OK                     # just below: no tokens, so no call either


def test_kernels_of_the_cache_read_by_ordinary_loads():
    """Each is resident while the kernel before it may still write what it will read, so nothing of it may go through
    the read-only path."""
    import glob
    import os
    import re
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_base_lora_gb300", "csrc")
    files = glob.glob(os.path.join(root, "k_kv_*.cu")) + glob.glob(os.path.join(root, "kv_*"))
    assert len(files) >= 6
    for f in files:
        with open(f) as t:
            code = re.sub(r"//.*", "", t.read())
        assert not re.search(r"__ldg\(|__restrict__|ld\.global\.nc", code), f
