"""The 8-bit K/V cache without a GPU: its oracle pinned by hand-worked examples, the binding's
struct against the header, workspace sizes, and the refusals that come before any CUDA call."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import kv8 as O
from test_abi import _header_struct_fields

HAVE_NVCC = shutil.which("nvcc") is not None or os.path.exists("/usr/local/cuda/bin/nvcc")
needs_lib = pytest.mark.skipif(not HAVE_NVCC, reason="nvcc is needed to build libhsa.so")


# ------------------------------------------------------------------------------- the oracle

def test_e4m3_codes_by_hand():
    # 1 = 2^0 * 1.000 -> exponent field 7; 448 = 2^8 * 1.75; 2^-9 the smallest subnormal
    assert list(O.e4m3_code([0.0, 1.0, -1.0, 448.0, 2.0 ** -9, 1e9])) == [0, 56, 184, 126, 1, 126]
    assert np.array_equal(O.code_values("e4m3", np.array([56, 184, 126, 1], np.uint8)),
                          [1.0, -1.0, 448.0, 2.0 ** -9])
    # ties go to the even code: 17 between 16 and 18, 19 between 18 and 20
    assert np.array_equal(O.code_values("e4m3", O.e4m3_code([17.0, 19.0])), [16.0, 20.0])


def test_write_by_hand_grows_a_block():
    c, s = np.zeros((16, 128), np.int8), np.float32(0)
    row = np.zeros((1, 128), np.float32)
    row[0, :3] = [127.0, -63.5, 2.0]
    c, s = O.write_block("int8", c, s, row, 0)
    assert s == 1.0 and list(c[0, :4]) == [127, -64, 2, 0]  # -63.5 to the even -64
    row[0, :3] = [254.0, 1.0, -3.0]
    c, s = O.write_block("int8", c, s, row, 1)
    # the scale doubles: 127 / 2 = 63.5 -> 64 (even), -64 / 2 = -32, 2 / 2 = 1
    assert s == 2.0 and list(c[0, :3]) == [64, -32, 1]
    assert list(c[1, :3]) == [127, 0, -2]  # 0.5 -> 0, -1.5 -> -2
    row[0, :3] = [1.0, 4.0, -5.0]
    before = c.copy()
    c, s = O.write_block("int8", c, s, row, 2)
    assert s == 2.0 and np.array_equal(c[:2], before[:2]) and list(c[2, :3]) == [0, 2, -2]
    c, s = O.write_block("int8", c, s, row, 0)  # from the first slot on: a scale of its own
    assert s == np.float32(5.0) / np.float32(127.0) and c[0, 2] == -127


def test_write_of_values_that_are_no_numbers():
    row = np.array([[np.inf, -np.inf, np.nan, 10.0] + [0.0] * 124], np.float32)
    c, s = O.write_block("int8", np.zeros((16, 128), np.int8), np.float32(0), row, 0)
    assert s == np.float32(10) / np.float32(127) and list(c[0, :4]) == [127, -127, 0, 127]


def test_attention_of_two_tokens_by_hand():
    q = np.zeros((1, 128))
    q[0, 0] = 1.0
    k = np.zeros((2, 128))
    k[1, 0] = np.log(3.0)
    v = np.zeros((2, 128))
    v[0, 5], v[1, 5] = 8.0, 4.0
    out, lse, _ = O.attend(q, k, v, np.ones((1, 2), bool), 1.0)  # weights 1/4 and 3/4
    assert out[0, 5] == pytest.approx(5.0) and lse[0] == pytest.approx(np.log(4.0))
    out, lse, _ = O.attend(q, k, v, np.zeros((1, 2), bool), 1.0)
    assert not out.any() and np.isneginf(lse[0])


# ------------------------------------------------------------------------------ the library

@pytest.fixture(scope="module")
def lib():
    from kv_cache_int8_gb300 import build, hsa
    build.build()
    return hsa


def dims(lib, **kw):
    return lib.Dims(**{**dict(batch=2, hq=32, hkv=8, max_pages_per_seq=64, num_pages=128, k2=4,
                              sink=16, window=32), **kw})


def test_binding_struct_matches_the_header():
    from kv_cache_int8_gb300 import hsa
    ctype = {"int32_t": ctypes.c_int32, "ptr": ctypes.c_void_p}
    want = [("ptr", n) for n in ("k", "v", "k_scale", "v_scale")] + [("int32_t", "format")]
    got = _header_struct_fields("hsa_kv8")
    assert got == want
    assert [(n, t) for n, t in hsa.hsa_kv8._fields_] == [(n, ctype[t]) for t, n in want]


@needs_lib
def test_workspace_sizes(lib):
    for op in (lib.HSA_OP_KV8_DECODE, lib.HSA_OP_KV8_PREFILL):
        assert lib.hsa_workspace_bytes(dims(lib), op) > 256
        for hq in (8, 24, 40, 48, 56, 64):  # every group of 1 to 8
            assert lib.hsa_workspace_bytes(dims(lib, hq=hq), op) > 256
        for bad in (dict(hq=72), dict(hq=12), dict(head_dim=64), dict(page_size=32),
                    dict(kv_on_host=True), dict(batch=0), dict(batch=2000)):
            assert lib.hsa_workspace_bytes(dims(lib, **bad), op) == 0


class Ws:
    def __init__(self, ptr, n):
        self.ptr, self.n = ptr, n

    def data_ptr(self):
        return self.ptr

    def numel(self):
        return self.n


OK = 1 << 20  # an aligned address that validation never follows


class Call:
    """Raw C calls with fake addresses: every argument valid but those given."""

    def __init__(self, lib, **kw):
        self.lib = lib
        self.a = dict(d=dims(lib), k=OK, v=OK, ks=OK, vs=OK, format=0, x=OK, y=OK, xs=8 * 128,
                      ys=8 * 128, qs=32 * 128, cu=OK, total=100, table=OK, lens=OK, idx=OK,
                      cnt=OK, out=OK, lse=OK, ws=OK, ws_bytes=1 << 40)
        self.a.update(kw)

    def __getattr__(self, name):
        return self.a[name]

    def run(self, fn):
        c = self.lib.load()
        d = ctypes.byref(self.d.c())
        kv = ctypes.byref(self.lib.hsa_kv8(self.k, self.v, self.ks, self.vs, self.format))
        if fn in ("write", "read"):
            return getattr(c, "hsa_kv8_" + fn)(d, kv, self.x, self.xs, self.y, self.ys, self.cu,
                                               self.total, self.table, self.lens, self.ws,
                                               self.ws_bytes, None)
        if fn == "decode":
            return c.hsa_kv8_decode(d, kv, self.x, self.table, self.lens, self.out, self.lse,
                                    self.ws, self.ws_bytes, None)
        if fn == "attend":
            return c.hsa_kv8_attend(d, kv, self.x, self.table, self.lens, self.idx, self.cnt,
                                    self.out, self.lse, self.ws, self.ws_bytes, None)
        return c.hsa_kv8_prefill(d, kv, self.x, self.qs, self.cu, self.total, self.table,
                                 self.lens, self.out, self.lse, self.ws, self.ws_bytes, None)


ALL = ("write", "read", "decode", "attend", "prefill")
INVALID, UNSUPPORTED, SMALL = 1, 2, 5


@needs_lib
@pytest.mark.parametrize("fns,bad,code", [
    (ALL, dict(k=None), INVALID), (ALL, dict(v=OK + 16), INVALID), (ALL, dict(ks=OK + 4), INVALID),
    (ALL, dict(vs=None), INVALID), (ALL, dict(format=2), INVALID), (ALL, dict(x=None), INVALID),
    (ALL, dict(x=OK + 8), INVALID), (ALL, dict(table=None), INVALID),
    (ALL, dict(lens=None), INVALID), (ALL, dict(table=OK + 2), INVALID),
    (("write", "read"), dict(y=None), INVALID), (("write", "read"), dict(xs=1020), INVALID),
    (("write", "read"), dict(ys=1016), INVALID), (("prefill",), dict(qs=4092), INVALID),
    (("prefill",), dict(qs=31 * 128), INVALID),
    (("write", "read", "prefill"), dict(total=-1), INVALID),
    (("write", "read", "prefill"), dict(cu=None), INVALID),  # no offsets: batch rows
    (("write", "read", "prefill"), dict(cu=OK + 2), INVALID),
    (("write", "read", "prefill"), dict(total=(1 << 31) - 1), UNSUPPORTED),
    (("decode", "attend", "prefill"), dict(out=None), INVALID),
    (("decode", "attend", "prefill"), dict(out=OK + 4), INVALID),
    (("decode", "attend", "prefill"), dict(lse=OK + 2), INVALID),
    (("decode", "attend", "prefill"), dict(ws=None), INVALID),
    (("decode", "attend", "prefill"), dict(ws=OK + 128), INVALID),
    (("decode", "attend", "prefill"), dict(ws_bytes=4096), SMALL),
    (("write", "read"), dict(ws=OK + 128), INVALID),
    (("write", "read"), dict(ws_bytes=128), SMALL),
    (("attend",), dict(cnt=None), INVALID), (("attend",), dict(idx=None), INVALID),
    (("attend",), dict(idx=OK + 2), INVALID),
])
def test_refusals_of_arguments(lib, fns, bad, code):
    for fn in fns:
        assert Call(lib, **bad).run(fn) == code, fn


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(hq=72), UNSUPPORTED), (dict(hq=30), INVALID), (dict(head_dim=64), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(batch=0), INVALID), (dict(batch=1025), UNSUPPORTED),
    (dict(kv_on_host=True), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 30), UNSUPPORTED), (dict(sm_scale=float("nan")), INVALID),
    (dict(window=-1), INVALID), (dict(per_head=2), INVALID),
])
def test_refusals_of_descriptors(lib, kw, code):
    for fn in ALL:
        assert Call(lib, d=dims(lib, **kw)).run(fn) == code, fn


@needs_lib
def test_too_many_visits_are_refused(lib):
    # rows x (kept blocks + sink + window blocks) beyond 32 bits
    d = dims(lib, hq=64, hkv=8, per_head=1, k2=1 << 27)
    assert Call(lib, d=d).run("attend") == UNSUPPORTED
    assert Call(lib, d=dims(lib, k2=0), idx=None, ws_bytes=64).run("attend") == SMALL


@needs_lib
def test_no_rows_are_no_call(lib):
    for fn in ("write", "read", "prefill"):
        assert Call(lib, total=0).run(fn) == 0
        assert Call(lib, total=0, x=None, y=None, out=None).run(fn) == 0


def test_the_binding_refuses_other_tensors():
    from kv_cache_int8_gb300 import hsa
    k = torch.zeros(4, 2, 16, 128, dtype=torch.int8)
    s = torch.zeros(4, 2)
    hsa.KV8(k, k.clone(), s, s.clone())
    for bad in ((k, k.view(torch.float8_e4m3fn), s, s), (k.float(), k.float(), s, s),
                (k, k[:3], s, s), (k, k, s, s[:3]), (k, k, s, s.double()),
                (k.transpose(0, 1), k.transpose(0, 1), s, s)):
        with pytest.raises(hsa.HsaError):
            hsa.KV8(*bad)
    d = dims(hsa, hq=4, hkv=2)
    cache = hsa.KV8(k, k.clone(), s, s.clone())
    rows = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    for x, y in ((rows.float(), rows), (rows[:, :1], rows), (rows, rows[:4]),
                 (rows.transpose(0, 1).contiguous().transpose(0, 1), rows),
                 (torch.zeros(5, 2, 256, dtype=torch.bfloat16)[..., ::2], rows)):
        with pytest.raises(hsa.HsaError):
            hsa.hsa_kv8_write(d, cache, x, y, None, None, None)


def _aligned(shape, dtype):
    """A zero CPU tensor on a 256-byte boundary (what the library's checks ask of device memory)."""
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    raw = torch.zeros(n + 256, dtype=torch.uint8)
    off = -raw.data_ptr() % 256
    return raw[off:off + n].view(dtype).view(shape)


class NoLibrary:
    """In the library's place: counts the calls that the binding lets through, runs none."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def binding(monkeypatch):
    from kv_cache_int8_gb300 import hsa
    lib = NoLibrary()
    monkeypatch.setattr(hsa, "_LIB", lib)
    monkeypatch.setattr(hsa, "_stream", lambda stream=None: 0)
    return hsa, lib


def binding_calls(hsa, d, cache, **kw):
    """The five calls of the binding with valid tensors of d's sizes, but those given."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    B, T = d.batch, 5
    a = dict(k=torch.zeros(T, d.hkv, 128, dtype=bf), v=torch.zeros(T, d.hkv, 128, dtype=bf),
             rows=torch.zeros(T, d.hq, 128, dtype=bf), rows_out=torch.zeros(T, d.hq, 128, dtype=bf),
             rows_lse=torch.zeros(T, d.hq, dtype=f32),
             cu=torch.zeros(B + 1, dtype=i32), table=torch.zeros(B, d.max_pages_per_seq, dtype=i32),
             lens=torch.zeros(B, dtype=i32), q=torch.zeros(B, d.hq, 128, dtype=bf),
             idx=torch.zeros(B, d.hkv, d.k2, dtype=i32), cnt=torch.zeros(B, d.hkv, dtype=i32),
             out=torch.zeros(B, d.hq, 128, dtype=f32), lse=torch.zeros(B, d.hq, dtype=f32),
             ws=torch.zeros(64, dtype=torch.uint8))
    a.update(kw)
    lists = (a["cu"], a["table"], a["lens"])
    return {
        "write": lambda: hsa.hsa_kv8_write(d, cache, a["k"], a["v"], *lists),
        "read": lambda: hsa.hsa_kv8_read(d, cache, a["k"], a["v"], *lists),
        "decode": lambda: hsa.hsa_kv8_decode(d, cache, a["q"], a["table"], a["lens"], a["out"],
                                             a["lse"], a["ws"]),
        "attend": lambda: hsa.hsa_kv8_attend(d, cache, a["q"], a["table"], a["lens"], a["idx"],
                                             a["cnt"], a["out"], a["lse"], a["ws"]),
        "prefill": lambda: hsa.hsa_kv8_prefill(d, cache, a["rows"], *lists, a["rows_out"],
                                               a["rows_lse"], a["ws"]),
    }


def cpu_cache(hsa, pages, hkv):
    return hsa.KV8(*(_aligned((pages, hkv, 16, 128), torch.int8) for _ in range(2)),
                   *(_aligned((pages, hkv), torch.float32) for _ in range(2)))


def test_the_binding_refuses_a_cache_of_other_sizes(binding):
    hsa, lib = binding
    d = dims(hsa, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    for pages, hkv in ((8, 2), (9, 2)):  # the descriptor may leave pages out
        for name, call in binding_calls(hsa, d, cpu_cache(hsa, pages, hkv)).items():
            call()
            assert lib.calls.pop() == "hsa_kv8_" + name
    for pages, hkv in ((7, 2), (8, 1), (8, 4), (1, 2)):
        for name, call in binding_calls(hsa, d, cpu_cache(hsa, pages, hkv)).items():
            with pytest.raises(hsa.HsaError):
                call()
            assert not lib.calls, name


def test_the_binding_refuses_arrays_that_it_would_misread(binding):
    """The attentions read and write their arrays densely: a slice of a fused projection, another
    type or another size would be misread or written past."""
    hsa, lib = binding
    d = dims(hsa, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    cache = cpu_cache(hsa, 8, 2)
    bf, f32 = torch.bfloat16, torch.float32
    fused = torch.zeros(3, 8, 128, dtype=bf)
    for good in (dict(), dict(q=fused[:, :4].contiguous()), dict(out=torch.zeros(3, 512)),
                 dict(q=torch.zeros(3, 1, 4, 128, dtype=bf)), dict(lse=None, rows_lse=None)):
        for name, call in binding_calls(hsa, d, cache, **good).items():
            call()
            assert lib.calls.pop() == "hsa_kv8_" + name
    for bad in (dict(q=fused[:, :4]), dict(q=torch.zeros(3, 4, 128)),
                dict(q=fused[:2, :4].contiguous()), dict(out=torch.zeros(3, 4, 128, dtype=bf)),
                dict(q=torch.zeros(3, 4, 256, dtype=bf)[..., ::2]),
                dict(out=torch.zeros(3, 8, 128)[:, :4]), dict(out=torch.zeros(3, 4, 64)),
                dict(out=torch.zeros(3, 4, 128, dtype=torch.float64)), dict(lse=torch.zeros(3)),
                dict(lse=torch.zeros(3, 4, dtype=bf)), dict(lse=torch.zeros(3, 8)[:, ::2])):
        calls = binding_calls(hsa, d, cache, **bad)
        for name in ("decode", "attend"):
            with pytest.raises(hsa.HsaError):
                calls[name]()
    for bad in (torch.zeros(5, 3), torch.zeros(5, 4, dtype=bf), torch.zeros(5, 8)[:, :4]):
        with pytest.raises(hsa.HsaError):
            binding_calls(hsa, d, cache, rows_lse=bad)["prefill"]()
    assert not lib.calls


def test_the_binding_refuses_lists_of_another_type(binding):
    """int64 lists (torch.cumsum's, for one, of int32 lengths) would be read as twice as many
    int32, every other one 0."""
    hsa, lib = binding
    d = dims(hsa, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    cache = cpu_cache(hsa, 8, 2)
    lens = torch.tensor([2, 3, 4], dtype=torch.int32)
    i32 = torch.int32
    for good in (dict(cu=torch.zeros(9, dtype=i32)), dict(cu=None)):
        for name in ("write", "read", "prefill"):
            binding_calls(hsa, d, cache, **good)[name]()
            assert lib.calls.pop() == "hsa_kv8_" + name
    for bad in (torch.cumsum(lens, 0), torch.zeros(4), torch.zeros(3, dtype=i32),
                torch.zeros(8, dtype=i32)[::2]):
        for name in ("write", "read", "prefill"):
            with pytest.raises(hsa.HsaError):
                binding_calls(hsa, d, cache, cu=bad)[name]()
    for bad, names in ((dict(lens=lens.long()), ALL), (dict(table=torch.zeros(3, 4).long()), ALL),
                       (dict(idx=torch.zeros(3, 2, 4).long()), ("attend",)),
                       (dict(cnt=torch.zeros(3, 2)), ("attend",))):
        for name in names:
            with pytest.raises(hsa.HsaError):
                binding_calls(hsa, d, cache, **bad)[name]()
    assert not lib.calls


def test_a_single_row_may_have_any_stride(binding, monkeypatch):
    """One token taken out of a [heads][tokens][128] tensor: its rows are contiguous, the stride
    between them is the heads'."""
    hsa, lib = binding
    d = dims(hsa, batch=1, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    cache = cpu_cache(hsa, 8, 2)
    got = []
    lib.hsa_kv8_write = lambda *a: got.append((a[7], a[3], a[5])) or 0
    lib.hsa_kv8_prefill = lambda *a: got.append((a[5], a[3])) or 0
    one = torch.zeros(2, 1, 128, dtype=torch.bfloat16).transpose(0, 1)
    many = torch.zeros(7, 8, 128, dtype=torch.bfloat16)
    assert one.stride() == (128, 128, 1)
    for k in (one, many[:1, 2:4], many[3:4, :2], one.expand(1, 2, 128)):
        binding_calls(hsa, d, cache, k=k, v=one, cu=None)["write"]()
        assert got.pop() == (1, 256, 256)
    q = torch.zeros(4, 1, 128, dtype=torch.bfloat16).transpose(0, 1)
    binding_calls(hsa, d, cache, rows=q, rows_out=torch.zeros(1, 4, 128, dtype=torch.bfloat16),
                  rows_lse=None, cu=None)["prefill"]()
    assert got.pop() == (1, 512)
    binding_calls(hsa, d, cache, k=many[:5, 2:4], v=many[:5, 4:6])["write"]()
    assert got.pop() == (5, 1024, 1024)
