"""Rotary positions and drafted tokens without a GPU: the oracle by hand, the binding's structs
against the header, and the refusals that come before any CUDA call."""
import copy
import ctypes
import dataclasses
import pickle

import numpy as np
import pytest
import torch

from kv_cache_int8_gb300 import hsa
from oracle import draft as R
from oracle import kv8 as O
from test_abi import _header_struct_fields
from test_kv8_abi import OK, _aligned, binding, cpu_cache, dims, lib, needs_lib  # noqa: F401

INVALID, UNSUPPORTED, SMALL = 1, 2, 5


# ------------------------------------------------------------------------------- the oracle

def test_turn_by_hand():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, :6] = [1, 2, 3, 4, 5, 6]
    quarter = np.array([[0.0, 1.0, 1.0, 0.0]], np.float32)  # pair 0 by a quarter, pair 1 not
    y = R.turn(x, quarter, neighbours=False)[0, 0]  # pairs (0, 2) and (1, 3)
    assert list(y[:6]) == [-3, 2, 1, 4, 5, 6]
    y = R.turn(x, quarter, neighbours=True)[0, 0]  # pairs (0, 1) and (2, 3)
    assert list(y[:6]) == [-2, 1, 3, 4, 5, 6]


def test_frequencies_by_hand():
    assert list(R.frequencies(4, 100.0)) == [1.0, 0.1]
    assert list(R.frequencies(4, 100.0, 1, 4.0)) == [0.25, 0.025]
    # turns within 20 pi tokens: 10 (kept) and 1 (slowed); within 5 pi: 2.5, half way of 1 to 4
    np.testing.assert_allclose(R.frequencies(4, 100.0, 2, 8.0, 1.0, 4.0, 20 * np.pi), [1.0, 0.0125])
    np.testing.assert_allclose(R.frequencies(4, 100.0, 2, 8.0, 1.0, 4.0, 5 * np.pi),
                               [0.5 + 0.5 / 8, 0.0125])


def test_branches_by_hand():
    assert R.branches([-1, 0, 0, 1, -1]).astype(int).tolist() == [
        [1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [0, 0, 0, 0, 1]]
    assert R.depths([-1, 0, 0, 1, -1]).tolist() == [0, 1, 1, 2, 0]
    assert R.seen(4, [-1, 0]).astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]


def test_keep_by_hand():
    c = O.empty("int8", 2, 1)
    rows = np.zeros((20, 1, 128), np.float32)
    rows[:, 0, 0] = 127.0 * np.arange(1, 21)  # token t: 127 (t + 1); scales 16 and 20
    O.write(c, rows, rows, [1, 0], 0)
    assert c["ks"][1, 0] == 16 and c["ks"][0, 0] == 20
    # the last 6 tokens (14 .. 19), of which nodes 1, 3 and 5 (tokens 15, 17, 19) stay
    assert R.keep(c, [1, 0], 20, 6, [1, 3, 5]) == 17
    # block 0: tokens 0 .. 13, then 15 and 17; token 17 was round(127 * 18 / 20) = 114 of scale 20
    s = np.float32(114 * 20) / np.float32(127)
    assert c["ks"][1, 0] == s and c["k"][1, 0, 15, 0] == 127
    assert c["k"][1, 0, 14, 0] == np.rint(127 * 16 / s)
    assert c["k"][1, 0, 13, 0] == np.rint(np.rint(127 * 14 / 16) * 16 / s)
    # block 1: token 19 alone, in slot 0, under a scale of its own
    assert c["k"][0, 0, 0, 0] == 127 and c["ks"][0, 0] == 20
    before = {n: c[n].copy() for n in ("k", "ks")}
    assert R.keep(c, [1, 0], 17, 3, []) == 14
    assert all(np.array_equal(before[n], c[n]) for n in before)


@pytest.mark.parametrize("fmt", ("int8", "e4m3"))
def test_the_mark_of_nodes_that_are_not_kept(fmt):
    """They leave a block's scale raised and its older tokens rounded again, by half a step of the
    new scale (int8: s / 2; E4M3: 2^-4 of a value, 2^-10 s among its smallest) beside fp32's own
    roundings; nodes that are not larger leave every bit as it was."""
    rng = np.random.default_rng(5)
    c = O.empty(fmt, 2, 3)
    pages = np.array([1, 0])

    def first():
        return np.stack([O.values(c, "k", pages, 11, h) for h in range(3)], 1)

    x = rng.standard_normal((11, 3, 128)).astype(np.float32)
    O.write(c, x, x, pages, 0)
    grown = 0
    for size in (1.0, 0.5, 1.1, 0.9, 3.0, 1.0, 100.0, 2.0 ** 30):
        codes, scale, was = c["k"].copy(), c["ks"].copy(), first()
        y = (size * rng.uniform(-4, 4, (9, 3, 128))).astype(np.float32)
        O.write(c, y, y, pages, 11)
        assert R.keep(c, pages, 20, 9, []) == 11
        largest = np.abs(y[:5]).max((0, 2)) / O.LEVELS[fmt]  # of the nodes in the block
        np.testing.assert_array_equal(c["ks"][1], np.maximum(scale[1], largest))
        s = c["ks"][1][None, :, None].astype(np.float64)
        half = s / 2 if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** -10 * s)
        assert (np.abs(first() - was) <= half + 2.0 ** -22 * np.abs(was)).all()
        for h in range(3):
            if c["ks"][1, h] == scale[1, h]:
                np.testing.assert_array_equal(c["k"][1, h, :11], codes[1, h, :11])
            else:
                grown += 1
    assert grown >= 9  # (3.0, 100.0 and 2^30 under every head)


# ------------------------------------------------------------------------------ the library

def test_binding_structs_match_the_header():
    from kv_cache_int8_gb300 import hsa
    ctype = {"int32_t": ctypes.c_int32, "ptr": ctypes.c_void_p, "double": ctypes.c_double}
    got = _header_struct_fields("hsa_rotary")
    assert got == [("ptr", "table"), ("int32_t", "rows"), ("int32_t", "dim"),
                   ("int32_t", "neighbours")]
    assert [(n, t) for n, t in hsa.hsa_rotary._fields_] == [(n, ctype[t]) for t, n in got]
    assert [n for n, _ in hsa.hsa_rotary_angles._fields_] == [
        "base", "factor", "low", "high", "original", "magnitude", "scaling"]
    assert ctypes.sizeof(hsa.hsa_rotary_angles) == 56


@needs_lib
def test_tree_workspace(lib):  # noqa: F811
    n = lib.hsa_workspace_bytes(dims(lib), lib.HSA_OP_KV8_TREE)
    assert 256 < n <= lib.hsa_workspace_bytes(dims(lib), lib.HSA_OP_KV8_PREFILL)
    for hq in (8, 24, 40, 48, 56, 64):
        assert lib.hsa_workspace_bytes(dims(lib, hq=hq), lib.HSA_OP_KV8_TREE) == n
    for bad in (dict(hq=72), dict(hq=12), dict(head_dim=64), dict(kv_on_host=True),
                dict(batch=2000)):
        assert lib.hsa_workspace_bytes(dims(lib, **bad), lib.HSA_OP_KV8_TREE) == 0


class Call:
    """Raw C calls with fake addresses: every argument valid but those given."""

    def __init__(self, lib, **kw):  # noqa: F811
        self.lib = lib
        self.a = dict(d=dims(lib), kk=OK, format=0, rot=True, angles=OK, rows=1000, dim=128, nb=0,
                      q=OK, qs=32 * 128, qo=2 * OK, qos=32 * 128, k=OK, ks=8 * 128, ko=2 * OK,
                      kos=8 * 128, v=OK, vs=8 * 128, pos=OK, parents=OK, cu=OK, total=100, table=OK,
                      lens=OK, out=4 * OK, lse=OK, idx=OK, stride=9, cnt=3 * OK, new=2 * OK, ws=OK,
                      ws_bytes=1 << 40)
        self.a.update(kw)

    def __getattr__(self, name):
        return self.a[name]

    def run(self, fn):
        c = self.lib.load()
        d = ctypes.byref(self.d.c()) if self.d else None
        kv = ctypes.byref(self.lib.hsa_kv8(self.kk, OK, OK, OK, self.format))
        r = ctypes.byref(self.lib.hsa_rotary(self.angles, self.rows, self.dim, self.nb))
        r = r if self.rot else None
        ws = (self.ws, self.ws_bytes, None)
        if fn == "rotate":
            return c.hsa_rotate(d, r, self.q, self.qs, self.qo, self.qos, self.k, self.ks, self.ko,
                                self.kos, self.pos, self.cu, self.total, self.lens, *ws)
        if fn == "write_rotated":
            return c.hsa_kv8_write_rotated(d, kv, r, self.q, self.qs, self.qo, self.qos, self.k,
                                           self.ks, self.v, self.vs, self.pos, self.cu, self.total,
                                           self.table, self.lens, *ws)
        if fn == "tree":
            return c.hsa_kv8_tree(d, kv, self.q, self.qs, self.parents, self.cu, self.total,
                                  self.table, self.lens, self.out, self.lse, *ws)
        return c.hsa_kv8_keep(d, kv, self.idx, self.stride, self.cnt, self.cu, self.table,
                              self.lens, self.new, *ws)


ALL = ("rotate", "write_rotated", "tree", "keep")
ROTARY, CACHE, ROWS = ALL[:2], ALL[1:], ALL[:3]


@needs_lib
@pytest.mark.parametrize("fns,bad,code", [
    (ALL, dict(d=None), INVALID),
    (ROTARY, dict(rot=False), INVALID), (ROTARY, dict(angles=None), INVALID),
    (ROTARY, dict(angles=OK + 8), INVALID), (ROTARY, dict(rows=0), INVALID),
    (ROTARY, dict(nb=2), INVALID), (ROTARY, dict(dim=0), UNSUPPORTED),
    (ROTARY, dict(dim=132), UNSUPPORTED), (ROTARY, dict(dim=136), UNSUPPORTED),
    (ROTARY, dict(dim=-8), UNSUPPORTED), (ROTARY, dict(dim=12), UNSUPPORTED),
    (CACHE, dict(kk=None), INVALID), (CACHE, dict(kk=OK + 16), INVALID),
    (CACHE, dict(format=2), INVALID), (CACHE, dict(table=None), INVALID),
    (CACHE, dict(table=OK + 2), INVALID), (CACHE, dict(lens=None), INVALID),
    (ALL, dict(lens=OK + 2), INVALID), (ALL, dict(cu=OK + 2), INVALID),
    (ROWS, dict(total=-1), INVALID), (ROWS, dict(total=(1 << 31) - 1), UNSUPPORTED),
    (("write_rotated", "tree"), dict(cu=None), INVALID),  # no offsets: batch rows
    (("rotate",), dict(cu=None, pos=None), INVALID), (("rotate",), dict(lens=None, pos=None), INVALID),
    (ROTARY, dict(pos=OK + 2), INVALID), (("tree",), dict(parents=OK + 2), INVALID),
    (("rotate", "tree"), dict(q=None), INVALID), (ROWS, dict(q=OK + 8), INVALID),
    (ROWS, dict(qs=4092), INVALID), (ROWS, dict(qs=31 * 128), INVALID),
    (ROTARY, dict(qo=None), INVALID), (ROTARY, dict(q=None), INVALID),
    (ROTARY, dict(qo=2 * OK + 8), INVALID), (ROTARY, dict(qos=4088), INVALID),
    (ROTARY, dict(qo=OK, qos=33 * 128), INVALID),  # in place under another stride
    (("rotate",), dict(ko=OK, kos=9 * 128), INVALID), (("rotate",), dict(k=None), INVALID),
    (("rotate",), dict(ko=None), INVALID), (("write_rotated",), dict(k=None), INVALID),
    (("write_rotated",), dict(v=None), INVALID), (ROTARY, dict(k=OK + 8), INVALID),
    (ROTARY, dict(ks=1020), INVALID), (("write_rotated",), dict(vs=1016), INVALID),
    (("tree",), dict(out=None), INVALID), (("tree",), dict(out=OK + 8), INVALID),
    (("tree",), dict(lse=OK + 2), INVALID), (("tree",), dict(ws=None), INVALID),
    (("tree",), dict(ws_bytes=4096), SMALL), (ALL, dict(ws=OK + 128), INVALID),
    (ALL, dict(ws_bytes=128), SMALL),
    (("keep",), dict(idx=None), INVALID), (("keep",), dict(idx=OK + 2), INVALID),
    (("keep",), dict(stride=-1), INVALID), (("keep",), dict(cnt=None), INVALID),
    (("keep",), dict(cnt=OK + 2), INVALID), (("keep",), dict(new=OK), INVALID),
    (("keep",), dict(new=3 * OK), INVALID), (("keep",), dict(new=5 * OK, idx=5 * OK), INVALID),
    (("keep",), dict(new=5 * OK, cu=5 * OK), INVALID), (("tree",), dict(out=OK), INVALID),
    (("keep",), dict(new=OK + 2), INVALID),
])
def test_refusals_of_arguments(lib, fns, bad, code):  # noqa: F811
    for fn in fns:
        assert Call(lib, **bad).run(fn) == code, fn


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(hq=72), UNSUPPORTED), (dict(hq=30), INVALID), (dict(head_dim=64), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(batch=0), INVALID), (dict(batch=1025), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(sm_scale=float("nan")), INVALID),
])
def test_refusals_of_descriptors(lib, kw, code):  # noqa: F811
    for fn in ALL:
        assert Call(lib, d=dims(lib, **kw)).run(fn) == code, fn
    for fn in CACHE:
        assert Call(lib, d=dims(lib, kv_on_host=True)).run(fn) == UNSUPPORTED, fn


@needs_lib
def test_no_rows_are_no_call(lib):  # noqa: F811
    for fn in ROWS:
        assert Call(lib, total=0).run(fn) == 0
        assert Call(lib, total=0, q=None, qo=None, k=None, ko=None, v=None, out=None).run(fn) == 0


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(base=0.0), INVALID), (dict(base=float("inf")), INVALID), (dict(scaling=3), INVALID),
    (dict(scaling=1, factor=0.0), INVALID), (dict(scaling=2, low=4.0), INVALID),
    (dict(scaling=2, original=0.0), INVALID), (dict(magnitude=float("nan")), INVALID),
    (dict(rows=0), INVALID), (dict(dim=4), UNSUPPORTED), (dict(dim=130), UNSUPPORTED),
    (dict(table=None), INVALID), (dict(table=OK + 4), INVALID),
])
def test_refusals_of_tables(lib, kw, code):  # noqa: F811
    a = dict(base=1e4, factor=8.0, low=1.0, high=4.0, original=8192.0, magnitude=1.0, scaling=0,
             table=OK, rows=16, dim=128)
    a.update(kw)
    s = lib.hsa_rotary_angles(a["base"], a["factor"], a["low"], a["high"], a["original"],
                              a["magnitude"], a["scaling"])
    assert lib.load().hsa_rotary_table(ctypes.byref(s), a["table"], a["rows"], a["dim"],
                                       None) == code
    assert lib.load().hsa_rotary_table(None, OK, 16, 128, None) == INVALID


def calls(hsa, d, cache, **kw):
    """The binding's calls with valid tensors of d's sizes, but those given."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    B, T = d.batch, 5
    a = dict(rotary=hsa.Rotary(_aligned((64, 32), f32)), q=torch.zeros(T, d.hq, 128, dtype=bf),
             q_out=torch.zeros(T, d.hq, 128, dtype=bf), k=torch.zeros(T, d.hkv, 128, dtype=bf),
             k_out=torch.zeros(T, d.hkv, 128, dtype=bf), v=torch.zeros(T, d.hkv, 128, dtype=bf),
             pos=torch.zeros(T, dtype=i32), parents=torch.zeros(T, dtype=i32),
             cu=torch.zeros(B + 1, dtype=i32), table=torch.zeros(B, d.max_pages_per_seq, dtype=i32),
             lens=torch.zeros(B, dtype=i32), out=torch.zeros(T, d.hq, 128, dtype=bf),
             lse=torch.zeros(T, d.hq), idx=torch.zeros(B, 4, dtype=i32),
             cnt=torch.zeros(B, dtype=i32), new=torch.zeros(B, dtype=i32),
             ws=torch.zeros(64, dtype=torch.uint8))
    a.update(kw)
    return {
        "hsa_rotate": lambda: hsa.hsa_rotate(d, a["rotary"], a["q"], a["q_out"], a["k"], a["k_out"],
                                             a["pos"], a["cu"], a["lens"]),
        "hsa_kv8_write_rotated": lambda: hsa.hsa_kv8_write_rotated(
            d, cache, a["rotary"], a["q"], a["q_out"], a["k"], a["v"], a["pos"], a["cu"],
            a["table"], a["lens"]),
        "hsa_kv8_tree": lambda: hsa.hsa_kv8_tree(d, cache, a["q"], a["parents"], a["cu"],
                                                 a["table"], a["lens"], a["out"], a["lse"],
                                                 a["ws"]),
        "hsa_kv8_keep": lambda: hsa.hsa_kv8_keep(d, cache, a["idx"], a["cnt"], a["cu"], a["table"],
                                                 a["lens"], a["new"]),
    }


def test_the_binding_refuses_what_it_would_misread(binding):  # noqa: F811
    hsa, fake = binding
    d = dims(hsa, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    cache = cpu_cache(hsa, 8, 2)
    bf, i32 = torch.bfloat16, torch.int32
    fused = torch.zeros(5, 8, 128, dtype=bf)
    rot, wr, tree, keep = ("hsa_rotate", "hsa_kv8_write_rotated", "hsa_kv8_tree", "hsa_kv8_keep")
    for good in (dict(), dict(q=fused[:, :4], q_out=fused[:, :4]), dict(pos=None), dict(cu=None),
                 dict(k=fused[:, 4:6], v=fused[:, 6:]), dict(parents=None), dict(lse=None),
                 dict(new=None), dict(idx=torch.zeros(3, 0, dtype=i32))):
        for name, call in calls(hsa, d, cache, **good).items():
            call()
            assert fake.calls.pop() == name
    both = dict(q=None, q_out=None)
    calls(hsa, d, cache, **both)[wr]()
    calls(hsa, d, cache, k=None, k_out=None)[rot]()
    fake.calls.clear()
    for bad, names in (
            (dict(q=fused[:, :4].float()), (rot, wr, tree)), (dict(q=fused[:4, :4]), (rot, wr, tree)),
            (dict(q=fused[:, :3]), (rot, wr, tree)), (dict(q=fused[..., ::2]), (rot, wr, tree)),
            (dict(q_out=fused[:4, :4]), (rot, wr)), (dict(q_out=None), (rot, wr)),
            (dict(k=fused[:, :4]), (rot, wr)), (dict(k=fused[:4, :2]), (rot, wr)),
            (dict(k_out=None), (rot,)), (dict(v=fused[:, :1]), (wr,)),
            (dict(pos=torch.zeros(5).long()), (rot, wr)), (dict(pos=torch.zeros(4, dtype=i32)), (rot, wr)),
            (dict(pos=torch.zeros(10, dtype=i32)[::2]), (rot, wr)),
            (dict(parents=torch.zeros(5).long()), (tree,)),
            (dict(parents=torch.zeros(4, dtype=i32)), (tree,)),
            (dict(cu=torch.zeros(4).long()), (rot, wr, tree, keep)),
            (dict(cu=torch.zeros(3, dtype=i32)), (rot, wr, tree, keep)),
            (dict(lens=torch.zeros(3).long()), (rot, wr, tree, keep)),
            (dict(table=torch.zeros(3, 4).long()), (wr, tree, keep)),
            (dict(out=torch.zeros(5, 4, 128)), (tree,)), (dict(out=fused[:, :4]), (tree,)),
            (dict(lse=torch.zeros(5, 8)[:, ::2]), (tree,)),
            (dict(idx=torch.zeros(3, 4).long()), (keep,)), (dict(idx=torch.zeros(2, 4, dtype=i32)), (keep,)),
            (dict(idx=torch.zeros(3, 8, dtype=i32)[:, ::2]), (keep,)),
            (dict(cnt=torch.zeros(2, dtype=i32)), (keep,)), (dict(cnt=torch.zeros(3).long()), (keep,)),
            (dict(new=torch.zeros(2, dtype=i32)), (keep,))):
        made = calls(hsa, d, cache, **bad)
        for name in names:
            with pytest.raises(hsa.HsaError):
                made[name]()
    for small in (cpu_cache(hsa, 7, 2), cpu_cache(hsa, 8, 1)):
        for name in (wr, tree, keep):
            with pytest.raises(hsa.HsaError):
                calls(hsa, d, small)[name]()
    for bad in (torch.zeros(4, 32, dtype=torch.float64), torch.zeros(32), torch.zeros(4, 64)[:, ::2]):
        with pytest.raises(hsa.HsaError):
            hsa.Rotary(bad)
    assert not fake.calls


def test_a_descriptor_keeps_its_struct_until_a_field_is_set():
    d = hsa.Dims(batch=2, hq=8, hkv=2, max_pages_per_seq=4, num_pages=9)
    held = d.ref()
    assert d.ref() is held and held._obj.batch == 2
    twins = [copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d)),
             dataclasses.replace(d, batch=3)]
    d.batch = 5
    assert d.ref()._obj.batch == 5 and held._obj.batch == 2
    assert [t.ref()._obj.batch for t in twins] == [2, 2, 2, 3]
    assert twins[0] == twins[1] != d


def test_a_table_is_made_on_a_gpu():
    with pytest.raises(hsa.HsaError):
        hsa.hsa_rotary_table(16, 128, device="cpu")


def test_a_descriptor_has_its_fields_alone():
    """What derives one descriptor from another's fields finds nothing else among them."""
    d = hsa.Dims(batch=2, hq=8, hkv=2, max_pages_per_seq=4, num_pages=9)
    names = [f.name for f in dataclasses.fields(d)]
    d.ref()
    assert list(vars(d)) == names
    other = hsa.Dims(**{**d.__dict__, "batch": 3})
    assert other.ref()._obj.batch == 3 and d.ref()._obj.batch == 2
    pickle.dumps(vars(d))
    d.chunk = 128
    assert d.ref()._obj.chunk == 128
    del d.chunk  # (the class's value again)
    assert d.ref()._obj.chunk == 64


def test_a_descriptor_set_while_its_struct_is_made():
    """A struct of fields that another thread sets meanwhile is not held: neither one whose fields
    were read before the set and that is there after it, nor one made between a field's value and
    the end of the call that sets it."""
    class Slow(hsa.Dims):
        def c(self):
            made = super().c()
            if hook:
                hook.pop()()
            return made

    d, hook = Slow(batch=2, hq=8, hkv=2, max_pages_per_seq=4, num_pages=9), []
    hook.append(lambda: setattr(d, "batch", 5))
    assert d.ref()._obj.batch == 2
    assert d.ref()._obj.batch == 5
    twin = copy.copy(d)
    hook.append(lambda: setattr(twin, "batch", 6))
    twin.ref()
    assert twin.ref()._obj.batch == 6 and d.ref()._obj.batch == 5

    class Early(hsa.Dims):  # asked for its struct as soon as a field may have changed
        def __setattr__(self, name, value):
            super().__setattr__(name, value)
            if watched:
                watched.append(self.ref()._obj.batch)

    watched = []
    e = Early(batch=2, hq=8, hkv=2, max_pages_per_seq=4, num_pages=9)
    e.ref()
    watched.append(0)
    e.batch = 7
    assert watched == [0, 7]

    class Between(int):  # a value that asks for the struct while it replaces the one before
        def __del__(self):
            d.ref()

    d.num_pages = Between(9)
    d.num_pages = 11
    assert d.ref()._obj.num_pages == 11


class On:
    """A tensor as if it lay on another device (-1: the host), pinned or not."""

    def __init__(self, t, device, pinned=False):
        self.t, self.device_index, self.pinned = t, device, pinned

    def get_device(self):
        return self.device_index

    def is_pinned(self):
        return self.pinned

    def __getattr__(self, name):
        return getattr(self.t, name)


def on_devices(hsa, monkeypatch, current=0):
    monkeypatch.setattr(hsa, "_DEVICE", lambda: current)
    d = dims(hsa, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    bf, i32 = torch.bfloat16, torch.int32
    cache = cpu_cache(hsa, 8, 2)
    cache.device = 0
    rotary = hsa.Rotary(_aligned((64, 32), torch.float32))
    rotary.device = 0
    rows = dict(q=torch.zeros(5, 4, 128, dtype=bf), q_out=torch.zeros(5, 4, 128, dtype=bf),
                k=torch.zeros(5, 2, 128, dtype=bf), k_out=torch.zeros(5, 2, 128, dtype=bf),
                v=torch.zeros(5, 2, 128, dtype=bf), out=torch.zeros(5, 4, 128, dtype=bf),
                lse=torch.zeros(5, 4), ws=torch.zeros(64, dtype=torch.uint8))
    lists = dict(pos=torch.zeros(5, dtype=i32), parents=torch.zeros(5, dtype=i32),
                 cu=torch.zeros(4, dtype=i32), table=torch.zeros(3, 4, dtype=i32),
                 lens=torch.zeros(3, dtype=i32), idx=torch.zeros(3, 4, dtype=i32),
                 cnt=torch.zeros(3, dtype=i32), new=torch.zeros(3, dtype=i32))
    return d, cache, rotary, rows, lists


# what each call reads and writes
TAKES = {
    "hsa_rotate": "q q_out k k_out pos",
    "hsa_kv8_write_rotated": "q q_out k v pos cu table lens",
    "hsa_kv8_tree": "q out lse ws parents cu table lens",
    "hsa_kv8_keep": "idx cnt cu table lens new",
}


def test_tensors_of_another_device_are_refused(binding, monkeypatch):  # noqa: F811
    """The library sees addresses alone: it would follow one of host memory, or of another GPU's."""
    hsa, fake = binding  # noqa: F811
    d, cache, rotary, rows, lists = on_devices(hsa, monkeypatch)
    every = {**rows, **lists}

    def made(**kw):
        a = {n: On(t, 0) for n, t in every.items()}
        a.update(kw)
        return calls(hsa, d, cache, rotary=rotary, **a)

    for name, takes in TAKES.items():
        made()[name]()
        assert fake.calls.pop() == name
        for n in takes.split():
            for device in (-1, 1):
                with pytest.raises(hsa.HsaError):
                    made(**{n: On(every[n], device)})[name]()
            pinned = made(**{n: On(every[n], -1, True)})[name]
            if n in lists:
                pinned()
                assert fake.calls.pop() == name
            else:
                with pytest.raises(hsa.HsaError):
                    pinned()
    for n in ("cu", "lens"):  # read by a rotation without positions only
        with pytest.raises(hsa.HsaError):
            made(pos=None, **{n: On(every[n], -1)})["hsa_rotate"]()
    monkeypatch.setattr(hsa, "_DEVICE", lambda: 1)
    for name in TAKES:
        with pytest.raises(hsa.HsaError):
            made()[name]()
    assert not fake.calls
    with pytest.raises(hsa.HsaError):
        hsa.KV8(cache.k, cache.v, cache.k_scale, On(cache.v_scale, 0))


@needs_lib
def test_host_tensors_are_refused_by_the_library_itself(lib):  # noqa: F811
    """Also where all of them lie there. (None of these calls reaches a GPU.)"""
    d = dims(lib, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    for name, call in calls(lib, d, cpu_cache(lib, 8, 2)).items():
        with pytest.raises(lib.HsaError) as e:
            call()
        assert e.value.code == INVALID, name


def test_lists_of_other_sizes_are_refused(binding):  # noqa: F811
    hsa, fake = binding  # noqa: F811
    d = dims(hsa, batch=3, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    cache, i32 = cpu_cache(hsa, 8, 2), torch.int32
    names = ("hsa_kv8_write_rotated", "hsa_kv8_tree", "hsa_kv8_keep")
    for good in (dict(table=torch.zeros(64, 4, dtype=i32)), dict(table=torch.zeros(12, dtype=i32)),
                 dict(lens=torch.zeros(64, dtype=i32)), dict(lens=torch.zeros(3, 1, dtype=i32))):
        for name in names:
            calls(hsa, d, cache, **good)[name]()
            assert fake.calls.pop() == name
    for bad in (dict(table=torch.zeros(2, 4, dtype=i32)), dict(table=torch.zeros(3, 8, dtype=i32)[:, :4]),
                dict(table=torch.zeros(3, 8, dtype=i32)), dict(table=torch.zeros(4, 3, dtype=i32)),
                dict(table=torch.zeros(11, dtype=i32)), dict(lens=torch.zeros(2, dtype=i32)),
                dict(lens=torch.zeros(6, dtype=i32)[::2])):
        for name in names:
            with pytest.raises(hsa.HsaError):
                calls(hsa, d, cache, **bad)[name]()
    for lens in (torch.zeros(2, dtype=i32), torch.zeros(6, dtype=i32)[::2]):
        with pytest.raises(hsa.HsaError):
            calls(hsa, d, cache, pos=None, lens=lens)["hsa_rotate"]()
    one = dims(hsa, batch=1, hq=4, hkv=2, num_pages=8, max_pages_per_seq=4)
    calls(hsa, one, cache, idx=torch.zeros(1, 4, dtype=i32), table=torch.zeros(1, 8, dtype=i32))[names[2]]()
    assert fake.calls == [names[2]]
