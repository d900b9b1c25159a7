"""Rotary positions and drafted tokens on the 8-bit K/V cache, on the GPU: rows and codes bit for
bit against the numpy oracle, attention against 64 bits within derived bounds."""
import numpy as np
import pytest
import torch

from kv8_harness import (D, PAGE, Batch, assert_rows, assert_same_cache, bf16, codes_of,
                         to_bf16)
from kv_cache_int8_gb300 import hsa
from oracle import draft as R
from oracle import kv8 as O

pytestmark = pytest.mark.gpu

FORMATS = ("int8", "e4m3")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(new):
    return i32(np.concatenate([[0], np.cumsum(new)]))


def places(lens, new):
    return np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)] or [[]]).astype(np.int64)


def err_word():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def bits(t):
    return t.view(torch.int16).cpu().numpy()


def angle_table(rows, dim, base=10000.0, magnitude=1.0):
    return R.table(rows, R.frequencies(dim, base), magnitude).astype(np.float32)


def to_bf16_bits(x):
    """fp32 values to bf16 bit patterns as the rounding instruction makes them."""
    return bits(torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16))


# ------------------------------------------------------------------------------ the table

@pytest.mark.parametrize("dim,kw", [
    (128, dict()), (8, dict(base=500000.0)), (64, dict(scaling=1, factor=4.0, magnitude=1.25)),
    (96, dict(scaling=2, factor=8.0, base=500000.0)),
    (120, dict(scaling=2, factor=40.0, low=1.0, high=32.0, original=4096.0, magnitude=0.5)),
])
def test_rotary_table(dim, kw):
    """Half a step of fp32: the numbers of [2^(e - 1), 2^e) lie 2^(e - 24) apart, so values up to a
    magnitude of at most 2^e are off by at most 2^(e - 25) (magnitude 1.25, values above 1: 2^-24,
    not 1.25 2^-25). Angles up to 2^20 radians are known to a few units of 2^-53, so to 2^-31
    together."""
    rows = (1 << 20) + 3
    got = hsa.hsa_rotary_table(rows, dim, **kw)
    assert got.shape == (rows, dim)
    pick = np.concatenate([np.arange(300), np.arange(rows - 300, rows),
                           np.random.default_rng(1).integers(rows, size=500)])
    magnitude = kw.pop("magnitude", 1.0)
    f = R.frequencies(dim, kw.pop("base", 10000.0), **kw)
    a = pick[:, None] * f
    want = magnitude * np.concatenate([np.cos(a), np.sin(a)], -1)
    err = np.abs(got[torch.from_numpy(pick).cuda()].cpu().numpy() - want)
    assert err.max() <= 2.0 ** (np.ceil(np.log2(magnitude)) - 25) + magnitude * 2.0 ** -31


# ------------------------------------------------------------------------------- rotation

@pytest.mark.parametrize("neighbours", (False, True))
@pytest.mark.parametrize("hq,hkv,dim,lens,new", [
    (1, 1, 8, [1], [1]), (32, 8, 128, [5], [1]), (4, 1, 64, [1, 17, 300], [1, 16, 0]),
    (24, 3, 96, [70, 9], [33, 9]), (17, 17, 120, [40], [7]), (40, 8, 16, [3] * 100, [2] * 100),
    (64, 8, 32, [2000], [1999]), (8, 4, 128, [1] * 1024, [1] * 1024),
])
def test_rotation(neighbours, hq, hkv, dim, lens, new):
    rng = np.random.default_rng(dim + len(lens))
    T = sum(new)
    q, k = (bf16(rng.standard_normal((T, h, D))) for h in (hq, hkv))
    t = angle_table(max(lens), dim)
    rot = hsa.Rotary(torch.from_numpy(t).cuda(), neighbours)
    d = hsa.Dims(batch=len(lens), hq=hq, hkv=hkv, max_pages_per_seq=1, num_pages=1)
    at = t[places(lens, new)]
    want_q, want_k = (to_bf16_bits(R.turn(x, at, neighbours)) for x in (q, k))
    gq, gk = to_bf16(q), to_bf16(k)
    oq, ok = torch.empty_like(gq), torch.empty_like(gk)
    err = err_word()
    hsa.hsa_rotate(d, rot, gq, oq, gk, ok, None, cu_of(new), i32(lens), err)
    np.testing.assert_array_equal(bits(oq), want_q)
    np.testing.assert_array_equal(bits(ok), want_k)
    # positions given, in place, queries alone
    hsa.hsa_rotate(d, rot, gq, gq, None, None, i32(places(lens, new)), None, None, err)
    np.testing.assert_array_equal(bits(gq), want_q)
    if new == [1] * len(lens):
        oq.zero_()
        hsa.hsa_rotate(d, rot, to_bf16(q), oq, gk, gk, None, None, i32(lens), err)
        np.testing.assert_array_equal(bits(oq), want_q)
        np.testing.assert_array_equal(bits(gk), want_k)
    assert hsa.hsa_read_device_error(err) == 0


def test_rotation_of_slices_of_numbers_that_are_none_and_of_rows_of_no_sequence():
    """Slices of a fused projection in place; infinities, NaN and the largest numbers stay in their
    pairs; rows behind the last sequence stay as they were; a graph and another stream."""
    hq, hkv, dim, lens, new = 6, 2, 64, [100, 50, 20], [30, 0, 20]
    T, rng = 50, np.random.default_rng(3)
    x = bf16(rng.standard_normal((T + 7, hq + 2 * hkv, D)))
    x[3, 1, 5], x[7, 6, 40], x[8, 0, 0], x[9, 7, 127], x[10, 2, 33] = (
        np.inf, -np.inf, np.nan, np.inf, 3.38e38)
    x = bf16(x)
    t = angle_table(100, dim)
    for neighbours in (False, True):
        rot = hsa.Rotary(torch.from_numpy(t).cuda(), neighbours)
        d = hsa.Dims(batch=3, hq=hq, hkv=hkv, max_pages_per_seq=1, num_pages=1)
        fused = [to_bf16(x) for _ in range(3)]
        want = x.copy()
        want[:T, :hq + hkv] = R.turn(x[:T, :hq + hkv], t[places(lens, new)], neighbours)
        args = [(d, rot, f[:, :hq], f[:, :hq], f[:, hq:hq + hkv], f[:, hq:hq + hkv], None,
                 cu_of(new), i32(lens)) for f in fused]
        hsa.hsa_rotate(*args[0])
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            hsa.hsa_rotate(*args[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hsa.hsa_rotate(*args[2])
        graph.replay()
        torch.cuda.synchronize()
        for f in fused:
            got = f.float().cpu().numpy()
            w = torch.from_numpy(want).to(torch.bfloat16).float().numpy()
            np.testing.assert_array_equal(np.isnan(got), np.isnan(w))
            np.testing.assert_array_equal(got[~np.isnan(w)], w[~np.isnan(w)])


def test_positions_outside_the_table_are_reported():
    d = hsa.Dims(batch=2, hq=2, hkv=1, max_pages_per_seq=1, num_pages=1)
    t = angle_table(50, 128)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    rng = np.random.default_rng(4)
    q = bf16(rng.standard_normal((6, 2, D)))
    err = err_word()
    for pos, cu, lens, ok in (([0, 49, 50, -1, 7, 1 << 30], None, None, [0, 1, 4]),
                              (None, [0, 4, 6], [52, 10], [0, 1, 4, 5]),
                              (None, [0, 4, 6], [3, 10], [4, 5]),  # more rows than tokens
                              (None, [0, 4, 7], [10, 10], [0, 1, 2, 3])):
        out = torch.full((6, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        hsa.hsa_rotate(d, rot, to_bf16(q), out, None, None, None if pos is None else i32(pos),
                       None if cu is None else i32(cu), None if lens is None else i32(lens), err)
        assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
        at = np.array(pos if pos is not None else [*range(lens[0] - 4, lens[0]), 8, 9])
        for r in range(6):
            if r in ok:
                w = to_bf16_bits(R.turn(q[r:r + 1], t[at[r:r + 1]], False))
                np.testing.assert_array_equal(bits(out[r:r + 1]), w)
            else:
                assert (out[r] == 9.0).all()


# ------------------------------------------------------------------------- rotated writes

def rows_of(s, n, heads):
    return bf16(s.rng.standard_normal((n, heads, D)))


def oracle_write(s, lens, new, k, v, t, positions, neighbours):
    """The oracle's cache after the new tokens; the positions default to the places."""
    at = 0
    pos = places(lens, new) if positions is None else np.asarray(positions)
    for b, (n, m) in enumerate(zip(lens, new)):
        if m:
            turned = R.turn(k[at:at + m], t[pos[at:at + m]], neighbours)
            O.write(s.cache, turned, v[at:at + m], s.table[b], n - m)
        at += m


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,dim,neighbours,before,new", [
    (1, 1, 128, False, [0], [1]), (32, 8, 128, False, [37], [1]), (8, 2, 64, True, [15, 16], [1, 1]),
    (12, 2, 96, False, [0, 5, 250, 31], [16, 12, 0, 33]), (8, 8, 8, True, [1, 2], [200, 15]),
    (24, 8, 120, False, [3] * 40, [2] * 40), (4, 4, 128, True, [9], [300]),
])
def test_rotated_write(fmt, hq, hkv, dim, neighbours, before, new):
    lens = [a + n for a, n in zip(before, new)]
    s = Batch(lens, hq, hkv, fmt, seed=dim + len(new), extra_pages=1, fill=False)
    for b, a in enumerate(before):
        if a:
            O.write(s.cache, s.rows(a, True), s.rows(a), s.table[b], 0)
    cache, d, T = s.gpu_cache(), s.dims(), sum(new)
    t = angle_table(max(lens) + 9, dim)
    rot = hsa.Rotary(torch.from_numpy(t).cuda(), neighbours)
    q, k, v = rows_of(s, T, hq), rows_of(s, T, hkv) * np.float32(3), rows_of(s, T, hkv)
    k = bf16(k)
    qkv = to_bf16(np.concatenate([q, k, v], 1))
    sl = (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    cu = None if new == [1] * len(new) else cu_of(new)
    err = err_word()
    oracle_write(s, lens, new, k, v, t, None, neighbours)
    hsa.hsa_kv8_write_rotated(d, cache, rot, sl[0], out, sl[1], sl[2], None, cu, s.gpu_table(),
                              s.gpu_lens(), err)
    assert_same_cache(cache, s.cache)
    want = to_bf16_bits(R.turn(q, t[places(lens, new)], neighbours))
    np.testing.assert_array_equal(bits(out), want)
    # written again at other positions, without queries, then queries turned in place
    pos = s.rng.integers(0, max(lens) + 9, T)
    oracle_write(s, lens, new, k, v, t, pos, neighbours)
    hsa.hsa_kv8_write_rotated(d, cache, rot, None, None, sl[1], sl[2], i32(pos), cu,
                              s.gpu_table(), s.gpu_lens(), err)
    assert_same_cache(cache, s.cache)
    oracle_write(s, lens, new, k, v, t, pos, neighbours)
    hsa.hsa_kv8_write_rotated(d, cache, rot, sl[0], sl[0], sl[1], sl[2], i32(pos), cu,
                              s.gpu_table(), s.gpu_lens(), err)
    assert_same_cache(cache, s.cache)
    np.testing.assert_array_equal(bits(qkv[:, :hq]), to_bf16_bits(R.turn(q, t[pos], neighbours)))
    assert hsa.hsa_read_device_error(err) == 0


@pytest.mark.parametrize("fmt,hq,hkv,dim,neighbours,before,new", [
    ("int8", 5, 5, 128, False, [7, 0], [4000, 2600]), ("e4m3", 8, 8, 64, True, [100, 3, 0], [5000, 1, 1600]),
    ("int8", 8, 8, 24, False, [5], [9000]), ("e4m3", 3, 3, 128, True, [33, 0, 2], [9, 0, 11000]),
])
def test_rotated_write_of_long_prompts(fmt, hq, hkv, dim, neighbours, before, new):
    """Enough blocks that a warp takes several heads, runs that do not divide the heads among them."""
    test_rotated_write(fmt, hq, hkv, dim, neighbours, before, new)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rotated_write_token_by_token_from_a_graph(fmt):
    """A decode loop whose one graph replays: the scale of a block grows, its codes follow."""
    s = Batch([0, 0], 4, 2, fmt, seed=5, fill=False, extra_pages=3)
    s.table[:, :3] = s.rng.permutation(6).reshape(2, 3)
    s.num_pages = 6
    s.cache = O.empty(fmt, 6, 2)
    d, cache = s.dims(), s.gpu_cache()
    t = angle_table(64, 128)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    q = torch.empty(2, 4, D, dtype=torch.bfloat16, device="cuda")
    k, v, out = q[:, :2].clone(), q[:, :2].clone(), torch.empty_like(q)
    lens = i32([1, 8])
    args = (d, cache, rot, q, out, k, v, None, None, s.gpu_table(), lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hsa.hsa_kv8_write_rotated(*args)
    for step in range(36):
        x = [bf16(s.rng.standard_normal((2, h, D)) * 1.1 ** step) for h in (4, 2, 2)]
        for dst, src in zip((q, k, v), x):
            dst.copy_(to_bf16(src))
        n = [1 + step, 8 + step]
        lens.copy_(i32(n))
        graph.replay()
        oracle_write(s, n, [1, 1], x[1], x[2], t, None, False)
        np.testing.assert_array_equal(bits(out), to_bf16_bits(
            R.turn(x[0], t[np.array(n) - 1], False)))
    assert_same_cache(cache, s.cache)


def test_rotated_write_of_awkward_values():
    """Infinities, NaN, numbers that overflow as they turn, zeros and the smallest: the rules of
    the plain write on the turned values."""
    for fmt in FORMATS:
        for neighbours in (False, True):
            s = Batch([33], 2, 1, fmt, seed=6, fill=False)
            k, v = rows_of(s, 33, 1), rows_of(s, 33, 1)
            k[0, 0, 3], k[1, 0, 70], k[2, 0, 9], v[3, 0, 1] = np.inf, -np.inf, np.nan, np.nan
            k[16:32] = 0
            k[17, 0, 0:128:16] = bf16(1e-39)
            k[32, 0, :] = bf16(3.38e38)
            t = angle_table(64, 128)
            rot = hsa.Rotary(torch.from_numpy(t).cuda(), neighbours)
            cache = s.gpu_cache()
            oracle_write(s, [33], [33], k, v, t, None, neighbours)
            hsa.hsa_kv8_write_rotated(s.dims(), cache, rot, None, None, to_bf16(k), to_bf16(v),
                                      None, cu_of([33]), s.gpu_table(), s.gpu_lens())
            assert_same_cache(cache, s.cache)


def test_rotated_writes_that_do_not_fit_are_reported():
    """A position outside the table leaves its token's block and query row as they were; a bad page
    its block; a bad length its sequence."""
    s = Batch([40, 20, 33], 2, 2, "int8", seed=7)
    new = [30, 20, 33]
    T = sum(new)
    q, k, v = rows_of(s, T, 2), rows_of(s, T, 2), rows_of(s, T, 2)
    t = angle_table(64, 32)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    pos = places(s.lens, new)
    pos[25] = 64  # sequence 0, token 35: block 2
    pos[52] = -1  # sequence 2, token 2: block 0
    err = err_word()
    out = torch.full((T, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    cache = s.gpu_cache()
    table = s.gpu_table()
    table[1, 1] = s.num_pages  # sequence 1, block 1
    held = {n: a.copy() for n, a in s.cache.items() if n != "fmt"}
    good = np.where((pos < 0) | (pos > 63), 0, pos)
    oracle_write(s, s.lens, new, k, v, t, good, False)
    for b, j in ((0, 2), (2, 0), (1, 1)):
        for n in held:
            s.cache[n][s.table[b, j]] = held[n][s.table[b, j]]
    hsa.hsa_kv8_write_rotated(s.dims(), cache, rot, to_bf16(q), out, to_bf16(k), to_bf16(v),
                              i32(pos), cu_of(new), table, s.gpu_lens(), err)
    assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
    assert_same_cache(cache, s.cache)
    want = to_bf16_bits(R.turn(q, t[good], False))
    keep = np.ones(T, bool)
    keep[[25, 52]] = False
    np.testing.assert_array_equal(bits(out)[keep], want[keep])
    assert (out[25] == 9.0).all() and (out[52] == 9.0).all()
    for lens, cu in (([40, -5, 33], [0, 30, 50, 83]), ([40, 20, 33], [0, 30, 20, 83]),
                     ([40, 20, 33], [0, 30, 50, 84]), ([40, 20, 49], [-1, 30, 50, 83])):
        hsa.hsa_kv8_write_rotated(s.dims(), cache, rot, None, None, to_bf16(k), to_bf16(v), None,
                                  i32(cu), s.gpu_table(), i32(lens), err)
        assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK


# ------------------------------------------------------------------------- tree attention

def run_tree(s, q, parents, new, lens=None, ws=None, **kw):
    d = s.dims(**kw)
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE) if ws is None else ws
    T = sum(new)
    out = torch.full((T, s.hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, s.hq), float("nan"), device="cuda")
    up = None if parents is None else i32([p for t in parents for p in t])
    hsa.hsa_kv8_tree(d, s.gpu_cache(), to_bf16(q), up, cu_of(new), s.gpu_table(), s.gpu_lens(lens),
                     out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check_tree(s, q, parents, new, out, lse, sm_scale=D ** -0.5, lens=None):
    g = s.hq // s.hkv
    at = 0
    for b, (n, m) in enumerate(zip(s.lens if lens is None else lens, new)):
        up = range(-1, m - 1) if parents is None else parents[b]
        seen = R.seen(n, up) if m else None
        for h in range(s.hkv if m else 0):
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            for j in range(h * g, (h + 1) * g):
                want, wl, tol = O.attend(q[at:at + m, j], k, v, seen, sm_scale)
                # weights are rounded to fp16 before the product with V (half a step 2^-11 of
                # each, so that much of the largest value), the result to bf16
                tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(v).max()
                assert_rows(out[at:at + m, j], None if lse is None else lse[at:at + m, j], want, wl,
                            tol, 2.0 ** -8)
        at += m


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,lens,new", [
    (1, 1, [1], [1]), (4, 1, [64], [64]), (8, 1, [128, 129], [128, 1]), (8, 8, [300], [40]),
    (4, 1, [300], [256]), (3, 1, [500, 90], [170, 90]), (14, 2, [400], [77]),
    (16, 2, [1, 17, 260, 1000], [1, 16, 0, 130]), (32, 8, [1500], [25]), (2, 1, [700], [256]),
    (64, 8, [333, 700], [1, 17]), (5, 1, [2048], [60]), (8, 2, [40] * 33, [3] * 33),
    (8, 1, [5000], [16]), (8, 1, [129, 128, 127, 256], [8, 8, 8, 8]), (6, 1, [2000], [200]),
    (32, 8, [16], [16]), (1, 1, [4000], [255]), (7, 1, [900, 1], [1, 1]),
])
def test_tree(fmt, hq, hkv, lens, new):
    s = Batch(lens, hq, hkv, fmt, seed=len(lens) + hq, extra_pages=1)
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    parents = [R.tree(s.rng, m, True) for m in new]
    out, lse = run_tree(s, q, parents, new)
    check_tree(s, q, parents, new, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_trees_of_every_shape(fmt):
    """A chain, a star, a comb, only roots, a chain given by no parents at all."""
    new = [40] * 4
    s = Batch([300, 40, 128, 90], 8, 2, fmt, seed=31)
    q = bf16(s.rng.standard_normal((160, 8, D)))
    parents = [list(range(-1, 39)), [-1] + [0] * 39, [-1] + [i // 2 * 2 for i in range(39)],
               [-1] * 40]
    out, lse = run_tree(s, q, parents, new)
    check_tree(s, q, parents, new, out, lse)
    out, lse = run_tree(s, q, None, new)
    check_tree(s, q, None, new, out, lse)


def test_tree_of_one_node_a_sequence_is_a_decode():
    """Without offsets; the same rows as the decode attention's within both roundings."""
    s = Batch([300, 17, 1, 1000], 8, 2, "e4m3", seed=32)
    q = bf16(s.rng.standard_normal((4, 8, D)))
    d = s.dims()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)  # serves all attentions
    out = torch.empty(4, 8, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 8, device="cuda")
    hsa.hsa_kv8_tree(d, s.gpu_cache(), to_bf16(q), i32([-1] * 4), None, s.gpu_table(),
                     s.gpu_lens(), out, lse, ws)
    check_tree(s, q, [[-1]] * 4, [1] * 4, out.float().cpu().numpy(), lse.cpu().numpy())
    full = torch.empty(4, 8, D, device="cuda")
    hsa.hsa_kv8_decode(d, s.gpu_cache(), to_bf16(q), s.gpu_table(), s.gpu_lens(), full, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    want = full.cpu().numpy()
    top = max(np.abs(O.values(s.cache, "v", s.table[b], n, h)).max()
              for b, n in enumerate(s.lens) for h in range(2))
    assert (np.abs(out.float().cpu().numpy() - want) <= 2.0 ** -10 * top + 2.0 ** -8 * np.abs(want)).all()


def test_tree_of_slices_streams_and_graphs():
    """Queries as slices of a fused projection, rows behind the last sequence left alone; the same
    bits on another stream and from a graph."""
    hq, hkv, new = 8, 2, [70, 0, 33]
    s = Batch([600, 20, 33], hq, hkv, "int8", seed=33)
    T = sum(new)
    q = bf16(s.rng.standard_normal((T, hq, D)))
    parents = [R.tree(s.rng, m) for m in new]
    fused = torch.full((T + 9, hq + 2 * hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:T, :hq] = to_bf16(q)
    up = i32([p for t in parents for p in t] + [7] * 9)
    d, cache = s.dims(), s.gpu_cache()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)
    outs = [torch.full((T + 9, hq, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    args = (d, cache, fused[:, :hq], up, cu_of(new), s.gpu_table(), s.gpu_lens())
    hsa.hsa_kv8_tree(*args, outs[0], None, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        hsa.hsa_kv8_tree(*args, outs[1], None, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hsa.hsa_kv8_tree(*args, outs[2], None, ws)
        hsa.hsa_kv8_tree(*args, outs[3], None, ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert hsa.hsa_read_device_error(ws) == 0
    for o in outs:
        assert torch.equal(o, outs[0]) and (o[T:] == 5.0).all()
    check_tree(s, q, parents, new, outs[0][:T].float().cpu().numpy(), None)


def test_tree_reports_what_does_not_fit():
    """Parents that are no earlier nodes, bad pages, lengths and offsets, too many nodes: reported,
    and the other sequences' rows right."""
    hq, hkv, new = 4, 1, [10, 20, 30]
    s = Batch([200, 100, 300], hq, hkv, "int8", seed=34)
    q = bf16(s.rng.standard_normal((60, hq, D)))
    parents = [R.tree(s.rng, m) for m in new]
    flat = [p for t in parents for p in t]
    d, cache = s.dims(), s.gpu_cache()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)

    def call(up=flat, cu=(0, 10, 30, 60), lens=s.lens, table=None):
        out = torch.full((60, hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((60, hq), 5.0, device="cuda")
        hsa.hsa_kv8_tree(d, cache, to_bf16(q), i32(up), i32(list(cu)),
                         s.gpu_table() if table is None else table, i32(lens), out, lse, ws)
        assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK
        assert torch.isfinite(out).all()
        return out.float().cpu().numpy(), lse.cpu().numpy()

    for bad in (-2, 5, 6, 1 << 30, -(1 << 31)):  # of node 5 of sequence 1: counts as -1
        up = list(flat)
        up[15] = bad
        out, lse = call(up)
        fixed = [parents[0], [p if i != 5 else -1 for i, p in enumerate(parents[1])], parents[2]]
        check_tree(s, q, fixed, new, out, lse)
    table = s.gpu_table()
    table[1, 2] = s.num_pages
    out, lse = call(table=table)
    for rows, m, b in ((slice(0, 10), 10, 0), (slice(30, 60), 30, 2)):
        one = Batch.__new__(Batch)
        one.__dict__.update(s.__dict__, lens=[s.lens[b]], table=s.table[b:b + 1])
        check_tree(one, q[rows], [parents[b]], [m], out[rows], lse[rows])
    for kw in (dict(lens=[200, 19, 300]), dict(lens=[200, -7, 300]), dict(lens=[200, 1 << 30, 300])):
        out, lse = call(**kw)
        assert (out[10:30] == 0).all() and np.isneginf(lse[10:30]).all()
        one = Batch.__new__(Batch)
        one.__dict__.update(s.__dict__, lens=[300], table=s.table[2:])
        check_tree(one, q[30:], [parents[2]], [30], out[30:], lse[30:])
    for cu in ((0, 10, 5, 60), (0, 10, 30, 61), (-4, 10, 30, 60)):
        call(cu=cu)
    # 257 nodes
    s = Batch([300, 30], 2, 1, "int8", seed=35)
    q = bf16(s.rng.standard_normal((262, 2, D)))
    d, cache = s.dims(), s.gpu_cache()
    out = torch.full((262, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((262, 2), 5.0, device="cuda")
    hsa.hsa_kv8_tree(d, cache, to_bf16(q), None, cu_of([257, 5]), s.gpu_table(), s.gpu_lens(), out,
                     lse, ws)
    assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK
    assert (out[:257] == 0).all() and torch.isneginf(lse[:257]).all()
    one = Batch.__new__(Batch)
    one.__dict__.update(s.__dict__, lens=[30], table=s.table[1:])
    check_tree(one, q[257:], None, [5], out[257:].float().cpu().numpy(), lse[257:].cpu().numpy())


@pytest.mark.parametrize("hq,hkv,n,m", [(8, 2, 600, 9), (8, 1, 5000, 16), (4, 4, 300, 100)])
def test_queries_that_are_not_finite_stay_in_their_rows(hq, hkv, n, m):
    s = Batch([n], hq, hkv, "int8", seed=36)
    q = bf16(s.rng.standard_normal((m, hq, D)))
    clean = q.copy()
    q[1, 0, 3], q[4, hq - 1, 100], q[m - 1, 1, 0] = np.inf, np.nan, -np.inf
    bad = ~np.isfinite(q).all(-1)
    parents = [R.tree(s.rng, m)]
    out, lse = run_tree(s, q, parents, [m])
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad]).all()
    ref_out, ref_lse = run_tree(s, clean, parents, [m])
    check_tree(s, clean, parents, [m], ref_out, ref_lse)
    at = ~bad
    got, want = out[at], ref_out[at]
    assert np.isfinite(got).all()
    # the rows' own weights are the same but for the scale that a block of rows shares
    assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * np.abs(want).max()).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", (3, 20))
def test_tree_over_blocks_of_zeros_and_of_unlike_scales(fmt, m):
    """V blocks of zeros count in the sums, K blocks of zeros give equal logits; scales of V that
    differ by 2^60 between blocks, queries by 2^40 and more between heads."""
    s = Batch([16 * 40 + 5], 4, 1, fmt, seed=37, fill=False)
    n = s.lens[0]
    k, v = s.rows(n), s.rows(n)
    block = np.arange(n) // PAGE
    v[block % 3 == 0] = 0
    v[block % 3 == 1] *= np.float32(2.0 ** -60)
    k[block % 4 == 1] = 0
    k[block == 40] = 0
    O.write(s.cache, k, v, s.table[0], 0)
    q = bf16(s.rng.standard_normal((m, 4, D)))
    q[:, 1] *= np.float32(2.0 ** -40)
    q[:, 2] *= np.float32(2.0 ** 20)  # one token takes all
    q[:, 3] = 0
    kk, vv = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    parents = R.tree(s.rng, m)
    out, lse = run_tree(s, q, [parents], [m])
    assert np.isfinite(out).all()
    for j in (0, 1, 3):  # at 2^20 the logits themselves are only known to a few units
        want, wl, tol = O.attend(q[:, j], kk, vv, R.seen(n, parents), D ** -0.5)
        tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
        assert_rows(out[:, j], lse[:, j], want, wl, tol, 2.0 ** -8)


def far_scales(s, b, kind):
    """V of sequence b by blocks: zeros, tiny, large, or everything in turn."""
    n = s.lens[b]
    k, v = s.rows(n), s.rows(n)
    block = (np.arange(n) // PAGE)[:, None, None]
    f = {"zero": 0.0 * block, "tiny": np.where(block % 7 == 3, 2.0 ** -100, 2.0 ** -90),
         "large": np.where(block % 5 == 1, 2.0 ** 100, 2.0 ** 70),
         "turns": np.choose(block % 4, [0.0, 2.0 ** -80, 1.0, 2.0 ** 90]),
         "late": np.where(block < block.max() * 0.6, 1.0, 2.0 ** 80)}[kind]
    O.write(s.cache, k, bf16(v * f), s.table[b], 0)


@pytest.mark.parametrize("kind", ("zero", "tiny", "large", "turns", "late"))
@pytest.mark.parametrize("hq,hkv,lens,m", [(4, 1, [2000], 5), (8, 1, [700, 3000], 16),
                                           (2, 2, [400], 60), (32, 8, [1200], 3)])
def test_tree_sums_where_v_is_zero_tiny_or_large(kind, hq, hkv, lens, m):
    """lse does not depend on V; results are right against the largest value that is seen."""
    s = Batch(lens, hq, hkv, "int8", seed=38, fill=False)
    for b in range(len(lens)):
        far_scales(s, b, kind)
    new = [m] * len(lens)
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    parents = [R.tree(s.rng, m) for _ in new]
    out, lse = run_tree(s, q, parents, new)
    check_tree(s, q, parents, new, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rise", (40.0, -40.0, 0.0))
def test_tree_whose_scores_grow_along_the_context(fmt, rise):
    """The running maximum moves at every tile, or never after the first; one token that takes
    everything at every place of a tile."""
    n, m = 1500, 12
    s = Batch([n], 8, 1, fmt, seed=39, fill=False)
    k, v = s.rows(n), s.rows(n)
    k[:, :, 0] = bf16(np.linspace(-1, 1, n)[:, None] * rise) + 0 * k[:, :, 0]
    O.write(s.cache, bf16(k), v, s.table[0], 0)
    q = bf16(s.rng.standard_normal((m, 8, D)))
    q[..., 0] = 8.0
    parents = [R.tree(s.rng, m)]
    out, lse = run_tree(s, q, parents, [m])
    check_tree(s, q, parents, [m], out, lse)


def test_one_token_takes_everything_at_every_place():
    n, m = 300, 16
    for at in (*range(0, 130, 9), 127, 128, 255, 256, 283, 284, 285, 299):
        s = Batch([n], 8, 1, "int8", seed=40, fill=False)
        k, v = s.rows(n) * np.float32(0.1), s.rows(n)
        k[at, 0, :16] = 100.0
        O.write(s.cache, bf16(k), v, s.table[0], 0)
        q = bf16(np.abs(s.rng.standard_normal((m, 8, D))))
        parents = [R.tree(s.rng, m)]
        out, lse = run_tree(s, q, parents, [m])
        check_tree(s, q, parents, [m], out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("power", (14, 20, 24, 30, 60, 100, 120))
@pytest.mark.parametrize("m", (2, 16))
def test_scores_of_any_size(fmt, power, m):
    """Queries up to 2^120: one token of a row has the largest score by far (its key is twice the
    others' largest along the query), so the row is that token's value but for fp16's and bf16's
    rounding, and lse its score within fp32's own roundings of it."""
    n = 700
    s = Batch([n], 8, 1, fmt, seed=44, fill=False)
    k, v = s.rows(n), s.rows(n)
    k[:, :, 0] = 1.0
    k[333, 0, 0] = 4.0
    O.write(s.cache, bf16(k), v, s.table[0], 0)
    q = np.zeros((m, 8, D), np.float32)
    q[..., 0] = 2.0 ** power
    q[m - 1, 3, 0] = -2.0 ** power  # (all scores alike but for one that is far below)
    parents = [R.tree(s.rng, m)]
    out, lse = run_tree(s, q, parents, [m])
    kk, vv = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    score = kk[333, 0] * 2.0 ** power * D ** -0.5
    rows = np.ones((m, 8), bool)
    rows[m - 1, 3] = False
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    # the weight of the one token is a power of two but for the sum's rounding: bf16's half step
    err = np.abs(out[rows] - vv[333])
    assert (err <= 2.0 ** -8 * np.abs(vv[333]) + 2.0 ** -20 * np.abs(vv[333]).max()).all()
    # factor, scale, product and logarithm: six roundings of the score, 2^-24 each
    assert (np.abs(lse[rows] - score) <= 6 * 2.0 ** -24 * score + 1e-5).all()


@pytest.mark.parametrize("hq,hkv,batch,m", [(8, 8, 300, 2), (4, 1, 1024, 1), (8, 1, 600, 5)])
def test_trees_of_large_batches(hq, hkv, batch, m):
    """Ragged batches of hundreds; a sample of the sequences against the oracle."""
    rng = np.random.default_rng(41)
    lens = [int(x) for x in rng.integers(m, 200, batch)]
    new = [int(rng.integers(0, m + 1)) for _ in lens]
    s = Batch(lens, hq, hkv, "int8", seed=41)
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    parents = [R.tree(s.rng, n, True) for n in new]
    out, lse = run_tree(s, q, parents, new)
    assert np.isfinite(out).all()
    at = np.concatenate([[0], np.cumsum(new)])
    for b in (*range(0, batch, 37), 255, 256, 257, batch - 1):
        if new[b] == 0:
            continue
        one = Batch.__new__(Batch)
        one.__dict__.update(s.__dict__, lens=[lens[b]], table=s.table[b:b + 1])
        r = slice(at[b], at[b + 1])
        check_tree(one, q[r], [parents[b]], [new[b]], out[r], lse[r])


def plain_tree(cache, table, n, q, seen, g):
    """out and lse of one sequence in fp64 on the GPU (long contexts): q [m][hq][128]."""
    m, hq, _ = q.shape
    outs, sums = [], []
    for h in range(hq // g):
        k, v = (getattr(cache, w).view(torch.int8)[table, h].view(cache.k.dtype).float().double() *
                getattr(cache, w + "_scale")[table, h].double()[:, None, None] for w in "kv")
        k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
        x = q[:, h * g:(h + 1) * g].double().transpose(0, 1) @ k.T * D ** -0.5
        x.masked_fill_(~seen, -float("inf"))
        lse = torch.logsumexp(x, -1)
        outs.append((torch.exp(x - lse[..., None]) @ v).transpose(0, 1))
        sums.append(lse.T)
    return torch.cat(outs, 1), torch.cat(sums, 1)


@pytest.mark.parametrize("fp8", (False, True))
@pytest.mark.parametrize("hq,hkv,n,m", [(8, 1, 1 << 20, 16), (4, 1, 700001, 5), (8, 8, 100003, 7),
                                        (8, 2, 300000, 70)])
def test_long_contexts(fp8, hq, hkv, n, m):
    """Stretches longer than the products add up by themselves (their sums round to zero, 2^-23 a
    product of 16 tokens: at most 2048 of them, 2^-12). The weights' fp16 rounding, up to 2^-11 of
    each, is a random sum over at least 1e5 / e weights (logits of variance 1), 1e-5; logits and
    fp32 sums 1e-5 more: 2^-14 together. Values of mean 2 against 64 bits."""
    pages = -(-n // PAGE)
    d = hsa.Dims(batch=1, hq=hq, hkv=hkv, max_pages_per_seq=pages, num_pages=pages)
    g = torch.Generator(device="cuda").manual_seed(7)
    cache = hsa.KV8.zeros(d, fp8)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    lens, cu = i32([n]), i32([0, n])
    k = torch.randn(n, hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    v = (torch.randn(n, hkv, D, generator=g, device="cuda") + 2.0).to(torch.bfloat16)
    hsa.hsa_kv8_write(d, cache, k, v, cu, table, lens)
    del k, v
    q = torch.randn(m, hq, D, generator=g, device="cuda").to(torch.bfloat16)
    parents = R.tree(np.random.default_rng(8), m)
    seen = torch.from_numpy(R.seen(n, parents)).cuda()
    out = torch.empty(m, hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(m, hq, device="cuda")
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)
    hsa.hsa_kv8_tree(d, cache, q, i32(parents), i32([0, m]), table, lens, out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    want, wl = plain_tree(cache, table[0].long(), n, q, seen, hq // hkv)
    # rounding to bf16 keeps the order, so a result within delta of the right one rounds to a
    # number between the ends' (a mean over results says less: they lie so near to 2 that bf16
    # rounds them all the same way)
    delta = 2.0 ** -12 + 2.0 ** -14
    assert (want > 1.0).all()
    low, high = (want * (1 - delta)).to(torch.bfloat16), (want * (1 + delta)).to(torch.bfloat16)
    assert ((out >= low) & (out <= high)).all()
    assert float((lse.double() - wl).abs().max()) <= 1e-5


def test_pages_shared_between_sequences():
    """Two drafts over one context: the page tables share its pages."""
    n, m = 160 + 12, 12
    s = Batch([n, 12], 8, 2, "int8", seed=42, extra_pages=10)
    s.table[1, :10] = s.table[0, :10]
    s.table[1, 10] = s.num_pages - 1
    s.lens[1] = n
    rows = s.rows(m), s.rows(m)
    O.write(s.cache, *rows, s.table[1], 160)
    q = bf16(s.rng.standard_normal((2 * m, 8, D)))
    parents = [R.tree(s.rng, m), R.tree(s.rng, m)]
    out, lse = run_tree(s, q, parents, [m, m])
    check_tree(s, q, parents, [m, m], out, lse)


def test_tree_of_another_softmax_scale():
    s = Batch([333], 8, 2, "e4m3", seed=43)
    q = bf16(s.rng.standard_normal((9, 8, D)))
    parents = [R.tree(s.rng, 9)]
    out, lse = run_tree(s, q, parents, [9], sm_scale=0.02)
    check_tree(s, q, parents, [9], out, lse, sm_scale=float(np.float32(0.02)))


# ---------------------------------------------------------------------- kept branches

def random_branch(rng, m, a):
    return sorted(rng.choice(m, a, replace=False).tolist())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hkv,lens,new,kept", [
    (1, [1], [1], [1]), (1, [1], [1], [0]), (8, [137], [25], [5]), (2, [16, 17, 32], [16, 1, 16], [3, 1, 16]),
    (3, [300, 40, 64, 7], [60, 40, 33, 0], [9, 33, 17, 0]), (8, [500], [300], [200]),
    (1, [90] * 200, [20] * 200, [4] * 200), (2, [1000], [1000], [77]),
])
def test_keep(fmt, hkv, lens, new, kept):
    s = Batch(lens, hkv, hkv, fmt, seed=50 + len(lens), extra_pages=1)
    d, cache, err = s.dims(), s.gpu_cache(), err_word()
    most = max(kept)
    idx = np.full((len(lens), most), 12345, dtype=np.int32)  # behind the kept ones: anything
    for b, (m, a) in enumerate(zip(new, kept)):
        idx[b, :a] = random_branch(s.rng, m, a)
    new_lens = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    hsa.hsa_kv8_keep(d, cache, i32(idx), i32(kept), cu_of(new), s.gpu_table(), s.gpu_lens(),
                     new_lens, err)
    want = [R.keep(s.cache, s.table[b], n, m, idx[b, :a])
            for b, (n, m, a) in enumerate(zip(lens, new, kept))]
    assert hsa.hsa_read_device_error(err) == 0
    assert new_lens.tolist() == want
    assert_same_cache(cache, s.cache)


@pytest.mark.parametrize("fmt", FORMATS)
def test_keeping_what_lies_in_place_changes_nothing_within_a_block(fmt):
    """The first nodes, all in the block of older tokens: codes and scales stay bit for bit."""
    s = Batch([30], 2, 2, fmt, seed=60)
    d, cache = s.dims(), s.gpu_cache()
    hsa.hsa_kv8_keep(d, cache, i32([list(range(10))]), i32([10]), cu_of([12]), s.gpu_table(),
                     s.gpu_lens())
    assert_same_cache(cache, s.cache)


def test_keep_of_unlike_and_zero_blocks():
    """Values move between blocks whose scales differ by 2^60; blocks of zeros keep scale 0."""
    for fmt in FORMATS:
        s = Batch([120], 1, 1, fmt, seed=61, fill=False)
        k, v = s.rows(120), s.rows(120)
        block = np.arange(120) // PAGE
        k[block % 2 == 0] *= np.float32(2.0 ** -60)
        v[block % 3 == 1] = 0
        O.write(s.cache, k, v, s.table[0], 0)
        cache, idx = s.gpu_cache(), list(range(0, 90, 3))
        hsa.hsa_kv8_keep(s.dims(), cache, i32([idx]), i32([30]), cu_of([90]), s.gpu_table(),
                         s.gpu_lens())
        R.keep(s.cache, s.table[0], 120, 90, idx)
        assert_same_cache(cache, s.cache)


def test_keep_reports_what_does_not_fit():
    """Indices out of order or range, too many, bad pages and lengths: the sequence stays as it
    was, the others move."""
    lens, new = [70, 90, 100], [20, 30, 40]
    good = [[1, 5], [0, 3, 29], [2, 39]]

    def call(b, idx=None, n=None, length=None, page=None):
        s = Batch(lens, 2, 2, "int8", seed=62)
        d, cache, err = s.dims(), s.gpu_cache(), err_word()
        flat = np.full((3, 4), -1, dtype=np.int32)
        for i, g in enumerate(good):
            flat[i, :len(g)] = g
        count = [len(g) for g in good]
        if idx is not None:
            flat[b, :len(idx)] = idx
            count[b] = len(idx)
        if n is not None:
            count[b] = n
        table = s.gpu_table()
        now = list(lens)
        if length is not None:
            now[b] = length
        if page is not None:
            table[b, page] = -1
        out = torch.full((3,), -9, dtype=torch.int32, device="cuda")
        hsa.hsa_kv8_keep(d, cache, i32(flat), i32(count), cu_of(new), table, i32(now), out, err)
        assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
        want = [now[i] if i == b else R.keep(s.cache, s.table[i], lens[i], new[i], good[i])
                for i in range(3)]
        assert out.tolist() == want
        assert_same_cache(cache, s.cache)

    call(0, idx=[5, 1])
    call(1, idx=[3, 3])
    call(1, idx=[-1, 3])
    call(2, idx=[2, 40])
    call(0, idx=[0, 1 << 30])
    call(0, n=5)  # longer than the row of indices
    call(1, n=-1)
    call(2, n=1 << 30)
    call(0, length=19)
    call(1, length=-(1 << 31))
    call(2, length=1 << 30)
    call(0, page=3)  # receives tokens
    call(2, page=6)  # only read from


# -------------------------------------------------------------------------- all together

@pytest.mark.parametrize("fmt", FORMATS)
def test_a_loop_of_drafted_tokens(fmt):
    """Prompts written with positions; then rounds of: a tree drafted behind each sequence, written
    at depths, attended, a branch kept; at the end a plain decode over what was kept. Every step
    against the oracle. The cache of a step is the GPU's own (its codes are checked bit for bit)."""
    hq, hkv, dim, B = 8, 2, 64, 3
    lens = [50, 17, 128]
    s = Batch([n + 120 for n in lens], hq, hkv, fmt, seed=70, fill=False)
    rng, t = s.rng, angle_table(400, 64)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    d, cache, table = s.dims(), s.gpu_cache(), s.gpu_table()
    ws, err = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL), err_word()
    lens_dev = i32(lens)

    def write(new, positions):
        q, k, v = (bf16(rng.standard_normal((sum(new), h, D))) for h in (hq, hkv, hkv))
        out = torch.empty(sum(new), hq, D, dtype=torch.bfloat16, device="cuda")
        hsa.hsa_kv8_write_rotated(d, cache, rot, to_bf16(q), out, to_bf16(k), to_bf16(v),
                                  None if positions is None else i32(positions), cu_of(new), table,
                                  lens_dev, err)
        oracle_write(s, lens, new, k, v, t, positions, False)
        assert_same_cache(cache, s.cache)
        return out

    write(lens, None)
    for new in ([9, 25, 1], [33, 0, 12], [2, 7, 16], [16, 16, 16]):
        parents = [R.tree(rng, m) for m in new]
        pos = np.concatenate([n + R.depths(p) for n, p in zip(lens, parents) if p])
        lens = [n + m for n, m in zip(lens, new)]
        lens_dev = i32(lens)
        q = write(new, pos)
        out = torch.empty_like(q)
        lse = torch.empty(sum(new), hq, device="cuda")
        hsa.hsa_kv8_tree(d, cache, q, i32([p for u in parents for p in u]), cu_of(new), table,
                         lens_dev, out, lse, ws)
        check_tree(s, q.float().cpu().numpy(), parents, new, out.float().cpu().numpy(),
                   lse.cpu().numpy(), lens=lens)
        # the branch that ends in a random node
        idx = np.full((B, max(new)), -1, dtype=np.int32)
        kept = []
        for b, u in enumerate(parents):
            path = np.flatnonzero(R.branches(u)[rng.integers(len(u))]) if u else []
            idx[b, :len(path)] = path
            kept.append(len(path))
        after = torch.empty(B, dtype=torch.int32, device="cuda")
        hsa.hsa_kv8_keep(d, cache, i32(idx), i32(kept), cu_of(new), table, lens_dev, after, err)
        lens = [R.keep(s.cache, s.table[b], lens[b], new[b], idx[b, :kept[b]]) for b in range(B)]
        assert after.tolist() == lens
        assert_same_cache(cache, s.cache)
        lens_dev = after
    q = bf16(rng.standard_normal((B, hq, D)))
    out, lse = torch.empty(B, hq, D, device="cuda"), torch.empty(B, hq, device="cuda")
    hsa.hsa_kv8_decode(d, cache, to_bf16(q), table, lens_dev, out, lse, ws)
    for b in range(B):
        for j in range(hq):
            k, v = (O.values(s.cache, w, s.table[b], lens[b], j // (hq // hkv)) for w in "kv")
            want, wl, tol = O.attend(q[b, j:j + 1], k, v, np.ones((1, lens[b]), bool), D ** -0.5)
            assert_rows(out[b, j:j + 1].cpu(), lse[b, j:j + 1].cpu(), want, wl, tol)
    assert hsa.hsa_read_device_error(ws) == 0 and hsa.hsa_read_device_error(err) == 0


class Step:
    """A verification step's arrays: write with positions, attend the trees, keep a branch."""

    def __init__(self, seed, lens, new, hq=8, hkv=2, fmt="int8"):
        s = Batch([n + m for n, m in zip(lens, new)], hq, hkv, fmt, seed=seed)
        T, self.d, self.cache, self.table = sum(new), s.dims(), s.gpu_cache(), s.gpu_table()
        self.rot = hsa.Rotary(torch.from_numpy(angle_table(2048, D)).cuda())
        self.x = [to_bf16(bf16(s.rng.standard_normal((T, h, D)))) for h in (hq, hkv, hkv)]
        trees = [R.tree(s.rng, m) for m in new]
        self.up = i32([p for t in trees for p in t])
        self.at = i32(np.concatenate([n + R.depths(t) for n, t in zip(lens, trees) if t]))
        paths = [np.flatnonzero(R.branches(t)[-1]) if t else [] for t in trees]
        idx = np.full((len(lens), max(map(len, paths))), -1, dtype=np.int32)
        for b, path in enumerate(paths):
            idx[b, :len(path)] = path
        self.idx, self.kept, self.cu = i32(idx), i32([len(path) for path in paths]), cu_of(new)
        self.lens = s.gpu_lens()
        self.ws = hsa.workspace(self.d, hsa.HSA_OP_KV8_PREFILL)
        self.q, self.out = (torch.zeros(T, hq, D, dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.lse = torch.zeros(T, hq, device="cuda")
        self.after = torch.zeros(len(lens), dtype=torch.int32, device="cuda")

    def run(self):
        hsa.hsa_kv8_write_rotated(self.d, self.cache, self.rot, self.x[0], self.q, self.x[1],
                                  self.x[2], self.at, self.cu, self.table, self.lens, self.ws)
        hsa.hsa_kv8_tree(self.d, self.cache, self.q, self.up, self.cu, self.table, self.lens,
                         self.out, self.lse, self.ws)
        hsa.hsa_kv8_keep(self.d, self.cache, self.idx, self.kept, self.cu, self.table, self.lens,
                         self.after, self.ws)

    def state(self):
        c = self.cache
        return [t.clone().view(torch.uint8) for t in
                (self.q, self.out, self.lse, self.after, c.k, c.v, c.k_scale, c.v_scale)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_verification_steps_at_once():
    """Two batches on two streams, each with its workspace: the bits of one after the other."""
    make = [lambda: Step(90, [700, 33, 1500], [25, 7, 60]),
            lambda: Step(91, [260] * 40, [9] * 40, hq=16, hkv=8, fmt="e4m3")]
    want = []
    for m in make:
        s = m()
        for _ in range(6):
            s.run()
        torch.cuda.synchronize()
        want.append(s.state())
    steps, streams = [m() for m in make], [torch.cuda.Stream() for _ in make]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert hsa.hsa_read_device_error(s.ws) == 0
        assert same(s.state(), w)


def test_a_captured_verification_step():
    """A step captured once and replayed over new tokens, trees, lengths and kept branches; between
    the replays another graph's prompt attention uses the same workspace."""
    lens, new = [300, 64, 1000, 17], [20, 0, 64, 5]
    s = Step(92, lens, new)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    prompt = torch.zeros_like(s.out)
    with torch.cuda.graph(graph):
        s.run()
    with torch.cuda.graph(other):
        hsa.hsa_kv8_prefill(s.d, s.cache, s.x[0], s.cu, s.table, s.lens, prompt, None, s.ws)
    for seed, now, m in ((93, [310, 60, 1000, 5], [3, 4, 70, 12]), (94, lens, new),
                         (95, [1, 50, 31, 20], [89, 0, 0, 0])):
        e = Step(seed, now, m)  # run as it is, in memory of its own
        for mine, its in zip(s.x + [s.up, s.at, s.cu, s.lens, s.kept],
                             e.x + [e.up, e.at, e.cu, e.lens, e.kept]):
            mine.copy_(its)
        # (branches as long as the captured step's rows of indices)
        s.idx.fill_(-1)
        short = min(s.idx.shape[1], e.idx.shape[1])
        s.idx[:, :short] = e.idx[:, :short]
        e.kept.clamp_(max=short)
        s.kept.copy_(e.kept)
        e.d, e.table, held = s.d, s.table, s.state()[4:]
        e.cache = hsa.KV8(s.cache.k.clone(), s.cache.v.clone(), s.cache.k_scale.clone(),
                          s.cache.v_scale.clone())
        e.run()
        want = torch.zeros_like(prompt)
        hsa.hsa_kv8_prefill(e.d, e.cache, e.x[0], e.cu, e.table, e.lens, want, None, e.ws)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert hsa.hsa_read_device_error(s.ws) == 0 and hsa.hsa_read_device_error(e.ws) == 0
        assert same(s.state(), e.state()) and torch.equal(prompt, want)
        assert not same(s.state()[4:], held)


def test_rotated_rows_go_into_the_bf16_cache():
    """hsa_rotate in front of the bf16 path: the append stores the turned key."""
    lens, hq, hkv = [100, 33], 8, 2
    rng, t = np.random.default_rng(80), angle_table(128, 128)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    d = hsa.Dims(batch=2, hq=hq, hkv=hkv, max_pages_per_seq=7, num_pages=14)
    x = [to_bf16(bf16(rng.standard_normal((2, h, D)))) for h in (hq, hkv, hkv)]
    q, k, v = (y.clone() for y in x)
    hsa.hsa_rotate(d, rot, q, q, k, k, None, None, i32(lens))
    at = t[np.array(lens) - 1]
    for got, y in ((q, x[0]), (k, x[1])):
        np.testing.assert_array_equal(
            bits(got), to_bf16_bits(R.turn(y.float().cpu().numpy(), at, False)))
    caches = [torch.zeros(14, hkv, PAGE, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kq = torch.zeros(14, hkv, PAGE, D, dtype=torch.int8, device="cuda")
    table = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7)
    hsa.hsa_append_kv(d, k, v, *caches, kq, torch.ones(2, hkv, D, device="cuda"), table, i32(lens))
    for b, n in enumerate(lens):
        page, slot = int(table[b, (n - 1) // PAGE]), (n - 1) % PAGE
        assert torch.equal(caches[0][page, :, slot], k[b])
        assert torch.equal(caches[1][page, :, slot], v[b])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("front,n,before", [(1, 1, 0), (3, 25, 5), (16, 16, 16), (40, 100, 7), (37, 0, 20)])
def test_one_sequence_behind_rows_of_none(fmt, front, n, before):
    """A single sequence's offsets may begin behind rows of no sequence, and rows may lie behind it:
    the calls that find a row's or a block's sequence leave both as they are."""
    hq, hkv, dim, behind = 8, 2, 128, 9
    s = Batch([before + n], hq, hkv, fmt, seed=front, fill=False)
    held = s.rows(before), s.rows(before)
    if before:
        O.write(s.cache, *held, s.table[0], 0)
    total = front + n + behind
    q = bf16(s.rng.standard_normal((total, hq, D)))
    k, v = (bf16(s.rng.standard_normal((total, hkv, D))) for _ in "kv")
    t = angle_table(before + n + 1, dim)
    rot = hsa.Rotary(torch.from_numpy(t).cuda(), False)
    d, caches, err = s.dims(), [s.gpu_cache(), s.gpu_cache()], err_word()
    cu, table, lens = i32([front, front + n]), s.gpu_table(), s.gpu_lens()
    mine = slice(front, front + n)
    at = t[np.arange(before, before + n)]
    plain = {name: c.copy() if isinstance(c, np.ndarray) else c for name, c in s.cache.items()}
    if n:
        O.write(plain, k[mine], v[mine], s.table[0], before)
        O.write(s.cache, R.turn(k[mine], at, False), v[mine], s.table[0], before)
    gq, gk, gv = to_bf16(q), to_bf16(k), to_bf16(v)
    hsa.hsa_kv8_write(d, caches[0], gk, gv, cu, table, lens, err)
    assert_same_cache(caches[0], plain)
    out = torch.full_like(gq, 9.0)
    hsa.hsa_kv8_write_rotated(d, caches[1], rot, gq, out, gk, gv, None, cu, table, lens, err)
    assert_same_cache(caches[1], s.cache)
    turned = torch.full_like(gq, 9.0), torch.full_like(gk, 9.0)
    hsa.hsa_rotate(d, rot, gq, turned[0], gk, turned[1], None, cu, lens, err)
    for got, x in ((out, q), (turned[0], q), (turned[1], k)):
        np.testing.assert_array_equal(bits(got[mine]), to_bf16_bits(R.turn(x[mine], at, False)))
        assert (got[:front] == 9.0).all() and (got[front + n:] == 9.0).all()
    back = torch.full_like(gk, 9.0), torch.full_like(gv, 9.0)
    hsa.hsa_kv8_read(d, caches[0], *back, cu, table, lens, err)
    for got, which in zip(back, "kv"):
        want = np.stack([O.values(plain, which, s.table[0], before + n, h) for h in range(hkv)], 1)
        np.testing.assert_array_equal(bits(got[mine]), to_bf16_bits(want[before:]))
        assert (got[:front] == 9.0).all() and (got[front + n:] == 9.0).all()
    assert hsa.hsa_read_device_error(err) == 0


@pytest.mark.parametrize("given", ("stream", "handle"))
def test_a_table_made_on_another_stream(given):
    """Memory that the current stream gave back while its work on it was still to come does not
    become the other stream's table."""
    rows, dim = 5000, 128
    want = hsa.hsa_rotary_table(rows, dim)
    other = torch.cuda.Stream()
    torch.cuda._sleep(1)
    held = torch.empty(rows, dim, device="cuda").fill_(1.0)  # (every kernel is loaded)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    held.fill_(7.0)
    del held
    table = hsa.hsa_rotary_table(rows, dim, stream=other if given == "stream" else other.cuda_stream)
    other.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(table, want)
    zero = hsa.hsa_rotary_table(rows, dim, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(zero, want)


def sawtooth_context(d, n, fp8, far, period):
    """A cache of n tokens whose scores (under a query of 31 in channel 0) rise by 8.2 over every
    `period` tokens, values of mean 2; `far`: one block in a period with values 2^-60 of that."""
    g = torch.Generator(device="cuda").manual_seed(17)
    cache = hsa.KV8.zeros(d, fp8)
    table = torch.randperm(d.num_pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    t = torch.arange(n, device="cuda")
    k = torch.randn(n, d.hkv, D, generator=g, device="cuda")
    k[:, :, 0] = (t % period / period * 3.0)[:, None]
    k = k.to(torch.bfloat16)
    v = (torch.randn(n, d.hkv, D, generator=g, device="cuda") + 2.0).to(torch.bfloat16)
    if far:
        v[t // PAGE % (period // PAGE) == 7] *= 2.0 ** -60
    hsa.hsa_kv8_write(d, cache, k, v, i32([0, n]), table, i32([n]))
    return cache, table, g


@pytest.mark.parametrize("fp8", (False, True))
@pytest.mark.parametrize("far", (False, True))
@pytest.mark.parametrize("hq,hkv,n,m", [(64, 8, 700001, 16), (64, 64, 200003, 20), (64, 16, 640007, 11)])
def test_stretches_longer_than_the_products_add_up(fp8, far, hq, hkv, n, m):
    """A CTA has more tiles of a row block in one stretch than its products add up by themselves
    (256 with two streams of rows, 512 with one), so it takes them in pieces that follow one
    another. The scores' sawtooth is a little longer than a stretch: its top, which a stretch's
    maximum follows by the lag, is in the first piece of some stretches and in the second of
    others. far: the second form of the step in the pieces that have such a block.

    Tolerances as for long contexts, products at their limit (2048 of them round to zero, 2^-23
    each: 2^-12); the weights' fp16 rounding is a random sum over 1e4 weights or more (a sixth of
    a sawtooth is within e of its top; logits of variance 1): 2^-11 / 1e2, 5e-6. lse: logits of
    magnitudes up to 40 in 8 products that round to zero, 4e-5, and sums of 2e-5."""
    group = hq // hkv
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    tiles, limit = -(-n // 128), 256 if group * m > 64 else 512
    assert tiles * hkv > 1.02 * limit * min(ctas, 256)  # (row blocks beside their tiles: 1 %)
    pages = -(-n // PAGE)
    d = hsa.Dims(batch=1, hq=hq, hkv=hkv, max_pages_per_seq=pages, num_pages=pages)
    cache, table, g = sawtooth_context(d, n, fp8, far, (limit + 45) * 128)
    q = torch.randn(m, hq, D, generator=g, device="cuda")
    q[..., 0] = 31.0
    q = q.to(torch.bfloat16)
    parents = R.tree(np.random.default_rng(18), m)
    seen = torch.from_numpy(R.seen(n, parents)).cuda()
    out = torch.empty(m, hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(m, hq, device="cuda")
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)
    hsa.hsa_kv8_tree(d, cache, q, i32(parents), i32([0, m]), table, i32([n]), out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    want, wl = plain_tree(cache, table[0].long(), n, q, seen, group)
    delta = 2.0 ** -12 + 2.0 ** -14
    assert (want > 1.0).all()
    low, high = (want * (1 - delta)).to(torch.bfloat16), (want * (1 + delta)).to(torch.bfloat16)
    assert ((out >= low) & (out <= high)).all()
    assert float((lse.double() - wl).abs().max()) <= 1e-4
    again = torch.empty_like(out)
    hsa.hsa_kv8_tree(d, cache, q, i32(parents), i32([0, m]), table, i32([n]), again, lse, ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("fp8", (False, True))
@pytest.mark.parametrize("low,high", [(20.0, 33.0), (33.0, 33.8)])
def test_weights_far_below_the_largest(fp8, low, high):
    """One token takes nearly everything, and its value is 0: the result is what the others, 2^-low
    to 2^-high of it, leave. (19 sequences of 8 heads over one context: a row block for each CTA
    of 152, so no part has a maximum of its own.)

    P is off by 2^-11 of itself or 2^-32 of the row's largest weight times scale: n times that, times
    the codes, is n 2^-32 of the largest value. Of the tail's sum: the products' rounding to zero
    2^-12, scores of 33 (log2) in three roundings of 2^-24 and ex2's 2^-22, 2^-17 together. Of the
    sum of weights: a lane adds one number a step of 128 tokens, each rounded by 2^-24. The result
    to bf16, 2^-8."""
    n, batch, hq, hkv = 65536, 19, 32, 8
    pages = n // PAGE
    d = hsa.Dims(batch=batch, hq=hq, hkv=hkv, max_pages_per_seq=pages, num_pages=pages)
    g = torch.Generator(device="cuda").manual_seed(23)
    cache = hsa.KV8.zeros(d, fp8)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    k = torch.randn(n, hkv, D, generator=g, device="cuda")
    drop = low + (high - low) * torch.rand(n, generator=g, device="cuda")
    drop[1234] = 0.0
    k[:, :, 0] = (4.0 - 4.0 / 33.0 * drop)[:, None]
    v = torch.randn(n, hkv, D, generator=g, device="cuda") + 2.0
    v[1234] = 0.0
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    one = hsa.Dims(batch=1, hq=hq, hkv=hkv, max_pages_per_seq=pages, num_pages=pages)
    hsa.hsa_kv8_write(one, cache, k, v, i32([0, n]), table[None].contiguous(), i32([n]))
    q = torch.zeros(batch, hq, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 33.0 / 4.0 * np.log(2.0) * D ** 0.5
    out = torch.empty_like(q)
    lse = torch.empty(batch, hq, device="cuda")
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)
    hsa.hsa_kv8_tree(d, cache, q, None, i32(range(batch + 1)), table.expand(batch, -1).contiguous(),
                     i32([n] * batch), out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    seen = torch.ones(1, n, dtype=torch.bool, device="cuda")
    want, wl = plain_tree(cache, table.long(), n, q[:1], seen, hq // hkv)
    largest = float(cache.v_scale.max()) * (448.0 if fp8 else 127.0)
    page, slot = int(table[1234 // PAGE]), 1234 % PAGE
    key = (cache.k.view(torch.int8)[page, :, slot].view(cache.k.dtype).float().double() *
           cache.k_scale[page, :, None].double()).repeat_interleave(hq // hkv, 0)
    others = 1.0 - torch.exp((q[0].double() * key).sum(-1) * D ** -0.5 - wl)  # [1][hq]
    sums = n / 128 * 2.0 ** -24
    tol = (2.0 ** -8 * want.abs() + n * 2.0 ** -32 * largest +
           (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -17 + sums) * largest * others[..., None])
    assert 0.0 < float(others.min()) and float(others.max()) < 0.02
    assert ((out.double() - want).abs() <= tol).all()
    assert float((lse.double() - wl).abs().max()) <= 23 * 4 * 2.0 ** -24 + 2.0 ** -20 + sums


@pytest.mark.parametrize("fmt", FORMATS)
def test_accepted_rows_written_again_leave_no_mark(fmt):
    """The block of the context's last tokens copied before a tree is written and copied back behind
    its verification, then the accepted rows written again: the cache of the accepted tokens alone,
    bit for bit, whatever was drafted in between (nodes ten times as large)."""
    hq, hkv, dim, rng = 4, 2, 128, np.random.default_rng(90)
    lens = [50, 16, 7]
    s = Batch([n + 100 for n in lens], hq, hkv, fmt, seed=91, fill=False)
    t = angle_table(300, dim)
    rot = hsa.Rotary(torch.from_numpy(t).cuda())
    d, cache, table, err = s.dims(), s.gpu_cache(), s.gpu_table(), err_word()
    arrays = (cache.k.view(torch.int8), cache.v.view(torch.int8), cache.k_scale, cache.v_scale)

    def write(lens, new, rows, positions):
        q = torch.empty(sum(new), hq, D, dtype=torch.bfloat16, device="cuda")
        hsa.hsa_kv8_write_rotated(d, cache, rot, q, q, *(to_bf16(x) for x in rows), i32(positions),
                                  cu_of(new), table, i32(lens), err)

    def normal(n, size=1.0):
        return [bf16(size * rng.standard_normal((n, hkv, D))) for _ in "kv"]

    rows = normal(sum(lens))
    write(lens, lens, rows, places(lens, lens))
    oracle_write(s, lens, lens, *rows, t, places(lens, lens), False)
    for new in ([9, 25, 1], [33, 3, 12], [2, 7, 16]):
        pages = torch.stack([table[b, n // PAGE] for b, n in enumerate(lens) if n % PAGE]).long()
        held = [a[pages].clone() for a in arrays]
        trees = [R.tree(rng, m) for m in new]
        rows = normal(sum(new), 10.0)
        at = np.concatenate([n + R.depths(p) for n, p in zip(lens, trees)])
        write([n + m for n, m in zip(lens, new)], new, rows, at)
        for a, h in zip(arrays, held):
            a[pages] = h
        paths = [np.flatnonzero(R.branches(u)[rng.integers(len(u))]) for u in trees]
        first = np.concatenate([[0], np.cumsum(new)])
        taken = np.concatenate([first[b] + p for b, p in enumerate(paths)])
        kept = [len(p) for p in paths]
        lens = [n + m for n, m in zip(lens, kept)]
        accepted = [x[taken] for x in rows]
        write(lens, kept, accepted, at[taken])
        oracle_write(s, lens, kept, *accepted, t, at[taken], False)
        got = codes_of(cache)
        for b, n in enumerate(lens):
            page = s.table[b, np.arange(n) // PAGE]
            for name in ("k", "v"):
                np.testing.assert_array_equal(got[name][page, :, np.arange(n) % PAGE],
                                              s.cache[name][page, :, np.arange(n) % PAGE])
                np.testing.assert_array_equal(got[name + "s"][page], s.cache[name + "s"][page])
    assert hsa.hsa_read_device_error(err) == 0
