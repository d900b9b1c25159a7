"""The 8-bit K/V cache on the GPU against its numpy oracle: writes bit for bit, values read
back bit for bit, decode attention (dense and over kept blocks) within derived fp32 bounds."""
import numpy as np
import pytest
import torch

from kv8_harness import (D, PAGE, Batch, assert_rows, assert_same_cache, bf16, codes_of, to_bf16)
from kv_cache_int8_gb300 import hsa
from oracle import kv8 as O

pytestmark = pytest.mark.gpu

FORMATS = ["int8", "e4m3"]


def error_word():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def cu_of(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------- write

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hkv,before,new", [
    (1, [0], [1]), (1, [0], [16]), (2, [0], [17]), (1, [5], [3]), (8, [15, 16, 17], [1, 1, 1]),
    (2, [0, 0, 100, 31, 7], [40, 0, 33, 1, 9]), (3, [1, 250], [300, 5]), (4, [12] * 9, [4] * 9),
])
def test_write_matches_the_definition(fmt, hkv, before, new):
    lens = [a + n for a, n in zip(before, new)]
    s = Batch(lens, hkv, hkv, fmt, seed=hkv, fill=False)
    for b, a in enumerate(before):  # older tokens, of half the size: most scales will grow
        if a:
            O.write(s.cache, bf16(0.5 * s.rows(a)), bf16(0.5 * s.rows(a)), s.table[b], 0)
    cache = s.gpu_cache()
    k, v = s.rows(sum(new), True), s.rows(sum(new))
    at = 0
    for b, n in enumerate(new):
        O.write(s.cache, k[at:at + n], v[at:at + n], s.table[b], before[b])
        at += n
    err = error_word()
    hsa.hsa_kv8_write(s.dims(), cache, to_bf16(k), to_bf16(v), cu_of(new), s.gpu_table(),
                      s.gpu_lens(), err)
    assert hsa.hsa_read_device_error(err) == 0
    assert_same_cache(cache, s.cache)


@pytest.mark.parametrize("fmt", FORMATS)
def test_token_by_token_writes(fmt):
    """A decode loop's appends without offsets; rows are slices of one fused projection."""
    hkv, steps = 2, 37
    s = Batch([steps, steps + 11, steps + 16], 4, hkv, fmt, seed=5, fill=False)
    for b, a in ((1, 11), (2, 16)):
        O.write(s.cache, s.rows(a), s.rows(a), s.table[b], 0)
    cache, table = s.gpu_cache(), s.gpu_table()
    for i in range(steps):
        qkv = bf16(s.rng.standard_normal((3, 4 + 2 * hkv, D)) * (1 + i % 5))
        dev = to_bf16(qkv)
        hsa.hsa_kv8_write(s.dims(), cache, dev[:, 4:4 + hkv], dev[:, 4 + hkv:], None, table,
                          s.gpu_lens([i + 1, i + 12, i + 17]))
        for b, a in enumerate((0, 11, 16)):
            O.write(s.cache, qkv[b:b + 1, 4:4 + hkv], qkv[b:b + 1, 4 + hkv:], s.table[b], a + i)
    assert_same_cache(cache, s.cache)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_of_awkward_values(fmt):
    """Zero blocks, the smallest and largest numbers, infinities and NaN, ties between codes."""
    s = Batch([16 * 7], 1, 1, fmt, fill=False)
    x = np.zeros((16 * 7, 1, D), np.float32)
    x[16:32] = bf16(s.rng.standard_normal((16, 1, D)) * 2.0 ** -130)
    x[32:48] = bf16(s.rng.standard_normal((16, 1, D)) * 2.0 ** 120)
    x[48:64] = s.rows(16)
    x[50, 0, 3], x[51, 0, 4], x[52, 0, 5] = np.inf, -np.inf, np.nan
    x[64:80] = np.nan
    x[70, 0, 0] = np.inf
    x[80:96] = bf16(np.arange(16 * D).reshape(16, 1, D) % 255 - 127) / 2  # halves of codes
    x[80, 0, 0] = 127
    x[96:112] = bf16(np.arange(16 * D).reshape(16, 1, D) % 448)
    x[96, 0, 0] = 448
    cache = s.gpu_cache()
    O.write(s.cache, x, -x, s.table[0], 0)
    hsa.hsa_kv8_write(s.dims(), cache, to_bf16(x), to_bf16(-x), cu_of([len(x)]), s.gpu_table(),
                      s.gpu_lens())
    assert_same_cache(cache, s.cache)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rewriting_a_rejected_draft(fmt):
    """Positions written twice: the block keeps its scale, the older tokens their codes."""
    s = Batch([30], 1, 1, fmt, seed=9, fill=False)
    O.write(s.cache, s.rows(20), s.rows(20), s.table[0], 0)
    cache = s.gpu_cache()
    for scale in (3.0, 0.25):
        k, v = bf16(scale * s.rows(10)), bf16(scale * s.rows(10))
        O.write(s.cache, k, v, s.table[0], 20)
        hsa.hsa_kv8_write(s.dims(), cache, to_bf16(k), to_bf16(v), cu_of([10]), s.gpu_table(),
                          s.gpu_lens())
        assert_same_cache(cache, s.cache)


def test_quantisation_error_of_whole_blocks():
    """Half a step: int8 amax / 254, E4M3 2^-4 of the value (2^-10 of the scale when small)."""
    for fmt in FORMATS:
        s = Batch([640], 1, 1, fmt, seed=3, fill=False)
        k, v = s.rows(640, True), s.rows(640)
        cache = s.gpu_cache()
        hsa.hsa_kv8_write(s.dims(), cache, to_bf16(k), to_bf16(v), cu_of([640]), s.gpu_table(),
                          s.gpu_lens())
        got = {**codes_of(cache), "fmt": fmt}
        for name, x in (("k", k), ("v", v)):
            y = O.values(got, name, s.table[0], 640, 0).reshape(40, 16, D)
            x = x[:, 0].reshape(40, 16, D).astype(np.float64)
            scale = np.abs(x).max((1, 2), keepdims=True) / float(O.LEVELS[fmt])
            half = scale / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4,
                                                              scale * 2.0 ** -10)
            # s, 1 / s and x * inv are each rounded once: x * inv is off by up to 3 * 2^-24 of
            # itself, at most 127 * 3 * 2^-24 = 2.3e-5 steps of an int8 code (4.6e-5 of half a
            # step) and less of an E4M3 one
            assert (np.abs(y - x) <= half * (1 + 5e-5)).all()


# ----------------------------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hkv,lens,new", [
    (1, [1], [1]), (2, [100, 16, 7, 333], [100, 16, 7, 333]), (8, [50, 200], [3, 65]),
    (4, [33, 20, 64], [0, 20, 1]),
])
def test_read_returns_the_values(fmt, hkv, lens, new):
    s = Batch(lens, hkv, hkv, fmt, seed=2)
    T = sum(new)
    big = torch.full((T, 3 * hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    hsa.hsa_kv8_read(s.dims(), s.gpu_cache(), big[:, hkv:2 * hkv], big[:, 2 * hkv:], cu_of(new),
                     s.gpu_table(), s.gpu_lens())
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for h in range(hkv):
            for name, off in (("k", hkv), ("v", 2 * hkv)):
                want = O.values(s.cache, name, s.table[b], n, h)[n - m:]
                got = big[at:at + m, off + h].float().cpu().numpy()
                np.testing.assert_array_equal(got, bf16(want.astype(np.float32)))
        at += m
    assert (big[:, :hkv] == 7.0).all()  # between the rows: as it was


# ------------------------------------------------------------------------- decode attention

def run_decode(s, q, kept=None, **kw):
    d = s.dims(**kw)
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_DECODE)
    out = torch.full((len(s.lens), s.hq, D), float("nan"), device="cuda")
    lse = torch.full((len(s.lens), s.hq), float("nan"), device="cuda")
    args = (d, s.gpu_cache(), to_bf16(q), s.gpu_table(), s.gpu_lens())
    if kept is None:
        hsa.hsa_kv8_decode(*args, out, lse, ws)
    else:
        hsa.hsa_kv8_attend(*args, *kept, out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    assert int(ws[256:256 + 4 * 768].sum()) == 0  # counters left at zero
    return out.cpu().numpy(), lse.cpu().numpy()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,lens", [
    (1, 1, [1]), (4, 1, [16]), (8, 1, [17, 1000]), (3, 3, [15, 130, 2]), (10, 2, [257]),
    (14, 2, [600, 0, 31]), (32, 8, [4096]), (24, 4, [0, 0]), (64, 8, [129, 2000, 1, 777]),
    (8, 8, [300] * 40),
])
def test_dense_decode(fmt, hq, hkv, lens):
    s = Batch(lens, hq, hkv, fmt, seed=hq, extra_pages=2)
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    out, lse = run_decode(s, q)
    g = hq // hkv
    for b, n in enumerate(lens):
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            want, wl, tol = O.attend(q[b, rows], k, v, np.ones((g, n), bool), D ** -0.5)
            assert_rows(out[b, rows], lse[b, rows], want, wl, tol)


@pytest.mark.parametrize("hq,hkv,lens", [
    (4, 1, [1 + i % 20 for i in range(300)]),            # a warp a row
    (6, 2, [10 + (i * 13) % 330 for i in range(170)]),   # four warps a row
    (2, 1, [17] * 160 + [6000, 0, 3]),                   # a CTA for them all, the long row cut
])
@pytest.mark.parametrize("kept", [False, True])
def test_decode_of_more_rows_than_ctas(hq, hkv, lens, kept):
    s = Batch(lens, hq, hkv, "e4m3", seed=hq)
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    args, kw = None, {}
    if kept:
        idx = np.tile(np.array([0, 1, 5], np.int32), (len(lens), hkv, 1))
        cnt = np.full((len(lens), hkv), 3, np.int32)
        args, kw = (torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()), dict(
            sink=3, window=9, k2=3)
    out, lse = run_decode(s, q, args, **kw)
    g = hq // hkv
    for b in list(range(0, len(lens), 17)) + [len(lens) - 3, len(lens) - 2, len(lens) - 1]:
        n = lens[b]
        t = np.arange(n)
        seen = np.ones(n, bool)
        if kept:
            seen = (t < 3) | (t >= n - 9) | np.isin(t // PAGE, [0, 1, 5])
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            want, wl, tol = O.attend(q[b, rows], k, v, np.tile(seen, (g, 1)), D ** -0.5)
            assert_rows(out[b, rows], lse[b, rows], want, wl, tol)


def test_dense_decode_of_extreme_queries_and_scale():
    """Queries from 2^-40 to 2^30 in one group (the fp16 operands carry a power of two a head),
    zero queries, a given softmax scale, logits far apart."""
    s = Batch([500, 37], 8, 1, "int8", seed=4)
    q = bf16(s.rng.standard_normal((2, 8, D)))
    q *= (2.0 ** np.array([-40, -20, -3, 0, 2, 4, -100, 0], np.float32))[:, None]
    q[:, 7] = 0
    q[1, 4] *= np.float32(2.0 ** 26)  # one token takes everything
    out, lse = run_decode(s, q, sm_scale=0.25)
    for b, n in enumerate(s.lens):
        k, v = (O.values(s.cache, w, s.table[b], n, 0) for w in "kv")
        want, wl, tol = O.attend(q[b], k, v, np.ones((8, n), bool), 0.25)
        assert_rows(out[b], lse[b], want, wl, tol)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("per_head", [0, 1])
@pytest.mark.parametrize("sink,window,k2,lens", [
    (0, 0, 4, [200, 64]), (4, 1, 8, [1000, 3, 5]), (20, 40, 0, [50, 61, 300]),
    (64, 256, 16, [2048, 319, 0, 321]), (16, 37, 200, [5000]), (0, 0, 0, [90]),
])
def test_attend_over_kept_blocks(fmt, per_head, sink, window, k2, lens):
    hq, hkv = 8, 2
    g, rows = hq // hkv, hq if per_head else hkv
    s = Batch(lens, hq, hkv, fmt, seed=k2 + 1)
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    idx = np.full((len(lens), rows, max(k2, 1)), -1, np.int32)
    cnt = np.zeros((len(lens), rows), np.int32)
    for b, n in enumerate(lens):
        for r in range(rows):
            m = min(k2, s.rng.integers(0, k2 + 1), -(-n // PAGE))
            # any blocks, those of the sink and the window too: they are clipped
            idx[b, r, :m] = np.sort(s.rng.permutation(-(-n // PAGE))[:m])
            cnt[b, r] = m
    out, lse = run_decode(s, q, (torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()),
                          sink=sink, window=window, k2=k2, per_head=per_head)
    for b, n in enumerate(lens):
        t = np.arange(n)
        for j in range(hq):
            h, r = j // g, j if per_head else j // g
            near = (t < sink) | (t >= n - window)
            far = np.isin(t // PAGE, idx[b, r, :cnt[b, r]]) & (t >= sink) & (t < n - window)
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            want, wl, tol = O.attend(q[b, j:j + 1], k, v, (near | far)[None], D ** -0.5)
            assert_rows(out[b, j:j + 1], lse[b, j:j + 1], want, wl, tol)


def test_selection_ids_outside_the_context_add_nothing():
    s = Batch([100], 2, 1, "int8", seed=6)
    q = bf16(s.rng.standard_normal((1, 2, D)))
    idx = torch.tensor([[[-5, 2, 6, 1 << 27, 40]]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[9]], dtype=torch.int32, device="cuda")  # more than k2
    out, lse = run_decode(s, q, (idx, cnt), sink=8, window=4, k2=5)
    t = np.arange(100)
    seen = (t < 8) | (t >= 96) | (t // PAGE == 2) | ((t // PAGE == 6) & (t < 96))
    k, v = (O.values(s.cache, w, s.table[0], 100, 0) for w in "kv")
    want, wl, tol = O.attend(q[0], k, v, np.tile(seen, (2, 1)), D ** -0.5)
    assert_rows(out[0], lse[0], want, wl, tol)


def test_decode_is_the_same_every_time_and_from_a_graph():
    """Bit-equal results call after call, on another stream, and replayed with new lengths."""
    s = Batch([3000, 17, 900], 16, 4, "e4m3", seed=8)
    q = to_bf16(s.rng.standard_normal((3, 16, D)))
    d, cache, table, lens = s.dims(), s.gpu_cache(), s.gpu_table(), s.gpu_lens()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_DECODE)
    outs = [torch.empty(3, 16, D, device="cuda") for _ in range(4)]
    for o in outs[:2]:
        hsa.hsa_kv8_decode(d, cache, q, table, lens, o, None, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        hsa.hsa_kv8_decode(d, cache, q, table, lens, outs[2], None, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hsa.hsa_kv8_decode(d, cache, q, table, lens, outs[3], None, ws)
    lens.copy_(torch.tensor([5, 1, 2], device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    short = outs[3].clone()
    lens.copy_(s.gpu_lens())
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert not torch.equal(short, outs[0])


# -------------------------------------------------------------------------- bad page tables

def test_bad_pages_and_lengths_are_reported_not_followed():
    s = Batch([40, 64, 50], 2, 1, "int8", seed=1)
    table = s.gpu_table()
    table[0, 1] = s.num_pages          # one past the pool
    lens = s.gpu_lens([40, 64, 16 * s.max_pages + 1])  # longer than its page-table row
    d, cache = s.dims(), s.gpu_cache()
    before = codes_of(cache)
    k = to_bf16(s.rows(40 + 64 + 4))
    cu = cu_of([40, 64, 4])
    err = error_word()
    hsa.hsa_kv8_write(d, cache, k, k, cu, table, lens, err)
    assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
    after = codes_of(cache)
    untouched = np.setdiff1d(np.arange(s.num_pages), np.r_[s.table[0, [0, 2]], s.table[1]])
    np.testing.assert_array_equal(after["k"][untouched], before["k"][untouched])
    outs = torch.full((108, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    hsa.hsa_kv8_read(d, cache, outs, outs.clone(), cu, table, lens, err)
    assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
    assert (outs[16:32] == 3.0).all() and (outs[104:] == 3.0).all()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_DECODE)
    out, lse = torch.empty(3, 2, D, device="cuda"), torch.empty(3, 2, device="cuda")
    q = to_bf16(s.rng.standard_normal((3, 2, D)))
    hsa.hsa_kv8_decode(d, cache, q, table, lens, out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK
    assert torch.isfinite(out).all() and (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    # rows that do not fit the arrays
    for bad in ([0, 40, 104, 200], [0, -3, 104, 108], [0, 40, 30, 108]):
        hsa.hsa_kv8_write(d, cache, k, k, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                          s.gpu_table(), s.gpu_lens(), err)
        assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK


# ------------------------------------------------------------------------ prompt attention

def run_prefill(s, q, new, **kw):
    d = s.dims(**kw)
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    T = sum(new)
    rows = to_bf16(q)
    out = torch.full((T, s.hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, s.hq), float("nan"), device="cuda")
    hsa.hsa_kv8_prefill(d, s.gpu_cache(), rows, cu_of(new), s.gpu_table(), s.gpu_lens(), out, lse,
                        ws)
    assert hsa.hsa_read_device_error(ws) == 0
    assert int(ws[256:256 + 4 * 768].sum()) == 0  # counters left at zero
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check_prefill(s, q, new, out, lse, sm_scale=D ** -0.5):
    g = s.hq // s.hkv
    at = 0
    for b, (n, m) in enumerate(zip(s.lens, new)):
        for h in range(s.hkv):
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            seen = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
            for j in range(h * g, (h + 1) * g):
                want, wl, tol = O.attend(q[at:at + m, j], k, v, seen, sm_scale)
                # probabilities are rounded to fp16 before the product with V (half a step
                # 2^-11 of each, so that much of the largest value), the result to bf16
                tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(v).max()
                assert_rows(out[at:at + m, j], None if lse is None else lse[at:at + m, j], want, wl,
                            tol, 2.0 ** -8)
        at += m


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,lens,new", [
    (1, 1, [1], [1]), (4, 1, [64], [64]), (8, 1, [128, 129], [128, 1]), (8, 8, [200], [200]),
    (4, 1, [300], [300]), (3, 1, [500, 90], [170, 90]), (14, 2, [400], [77]),
    (16, 2, [1, 17, 260, 1000], [1, 16, 0, 130]), (32, 8, [1500], [40]),
    (64, 8, [333, 700], [1, 65]), (5, 1, [2048], [700]), (8, 2, [40] * 33, [3] * 33),
])
def test_prefill(fmt, hq, hkv, lens, new):
    s = Batch(lens, hq, hkv, fmt, seed=len(lens) + hq, extra_pages=1)
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    out, lse = run_prefill(s, q, new)
    check_prefill(s, q, new, out, lse)


def test_prefill_of_strided_queries_leaves_other_rows_alone():
    """Queries as slices of a fused projection, rows behind the last sequence, no lse; the same
    bits again on another stream and from a replayed graph."""
    hq, hkv, new = 8, 2, [70, 0, 33]
    s = Batch([600, 20, 33], hq, hkv, "int8", seed=11)
    T = sum(new)
    q = bf16(s.rng.standard_normal((T, hq, D)))
    fused = torch.full((T + 9, hq + 2 * hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:T, :hq] = to_bf16(q)
    d, cache = s.dims(), s.gpu_cache()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    outs = [torch.full((T + 9, hq, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    args = (d, cache, fused[:, :hq], cu_of(new), s.gpu_table(), s.gpu_lens())
    hsa.hsa_kv8_prefill(*args, outs[0], None, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        hsa.hsa_kv8_prefill(*args, outs[1], None, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hsa.hsa_kv8_prefill(*args, outs[2], None, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert hsa.hsa_read_device_error(ws) == 0
    for o in outs:
        assert torch.equal(o, outs[0]) and (o[T:] == 5.0).all()
    check_prefill(s, q, new, outs[0][:T].float().cpu().numpy(), None)


def test_prefill_without_offsets_is_a_decode():
    s = Batch([300, 17, 1], 4, 2, "e4m3", seed=12)
    q = bf16(s.rng.standard_normal((3, 4, D)))
    d = s.dims()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    out = torch.empty(3, 4, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 4, device="cuda")
    hsa.hsa_kv8_prefill(d, s.gpu_cache(), to_bf16(q), None, s.gpu_table(), s.gpu_lens(), out, lse,
                        ws)
    check_prefill(s, q, [1, 1, 1], out.float().cpu().numpy(), lse.cpu().numpy())


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_over_blocks_of_zeros_and_of_unlike_scales(fmt):
    """V blocks of zeros count in the sums, K blocks of zeros give equal logits; scales of V
    that differ by 2^60 between blocks, queries by 2^60 between heads."""
    s = Batch([16 * 40 + 5], 4, 1, fmt, seed=13, fill=False)
    n = s.lens[0]
    k, v = s.rows(n), s.rows(n)
    block = np.arange(n) // PAGE
    v[block % 3 == 0] = 0
    v[block % 3 == 1] *= np.float32(2.0 ** -60)
    k[block % 4 == 1] = 0
    k[block == 40] = 0
    O.write(s.cache, k, v, s.table[0], 0)
    q = bf16(s.rng.standard_normal((8, 4, D)))
    q[:, 1] *= np.float32(2.0 ** -40)
    q[:, 2] *= np.float32(2.0 ** 20)  # one token takes all
    q[:, 3] = 0
    kk, vv = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    out, lse = run_decode(s, q[:1])
    want, wl, tol = O.attend(q[0], kk, vv, np.ones((4, n), bool), D ** -0.5)
    ok = [0, 1, 3]  # at 2^20 the logits themselves are only known to a few units
    assert_rows(out[0][ok], lse[0][ok], want[ok], wl[ok], {m: t[ok] for m, t in tol.items()})
    assert np.isfinite(out).all()
    out, lse = run_prefill(s, q, [8])
    for j in ok:
        seen = np.arange(n)[None] <= (n - 8 + np.arange(8))[:, None]
        want, wl, tol = O.attend(q[:, j], kk, vv, seen, D ** -0.5)
        tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
        assert_rows(out[:, j], lse[:, j], want, wl, tol, 2.0 ** -8)


def test_long_decode_keeps_its_digits():
    """2M tokens of one row: 54 blocks add up in each of 152 x 16 warps. 2-norm error against 64
    bits below 1e-6: 54 + 16 + 152 roundings of at most 2^-24 of a running sum, as random ones
    sqrt(222) * 2^-24 = 9e-7 where the running sum is already the result."""
    n, hkv = 1 << 21, 1
    d = hsa.Dims(batch=1, hq=4, hkv=hkv, max_pages_per_seq=n // 16, num_pages=n // 16, k2=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(n, hkv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    for fp8 in (False, True):
        cache = hsa.KV8.zeros(d, fp8)
        table = torch.randperm(n // 16, generator=g, device="cuda").to(torch.int32)[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        hsa.hsa_kv8_write(d, cache, x[0], x[1], cu, table, lens)
        q = torch.randn(1, 4, D, generator=g, device="cuda").to(torch.bfloat16)
        out, lse = torch.empty(1, 4, D, device="cuda"), torch.empty(1, 4, device="cuda")
        hsa.hsa_kv8_decode(d, cache, q, table, lens, out, lse,
                           hsa.workspace(d, hsa.HSA_OP_KV8_DECODE))
        val = [(c.view(torch.int8)[table[0].long()].view(c.dtype).float().double() *
                sc[table[0].long()].double()[..., None, None]).view(n, D)
               for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        logit = q[0].double() @ val[0].T * D ** -0.5
        want = torch.softmax(logit, -1) @ val[1]
        assert float((out[0].double() - want).norm() / want.norm()) < 1e-6
        assert float((lse[0].double() - torch.logsumexp(logit, -1)).abs().max()) < 2e-6


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_serving_loop(fmt):
    """Prompts written and attended, then tokens appended one by one with dense and kept
    attention, a drafted stretch verified and taken back: all four operators on one cache."""
    hq, hkv = 8, 2
    g = hq // hkv
    prompt = [150, 33, 64]
    s = Batch([n + 24 for n in prompt], hq, hkv, fmt, seed=21, fill=False)
    d = s.dims(sink=16, window=20, k2=3)
    cache, table = s.gpu_cache(), s.gpu_table()
    wp = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    wd = wp  # one workspace for all

    def values(b, n, h):
        return [O.values(s.cache, w, s.table[b], n, h) for w in "kv"]

    def extend(lens, new):  # writes and attends `new` tokens up to `lens`
        T = sum(new)
        qkv = bf16(s.rng.standard_normal((T, hq + 2 * hkv, D)))
        dev = to_bf16(qkv)
        k, v = dev[:, hq:hq + hkv], dev[:, hq + hkv:]
        dl = s.gpu_lens(lens)
        hsa.hsa_kv8_write(d, cache, k, v, cu_of(new), table, dl)
        out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
        hsa.hsa_kv8_prefill(d, cache, dev[:, :hq], cu_of(new), table, dl, out, None, wp)
        at = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            O.write(s.cache, qkv[at:at + m, hq:hq + hkv], qkv[at:at + m, hq + hkv:], s.table[b],
                    n - m)
            for h in range(hkv):
                kk, vv = values(b, n, h)
                seen = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
                for j in range(h * g, h * g + g):
                    want, _, tol = O.attend(qkv[at:at + m, j], kk, vv, seen, D ** -0.5)
                    tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
                    assert_rows(out[at:at + m, j].float().cpu(), None, want, None, tol, 2.0 ** -8)
            at += m

    extend(prompt, prompt)
    lens = list(prompt)
    for step in range(5):
        lens = [n + 1 for n in lens]
        qkv = bf16(s.rng.standard_normal((3, hq + 2 * hkv, D)))
        dev, dl = to_bf16(qkv), s.gpu_lens(lens)
        hsa.hsa_kv8_write(d, cache, dev[:, hq:hq + hkv], dev[:, hq + hkv:], None, table, dl)
        idx = np.tile(np.array([1, 2, 4], np.int32), (3, hkv, 1))
        cnt = torch.full((3, hkv), 3, dtype=torch.int32, device="cuda")
        q = dev[:, :hq].contiguous()
        dense, kept = (torch.empty(3, hq, D, device="cuda") for _ in range(2))
        hsa.hsa_kv8_decode(d, cache, q, table, dl, dense, None, wd)
        hsa.hsa_kv8_attend(d, cache, q, table, dl, torch.from_numpy(idx).cuda(), cnt, kept, None, wd)
        for b, n in enumerate(lens):
            O.write(s.cache, qkv[b:b + 1, hq:hq + hkv], qkv[b:b + 1, hq + hkv:], s.table[b], n - 1)
            t = np.arange(n)
            seen = (t < 16) | (t >= n - 20) | np.isin(t // PAGE, [1, 2, 4])
            for h in range(hkv):
                kk, vv = values(b, n, h)
                rows = slice(h * g, h * g + g)
                for got, mask in ((dense, np.ones(n, bool)), (kept, seen)):
                    want, _, tol = O.attend(qkv[b, rows], kk, vv, np.tile(mask, (g, 1)), D ** -0.5)
                    assert_rows(got[b, rows].cpu(), None, want, None, tol)
    extend([n + 7 for n in lens], [7, 7, 7])   # a draft ...
    extend([n + 4 for n in lens], [3, 2, 4])   # ... of which a part is kept and written anew
    assert_same_cache(cache, s.cache)
    assert hsa.hsa_read_device_error(wp) == 0


def test_codes_beyond_two_gigabytes():
    """Pages whose bytes lie past 2^31 in each code array."""
    hq, hkv, lens, new = 16, 8, [70, 33], [40, 5]
    s = Batch(lens, hq, hkv, "int8", seed=14)
    shift = 140000  # pages of 16 KiB
    small, n = s.gpu_cache(), s.num_pages
    codes = [torch.zeros(shift + n, hkv, 16, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(shift + n, hkv, device="cuda") for _ in range(2)]
    for big, old in zip(codes + scales, (small.k, small.v, small.k_scale, small.v_scale)):
        big[shift:] = old
    cache = hsa.KV8(*codes, *scales)
    table = s.gpu_table()
    table += shift
    d = s.dims()
    d = hsa.Dims(**{**d.__dict__, "num_pages": shift + n})
    k, v = s.rows(sum(new)), s.rows(sum(new))
    at = 0
    for b, m in enumerate(new):
        O.write(s.cache, k[at:at + m], v[at:at + m], s.table[b], lens[b] - m)
        at += m
    hsa.hsa_kv8_write(d, cache, to_bf16(k), to_bf16(v), cu_of(new), table, s.gpu_lens())
    assert_same_cache(hsa.KV8(codes[0][shift:], codes[1][shift:], scales[0][shift:].clone(),
                              scales[1][shift:].clone()), s.cache)
    assert not codes[0][:shift].any() and not scales[1][:shift].any()
    back = torch.empty(2, sum(lens), hkv, D, dtype=torch.bfloat16, device="cuda")
    hsa.hsa_kv8_read(d, cache, back[0], back[1], cu_of(lens), table, s.gpu_lens())
    want = O.values(s.cache, "v", s.table[1], lens[1], 3)
    np.testing.assert_array_equal(back[1, lens[0]:, 3].float().cpu().numpy(), bf16(want))
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    out = torch.empty(sum(new), hq, D, dtype=torch.bfloat16, device="cuda")
    hsa.hsa_kv8_prefill(d, cache, to_bf16(q), cu_of(new), table, s.gpu_lens(), out, None,
                        hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL))
    check_prefill(s, q, new, out.float().cpu().numpy(), None)
    rows = [new[0] - 1, sum(new) - 1]
    o32, lse = torch.empty(2, hq, D, device="cuda"), torch.empty(2, hq, device="cuda")
    hsa.hsa_kv8_decode(d, cache, to_bf16(q[rows]), table, s.gpu_lens(), o32, lse,
                       hsa.workspace(d, hsa.HSA_OP_KV8_DECODE))
    for b in range(2):
        for h in range(hkv):
            kk, vv = (O.values(s.cache, w, s.table[b], lens[b], h) for w in "kv")
            r = slice(2 * h, 2 * h + 2)
            want, wl, tol = O.attend(q[rows[b], r], kk, vv, np.ones((2, lens[b]), bool), D ** -0.5)
            assert_rows(o32[b, r].cpu(), lse[b, r].cpu(), want, wl, tol)


def test_a_large_batch():
    """1024 sequences, most short, one long: every operator."""
    lens = [1 + (i * 37) % 23 for i in range(1023)] + [700]
    new = [min(n, 1 + i % 3) for i, n in enumerate(lens)]
    s = Batch(lens, 4, 2, "e4m3", seed=15)
    q = bf16(s.rng.standard_normal((len(lens), 4, D)))
    out, lse = run_decode(s, q)
    for b in (0, 1, 500, 1022, 1023):
        for h in range(2):
            kk, vv = (O.values(s.cache, w, s.table[b], lens[b], h) for w in "kv")
            r = slice(2 * h, 2 * h + 2)
            want, wl, tol = O.attend(q[b, r], kk, vv, np.ones((2, lens[b]), bool), D ** -0.5)
            assert_rows(out[b, r], lse[b, r], want, wl, tol)
    q = bf16(s.rng.standard_normal((sum(new), 4, D)))
    out, lse = run_prefill(s, q, new)
    at = np.concatenate([[0], np.cumsum(new)])
    for b in (0, 2, 777, 1023):
        n, m = lens[b], new[b]
        for h in range(2):
            kk, vv = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            seen = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
            for j in (2 * h, 2 * h + 1):
                want, wl, tol = O.attend(q[at[b]:at[b + 1], j], kk, vv, seen, D ** -0.5)
                tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
                assert_rows(out[at[b]:at[b + 1], j], lse[at[b]:at[b + 1], j], want, wl, tol,
                            2.0 ** -8)


def test_prefill_reports_what_does_not_fit():
    s = Batch([40, 64, 50], 2, 1, "int8", seed=1)
    table = s.gpu_table()
    table[0, 1] = -7
    lens = s.gpu_lens([40, 64, 3])  # the third has fewer tokens than new ones
    d = s.dims()
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    q = to_bf16(s.rng.standard_normal((24, 2, D)))
    out = torch.full((24, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((24, 2), 9.0, device="cuda")
    hsa.hsa_kv8_prefill(d, s.gpu_cache(), q, cu_of([10, 10, 4]), table, lens, out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK
    assert torch.isfinite(out).all() and (out[20:] == 0).all() and torch.isneginf(lse[20:]).all()
    check = Batch([40, 64, 50], 2, 1, "int8", seed=1)
    kk, vv = (O.values(check.cache, w, check.table[1], 64, 0) for w in "kv")
    seen = np.arange(64)[None] <= (54 + np.arange(10))[:, None]
    want, wl, tol = O.attend(q[10:20, 0].float().cpu().numpy(), kk, vv, seen, D ** -0.5)
    tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
    assert_rows(out[10:20, 0].float().cpu(), lse[10:20, 0].cpu(), want, wl, tol, 2.0 ** -8)


def test_unlimited_sink_and_window_see_everything():
    s = Batch([300, 5], 4, 2, "int8", seed=16)
    q = bf16(s.rng.standard_normal((2, 4, D)))
    dense, dense_lse = run_decode(s, q)
    none = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    idx = torch.full((2, 2, 1), -1, dtype=torch.int32, device="cuda")
    big = 2 ** 31 - 1
    for kw in (dict(sink=big), dict(window=big), dict(sink=big, window=big)):
        out, lse = run_decode(s, q, (idx, none), k2=1, **kw)
        # the same products, at most 40 sums in another order: 40 * 2^-24 * max |v| (4.5)
        np.testing.assert_allclose(out, dense, rtol=0, atol=1.1e-5)
        np.testing.assert_allclose(lse, dense_lse, rtol=0, atol=1.1e-5)


@pytest.mark.parametrize("hq,hkv,lens", [
    (4, 2, [1, 20, 5000]),                               # CTAs share rows
    (4, 1, [1 + i % 20 for i in range(300)]),            # a warp a row
    (4, 2, [10 + (i * 13) % 330 for i in range(170)]),   # four warps a row
])
def test_queries_that_are_not_finite_stay_in_their_rows(hq, hkv, lens):
    """A NaN or an infinity in a query head makes that head's results NaN, however the rows are
    shared out, and no other's."""
    s = Batch(lens, hq, hkv, "int8", seed=17)
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    q[0, 1, 7], q[2, 3, 100], q[-1, 0, 0] = np.nan, np.inf, -np.inf
    bad = ~np.isfinite(q).all(-1)
    out, lse = run_decode(s, q)
    rows, row_lse = run_prefill(s, q, [1] * len(lens))
    for o, l in ((out, lse), (rows, row_lse)):
        np.testing.assert_array_equal(np.isnan(o).any(-1), bad)
        np.testing.assert_array_equal(np.isnan(l), bad)
    g = hq // hkv
    for b in (0, 2, len(lens) - 1):
        for j in range(hq):
            if not bad[b, j]:
                k, v = (O.values(s.cache, w, s.table[b], lens[b], j // g) for w in "kv")
                want, wl, tol = O.attend(q[b, j:j + 1], k, v, np.ones((1, lens[b]), bool),
                                         D ** -0.5)
                assert_rows(out[b, j:j + 1], lse[b, j:j + 1], want, wl, tol)


@pytest.mark.parametrize("fmt", FORMATS)
def test_prefill_where_one_token_takes_everything(fmt):
    """Each query's weight lies on one token, at any place of a tile: a maximum that misses it
    would push its probability out of fp16."""
    n, m = 700, 260
    s = Batch([n], 4, 1, fmt, seed=18)
    k = O.values(s.cache, "k", s.table[0], n, 0)
    q = np.empty((m, 4, D), np.float32)
    for i in range(m):
        for j in range(4):
            q[i, j] = 40.0 * k[(37 * i + 131 * j) % (n - m + i + 1)]
    q = bf16(q)
    out, lse = run_prefill(s, q, [m])
    check_prefill(s, q, [m], out, lse)


@pytest.mark.parametrize("rise", [0.02, 0.3, 3.0])
@pytest.mark.parametrize("m", [9, 20, 150])
def test_prefill_whose_scores_grow_along_the_context(m, rise):
    """Each half of a tile raises the maximum, by up to 64 tokens x `rise` x 100 x 0.01 x 128 /
    sqrt(128): the accumulator follows it before and between the products with V."""
    n = 900
    s = Batch([n], 4, 1, "int8", seed=19, fill=False)
    u = np.sign(s.rng.standard_normal(D)).astype(np.float32)
    k = bf16(np.arange(n, dtype=np.float32)[:, None, None] * 0.01 * u)
    O.write(s.cache, k, s.rows(n), s.table[0], 0)
    q = bf16(100.0 * rise * u * s.rng.uniform(0.5, 1.0, (m, 4, 1)))
    out, lse = run_prefill(s, q, [m])
    check_prefill(s, q, [m], out, lse)


@pytest.mark.parametrize("n,m", [(1, 1), (40, 3), (700, 260), (9000, 5)])
def test_prefill_of_infinities_against_codes_of_one_sign(n, m):
    """An infinity times key codes of the other sign makes every score of a row -inf, whether the
    row sees one token or many, in a whole row block or in parts of one (9000 tokens)."""
    s = Batch([n], 4, 2, "int8", seed=23, fill=False)
    k = s.rows(n)
    k[:, :, 7] = -np.abs(k[:, :, 7]) - 1.0  # a code below zero in every token
    O.write(s.cache, k, s.rows(n), s.table[0], 0)
    q = bf16(s.rng.standard_normal((m, 4, D)))
    q[0, 0, 7], q[-1, 1, 7], q[m // 2, 3, 7] = np.inf, np.inf, np.inf
    bad = ~np.isfinite(q).all(-1)
    out, lse = run_prefill(s, q, [m])
    np.testing.assert_array_equal(np.isnan(out).all(-1), bad)
    np.testing.assert_array_equal(np.isnan(out).any(-1), bad)
    np.testing.assert_array_equal(np.isnan(lse), bad)
    for h in range(2):
        kk, vv = (O.values(s.cache, w, s.table[0], n, h) for w in "kv")
        seen = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
        for j in (2 * h, 2 * h + 1):
            ok = ~bad[:, j]
            want, wl, tol = O.attend(q[ok, j], kk, vv, seen[ok], D ** -0.5)
            tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(vv).max()
            assert_rows(out[ok, j], lse[ok, j], want, wl, tol, 2.0 ** -8)


# Magnitudes of V's blocks (powers of two, None: zeros), repeated along the sequence.
V_MAGNITUDES = {"tiny": [-115], "zero": [None], "zero, then large": [None] * 30 + [60],
                "large, then tiny": [100] * 20 + [-110], "tiny, then large": [-110] * 20 + [100],
                "all kinds": [None, -100, 0, 50, 120], "zero within": [0, 0, None]}


def unlike_batch(lens, hq, hkv, fmt, magnitudes):
    s = Batch(lens, hq, hkv, fmt, seed=len(lens), fill=False)
    for b, n in enumerate(lens):
        v = s.rows(n)
        for i in range(0, n, PAGE):
            e = magnitudes[i // PAGE % len(magnitudes)]
            v[i:i + PAGE] *= np.float32(0.0 if e is None else 2.0 ** e)
        O.write(s.cache, s.rows(n), v, s.table[b], 0)
    return s


def unlike_bounds(q, k, v, seen, tol, levels, probability, floor):
    """Bounds of an output row by what its own tokens weigh, not by the largest value: every
    weight is off by twice the oracle's relative bound and by the rounding of its fp16 form,
    `probability` of itself, and never by less than `floor` of the heaviest token's (the fp16
    form's smallest step against the least that the heaviest one is carried as)."""
    x = np.where(seen, q @ k.T * D ** -0.5, -np.inf)
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    top = np.abs(v).max() if v.any() else 1.0
    rel = tol["out"] / top  # 2 (eps + sums)
    heaviest = (p * np.abs(v).max(-1)).max(-1)  # a value is at most `levels` scales
    return ((rel + probability)[:, None] * (p @ np.abs(v)) +
            (len(k) * floor * levels * heaviest)[:, None])


@pytest.mark.parametrize("kind", list(V_MAGNITUDES))
@pytest.mark.parametrize("fmt,hq,hkv,lens", [
    ("int8", 4, 1, [1, 645, 0, 5000]),                           # CTAs share rows
    ("e4m3", 7, 1, [16, 700]), ("int8", 8, 1, [3000]),
    ("e4m3", 4, 1, [1 + i % 60 for i in range(300)]),            # a warp a row
    ("int8", 6, 2, [10 + (i * 13) % 330 for i in range(170)]),   # four warps a row
])
def test_decode_sums_where_v_is_zero_tiny_or_large(kind, fmt, hq, hkv, lens):
    """The sum of the weights has nothing to do with V: no scale of V, nor any mixture of them,
    may push it out of fp32 or lose a part of it."""
    s = unlike_batch(lens, hq, hkv, fmt, V_MAGNITUDES[kind])
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    out, lse = run_decode(s, q)
    g = hq // hkv
    for b in list(range(0, len(lens), 23)) + [len(lens) - 1]:
        n = lens[b]
        if n == 0:
            continue
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            k, v = (O.values(s.cache, w, s.table[b], n, h) for w in "kv")
            seen = np.ones((g, n), bool)
            want, wl, tol = O.attend(q[b, rows], k, v, seen, D ** -0.5)
            # fp16 in two halves: nothing but its floor, 2^-25 against at least 2^10
            bound = unlike_bounds(q[b, rows].astype(np.float64), k, v, seen, tol,
                                  float(O.LEVELS[fmt]), 0.0, 2.0 ** -35)
            assert (np.abs(lse[b, rows] - wl) <= tol["lse"]).all(), (b, h)
            assert (np.abs(out[b, rows] - want) <= bound).all(), (b, h)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_over_a_million_tokens_of_zeros(fp8):
    """An empty V (a fresh cache's): 2^20 equal weights, whose sums are whole numbers; the
    logarithm and its two scalings are off by 2^-22 of ln 2^20 at most."""
    n = 1 << 20
    d = hsa.Dims(batch=1, hq=4, hkv=1, max_pages_per_seq=n // 16, num_pages=n // 16, k2=0)
    table = torch.arange(n // 16, device="cuda", dtype=torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = torch.ones(1, 4, D, device="cuda"), torch.empty(1, 4, device="cuda")
    q = torch.ones(1, 4, D, device="cuda", dtype=torch.bfloat16)
    hsa.hsa_kv8_decode(d, hsa.KV8.zeros(d, fp8), q, table, lens, out, lse,
                       hsa.workspace(d, hsa.HSA_OP_KV8_DECODE))
    assert not out.any()
    assert float((lse.double() - np.log(n)).abs().max()) <= np.log(n) * 2.0 ** -22


@pytest.mark.parametrize("kind", list(V_MAGNITUDES))
@pytest.mark.parametrize("fmt,hq,hkv,lens,new", [
    ("int8", 4, 1, [1, 645, 5000], [1, 30, 9]),   # row blocks in parts
    ("e4m3", 4, 2, [700], [400]), ("int8", 7, 1, [900, 40], [200, 40]),
])
def test_prefill_sums_where_v_is_zero_tiny_or_large(kind, fmt, hq, hkv, lens, new):
    s = unlike_batch(lens, hq, hkv, fmt, V_MAGNITUDES[kind])
    q = bf16(s.rng.standard_normal((sum(new), hq, D)))
    out, lse = run_prefill(s, q, new)
    g, at = hq // hkv, 0
    for b, (n, m) in enumerate(zip(lens, new)):
        seen = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
        for j in range(hq):
            k, v = (O.values(s.cache, w, s.table[b], n, j // g) for w in "kv")
            qj = q[at:at + m, j].astype(np.float64)
            want, wl, tol = O.attend(qj, k, v, seen, D ** -0.5)
            # fp16: half a step 2^-11, or its floor, 2^-25 against at least 2^7
            bound = unlike_bounds(qj, k, v, seen, tol, float(O.LEVELS[fmt]), 2.0 ** -11,
                                  2.0 ** -32)
            bound += 2.0 ** -8 * (np.abs(want) + bound)  # the bf16 result
            assert (np.abs(lse[at:at + m, j] - wl) <= tol["lse"]).all(), (b, j)
            assert (np.abs(out[at:at + m, j] - want) <= bound).all(), (b, j)
        at += m


def test_prefill_over_zeros_whose_first_scores_are_lower():
    """V all zero, 16 low scores, then 28K to 32K equal ones, in row blocks that are many enough to
    be taken whole: with a reference that stays behind by its permitted 2^8, the sums must not
    leave fp32. lse against 64 bits; the logits are exact but for the scale's rounding, and each
    of 256 tiles adds up with a rounding or two, as the logarithm and its scalings."""
    n, m = 1 << 15, 4096
    d = hsa.Dims(batch=1, hq=8, hkv=1, max_pages_per_seq=n // 16, num_pages=n // 16, k2=0)
    cache = hsa.KV8.zeros(d)
    cache.k_scale.fill_(1.0)
    cache.k[:, :, :, 0] = 1
    cache.k[0, :, :, 0] = 0
    table = torch.arange(n // 16, device="cuda", dtype=torch.int32)[None]
    q = torch.zeros(m, 8, D, device="cuda", dtype=torch.bfloat16)
    q[:, ::2, 0], q[:, 1::2, 0] = 56.0, 5.0  # times D^-1/2 log2 e: 7.1, just below the lag, and 0.64
    out = torch.ones(m, 8, D, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(m, 8, device="cuda")
    hsa.hsa_kv8_prefill(d, cache, q, cu_of([m]), table, torch.tensor([n], dtype=torch.int32,
                        device="cuda"), out, lse, hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL))
    assert not out.any()
    x = q[:, :, 0].double().cpu().numpy() * D ** -0.5
    ones = (n - m + np.arange(m) + 1 - 16)[:, None]
    want = np.log(16.0 + ones * np.exp(x))
    assert (np.abs(lse.cpu().numpy() - want) <= 600 * 2.0 ** -24 + 2.0 ** -22 * want).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prompts_lose_nothing_to_their_own_sums(fp8):
    """Equal scores over half a million tokens, V with a mean in each channel: 4096 token tiles
    add up in a row. A stretch of 256 (2048 products) may lose 2^-23 of the sum each, 2^-12 of
    the result (its values are of one sign; the weights, all of a scale that is a power of two,
    are not rounded); 2^-16 for the rest of the sums in fp32 and the division, and half a step of
    bf16."""
    n, m = 1 << 19, 8192
    d = hsa.Dims(batch=1, hq=8, hkv=1, max_pages_per_seq=n // 16, num_pages=n // 16, k2=0)
    cache = hsa.KV8.zeros(d, fp8)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 10 + 100 * torch.rand(D, generator=g, device="cuda") + 8 * torch.rand(
        n // 16, 1, 16, D, generator=g, device="cuda")
    cache.v.copy_(x.round().to(cache.v.dtype))
    cache.v_scale.fill_(2.0 ** -7)
    table = torch.randperm(n // 16, generator=g, device="cuda").to(torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.zeros(m, 8, D, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(m, 8, D, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(m, 8, device="cuda")
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    hsa.hsa_kv8_prefill(d, cache, q, cu_of([m]), table, lens, out, lse, ws)
    assert hsa.hsa_read_device_error(ws) == 0
    page = table[0].long()
    values = (cache.v.view(torch.int8)[page].view(cache.v.dtype).float().double() *
              cache.v_scale[page].double()[..., None, None]).view(n, D)
    seen = torch.arange(n - m + 1, n + 1, device="cuda", dtype=torch.float64)[:, None]
    want = values.cumsum(0)[n - m:] / seen
    step = torch.exp2(torch.floor(torch.log2(want)) - 7)  # of bf16
    for j in (0, 7):
        err = (out[:, j].double() - want).abs()
        assert bool((err <= step / 2 + want * (2.0 ** -12 + 2.0 ** -16)).all())
        assert float((lse[:, j].double() - seen[:, 0].log()).abs().max()) <= 14 * 2.0 ** -20


@pytest.mark.parametrize("hq,n,m", [(4, 40000, 700), (8, 70000, 90), (1, 36000, 40)])
def test_prompts_of_stretches_longer_than_the_products_add_up(hq, n, m):
    """More than 256 token tiles a row block, whole row blocks and parts, one tile of rows and
    two; normal scores, a few rows checked against 64 bits."""
    s = Batch([n], hq, 1, "int8", seed=24, fill=False)
    for name in ("k", "v"):
        s.cache[name][...] = s.rng.integers(-127, 128, s.cache[name].shape)
        s.cache[name + "s"][...] = s.rng.uniform(0.005, 0.02, s.cache[name + "s"].shape)
    # many copies of the sequence, so that a CTA's slice holds more than a stretch
    copies = 1 + 152 * 600 // (max(1, m * hq // 256) * (n // 128))
    s.lens, s.table = [n] * copies, np.tile(s.table, (copies, 1))
    q = bf16(s.rng.standard_normal((m * copies, hq, D)))
    out, lse = run_prefill(s, q, [m] * copies)
    k, v = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    for b in sorted({0, copies // 2, copies - 1}):
        for j in sorted({0, hq - 1}):
            i = np.unique([0, 1, m // 3, m // 2, m - 1])
            seen = np.arange(n)[None] <= (n - m + i)[:, None]
            want, wl, tol = O.attend(q[b * m + i, j], k, v, seen, D ** -0.5)
            # fp16 weights; 2048 products a stretch, 2^-23 of the running sum each, whose values
            # are no larger than max |v|
            tol["out"] = tol["out"] + (2.0 ** -11 + 2.0 ** -12) * np.abs(v).max()
            assert_rows(out[b * m + i, j], lse[b * m + i, j], want, wl, tol, 2.0 ** -8)


def test_many_layers_in_turn():
    """70 caches of one shape in turn, beside as many key-code caches of the scorer's: each call
    reads its own."""
    d = hsa.Dims(batch=1, hq=4, hkv=1, max_pages_per_seq=1, num_pages=1, k2=1, sink=0, window=1)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([9], dtype=torch.int32, device="cuda")
    q = torch.ones(1, 4, D, device="cuda", dtype=torch.bfloat16)
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_DECODE)
    layers = []
    for i in range(70):
        cache = hsa.KV8.zeros(d)
        cache.v.fill_(i)
        cache.v_scale.fill_(1.0)
        kq = torch.full((1, 1, 16, D), i, dtype=torch.int8, device="cuda")
        layers.append((cache, kq, torch.zeros(1, 4, D, device="cuda"),
                       torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")))
    k_scale = torch.ones(1, 1, D, device="cuda")
    for _ in range(2):
        for cache, kq, out, block_max in layers:
            hsa.hsa_score_blocks(d, q, kq, k_scale, table, lens, block_max)
            hsa.hsa_kv8_decode(d, cache, q, table, lens, out, None, ws)
    first = int(layers[1][3][0, 0, 0])
    assert first > 0
    for i, (_, _, out, block_max) in enumerate(layers):
        # 9 equal weights of one value: sums of whole numbers, one division
        np.testing.assert_allclose(out.cpu().numpy(), i, rtol=2.0 ** -21)
        assert abs(int(block_max[0, 0, 0]) - i * first) <= i  # scores grow with the codes


def test_lengths_far_below_zero_are_reported():
    """-2^31 less one new token is a large position in 32 bits: the sequence is left out all the
    same, and the others are not."""
    s = Batch([40, 40], 2, 1, "int8", seed=1)
    d, cache, table, err = s.dims(), s.gpu_cache(), s.gpu_table(), error_word()
    before = codes_of(cache)
    q = to_bf16(s.rng.standard_normal((6, 2, D)))
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    for n in (-2 ** 31, -2 ** 31 + 2, -1):
        lens = torch.tensor([n, 40], dtype=torch.int32, device="cuda")
        for cu in (cu_of([3, 3]), None):
            m = 3 if cu is not None else 1
            k = torch.full((2 * m, 1, D), 2.0, dtype=torch.bfloat16, device="cuda")
            hsa.hsa_kv8_read(d, cache, k, k.clone(), cu, table, lens, err)
            assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
            assert (k[:m] == 2.0).all() and not (k[m:] == 2.0).all()
            hsa.hsa_kv8_write(d, cache, k, k, cu, table, lens, err)
            assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
            out = torch.full((2 * m, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((2 * m, 2), 9.0, device="cuda")
            hsa.hsa_kv8_prefill(d, cache, q[:2 * m], cu, table, lens, out, lse, ws)
            assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK
            assert not out[:m].any() and torch.isneginf(lse[:m]).all()
            assert torch.isfinite(lse[m:]).all() and out[m:].any(-1).all()
    after = codes_of(cache)
    other = np.setdiff1d(np.arange(s.num_pages), s.table[1])
    for name in before:
        np.testing.assert_array_equal(after[name][other], before[name][other])


@pytest.mark.parametrize("lens,cu", [
    ([16], [5000, 5016]), ([16, 16], [900, 916, 932]), ([16, 4, 4], [0, 16, 16, 90000]),
    ([4] * 300, [0] * 300 + [-4]),
])
def test_offsets_outside_the_arrays_are_reported(lens, cu):
    """Wherever they lead: sequences behind every row, the only one, the last of many."""
    s = Batch(lens, 2, 1, "int8", seed=1)
    d, err = s.dims(), error_word()
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    k = torch.full((20, 1, D), 2.0, dtype=torch.bfloat16, device="cuda")
    cache = s.gpu_cache()
    hsa.hsa_kv8_read(d, cache, k, k.clone(), cu, s.gpu_table(), s.gpu_lens(), err)
    assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
    hsa.hsa_kv8_write(d, cache, k, k, cu, s.gpu_table(), s.gpu_lens(), err)
    assert hsa.hsa_read_device_error(err) == hsa.HSA_ERR_DEVICE_CHECK
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    q = to_bf16(s.rng.standard_normal((20, 2, D)))
    out = torch.full((20, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    hsa.hsa_kv8_prefill(d, cache, q, cu, s.gpu_table(), s.gpu_lens(), out, None, ws)
    assert hsa.hsa_read_device_error(ws) == hsa.HSA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("lo,hi", [(-126, -100), (-40, -30), (-10, 2), (30, 40), (100, 119)])
def test_decode_of_one_token_gives_its_value(lo, hi):
    """Weight 1 on one value, under any scale. log2 of the scale is off by an ulp, 2^-23 of itself,
    and enters as an exponent; two exponentials of 2^-22 and a few roundings of 2^-24."""
    n = 500
    d = hsa.Dims(batch=n, hq=3, hkv=1, max_pages_per_seq=1, num_pages=n, k2=0)
    cache = hsa.KV8.zeros(d)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache.v.copy_(torch.randint(-127, 128, cache.v.shape, generator=g, device="cuda"))
    scale = torch.exp2(lo + (hi - lo) * torch.rand(n, 1, generator=g, device="cuda")).clamp(min=2.0 ** -126)
    cache.v_scale.copy_(scale)
    q = torch.zeros(n, 3, D, device="cuda", dtype=torch.bfloat16)
    out, lse = torch.empty(n, 3, D, device="cuda"), torch.empty(n, 3, device="cuda")
    hsa.hsa_kv8_decode(d, cache, q, torch.arange(n, device="cuda", dtype=torch.int32)[:, None],
                       torch.ones(n, device="cuda", dtype=torch.int32), out, lse,
                       hsa.workspace(d, hsa.HSA_OP_KV8_DECODE))
    want = (cache.v[:, 0, 0].double() * scale.double())[:, None]
    rel = np.log(2) * 2.0 ** -23 * max(abs(lo), abs(hi)) + 2 * 2.0 ** -22 + 8 * 2.0 ** -24
    assert bool(((out.double() - want).abs() <= rel * want.abs() + 2.0 ** -149).all())
    assert float(lse.abs().max()) <= rel


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,per_head", [(7, 1, 0), (8, 1, 0), (24, 3, 1)])
@pytest.mark.parametrize("lens", [
    [1 + i % 20 for i in range(300)],             # a warp a row
    [10 + (i * 13) % 330 for i in range(170)],    # four warps a row
    [17] * 160 + [6000, 0, 3],                    # a CTA for them all, the long row cut
], ids=["warp", "four", "cta"])
def test_more_rows_than_ctas_of_every_kind(fmt, hq, hkv, per_head, lens):
    """Full and odd groups, a selection of its own for each query head, both formats, dense and
    over kept blocks, for each way in which rows are shared out."""
    s = Batch(lens, hq, hkv, fmt, seed=hq + len(lens))
    q = bf16(s.rng.standard_normal((len(lens), hq, D)))
    rows, g = hq if per_head else hkv, hq // hkv
    idx = np.empty((len(lens), rows, 3), np.int32)
    for r in range(rows):  # a row's own blocks
        idx[:, r] = [r % 3, 3 + r % 2, 7 + r]
    cnt = np.tile(np.arange(rows, dtype=np.int32) % 4, (len(lens), 1))
    kept = (torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda())
    results = [(run_decode(s, q), None),
               (run_decode(s, q, kept, sink=3, window=9, k2=3, per_head=per_head), kept)]
    for b in list(range(0, len(lens), 29)) + [len(lens) - 3, len(lens) - 2, len(lens) - 1]:
        n = lens[b]
        t = np.arange(n)
        for j in range(hq):
            k, v = (O.values(s.cache, w, s.table[b], n, j // g) for w in "kv")
            r = j if per_head else j // g
            near = (t < 3) | (t >= n - 9) | np.isin(t // PAGE, idx[b, r, :cnt[b, r]])
            for (out, lse), form in results:
                seen = np.ones(n, bool) if form is None else near
                want, wl, tol = O.attend(q[b, j:j + 1], k, v, seen[None], D ** -0.5)
                assert_rows(out[b, j:j + 1], lse[b, j:j + 1], want, wl, tol)


@pytest.mark.parametrize("fmt,hq,n,m", [("int8", 8, 131072, 3), ("e4m3", 4, 100001, 70),
                                        ("int8", 5, 60000, 128)])
def test_prompt_rows_joined_of_many_parts(fmt, hq, n, m):
    """Few new tokens over a long context: a row block in up to 152 parts, one tile or two."""
    s = Batch([n], hq, 1, fmt, seed=25, fill=False)
    for name in ("k", "v"):
        c = s.cache[name]
        c[...] = s.rng.integers(-100, 101, c.shape) if fmt == "int8" else O.e4m3_code(
            s.rng.standard_normal(c.shape, dtype=np.float32) * 100.0)
        s.cache[name + "s"][...] = s.rng.uniform(0.005, 0.02, s.cache[name + "s"].shape)
    q = bf16(s.rng.standard_normal((m, hq, D)))
    out, lse = run_prefill(s, q, [m])
    i = np.unique([0, 1, m // 2, m - 1])
    k, v = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    seen = np.arange(n)[None] <= (n - m + i)[:, None]
    for j in range(hq):
        want, wl, tol = O.attend(q[i, j], k, v, seen, D ** -0.5)
        tol["out"] = tol["out"] + 2.0 ** -11 * np.abs(v).max()
        assert_rows(out[i, j], lse[i, j], want, wl, tol, 2.0 ** -8)


def test_long_stretches_over_unlike_scales():
    """The sums' own frame (V of zeros, tiny and large) across stretches of 256 tiles and parts."""
    hq, n, m, copies = 4, 40000, 300, 60
    s = Batch([n], hq, 1, "int8", seed=26, fill=False)
    pages = s.cache["v"].shape[0]
    for name in ("k", "v"):
        s.cache[name][...] = s.rng.integers(-127, 128, s.cache[name].shape)
        s.cache[name + "s"][...] = s.rng.uniform(0.005, 0.02, (pages, 1))
    e = s.rng.choice([-110, -60, 0, 0, 0, 0, 50, 100], (pages, 1))
    s.cache["vs"] *= (2.0 ** e).astype(np.float32)
    zero = s.rng.random(pages) < 0.1
    s.cache["v"][zero], s.cache["vs"][zero] = 0, 0
    s.lens, s.table = [n] * copies, np.tile(s.table, (copies, 1))
    q = bf16(s.rng.standard_normal((m * copies, hq, D)))
    out, lse = run_prefill(s, q, [m] * copies)
    k, v = (O.values(s.cache, w, s.table[0], n, 0) for w in "kv")
    i = np.array([0, m // 2, m - 1])
    seen = np.arange(n)[None] <= (n - m + i)[:, None]
    for b in (0, 1, copies // 2, copies - 1):
        for j in (0, hq - 1):
            qj = q[b * m + i, j].astype(np.float64)
            want, wl, tol = O.attend(qj, k, v, seen, D ** -0.5)
            bound = unlike_bounds(qj, k, v, seen, tol, 127.0, 2.0 ** -11 + 2.0 ** -12, 2.0 ** -32)
            bound += 2.0 ** -8 * (np.abs(want) + bound)
            assert (np.abs(lse[b * m + i, j] - wl) <= tol["lse"]).all(), (b, j)
            assert (np.abs(out[b * m + i, j] - want) <= bound).all(), (b, j)


def test_prompt_rows_are_the_same_every_time():
    """Parts meet in the order of their slices, whichever CTA joins them: the same bits, call
    after call."""
    s = Batch([6000, 9000, 12000, 7000], 8, 2, "int8", seed=27, fill=False)
    for name in ("k", "v"):
        s.cache[name][...] = s.rng.integers(-127, 128, s.cache[name].shape)
    new = [7, 24, 11, 300]
    d, cache, table, lens, cu = s.dims(), s.gpu_cache(), s.gpu_table(), s.gpu_lens(), cu_of(new)
    ws = hsa.workspace(d, hsa.HSA_OP_KV8_PREFILL)
    q = to_bf16(s.rng.standard_normal((sum(new), 8, D)) * 0.1)
    first = None
    for _ in range(20):
        out = torch.empty(sum(new), 8, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(sum(new), 8, device="cuda")
        hsa.hsa_kv8_prefill(d, cache, q, cu, table, lens, out, lse, ws)
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert torch.isfinite(first[0]).all() and torch.isfinite(first[1]).all()
