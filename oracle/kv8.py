"""The 8-bit K/V cache in numpy, from its definition: codes and scales exactly (fp32 decisions),
attention in fp64. Independent of the CUDA library; test infrastructure only.

A cache is a dict: "fmt" ("int8" or "e4m3"), "k" / "v" codes [pages][hkv][16][128] (int8, or
uint8 bit patterns of E4M3), "ks" / "vs" fp32 scales [pages][hkv]."""
from __future__ import annotations

import numpy as np

PAGE, D = 16, 128
LEVELS = {"int8": np.float32(127), "e4m3": np.float32(448)}


def _e4m3_table() -> np.ndarray:
    """Values of the E4M3 codes 0 .. 126 (ascending; 127 is the NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = _e4m3_table()


def e4m3_code(x) -> np.ndarray:
    """Bit patterns of the E4M3 values nearest to x (finite), ties to the even code,
    saturating."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3[-1])
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == E4M3[hi], hi, code)
    code = np.where(a == E4M3[lo], lo, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def code_values(fmt: str, codes) -> np.ndarray:
    """The numbers that codes stand for (fp64, without the scale)."""
    if fmt == "int8":
        return codes.astype(np.float64)
    mag = np.concatenate([E4M3, [np.nan]])[codes & 127]
    return np.where(codes & 128, -mag, mag)


def encode(fmt: str, y) -> np.ndarray:
    """Codes of fp32 numbers y already multiplied by the inverse scale."""
    y = np.clip(np.asarray(y, dtype=np.float32), -LEVELS[fmt], LEVELS[fmt])
    return np.rint(y).astype(np.int8) if fmt == "int8" else e4m3_code(y)


def empty(fmt: str, pages: int, hkv: int) -> dict:
    t = np.int8 if fmt == "int8" else np.uint8
    return {"fmt": fmt, "k": np.zeros((pages, hkv, PAGE, D), t),
            "v": np.zeros((pages, hkv, PAGE, D), t), "ks": np.zeros((pages, hkv), np.float32),
            "vs": np.zeros((pages, hkv), np.float32)}


def write_block(fmt: str, codes, scale, rows, first: int):
    """One block [16][128]: rows [n][128] (fp32) become slots [first, first + n); slots before
    `first` hold older tokens. Returns (codes, scale)."""
    f32 = np.float32
    rows = np.asarray(rows, dtype=f32)
    fin = np.where(np.isfinite(rows), np.abs(rows), f32(0))
    s = f32(fin.max()) / LEVELS[fmt]
    if s < f32(2.0) ** f32(-126):
        s = f32(0)
    if first > 0:
        s = max(f32(scale), s)
    inv = f32(1) / s if s > 0 else f32(0)
    out = codes.copy()
    if first > 0 and s > scale:
        ratio = f32(scale) * inv
        out[:first] = encode(fmt, code_values(fmt, codes[:first]).astype(f32) * ratio)
    with np.errstate(invalid="ignore", over="ignore"):
        y = rows * inv
    y = np.where(np.isnan(rows) | np.isnan(y), f32(0), y)
    out[first:first + len(rows)] = encode(fmt, y)
    return out, f32(s)


def write(cache: dict, k_new, v_new, table, start: int) -> None:
    """Tokens [start, start + n) of one sequence (page-table row `table`) from rows
    [n][hkv][128], in place."""
    n, hkv = k_new.shape[0], k_new.shape[1]
    at = start
    while at < start + n:
        slot = at % PAGE
        m = min(PAGE - slot, start + n - at)
        page = table[at // PAGE]
        for x, c, s in ((k_new, "k", "ks"), (v_new, "v", "vs")):
            for h in range(hkv):
                cache[c][page, h], cache[s][page, h] = write_block(
                    cache["fmt"], cache[c][page, h], cache[s][page, h],
                    x[at - start:at - start + m, h], slot)
        at += m


def values(cache: dict, which: str, table, n: int, h: int) -> np.ndarray:
    """[n][128] fp64 values of a sequence's tokens under kv head h."""
    pages = table[:-(-n // PAGE)]
    c = code_values(cache["fmt"], cache[which][pages, h])
    c = c * cache[which + "s"][pages, h].astype(np.float64)[:, None, None]
    return c.reshape(-1, D)[:n]


def attend(q, k, v, seen, sm_scale: float):
    """q [r][128], k / v [n][128], seen [r][n] bool, fp64. Returns (out, lse, tol): tol bounds
    an fp32 evaluation's error of each output row. A row that sees nothing: 0, -inf."""
    q = np.asarray(q, dtype=np.float64)
    x = q @ k.T * sm_scale
    x = np.where(seen, x, -np.inf)
    m = x.max(-1, keepdims=True) if x.shape[1] else np.full((len(q), 1), -np.inf)
    m0 = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(x - m0)
    l = p.sum(-1, keepdims=True)
    out = np.divide(p @ v, l, out=np.zeros((len(q), v.shape[1])), where=l > 0)
    with np.errstate(divide="ignore"):
        lse = (m0 + np.log(l))[:, 0]
    # logits: 8 products of 16 terms, each summed with 17 roundings of at most 2^-24 of the sum
    # of magnitudes B, then 4 scalings; the exponential and its argument 2^-21 and 2^-23 |x|;
    # sums over n tokens: one rounding a 16-token block, 16 inside a block, 64 for the joins
    big = (np.abs(q) @ np.abs(k).T * abs(sm_scale) * seen).max(-1) if k.shape[0] else np.zeros(len(q))
    eps = (8 * 17 + 8) * 2.0 ** -24 * big + 2.0 ** -21
    top = np.abs(v).max() if v.size else 0.0
    sums = (len(k) / 16 + 80) * 2.0 ** -24
    return out, lse, {"out": top * 2 * (eps + sums), "lse": 2 * (eps + sums) + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))}
