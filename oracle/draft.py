"""Rotary positions and drafted tokens on the 8-bit K/V cache in numpy, from their definitions: the
rotation and the codes exactly (fp32 decisions), attention by oracle.kv8 in fp64. Independent of the
CUDA library; test infrastructure only."""
from __future__ import annotations

import numpy as np

from . import kv8 as O

PAGE, D = O.PAGE, O.D


def frequencies(dim: int, base: float, scaling: int = 0, factor: float = 1.0, low: float = 1.0,
                high: float = 4.0, original: float = 8192.0) -> np.ndarray:
    f = base ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    if scaling == 1:
        return f / factor
    if scaling == 2:
        w = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0, 1)
        return f * (w + (1 - w) / factor)
    return f


def table(rows: int, f, magnitude: float = 1.0) -> np.ndarray:
    """[rows][dim] in fp64: cosines, then sines."""
    a = np.arange(rows, dtype=np.float64)[:, None] * f
    return magnitude * np.concatenate([np.cos(a), np.sin(a)], -1)


def turn(x, angles, neighbours: bool) -> np.ndarray:
    """Rows x [n][heads][128] under the table rows angles [n][dim] fp32; every operation rounded to
    fp32."""
    x = np.asarray(x, dtype=np.float32)
    dim = angles.shape[1]
    i = np.arange(dim // 2)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + dim // 2)
    c, s = angles[:, None, :dim // 2], angles[:, None, dim // 2:]
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def branches(parents) -> np.ndarray:
    """[node][node]: whether the second is the first or one of its ancestors."""
    n = len(parents)
    seen = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return seen


def depths(parents) -> np.ndarray:
    return branches(parents).sum(-1) - 1


def seen(n: int, parents) -> np.ndarray:
    """[node][token]: what each of the last len(parents) of n tokens attends."""
    m = len(parents)
    return np.concatenate([np.ones((m, n - m), dtype=bool), branches(parents)], -1)


def tree(rng, n: int, roots: bool = False) -> list:
    """Parents of a random tree: node 0 hangs on the context, node i on an earlier one (with
    `roots` now and then on the context)."""
    return [-1 if i == 0 or (roots and rng.random() < 0.2) else int(rng.integers(i))
            for i in range(n)]


def keep(cache: dict, page_row, n: int, m: int, idx) -> int:
    """Moves the nodes idx of the last m of n tokens behind the first n - m; the new length."""
    idx = np.asarray(idx, dtype=np.int64)
    start, hkv = n - m, cache["k"].shape[1]
    if idx.size:
        at = start + idx
        pages, slots = np.asarray(page_row)[at // PAGE], at % PAGE
        rows = []
        for c, s in (("k", "ks"), ("v", "vs")):
            v = O.code_values(cache["fmt"], cache[c][pages, :, slots]).astype(np.float32)
            rows.append(v * cache[s][pages][..., None])
        assert rows[0].shape == (idx.size, hkv, D) and rows[0].dtype == np.float32
        O.write(cache, rows[0], rows[1], page_row, start)
    return start + idx.size
