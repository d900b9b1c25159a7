"""Shared helpers of the 8-bit K/V cache tests: seeded ragged batches, the cache on both sides."""
from __future__ import annotations

import numpy as np
import torch

from kv_cache_int8_gb300 import hsa
from oracle import kv8 as O

PAGE, D = 16, 128


def bf16(x) -> np.ndarray:
    """fp32 values rounded to bf16."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(
        torch.bfloat16).float().numpy()


def to_bf16(x, device="cuda") -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(device)


class Batch:
    """Sequences of the given lengths in a permuted page pool with `spare` unused pages; page
    tables padded with -1 beyond each sequence; the oracle's cache filled by whole-sequence
    writes of random K and V (outlier key channels)."""

    def __init__(self, lens, hq, hkv, fmt, seed=0, spare=3, extra_pages=0, fill=True):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hq, self.hkv, self.fmt = rng, list(lens), hq, hkv, fmt
        per = [-(-n // PAGE) for n in lens]
        self.max_pages = max(max(per), 1) + extra_pages
        self.num_pages = sum(per) + spare
        pool = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.max_pages), -1, dtype=np.int32)
        off = 0
        for b, p in enumerate(per):
            self.table[b, :p] = pool[off:off + p]
            off += p
        self.cache = O.empty(fmt, self.num_pages, hkv)
        # whatever lies in slots that no token has reached must not matter
        for name in ("k", "v"):
            c = self.cache[name]
            c[...] = rng.integers(-128, 128, c.shape).astype(np.int8).view(c.dtype)
            self.cache[name + "s"][...] = rng.uniform(0.5, 2.0, (self.num_pages, hkv))
        if fill:
            for b, n in enumerate(lens):
                if n:
                    O.write(self.cache, self.rows(n, True), self.rows(n), self.table[b], 0)

    def rows(self, n, outliers=False):
        x = self.rng.standard_normal((n, self.hkv, D), dtype=np.float32)
        if outliers:
            x[:, :, 5::32] *= 8.0
        return bf16(x)

    def dims(self, **kw) -> hsa.Dims:
        kw = {"sink": 0, "window": 0, "k2": 0, **kw}
        return hsa.Dims(batch=len(self.lens), hq=self.hq, hkv=self.hkv,
                        max_pages_per_seq=self.max_pages, num_pages=self.num_pages, **kw)

    def gpu_cache(self) -> hsa.KV8:
        c = self.cache
        codes = [torch.from_numpy(c[n].view(np.int8).copy()).cuda() for n in ("k", "v")]
        if self.fmt == "e4m3":
            codes = [t.view(torch.float8_e4m3fn) for t in codes]
        return hsa.KV8(*codes, torch.from_numpy(c["ks"].copy()).cuda(),
                       torch.from_numpy(c["vs"].copy()).cuda())

    def gpu_table(self):
        return torch.from_numpy(self.table).cuda()

    def gpu_lens(self, lens=None):
        return torch.tensor(self.lens if lens is None else lens, dtype=torch.int32, device="cuda")


def codes_of(cache: hsa.KV8) -> dict:
    """A device cache's arrays in the oracle's types."""
    t = np.uint8 if cache.k.dtype == torch.float8_e4m3fn else np.int8
    return {"k": cache.k.view(torch.int8).cpu().numpy().view(t),
            "v": cache.v.view(torch.int8).cpu().numpy().view(t),
            "ks": cache.k_scale.cpu().numpy(), "vs": cache.v_scale.cpu().numpy()}


def assert_same_cache(got: hsa.KV8, want: dict):
    for name, a in codes_of(got).items():
        np.testing.assert_array_equal(a.view(np.int8) if a.itemsize == 1 else a,
                                      want[name].view(np.int8) if a.itemsize == 1 else want[name],
                                      err_msg=name)


def assert_rows(got, lse, want, want_lse, tol, rounding=0.0):
    """Output rows within the oracle's bound (plus a relative rounding of the result)."""
    got = np.asarray(got, dtype=np.float64)
    assert np.isfinite(got).all()
    bound = tol["out"][:, None] + rounding * (np.abs(want) + tol["out"][:, None])
    err = np.abs(got - want)
    assert (err <= bound).all(), f"max error {err.max():.3e}, bound there {bound.flat[err.argmax()]:.3e}"
    if lse is not None:
        lse = np.asarray(lse, dtype=np.float64)
        none = np.isneginf(want_lse)
        assert (np.isneginf(lse) == none).all()
        assert (np.abs(lse[~none] - want_lse[~none]) <= tol["lse"][~none]).all()
