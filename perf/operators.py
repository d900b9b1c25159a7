"""The operators of the 8-bit K/V cache, as measured work: inputs, plain forms, exact values.

The cache holds the codes of K and V in 8 bits (int8 or FP8 E4M3), paged like the bf16 cache
([page][kv head][16][128]), with one fp32 scale for each 16-token block and kv head, for K and
for V apart. Four operators live on it:

  write    the new tokens' K and V (bf16) are quantised into their blocks as they arrive; a
           block that already holds tokens keeps the larger scale and its codes follow it
  read     the values of the last n tokens of each sequence, back in bf16
  decode   attention of one query token a sequence over its whole context (`dense`), or over
           the sink, the window and a list of kept blocks (`kept`)
  prefill  causal attention of the last n tokens of each sequence over the context

``own`` chooses between the plain form (elementary torch operations) and the framework's
kernels. Sizes follow the decode configurations of kv_cache_int8_gb300.workloads (32 or 64
query heads over 8 kv heads, 4 over 1; 8K to 128K tokens, permuted page pools).
"""
import math

import torch

own = False

PAGE, D = 16, 128
TINY = 2.0 ** -126  # scales below the smallest normal number count as zero
LEVELS = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a single long chat: the newest token joins a 128K context
        dict(name="write-step", op="write", fmt="int8", batch=1, hq=32, hkv=8, lo=131000,
             hi=131000, new_lo=1, new_hi=1),
        # one step of a serving batch at mixed positions inside their blocks
        dict(name="write-step-batch", op="write", fmt="e4m3", batch=256, hq=32, hkv=8, lo=300,
             hi=5000, new_lo=1, new_hi=1),
        # a batch of long prompts (and continued chats, starting inside a block) on arrival
        dict(name="write-prompts", op="write", fmt="int8", batch=8, hq=32, hkv=8, lo=9000,
             hi=23000, new_lo=8001, new_hi=22777),
        # a short tail read back, as for a draft model or a re-quantisation of the window
        dict(name="read-tail", op="read", fmt="int8", batch=1, hq=32, hkv=8, lo=8191, hi=8191,
             new_lo=1024, new_hi=1024),
        # whole contexts read back, as for moving sequences to another cache
        dict(name="read-whole", op="read", fmt="e4m3", batch=4, hq=32, hkv=8, lo=15000,
             hi=40000, new_lo=1 << 30, new_hi=1 << 30),
        # the tiny configuration: one kv head, 8192 tokens; latency of a single call
        dict(name="decode-tiny", op="decode", kind="dense", fmt="int8", batch=1, hq=4, hkv=1,
             lo=8192, hi=8192),
        # one 128K sequence, groups of 4 query heads
        dict(name="decode-128k", op="decode", kind="dense", fmt="e4m3", batch=1, hq=32, hkv=8,
             lo=131072, hi=131072),
        # the batched configuration: eight sequences of 32K to 128K tokens, groups of 8
        dict(name="decode-batch", op="decode", kind="dense", fmt="int8", batch=8, hq=64, hkv=8,
             lo=32768, hi=131072),
        # the pruned step's attention: sink 128, window 1024 and 128 kept blocks of 128K tokens
        dict(name="decode-kept", op="decode", kind="kept", fmt="int8", batch=1, hq=32, hkv=8,
             lo=131072, hi=131072, sink=128, window=1024, k2=128),
        # drafted tokens of a few chats verified together: rows of one tile, long contexts
        dict(name="prefill-verify", op="prefill", fmt="int8", batch=4, hq=32, hkv=8, lo=6000,
             hi=12000, new_lo=5, new_hi=33),
        # one chunk of a chunked prompt behind 30K tokens of context
        dict(name="prefill-chunk", op="prefill", fmt="e4m3", batch=1, hq=32, hkv=8, lo=32768,
             hi=32768, new_lo=2048, new_hi=2048),
        # a whole 8K prompt
        dict(name="prefill-prompt", op="prefill", fmt="int8", batch=1, hq=32, hkv=8, lo=8192,
             hi=8192, new_lo=8192, new_hi=8192),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prefill"])
    fmt = rng.choice(["int8", "e4m3"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    c = dict(op=op, fmt=fmt, hq=hkv * group, hkv=hkv)
    if op in ("write", "read"):
        c["batch"] = _log(rng, 1, 256)
        most = max(64, 140000 // c["batch"])  # tokens a sequence
        c["hi"] = _log(rng, 17, most)
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.3, 1.0)))
        c["new_hi"] = 1 if op == "write" and rng.random() < 0.4 else _log(rng, 1, c["hi"])
        c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.3, 1.0)))
    elif op == "decode":
        c["kind"] = rng.choice(["dense", "dense", "kept"])
        c["batch"] = _log(rng, 1, 64)
        most = max(64, 600000 // c["batch"])
        c["hi"] = _log(rng, 17, min(131072, most))
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.3, 1.0)))
        if c["kind"] == "kept":
            c.update(sink=rng.choice([0, 4, 64, 128]), window=rng.choice([1, 37, 256, 1024]),
                     k2=_log(rng, 1, 256))
    else:
        c["batch"] = _log(rng, 1, 8)
        c["hi"] = _log(rng, 17, 32768)
        # at most the products of the whole 8K prompt, padded sequences included
        most = max(1, int(0.9 * 8192 * 8192 * 32 / (c["batch"] * c["hi"] * c["hq"])))
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.3, 1.0)))
        c["new_hi"] = _log(rng, 1, min(most, c["hi"]))
        c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.3, 1.0)))
    return c


# ------------------------------------------------------------------------------ inputs

def _lengths(case):
    """Tokens (N_b) and new tokens (n_b) of each sequence: fixed by the case, spread over its
    ranges."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    lens = [lo + (hi - lo) * ((b * 619 + 211) % 997) // 996 for b in range(B)]
    if B > 1:
        lens[0], lens[-1] = hi, lo
    if "new_hi" not in case:
        return lens, [1] * B
    lo, hi = case["new_lo"], case["new_hi"]
    new = [lo + (hi - lo) * ((b * 389 + 307) % 991) // 990 for b in range(B)]
    return lens, [min(n, m) for n, m in zip(new, lens)]


def _quantise(x, fmt):
    """Codes (as the type they are stored in) and scales of full blocks x [..][16][128] fp32."""
    amax = x.abs().amax((-2, -1))
    s = amax / torch.full_like(amax, LEVELS[fmt])
    s = torch.where(s < TINY, torch.zeros_like(s), s)
    y = x * torch.where(s > 0, 1.0 / s, torch.zeros_like(s))[..., None, None]
    if fmt == "int8":
        return y.round().clamp(-127, 127).to(torch.int8), s
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), s


def _blocks(pages, hkv, gen, outliers):
    """Random blocks [pages][hkv][16][128]: normal values; for keys 4 channels of each head
    are 8 times larger."""
    x = torch.randn(pages, hkv, PAGE, D, generator=gen, device="cuda")
    if outliers:
        ch = torch.rand(hkv, D, generator=gen, device="cuda").argsort(-1)[:, :4]
        f = torch.ones(hkv, D, device="cuda").scatter_(1, ch, 8.0)
        x *= f[:, None, :]
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, hq, hkv, fmt = case["batch"], case["hq"], case["hkv"], case["fmt"]
    lens, new = _lengths(case)
    per = [-(-n // PAGE) for n in lens]
    pool = torch.randperm(sum(per), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
    off = 0
    for b, p in enumerate(per):
        table[b, :p] = pool[off:off + p]
        off += p
    st = dict(op=case["op"], kind=case.get("kind"), fmt=fmt, hq=hq, hkv=hkv, table=table,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), lens_host=lens,
              new_host=new, sm_scale=1.0 / math.sqrt(D), sink=case.get("sink", 0),
              window=case.get("window", 0), k2=case.get("k2", 0))
    for name in ("k", "v"):
        codes = torch.empty(sum(per), hkv, PAGE, D, device="cuda",
                            dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
        scale = torch.empty(sum(per), hkv, device="cuda")
        for p in range(0, sum(per), 4096):
            n = min(4096, sum(per) - p)
            codes[p:p + n], scale[p:p + n] = _quantise(_blocks(n, hkv, gen, name == "k"), fmt)
        st[name], st[name + "_scale"] = codes, scale
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
    st["total"] = T
    # one new token a sequence needs no offsets: row b is sequence b's token
    st["cu"] = (None if max(new) == 1 and min(new) == 1 else
                torch.tensor(cu, dtype=torch.int32, device="cuda"))
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] == "write":
        # K and V as slices of one projection's output [tokens][hq + 2 hkv][128]
        qkv = torch.empty(T, hq + 2 * hkv, D, **bf16)
        for t in range(0, T, 65536):
            n = min(65536, T - t)
            qkv[t:t + n] = torch.randn(n, hq + 2 * hkv, D, generator=gen, device="cuda")
        st["k_new"], st["v_new"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    elif case["op"] == "read":
        st["k_out"] = torch.empty(T, hkv, D, **bf16)
        st["v_out"] = torch.empty(T, hkv, D, **bf16)
    elif case["op"] == "decode":
        st["q"] = torch.randn(B, hq, D, generator=gen, device="cuda").to(torch.bfloat16)
        st["out"] = torch.empty(B, hq, D, device="cuda")
        st["lse"] = torch.empty(B, hq, device="cuda")
        if case["kind"] == "kept":
            # the kept blocks of a pruned step: distinct, ascending, -1 behind the last
            k2 = case["k2"]
            idx = torch.full((B, hkv, k2), -1, dtype=torch.int32, device="cuda")
            cnt = torch.zeros(B, hkv, dtype=torch.int32, device="cuda")
            for b in range(B):
                lo, hi = case["sink"] // PAGE, -(-max(lens[b] - case["window"], 0) // PAGE)
                if hi > lo:
                    pick = torch.rand(hkv, hi - lo, generator=gen, device="cuda").argsort(-1)
                    pick = (pick[:, :k2] + lo).sort(-1)[0]
                    idx[b, :, :pick.shape[1]] = pick.to(torch.int32)
                    cnt[b] = pick.shape[1]
            st["block_idx"], st["n_blocks"] = idx, cnt
    else:
        st["q"] = torch.randn(T, hq, D, generator=gen, device="cuda").to(torch.bfloat16)
        st["out"] = torch.empty(T, hq, D, **bf16)
        st["lse"] = torch.empty(T, hq, device="cuda")
    return st


# --------------------------------------------------------------------------- plain form

def _new_of(st):
    """(first new position, number of new tokens, first row) of each sequence."""
    lens = st["lens"].long()
    if st["cu"] is None:
        return lens - 1, torch.ones_like(lens), torch.arange(lens.numel(), device="cuda")
    cu = st["cu"].long()
    n = cu[1:] - cu[:-1]
    return lens - n, n, cu[:-1]


def _rows(st):
    """(sequence, position) of every new row."""
    start, _, first = _new_of(st)
    r = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(first.contiguous(), r, right=True) - 1
    return b, start[b] + r - first[b]


def _plain_write(st):
    start, n, first = _new_of(st)
    lens = st["lens"].long()
    touched = max((m - 1) // PAGE - (m - k) // PAGE + 1
                  for m, k in zip(st["lens_host"], st["new_host"]))
    last = (lens - 1) // PAGE
    # a sequence with fewer blocks than the others repeats its last one (the same values)
    p = torch.minimum(start[:, None] // PAGE + torch.arange(touched, device="cuda"), last[:, None])
    page = torch.gather(st["table"].long(), 1, p)
    pos = p[..., None] * PAGE + torch.arange(PAGE, device="cuda")  # [B][J][16]
    fresh = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    stale = pos < start[:, None, None]
    src = (first[:, None, None] + pos - start[:, None, None]).clamp(0, st["total"] - 1)
    has_old = stale.any(-1)[..., None]
    levels = LEVELS[st["fmt"]]
    for name in ("k", "v"):
        codes, scale = st[name].view(torch.int8), st[name + "_scale"]
        x = st[name + "_new"][src].float().transpose(2, 3)  # [B][J][H][16][128]
        new = fresh[:, :, None, :, None]
        finite = torch.where(new & torch.isfinite(x), x.abs(), torch.zeros_like(x))
        amax = finite.amax((-2, -1))
        s_new = amax / torch.full_like(amax, levels)
        s_new = torch.where(s_new < TINY, torch.zeros_like(s_new), s_new)
        s_old = scale[page]
        s = torch.where(has_old, torch.maximum(s_old, s_new), s_new)
        s = torch.where(fresh.any(-1)[..., None], s, s_old)
        inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))[..., None, None]
        was = codes[page]
        ratio = s_old[..., None, None] * inv
        grown = (s > s_old)[..., None, None]
        y = torch.where(torch.isnan(x), torch.zeros_like(x), x * inv)
        y = torch.where(torch.isnan(y), torch.zeros_like(y), y).clamp(-levels, levels)
        if st["fmt"] == "int8":
            put = y.round().to(torch.int8)
            moved = (was.float() * ratio).round().to(torch.int8)
        else:
            put = y.to(torch.float8_e4m3fn).view(torch.int8)
            moved = (was.view(torch.float8_e4m3fn).float() * ratio).to(
                torch.float8_e4m3fn).view(torch.int8)
        old = stale[:, :, None, :, None] & grown
        codes[page] = torch.where(new, put, torch.where(old, moved, was))
        scale[page] = s
    return st["k"], st["v"], st["k_scale"], st["v_scale"]


def _values(st, name, b, pos):
    """fp32 values of tokens (b, pos) for every kv head: [..][H][128]."""
    page = st["table"].long()[b, pos // PAGE]
    codes = st[name][page, :, pos % PAGE] if st["fmt"] == "int8" else \
        st[name].view(torch.uint8)[page, :, pos % PAGE].view(torch.float8_e4m3fn)
    return codes.float() * st[name + "_scale"][page][..., None]


def _plain_read(st):
    b, pos = _rows(st)
    for name in ("k", "v"):
        st[name + "_out"].copy_(_values(st, name, b, pos))
    return st["k_out"], st["v_out"]


def _softmax_values(s, seen, v):
    """softmax over the last axis of s where `seen`, times v, and the log of the sum."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(s - m)
    del s
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out, (m + torch.log(total))[..., 0]


def _plain_decode(st):
    B, hq, hkv = st["q"].shape[0], st["hq"], st["hkv"]
    lens = st["lens"].long()
    ar = lambda n: torch.arange(n, device="cuda")  # noqa: E731
    q = st["q"].float().view(B, hkv, hq // hkv, D)
    if st["kind"] == "dense":
        pos = ar(max(st["lens_host"])).expand(B, -1)
        seen = (pos < lens[:, None])[:, None]
        pos = torch.minimum(pos, lens[:, None] - 1)
        b = ar(B)[:, None]
        k = _values(st, "k", b, pos).transpose(1, 2)  # [B][H][L][128]
        v = _values(st, "v", b, pos).transpose(1, 2)
    else:
        # sink, window and kept blocks, in that order; each token once
        head = torch.minimum(lens, torch.full_like(lens, st["sink"]))
        tail = torch.maximum(lens - st["window"], head)
        blk = st["block_idx"].long()
        listed_ = ar(blk.shape[-1]) < st["n_blocks"].long()[..., None]
        kept = (blk.clamp(min=0)[..., None] * PAGE + ar(PAGE)).flatten(-2)
        kept_ok = listed_[..., None].expand(*listed_.shape, PAGE).flatten(-2)
        kept_ok = kept_ok & (kept >= st["sink"]) & (kept < (lens - st["window"])[:, None, None])
        a, w = ar(st["sink"]).expand(B, -1), tail[:, None] + ar(st["window"])
        a_ok, w_ok = a < head[:, None], w < lens[:, None]
        every = lambda t: t[:, None].expand(-1, hkv, -1)  # noqa: E731
        pos = torch.cat([every(a), every(w), kept], -1)
        seen = torch.cat([every(a_ok), every(w_ok), kept_ok], -1)
        pos = torch.where(seen, pos, torch.zeros_like(pos))
        page = st["table"].long()[ar(B)[:, None, None], pos // PAGE]
        h = ar(hkv)[None, :, None]
        pick = lambda n: (st[n].view(torch.int8)[page, h, pos % PAGE].view(st[n].dtype).float()  # noqa: E731
                          * st[n + "_scale"][page, h][..., None])
        k, v = pick("k"), pick("v")
    s = torch.matmul(q, k.transpose(-1, -2)) * st["sm_scale"]
    del k
    out, lse = _softmax_values(s, seen[:, :, None], v)
    return out.reshape(B, hq, D), lse.reshape(B, hq)


def _plain_prefill(st):
    start, n, first = _new_of(st)
    B, hq, hkv = start.numel(), st["hq"], st["hkv"]
    ar = lambda m: torch.arange(m, device="cuda")  # noqa: E731
    lens = st["lens"].long()
    most = max(st["new_host"])
    row = (first[:, None] + torch.minimum(ar(most), n[:, None] - 1)).clamp(0, st["total"] - 1)
    q = st["q"][row].float().view(B, most, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    pos = torch.minimum(ar(max(st["lens_host"])), lens[:, None] - 1)
    b = ar(B)[:, None]
    k = _values(st, "k", b, pos).transpose(1, 2)[:, :, None]  # [B][H][1][L][128]
    v = _values(st, "v", b, pos).transpose(1, 2)[:, :, None]
    at = start[:, None] + ar(most)
    seen = (ar(pos.shape[1]) <= torch.minimum(at, lens[:, None] - 1)[..., None])[:, None, None]
    s = torch.matmul(q, k.transpose(-1, -2))
    del k
    s *= st["sm_scale"]
    out, lse = _softmax_values(s, seen, v)
    bb, at = _rows(st)
    i = at - start[bb]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, most, hq, D)[bb, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, most, hq)[bb, i]
    return out.to(torch.bfloat16), lse


# ------------------------------------------------------------------------------ one pass

_WORKSPACES = {}  # one workspace for each (operation, size), as a serving loop keeps


def _handles(st):
    """The descriptor, the cache's handle and the workspace that a user's program keeps."""
    from kv_cache_int8_gb300 import hsa
    d = hsa.Dims(batch=len(st["lens_host"]), hq=st["hq"], hkv=st["hkv"],
                 max_pages_per_seq=st["table"].shape[1], num_pages=st["k"].shape[0],
                 k2=st["k2"], sink=st["sink"], window=st["window"])
    cache = hsa.KV8(st["k"], st["v"], st["k_scale"], st["v_scale"])
    ws = None
    if st["op"] in ("decode", "prefill"):
        op = hsa.HSA_OP_KV8_DECODE if st["op"] == "decode" else hsa.HSA_OP_KV8_PREFILL
        key = (op, hsa.hsa_workspace_bytes(d, op))
        ws = _WORKSPACES.get(key)
        if ws is None:
            ws = _WORKSPACES[key] = hsa.workspace(d, op)
    return hsa, d, cache, ws


def run(state):
    st = state
    op = st["op"]
    if own:
        if "handles" not in st:
            st["handles"] = _handles(st)
        hsa, d, cache, ws = st["handles"]
        if op == "write":
            hsa.hsa_kv8_write(d, cache, st["k_new"], st["v_new"], st["cu"], st["table"],
                              st["lens"])
            return st["k"], st["v"], st["k_scale"], st["v_scale"]
        if op == "read":
            hsa.hsa_kv8_read(d, cache, st["k_out"], st["v_out"], st["cu"], st["table"],
                             st["lens"])
            return st["k_out"], st["v_out"]
        if op == "decode" and st["kind"] == "dense":
            hsa.hsa_kv8_decode(d, cache, st["q"], st["table"], st["lens"], st["out"], st["lse"],
                               ws)
        elif op == "decode":
            hsa.hsa_kv8_attend(d, cache, st["q"], st["table"], st["lens"], st["block_idx"],
                               st["n_blocks"], st["out"], st["lse"], ws)
        else:
            hsa.hsa_kv8_prefill(d, cache, st["q"], st["cu"], st["table"], st["lens"], st["out"],
                                st["lse"], ws)
        return st["out"], st["lse"]
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode,
            "prefill": _plain_prefill}[op](st)


# ------------------------------------------------------------------------------ the work

def work(case):
    lens, new = _lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], sum(new)
    block = hkv * (PAGE * D + 4)  # bytes of one block of all heads, K or V, with its scale
    meta = 4 * (sum(-(-n // PAGE) for n in lens) + 2 * len(lens))
    if case["op"] == "write":
        # new rows in, their codes out; a block's scale in and out
        blocks = sum((m - 1) // PAGE - (m - k) // PAGE + 1 for m, k in zip(lens, new))
        return dict(bytes=2 * T * hkv * D * 3 + 2 * blocks * hkv * 8 + 8 * len(lens),
                    flops=2 * T * hkv * D * 3)
    if case["op"] == "read":
        return dict(bytes=2 * T * hkv * (D * 3) + 2 * T * hkv * 4 // PAGE, flops=2 * T * hkv * D)
    if case["op"] == "decode":
        if case["kind"] == "dense":
            tokens = [n * hkv for n in lens]
            blocks = sum(-(-n // PAGE) for n in lens)
        else:
            got = []
            for n in lens:
                lo, hi = case["sink"] // PAGE, -(-max(n - case["window"], 0) // PAGE)
                got.append(min(n, case["sink"] + case["window"] +
                               PAGE * min(case["k2"], max(hi - lo, 0))))
            tokens = [g * hkv for g in got]
            blocks = sum(-(-g // PAGE) for g in got)
            meta = 8 * blocks
        return dict(bytes=2 * blocks * block + meta + len(lens) * hq * (2 * D + 4 * D + 4),
                    flops=4 * D * (hq // hkv) * sum(tokens))
    # prefill: each row against the tokens up to its own
    seen = sum(k * (n - k) + k * (k + 1) // 2 for n, k in zip(lens, new))
    return dict(bytes=2 * sum(-(-n // PAGE) for n in lens) * block + meta +
                T * hq * (2 * D + 2 * D + 4), flops=4 * D * hq * seen)


# ---------------------------------------------------------------------- values in 64 bits

def _as_f32(x):
    """Each value of x (64 bits) rounded to fp32, in 64 bits."""
    return x.to(torch.float32).to(torch.float64)


def _e4m3(x):
    """Each value of x (64 bits, at most 448 in magnitude) rounded to E4M3, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def _exact_write(st):
    fmt, levels = st["fmt"], LEVELS[st["fmt"]]
    at = 0
    for b, (N, n) in enumerate(zip(st["lens_host"], st["new_host"])):
        first = N - n
        for name in ("k", "v"):
            store, scale = st[name], st[name + "_scale"]
            x = st[name + "_new"][at:at + n].double()  # [n][H][128]
            lo, hi = first // PAGE, (N - 1) // PAGE + 1
            pages = st["table"][b, lo:hi].long()
            full = torch.zeros((hi - lo) * PAGE, st["hkv"], D, dtype=torch.float64, device="cuda")
            full[first - lo * PAGE:first - lo * PAGE + n] = x
            full = full.view(hi - lo, PAGE, st["hkv"], D).transpose(1, 2)
            s = _as_f32(full.abs().amax((-2, -1)) / levels)
            s[s < TINY] = 0.0
            had = scale[pages].double()
            codes = (store.view(torch.int8)[pages].view(store.dtype)).float().double()
            if first % PAGE:
                s[0] = torch.maximum(s[0], had[0])
            inv = torch.where(s > 0, _as_f32(1.0 / s.clamp(min=TINY)), 0.0)[..., None, None]
            y = _as_f32(full * inv).clamp(-levels, levels)
            moved = _as_f32(codes * _as_f32(had[..., None, None] * inv))
            y, moved = (torch.round(t) if fmt == "int8" else _e4m3(t) for t in (y, moved))
            moved = torch.where((s > had)[..., None, None], moved, codes)
            slot = torch.arange(lo * PAGE, hi * PAGE, device="cuda").view(hi - lo, 1, PAGE, 1)
            y = torch.where(slot < first, moved, torch.where(slot < N, y, codes))
            back = y.float().to(store.dtype)
            store.view(torch.int8)[pages] = back.view(torch.int8)
            scale[pages] = s.float()
        at += n
    return st["k"], st["v"], st["k_scale"], st["v_scale"]


def _exact_tokens(st, name, b, lo, hi):
    """Values of tokens [lo, hi) of sequence b in 64 bits: [H][hi - lo][128]."""
    p0, p1 = lo // PAGE, -(-hi // PAGE)
    pages = st["table"][b, p0:p1].long()
    c = st[name].view(torch.int8)[pages].view(st[name].dtype).float().double()
    c *= st[name + "_scale"][pages].double()[..., None, None]
    c = c.transpose(0, 1).reshape(st["hkv"], -1, D)
    return c[:, lo - p0 * PAGE:hi - p0 * PAGE]


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "write":
        return _exact_write(st)
    hkv, G = st["hkv"], st["hq"] // st["hkv"]
    if st["op"] == "read":
        out = [torch.cat([_exact_tokens(st, name, b, N - n, N).transpose(0, 1)
                          for b, (N, n) in enumerate(zip(st["lens_host"], st["new_host"]))])
               for name in ("k", "v")]
        return out[0], out[1]
    outs, sums = [], []
    at = 0
    for b, (N, n) in enumerate(zip(st["lens_host"], st["new_host"])):
        q = st["q"][at:at + n].double().view(n, hkv, G, D).permute(1, 2, 0, 3)  # [H][G][n][128]
        at += n
        k, v = _exact_tokens(st, "k", b, 0, N), _exact_tokens(st, "v", b, 0, N)
        o = torch.empty(n, hkv, G, D, dtype=torch.float64, device="cuda")
        z = torch.empty(n, hkv, G, dtype=torch.float64, device="cuda")
        allowed = None
        if st["kind"] == "kept":
            t = torch.arange(N, device="cuda")
            allowed = ((t < st["sink"]) | (t >= N - st["window"])).repeat(hkv, 1)
            for h in range(hkv):
                keep = st["block_idx"][b, h, :int(st["n_blocks"][b, h])].long()
                inside = torch.zeros(-(-N // PAGE), dtype=torch.bool, device="cuda")
                inside[keep] = True
                allowed[h] |= inside[t // PAGE]
        for i in range(0, n, 512):
            j = min(n, i + 512)
            end = N - n + j
            logit = q[:, :, i:j] @ k[:, None, :end].transpose(-1, -2) * st["sm_scale"]
            where = torch.arange(N - n + i, N - n + j, device="cuda")[:, None]
            hide = torch.arange(end, device="cuda")[None] > where
            if allowed is not None:
                hide = hide[None, None] | ~allowed[:, None, None]
            logit.masked_fill_(hide, -math.inf)
            top = logit.amax(-1, keepdim=True)
            logit.sub_(top).exp_()
            total = logit.sum(-1, keepdim=True)
            o[i:j] = ((logit @ v[:, None, :end]) / total).permute(2, 0, 1, 3)
            z[i:j] = (top + torch.log(total))[..., 0].permute(2, 0, 1)
        outs.append(o.view(n, hkv * G, D))
        sums.append(z.view(n, hkv * G))
    return torch.cat(outs), torch.cat(sums)
