"""The operators of drafted tokens on the 8-bit K/V cache, as measured work: inputs, plain forms,
exact values.

A step that verifies drafted tokens puts positions on the new queries and keys, writes keys and
values into the cache, attends each drafted token to the context and to its own branch, and moves
the accepted branch into place. Four operators:

  rotate  rotary positions on rows of queries and keys (bf16 in, bf16 out): pairs of channels
          (i, i + r / 2), or neighbours, in the first r channels of a head, turned by the angles
          of a table of cosines and sines (frequencies scaled for long contexts)
  append  the same on the way into the cache: queries turned, keys turned and quantised, values
          quantised (their blocks' values are read back after it)
  tree    attention of drafted tokens: node i of a sequence sees the context in front of the
          drafted tokens, itself and its ancestors
  keep    the accepted nodes' keys and values move to the places behind the context, re-quantised
          under their new blocks' scales, and the sequences get their new lengths (the values of
          the blocks concerned are read back after it)

``own`` chooses between the plain form (elementary torch operations) and the framework's kernels.
Sizes follow the decode configurations of kv_cache_int8_gb300.workloads (32 or 64 query heads over
8 kv heads, 4 over 1; 8K to 128K tokens, permuted page pools).
"""
import math

import torch

own = False

PAGE, D = 16, 128
TINY = 2.0 ** -126  # scales below the smallest normal number count as zero
LEVELS = {"int8": 127.0, "e4m3": 448.0}
CONTEXT = 131072  # rows of a rotary table


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a long chat: the new token's queries and keys
        dict(name="rotate-step", op="rotate", batch=1, hq=32, hkv=8, lo=131000, hi=131000, new_lo=1,
             new_hi=1, rot=128, pairs="halves", tree=False),
        # long prompts and continued chats on arrival; half of each head, neighbouring channels
        dict(name="rotate-prompts", op="rotate", batch=8, hq=32, hkv=8, lo=9000, hi=23000,
             new_lo=8001, new_hi=22777, rot=64, pairs="neighbours", tree=False),
        # the newest token of a 128K context joins the cache
        dict(name="append-step", op="append", fmt="int8", batch=1, hq=32, hkv=8, lo=131000,
             hi=131000, new_lo=1, new_hi=1, rot=128, pairs="halves", tree=False),
        # one step of a serving batch at mixed positions inside their blocks
        dict(name="append-batch", op="append", fmt="e4m3", batch=256, hq=32, hkv=8, lo=300,
             hi=5000, new_lo=1, new_hi=1, rot=128, pairs="neighbours", tree=False),
        # drafted trees of a batch of chats: positions are depths, groups of 8 query heads
        dict(name="append-trees", op="append", fmt="e4m3", batch=64, hq=64, hkv=8, lo=300,
             hi=5000, new_lo=9, new_hi=33, rot=64, pairs="halves", tree=True),
        # a batch of long prompts (and continued chats, starting inside a block) on arrival
        dict(name="append-prompts", op="append", fmt="int8", batch=8, hq=32, hkv=8, lo=9000,
             hi=23000, new_lo=8001, new_hi=22777, rot=128, pairs="halves", tree=False),
        # the tiny configuration with eight drafted tokens: latency of a single call
        dict(name="tree-tiny", op="tree", fmt="int8", batch=1, hq=4, hkv=1, lo=8192, hi=8192,
             new_lo=8, new_hi=8, tree=True),
        # drafted trees of a few chats verified together, odd sizes
        dict(name="tree-chats", op="tree", fmt="int8", batch=4, hq=32, hkv=8, lo=6000, hi=12000,
             new_lo=5, new_hi=33, tree=True),
        # one drafted tree behind a 128K context
        dict(name="tree-long", op="tree", fmt="e4m3", batch=1, hq=32, hkv=8, lo=131072, hi=131072,
             new_lo=25, new_hi=25, tree=True),
        # the batched configuration: eight sequences of 32K to 128K tokens, groups of 8
        dict(name="tree-batch", op="tree", fmt="int8", batch=8, hq=64, hkv=8, lo=32768, hi=131072,
             new_lo=6, new_hi=17, tree=True),
        # the accepted branch of a single chat
        dict(name="keep-step", op="keep", fmt="int8", batch=1, hq=32, hkv=8, lo=8191, hi=8191,
             new_lo=25, new_hi=25, tree=True),
        # the accepted branches of a serving batch, large and small trees
        dict(name="keep-batch", op="keep", fmt="e4m3", batch=256, hq=32, hkv=8, lo=300, hi=5000,
             new_lo=9, new_hi=64, tree=True),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "tree", "tree", "tree", "keep"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    c = dict(op=op, hq=hkv * group, hkv=hkv, tree=op in ("tree", "keep") or rng.random() < 0.3)
    if op != "rotate":
        c["fmt"] = rng.choice(["int8", "e4m3"])
    if op in ("rotate", "append"):
        c["rot"] = rng.choice([32, 64, 96, 128])
        c["pairs"] = rng.choice(["halves", "neighbours"])
        c["batch"] = _log(rng, 1, 256)
        # tokens a sequence: at most the rows of the listed prompts
        most = max(64, 120000 * 40 // (max(40, c["hq"] + hkv) * c["batch"]))
        c["hi"] = _log(rng, 17, most)
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.3, 1.0)))
        c["new_hi"] = (_log(rng, 1, min(64, c["hi"])) if c["tree"] else
                       1 if rng.random() < 0.4 else _log(rng, 1, c["hi"]))
    else:
        c["batch"] = _log(rng, 1, 64 if op == "tree" else 256)
        c["hi"] = _log(rng, 65, min(131072, 500000 // c["batch"]))
        c["lo"] = max(65, int(c["hi"] * rng.uniform(0.3, 1.0)))
        # at most the products of the batched configuration, padded sequences included
        most = 8 * 131072 * 64 * 17 / (c["batch"] * c["hi"] * c["hq"])
        c["new_hi"] = _log(rng, 1, 64 if op == "keep" else max(1, min(64, int(most))))
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


def _table(rot):
    """Cosines, then sines, of every position's angles [CONTEXT][rot] fp32 (angles in 64 bits).
    Frequencies of base 500000; those that turn less than once in 8192 positions are 8 times
    slower, those that turn more than 4 times unchanged, with a blend in between."""
    f = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    blend = ((8192.0 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
    f = f * (blend + (1.0 - blend) / 8.0)
    a = torch.arange(CONTEXT, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def _kept(new):
    """Accepted nodes of each sequence: 0 to 8, as far as there are so many."""
    return [min(n, (b * 5 + 4) % 9) for b, n in enumerate(new)]


def _trees(new, gen):
    """Parents of every sequence's nodes: node 0 hangs on the context (-1), node i on one of the
    nodes in front of it, each as likely (about ln n deep)."""
    u = torch.rand(sum(new), generator=gen, device="cuda").tolist()
    parents, depths, at = [], [], 0
    for n in new:
        p = [-1] + [min(int(u[at + i] * i), i - 1) for i in range(1, n)]
        d = []
        for i in range(n):
            d.append(0 if p[i] < 0 else d[p[i]] + 1)
        parents.append(p)
        depths.append(d)
        at += n
    return parents, depths


def _offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, hq, hkv, op = case["batch"], case["hq"], case["hkv"], case["op"]
    lens, new = _lengths(case)
    cu = _offsets(new)
    T = cu[-1]
    i32 = dict(dtype=torch.int32, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    st = dict(op=op, hq=hq, hkv=hkv, lens=torch.tensor(lens, **i32), lens_host=lens, new_host=new,
              total=T, sm_scale=1.0 / math.sqrt(D))
    # one new token a sequence needs no offsets: row b is sequence b's token
    st["cu"] = None if max(new) == 1 and min(new) == 1 else torch.tensor(cu, **i32)
    depths = None
    if case["tree"] and op != "keep":
        parents, depths = _trees(new, gen)
        st["parents"] = torch.tensor([p for t in parents for p in t], **i32)
        st["parents_host"] = parents
    if op in ("rotate", "append"):
        st["rot"], st["neighbours"] = case["rot"], case["pairs"] == "neighbours"
        st["table"] = _table(case["rot"])
        st["positions"] = None
        if case["tree"]:
            st["positions"] = torch.tensor(
                [N - n + d for N, n, t in zip(lens, new, depths) for d in t], **i32)
        # queries, keys and values as slices of one projection's output [tokens][hq + 2 hkv][128]
        qkv = torch.empty(T, hq + 2 * hkv, D, **bf16)
        for t in range(0, T, 65536):
            n = min(65536, T - t)
            qkv[t:t + n] = torch.randn(n, hq + 2 * hkv, D, generator=gen, device="cuda")
        st["q"], st["k_new"], st["v_new"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["q_out"] = torch.empty(T, hq, D, **bf16)
        if op == "rotate":
            st["k_out"] = torch.empty(T, hkv, D, **bf16)
            return st
    st["fmt"] = case["fmt"]
    per = [-(-n // PAGE) for n in lens]
    pool = torch.randperm(sum(per), generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max(per)), -1, **i32)
    off = 0
    for b, p in enumerate(per):
        table[b, :p] = pool[off:off + p]
        off += p
    st["pages"] = table
    for name in ("k", "v"):
        codes = torch.empty(sum(per), hkv, PAGE, D, device="cuda",
                            dtype=torch.int8 if st["fmt"] == "int8" else torch.float8_e4m3fn)
        scale = torch.empty(sum(per), hkv, device="cuda")
        for p in range(0, sum(per), 4096):
            n = min(4096, sum(per) - p)
            codes[p:p + n], scale[p:p + n] = _quantise(_blocks(n, hkv, gen, name == "k"),
                                                       st["fmt"])
        st[name], st[name + "_scale"] = codes, scale
    if op == "tree":
        st["q"] = torch.randn(T, hq, D, generator=gen, device="cuda").to(torch.bfloat16)
        st["out"] = torch.empty(T, hq, D, **bf16)
        st["lse"] = torch.empty(T, hq, device="cuda")
        return st
    kept = new
    if op == "keep":
        # branches of the lengths that the case fixes: node 0 and later nodes, ascending
        kept = _kept(new)
        paths = []
        for n, m in zip(new, kept):
            more = torch.rand(n - 1, generator=gen, device="cuda").argsort()[:max(m - 1, 0)]
            paths.append([0] * (m > 0) + sorted(1 + i for i in more.tolist()))
        most = max(max(kept), 1)
        st["keep_idx"] = torch.tensor([p + [-1] * (most - len(p)) for p in paths], **i32)
        st["n_keep"] = torch.tensor(kept, **i32)
        st["paths_host"] = paths
        st["new_lens"] = torch.empty(B, **i32)
    # read back: the blocks that receive tokens, from their first slot on
    ends = [N - n + m for N, n, m in zip(lens, new, kept)]
    back = [(N - n) % PAGE + m for N, n, m in zip(lens, new, kept)]
    st["ends"] = torch.tensor(ends, **i32)
    st["ends_host"], st["kept_host"] = ends, kept
    st["cu_back"] = torch.tensor(_offsets(back), **i32)
    st["back_host"] = back
    st["total_back"] = sum(back)
    st["k_back"] = torch.empty(sum(back), hkv, D, **bf16)
    st["v_back"] = torch.empty(sum(back), hkv, D, **bf16)
    return st


# --------------------------------------------------------------------------- plain form

def _span(lens, cu):
    """(first new position, number of new tokens, first row) of each sequence."""
    lens = lens.long()
    if cu is None:
        return lens - 1, torch.ones_like(lens), torch.arange(lens.numel(), device="cuda")
    cu = cu.long()
    n = cu[1:] - cu[:-1]
    return lens - n, n, cu[:-1]


def _rows(lens, cu, total):
    """(sequence, position) of every row."""
    start, _, first = _span(lens, cu)
    r = torch.arange(total, device="cuda")
    b = torch.searchsorted(first.contiguous(), r, right=True) - 1
    return b, start[b] + r - first[b]


def _turn(st, x):
    """Rows x [tokens][heads][128] with their positions on, fp32."""
    r = st["rot"]
    pos = st["positions"]
    pos = _rows(st["lens"], st["cu"], st["total"])[1] if pos is None else pos.long()
    cs = st["table"][pos]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    x = x.float()
    if st["neighbours"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_store(st, start, n, src, x, codes, scale):
    """Quantises rows src [B][most] of x (fp32) into positions start .. start + n of each
    sequence."""
    B, most = src.shape
    levels, fmt = LEVELS[st["fmt"]], st["fmt"]
    end = start + n
    ar = lambda m: torch.arange(m, device="cuda")  # noqa: E731
    touched = (most + PAGE - 2) // PAGE + 1
    # a sequence with fewer blocks than the others repeats its last one (the same values); one
    # that receives nothing repeats the block in front of its end, where nothing changes
    last = (end - 1).clamp(min=0) // PAGE
    p = torch.minimum(start[:, None] // PAGE + ar(touched), last[:, None])
    page = torch.gather(st["pages"].long(), 1, p)
    pos = p[..., None] * PAGE + ar(PAGE)  # [B][J][16]
    fresh = (pos >= start[:, None, None]) & (pos < end[:, None, None])
    stale = pos < start[:, None, None]
    at = (pos - start[:, None, None]).clamp(0, most - 1)
    x = x[torch.gather(src, 1, at.flatten(1)).view(at.shape)].transpose(2, 3)  # [B][J][H][16][128]
    new = fresh[:, :, None, :, None]
    finite = torch.where(new & torch.isfinite(x), x.abs(), torch.zeros_like(x))
    amax = finite.amax((-2, -1))
    s_new = amax / torch.full_like(amax, levels)
    s_new = torch.where(s_new < TINY, torch.zeros_like(s_new), s_new)
    s_old = scale[page]
    s = torch.where(stale.any(-1)[..., None], torch.maximum(s_old, s_new), s_new)
    s = torch.where(fresh.any(-1)[..., None], s, s_old)
    inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))[..., None, None]
    was = codes.view(torch.int8)[page]
    ratio = s_old[..., None, None] * inv
    y = torch.where(torch.isnan(x), torch.zeros_like(x), x * inv)
    y = torch.where(torch.isnan(y), torch.zeros_like(y), y).clamp(-levels, levels)
    if fmt == "int8":
        put = y.round().to(torch.int8)
        moved = (was.float() * ratio).round().to(torch.int8)
    else:
        put = y.to(torch.float8_e4m3fn).view(torch.int8)
        moved = (was.view(torch.float8_e4m3fn).float() * ratio).to(
            torch.float8_e4m3fn).view(torch.int8)
    old = stale[:, :, None, :, None] & (s > s_old)[..., None, None]
    codes.view(torch.int8)[page] = torch.where(new, put, torch.where(old, moved, was))
    scale[page] = s


def _values(st, name, b, pos):
    """fp32 values of tokens (b, pos) for every kv head: [..][H][128]."""
    page = st["pages"].long()[b, pos // PAGE]
    codes = st[name].view(torch.int8)[page, :, pos % PAGE].view(st[name].dtype)
    return codes.float() * st[name + "_scale"][page][..., None]


def _plain_back(st):
    b, pos = _rows(st["ends"], st["cu_back"], st["total_back"])
    st["k_back"].copy_(_values(st, "k", b, pos))
    st["v_back"].copy_(_values(st, "v", b, pos))


def _plain_rotate(st):
    st["q_out"].copy_(_turn(st, st["q"]))
    st["k_out"].copy_(_turn(st, st["k_new"]))
    return st["q_out"], st["k_out"]


def _plain_append(st):
    st["q_out"].copy_(_turn(st, st["q"]))
    start, n, first = _span(st["lens"], st["cu"])
    src = first[:, None] + torch.arange(max(st["new_host"]), device="cuda")
    src = src.clamp(max=st["total"] - 1)
    _plain_store(st, start, n, src, _turn(st, st["k_new"]), st["k"], st["k_scale"])
    _plain_store(st, start, n, src, st["v_new"].float(), st["v"], st["v_scale"])
    _plain_back(st)
    return st["q_out"], st["k_back"], st["v_back"]


def _plain_keep(st):
    start, _, _ = _span(st["lens"], st["cu"])
    n = st["n_keep"].long()
    idx = st["keep_idx"].long()
    b = torch.arange(idx.shape[0], device="cuda")[:, None]
    pos = (start[:, None] + idx).clamp(min=0)
    src = torch.arange(idx.numel(), device="cuda").view(idx.shape)
    k = _values(st, "k", b, pos).flatten(0, 1)
    v = _values(st, "v", b, pos).flatten(0, 1)
    _plain_store(st, start, n, src, k, st["k"], st["k_scale"])
    _plain_store(st, start, n, src, v, st["v"], st["v_scale"])
    st["new_lens"].copy_(start + n)
    _plain_back(st)
    return st["k_back"], st["v_back"], st["new_lens"]


def _seen_nodes(st, first, n, most):
    """[B][node][node]: whether the second is the first or one of its ancestors."""
    i = torch.arange(most, device="cuda")
    up = st["parents"].long()[(first[:, None] + i).clamp(max=st["total"] - 1)]
    up = torch.where(i < n[:, None], up, torch.full_like(up, -1))
    m = ((up[..., None] == i) | (i[:, None] == i)).float()
    twice = lambda a: (a @ a).clamp(max=1.0)  # noqa: E731  (paths twice as long)
    return twice(twice(twice(twice(twice(twice(m)))))) > 0


def _plain_tree(st):
    start, n, first = _span(st["lens"], st["cu"])
    B, hq, hkv = start.numel(), st["hq"], st["hkv"]
    ar = lambda m: torch.arange(m, device="cuda")  # noqa: E731
    lens, most = st["lens"].long(), max(st["new_host"])
    row = (first[:, None] + torch.minimum(ar(most), n[:, None] - 1)).clamp(0, st["total"] - 1)
    q = st["q"][row].float().view(B, most, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    every = ar(max(st["lens_host"]))
    pos = torch.minimum(every, lens[:, None] - 1)
    b = ar(B)[:, None]
    k = _values(st, "k", b, pos).transpose(1, 2)[:, :, None]  # [B][H][1][L][128]
    v = _values(st, "v", b, pos).transpose(1, 2)[:, :, None]
    node = every - start[:, None]  # [B][L]
    reach = _seen_nodes(st, first, n, most)
    own_branch = torch.gather(reach, 2, node.clamp(0, most - 1)[:, None].expand(-1, most, -1))
    seen = ((node < 0)[:, None] | (own_branch & (node < n[:, None])[:, None]))[:, None, None]
    s = torch.matmul(q, k.transpose(-1, -2))
    del k
    s *= st["sm_scale"]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    s = torch.exp(s - top)
    total = s.sum(-1, keepdim=True)
    out = torch.matmul(s, v) / total
    lse = (top + torch.log(total))[..., 0]
    bb, at = _rows(st["lens"], st["cu"], st["total"])
    i = at - start[bb]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, most, hq, D)[bb, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, most, hq)[bb, i]
    return out.to(torch.bfloat16), lse


# ------------------------------------------------------------------------------ one pass

_WORKSPACES = {}  # one workspace for each size, as a serving loop keeps


def _handles(st):
    """The descriptor, the handles of the cache and of the rotary table, and the workspace that a
    user's program keeps."""
    from kv_cache_int8_gb300 import hsa
    pages = st.get("pages")
    d = hsa.Dims(batch=len(st["lens_host"]), hq=st["hq"], hkv=st["hkv"],
                 max_pages_per_seq=1 if pages is None else pages.shape[1],
                 num_pages=1 if pages is None else st["k"].shape[0])
    cache = None if pages is None else hsa.KV8(st["k"], st["v"], st["k_scale"], st["v_scale"])
    rotary = hsa.Rotary(st["table"], neighbours=st["neighbours"]) if "table" in st else None
    ws = None
    if st["op"] == "tree":
        size = hsa.hsa_workspace_bytes(d, hsa.HSA_OP_KV8_TREE)
        ws = _WORKSPACES.get(size)
        if ws is None:
            ws = _WORKSPACES[size] = hsa.workspace(d, hsa.HSA_OP_KV8_TREE)
    return hsa, d, cache, rotary, ws


def run(state):
    st = state
    op = st["op"]
    if own:
        if "handles" not in st:
            st["handles"] = _handles(st)
        hsa, d, cache, rotary, ws = st["handles"]
        if op == "rotate":
            hsa.hsa_rotate(d, rotary, st["q"], st["q_out"], st["k_new"], st["k_out"],
                           st["positions"], st["cu"], st["lens"])
            return st["q_out"], st["k_out"]
        if op == "tree":
            hsa.hsa_kv8_tree(d, cache, st["q"], st["parents"], st["cu"], st["pages"], st["lens"],
                             st["out"], st["lse"], ws)
            return st["out"], st["lse"]
        if op == "append":
            hsa.hsa_kv8_write_rotated(d, cache, rotary, st["q"], st["q_out"], st["k_new"],
                                      st["v_new"], st["positions"], st["cu"], st["pages"],
                                      st["lens"])
            hsa.hsa_kv8_read(d, cache, st["k_back"], st["v_back"], st["cu_back"], st["pages"],
                             st["lens"])
            return st["q_out"], st["k_back"], st["v_back"]
        hsa.hsa_kv8_keep(d, cache, st["keep_idx"], st["n_keep"], st["cu"], st["pages"],
                         st["lens"], st["new_lens"])
        hsa.hsa_kv8_read(d, cache, st["k_back"], st["v_back"], st["cu_back"], st["pages"],
                         st["new_lens"])
        return st["k_back"], st["v_back"], st["new_lens"]
    return {"rotate": _plain_rotate, "append": _plain_append, "tree": _plain_tree,
            "keep": _plain_keep}[op](st)


# ------------------------------------------------------------------------------ the work

def work(case):
    lens, new = _lengths(case)
    hq, hkv, T, op = case["hq"], case["hkv"], sum(new), case["op"]
    if op == "rotate":
        return dict(bytes=T * (hq + hkv) * D * 4 + T * case["rot"] * 4 + 8 * len(lens),
                    flops=3 * T * (hq + hkv) * case["rot"])
    blocks = sum((m - 1) // PAGE - (m - k) // PAGE + 1 for m, k in zip(lens, new))
    if op == "append":
        # rows in, queries and codes out, a block's scale in and out; the blocks read back
        back = sum((m - k) % PAGE + k for m, k in zip(lens, new))
        return dict(bytes=T * (hq * 4 + hkv * 6) * D + T * case["rot"] * 4 + 2 * blocks * hkv * 8 +
                    2 * back * hkv * D * 3 + 8 * len(lens),
                    flops=3 * T * (hq + hkv) * case["rot"] + 6 * T * hkv * D)
    if op == "keep":
        # the branches' codes in and out, scales; the blocks read back
        kept = _kept(new)
        back = sum((m - n) % PAGE + a for m, n, a in zip(lens, new, kept))
        return dict(bytes=2 * hkv * (sum(kept) * 2 * D + back * 3 * D + 12 * len(lens)),
                    flops=2 * hkv * D * (3 * sum(kept) + back))
    # tree: every node against the context and about ln n + 1 nodes
    blocks = sum(-(-n // PAGE) for n in lens)
    seen = sum(k * (n - k + math.log(k) + 1) for n, k in zip(lens, new))
    return dict(bytes=2 * blocks * hkv * (PAGE * D + 4) + 4 * (blocks + T + 2 * len(lens)) +
                T * hq * (4 * D + 4), flops=4 * D * hq * seen)


# ---------------------------------------------------------------------- values in 64 bits

def _as_f32(x):
    """Each value of x (64 bits) rounded to fp32, in 64 bits."""
    return x.to(torch.float32).to(torch.float64)


def _e4m3(x):
    """Each value of x (64 bits, at most 448 in magnitude) rounded to E4M3, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def _exact_turn(st, x, at, first, rounded):
    """Rows x of one sequence (64 bits, first row `at`, first position `first`) turned; with
    `rounded` every operation rounds to fp32, as the codes' definition has it."""
    r, n = st["rot"], x.shape[0]
    to = _as_f32 if rounded else (lambda t: t)
    pos = (torch.arange(first, first + n, device="cuda") if st["positions"] is None else
           st["positions"][at:at + n].long())
    cos = st["table"][pos, :r // 2].double()[:, None]
    sin = st["table"][pos, r // 2:].double()[:, None]
    i = torch.arange(r // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if st["neighbours"] else (i, i + r // 2)
    y = x.clone()
    y[..., ia] = to(to(x[..., ia] * cos) - to(x[..., ib] * sin))
    y[..., ib] = to(to(x[..., ib] * cos) + to(x[..., ia] * sin))
    return y


def _exact_store(st, name, b, first, x):
    """Rows x [n][H][128] (64 bits) into positions first .. first + n of sequence b."""
    n, fmt, levels = x.shape[0], st["fmt"], LEVELS[st["fmt"]]
    if n == 0:
        return
    store, scale = st[name], st[name + "_scale"]
    lo, hi = first // PAGE, (first + n - 1) // PAGE + 1
    pages = st["pages"][b, lo:hi].long()
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
    y = torch.where(slot < first, moved, torch.where(slot < first + n, y, codes))
    store.view(torch.int8)[pages] = y.float().to(store.dtype).view(torch.int8)
    scale[pages] = s.float()


def _exact_tokens(st, name, b, lo, hi):
    """Values of tokens [lo, hi) of sequence b in 64 bits: [H][hi - lo][128]."""
    p0, p1 = lo // PAGE, -(-hi // PAGE)
    pages = st["pages"][b, p0:p1].long()
    c = st[name].view(torch.int8)[pages].view(st[name].dtype).float().double()
    c *= st[name + "_scale"][pages].double()[..., None, None]
    c = c.transpose(0, 1).reshape(st["hkv"], -1, D)
    return c[:, lo - p0 * PAGE:hi - p0 * PAGE]


def _exact_back(st, name):
    return torch.cat([_exact_tokens(st, name, b, N - n, N).transpose(0, 1)
                      for b, (N, n) in enumerate(zip(st["ends_host"], st["back_host"]))])


def exact(case, seed):
    st = prepare(case, seed)
    spans = list(enumerate(zip(st["lens_host"], st["new_host"], _offsets(st["new_host"]))))
    if st["op"] == "rotate":
        return tuple(torch.cat([_exact_turn(st, st[name][at:at + n].double(), at, N - n, False)
                                for _, (N, n, at) in spans]) for name in ("q", "k_new"))
    if st["op"] == "append":
        q = torch.cat([_exact_turn(st, st["q"][at:at + n].double(), at, N - n, False)
                       for _, (N, n, at) in spans])
        for b, (N, n, at) in spans:
            k = _exact_turn(st, st["k_new"][at:at + n].double(), at, N - n, True)
            _exact_store(st, "k", b, N - n, k)
            _exact_store(st, "v", b, N - n, st["v_new"][at:at + n].double())
        return q, _exact_back(st, "k"), _exact_back(st, "v")
    if st["op"] == "keep":
        for b, (N, n, _) in spans:
            path = torch.tensor(st["paths_host"][b], dtype=torch.long, device="cuda")
            for name in ("k", "v"):
                x = _as_f32(_exact_tokens(st, name, b, N - n, N)[:, path].transpose(0, 1))
                _exact_store(st, name, b, N - n, x)
        return _exact_back(st, "k"), _exact_back(st, "v"), st["ends"]
    hkv, G = st["hkv"], st["hq"] // st["hkv"]
    outs, sums = [], []
    for b, (N, n, at) in spans:
        q = st["q"][at:at + n].double().view(n, hkv, G, D).permute(1, 2, 0, 3)  # [H][G][n][128]
        k, v = _exact_tokens(st, "k", b, 0, N), _exact_tokens(st, "v", b, 0, N)
        hide = torch.ones(n, n, dtype=torch.bool)
        for i, p in enumerate(st["parents_host"][b]):
            if p >= 0:
                hide[i] = hide[p]
            hide[i, i] = False
        logit = q @ k[:, None].transpose(-1, -2) * st["sm_scale"]
        logit[..., N - n:].masked_fill_(hide.cuda(), -math.inf)
        top = logit.amax(-1, keepdim=True)
        logit.sub_(top).exp_()
        total = logit.sum(-1, keepdim=True)
        o = (logit @ v[:, None]) / total
        outs.append(o.permute(2, 0, 1, 3).reshape(n, hkv * G, D))
        sums.append((top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(n, hkv * G))
    return torch.cat(outs), torch.cat(sums)
