"""Cases and plain forms of more operators around the compressed linear layers: the product in 8-bit
integers with a scale to each token and channel, rotary positions with several axes, and the pages of a
quantised K/V cache (given out, forked, taken back, compacted, and the accepted drafts' entries moved together).

`run(state)` computes an operator in elementary torch operations in 32 bits (`own` false) or through the
package's entry points (`own` true).  Widths and head layouts are those of this repository's layer sets:
4096 x 11008 (LLaMA-7B), 8192 -> 10240 and 8192 x 28672 (LLaMA-70B), 52 heads (6656).

Pages: `table` int32 [sequences, width] names each sequence's pages (-1 past its last one), `lens` int32
[sequences] its tokens, `refs` int32 [pages] how many sequences hold a page.  Free pages (refs 0) are given
out lowest first, to sequences in their order, at each to its places in order.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # qkv of one new token: the weights are read once, everything else is small
        dict(name="int8 1 token", op="int8", T=1, K=8192, N=10240, src="f16", dst="f32", clamp=0.0, bias=False),
        # up of a decode batch of 64 sequences
        dict(name="int8 decode batch", op="int8", T=64, K=8192, N=28672, src="bf16", dst="f32", clamp=0.0, bias=False),
        # down of a chunk of a prompt
        dict(name="int8 chunk", op="int8", T=256, K=28672, N=8192, src="bf16", dst="bf16", clamp=0.0, bias=False),
        # ragged sizes, the activations clamped on the way, fp32 in
        dict(name="int8 ragged", op="int8", T=777, K=4099, N=11005, src="f32", dst="f16", clamp=6.0, bias=True),
        # up of a prompt of 2048 tokens
        dict(name="int8 prompt", op="int8", T=2048, K=8192, N=28672, src="bf16", dst="bf16", clamp=0.0, bias=False),
        # q and k heads of one new token after an image, as the qkv layer leaves them (fp32)
        dict(name="axes 1 token", op="axes", T=1, hq=64, hkv=8, D=128, sections="16,24,24", order="blocks",
             layout="half", src="f32", dst="bf16"),
        # a prompt of text, an image and text: time, height and width take turns
        dict(name="axes prompt", op="axes", T=8192, hq=64, hkv=8, D=128, sections="24,20,20", order="turns",
             layout="half", src="bf16", dst="bf16"),
        # an image encoder's patches: height and width, heads of 80 channels
        dict(name="axes patches", op="axes", T=16383, hq=16, hkv=16, D=80, sections="20,20", order="blocks",
             layout="half", src="f16", dst="f16"),
        # one sequence's tree of 7 drafts: pages for it, the accepted path moved together, the rest taken back
        dict(name="pages step 1", op="step", B=1, n=7, L=500, width=64, pages=2000, page=16, heads=8, D=128, kind="int4"),
        # the same for 64 sequences of up to 8000 tokens with trees of 16
        dict(name="pages step 64", op="step", B=64, n=16, L=8000, width=160, pages=9000, page=64, heads=8, D=128,
             kind="int8"),
        # eight prompts with eight continuations each: pages shared but for the last, which is copied
        dict(name="pages fork", op="fork", B=64, n=8, L=8000, width=160, pages=2000, page=64, heads=32, D=128,
             kind="int8"),
        # a pool with many holes: its live pages moved to its start
        dict(name="pages compact", op="compact", B=96, n=4096, L=8000, width=128, pages=12000, page=64, heads=8, D=128,
             kind="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, half):
    """Pairs of 2, 3 or 4 axes, as text, and an order that they allow."""
    axes = rng.choice([2, 3, 3, 4])
    rest = [rng.randrange(1, max(2, half // axes)) for _ in range(axes - 1)]
    first = half - sum(rest)
    turns = all(a + 1 + axes * (s - 1) < half for a, s in enumerate(rest)) and rng.random() < 0.5
    return ",".join(str(v) for v in [first] + rest), "turns" if turns else "blocks"


def draw(rng):
    op = rng.choice(["int8", "int8", "int8", "axes", "axes", "step", "fork", "compact"])
    if op == "int8":
        K, N = _log(rng, 200, 28672), _log(rng, 200, 28672)
        if rng.random() < 0.6:
            K = -(-K // 128) * 128
        if rng.random() < 0.6:
            N = -(-N // 64) * 64
        T = max(1, min(_log(rng, 1, 8192), int(4.8e11 / (K * N))))
        return dict(op=op, T=T, K=K, N=N, src=rng.choice(["f32", "f16", "bf16"]), dst=rng.choice(["f32", "f16", "bf16"]),
                    clamp=rng.choice([0.0, 0.0, 4.0]), bias=rng.random() < 0.3)
    if op == "axes":
        hq, hkv = rng.choice([(32, 32), (64, 8), (52, 52), (16, 2), (16, 16)])
        D = rng.choice([64, 80, 128])
        sections, order = _sections(rng, rng.choice([D, D, D // 2]) // 2)
        return dict(op=op, T=_log(rng, 1, 8192), hq=hq, hkv=hkv, D=D, sections=sections, order=order,
                    layout=rng.choice(["half", "half", "interleaved"]), src=rng.choice(["f32", "f16", "bf16"]),
                    dst=rng.choice(["f16", "bf16"]))
    page = rng.choice([16, 32, 64, 128])
    shape = dict(page=page, heads=rng.choice([2, 8, 32, 52]), D=rng.choice([64, 128]), kind=rng.choice(["int8", "int4"]))
    B, L, n = _log(rng, 1, 64), _log(rng, 20, 8000), rng.choice([2, 7, 16, 64])
    if op == "fork":
        n = rng.choice([1, 2, 4, 8])
        B = n * -(-B // n)
    if op == "compact":
        n = rng.choice([100, 1000, 4096])
    width = (L + 64) // page + 2 + rng.randrange(20)
    # what the sequences hold, and as much again; a pool of at most 2 GB
    most = int(3e9 / (2 * page * shape["heads"] * shape["D"]))
    B = max(n if op == "fork" else 1, min(B, most // (3 * width)))
    B -= B % n if op == "fork" else 0
    return dict(op=op, B=B, n=n, L=L, width=width, pages=2 * B * width + rng.randrange(5, 500), **shape)


def _page_bytes(c):
    return c["page"] * c["heads"] * (2 * (c["D"] + 2) if c["kind"] == "int8" else 2 * (c["D"] // 2 + 2 * (c["D"] // 32)))


def _step_lens(c):
    """Tokens of each sequence, its drafts, and the drafts that are kept, first to last [B, most].  A kept draft lies at its
    own place or past the kept ones' places, so that a second pass over the same entries moves the same ones."""
    r = np.random.default_rng(7919 * c["B"] + 31 * c["n"] + c["L"])
    ctx = r.integers(max(1, c["L"] // 8), c["L"] + 1, c["B"])
    new = r.integers(max(1, c["n"] // 2), c["n"] + 1, c["B"])
    new[r.integers(c["B"])] = c["n"]
    most = max(1, c["n"] // 2)
    keep = r.integers(0, np.minimum(new, most) + 1)
    kept = np.full((c["B"], most), -1, np.int64)
    for b in range(c["B"]):
        k, same = int(keep[b]), int(r.integers(0, keep[b] + 1))
        far = np.sort(r.choice(np.arange(k, new[b]), min(k - same, new[b] - k), replace=False))
        path = np.concatenate([np.arange(k - len(far)), far])
        kept[b, :k] = path
    return ctx, new, kept


def _fork_lens(c):
    r = np.random.default_rng(104729 * c["B"] + 17 * c["n"] + c["L"])
    groups = c["B"] // c["n"]
    ctx = np.zeros(c["B"], np.int64)
    ctx[c["n"] - 1::c["n"]] = r.integers(max(1, c["L"] // 8), c["L"] + 1, groups)  # a group's prompt is its last sequence
    parents = np.repeat(np.arange(groups) * c["n"] + c["n"] - 1, c["n"])
    return ctx, parents


def _compact_tables(c, seed):
    """Tables over pages that lie anywhere; every fourth sequence shares its first pages with the one before."""
    r = np.random.default_rng(15485863 * c["B"] + c["L"] + c["pages"] + 1000003 * (seed % 1000003))
    lens = np.random.default_rng(c["B"] + c["L"]).integers(max(1, c["L"] // 8), min(c["L"], c["width"] * c["page"]) + 1, c["B"])
    table = np.full((c["B"], c["width"]), -1, np.int64)
    order, at = r.permutation(c["pages"]), 0
    for b in range(c["B"]):
        n = -(-int(lens[b]) // c["page"])
        table[b, :n] = order[at:at + n]
        at += n
        if b % 4 == 3:
            same = min(n, int(lens[b - 1]) // c["page"]) // 2
            table[b, :same] = table[b - 1, :same]
    return table, lens


def work(case):
    c = case
    if c["op"] == "int8":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": 1.0 * T * K * SIZE[c["src"]] + 1.0 * N * K + N * (8 if c["bias"] else 4) + 1.0 * T * N * SIZE[c["dst"]],
                "flops": 2.0 * T * K * N}
    if c["op"] == "axes":
        heads, s = c["hq"] + c["hkv"], [int(v) for v in c["sections"].split(",")]
        return {"bytes": c["T"] * (heads * c["D"] * (SIZE[c["src"]] + SIZE[c["dst"]]) + 8.0 * sum(s) + 4 * len(s)),
                "flops": 6.0 * c["T"] * heads * sum(s)}
    tables = 8.0 * c["B"] + 4.0 * c["pages"]
    if c["op"] == "step":
        ctx, new, kept = _step_lens(c)
        moved = int((kept >= 0).sum())
        return {"bytes": 2.0 * moved * _page_bytes(c) / c["page"] + tables + 4.0 * (kept.size + int(new.sum()) + c["B"]),
                "flops": 1.0 * c["pages"]}
    if c["op"] == "fork":
        ctx, parents = _fork_lens(c)
        part = int((ctx % c["page"] != 0).sum()) * (c["n"] - 1)
        return {"bytes": 2.0 * part * _page_bytes(c) + tables + 8.0 * c["B"] * c["width"], "flops": 1.0 * c["pages"]}
    table, lens = _compact_tables(c, 1)
    live = np.unique(table[table >= 0])
    moves = min(c["n"], int((live >= live.size).sum()))
    return {"bytes": 2.0 * moves * _page_bytes(c) + 8.0 * table.size + 8.0 * c["pages"] + 8.0 * c["n"], "flops": 1.0 * c["pages"]}


# -------------------------------------------------------------------- inputs
def _positions(T, axes, first):
    """Text, an image of about half the tokens, text: int64 [axes, T] (time, height, width; two axes have no time, four
    have the image's number last)."""
    n0, m = T // 4, T // 2
    side = max(1, int(math.sqrt(m)))
    i = np.arange(m)
    t = np.concatenate([np.arange(n0), np.full(m, n0), np.arange(T - n0 - m) + n0 + -(-max(m, 1) // side)])
    h = np.concatenate([np.arange(n0), n0 + i // side, t[n0 + m:]])
    w = np.concatenate([np.arange(n0), n0 + i % side, t[n0 + m:]])
    rows = [h, w] if axes == 2 else [t, h, w, (t >= n0).astype(np.int64) - first][:axes]
    return np.stack(rows) + first


def _table(P, sections, dev):
    """cos and sin of every position and pair [P, pairs, 2] (fp32 from 64 bits), one row of frequencies for all axes."""
    n = sum(sections)
    inv = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)
    a = torch.arange(P, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.stack([a.cos(), a.sin()], -1).to(torch.float32).contiguous()


def _ints(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev)


def _cache(s, gen, dev):
    """The cache's tensors: any codes, and scales of small positive values."""
    shape = (s["pages"], s["heads"], s["page"], s["D"] if s["kind"] == "int8" else s["D"] // 2)
    tail = () if s["kind"] == "int8" else (s["D"] // 32,)
    for name in ("k", "v"):
        s[name] = torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)
        s[name + "s"] = torch.rand(shape[:3] + tail, generator=gen, device=dev).half()


def _handles(s):
    """The layer, cache and pool objects that a program keeps around its tensors (the plain form works on the tensors)."""
    if own:
        import compressed_linear_amd as cla
        if s["op"] == "int8":
            s["layer"] = cla.Int8Linear(s["w"], s["sw"], bias=s["b"], clamp=s["clamp"] or None)
        elif s["op"] != "axes":
            s["cache"] = cla.KVCache(kind=s["kind"], k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"])
            s["pool"] = cla.PagePool(page_size=s["page"], block_table=s["table"], lens=s["lens"], refs=s["refs"])
    return s


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    s = dict(c)
    if c["op"] == "int8":
        T, K, N = c["T"], c["K"], c["N"]
        # activations with a few channels that carry larger values; weights quantised to their channel's largest
        gain = 1.0 + 9.0 * (torch.rand(K, generator=gen, device=dev) < 0.005)
        s["x"] = (torch.randn(T, K, generator=gen, device=dev) * gain).to(DT[c["src"]])
        w = torch.randn(N, K, generator=gen, device=dev)
        s["sw"] = w.abs().amax(-1) * (0.02 / 127.0)
        s["w"] = (w * (0.02 / s["sw"])[:, None]).round().clamp(-127, 127).to(torch.int8)
        s["b"] = torch.randn(N, generator=gen, device=dev) if c["bias"] else None
        return _handles(s)
    if c["op"] == "axes":
        sections = [int(v) for v in c["sections"].split(",")]
        qkv = torch.randn(c["T"], c["hq"] + 2 * c["hkv"], c["D"], generator=gen, device=dev).to(DT[c["src"]])
        s["x"] = qkv[:, :c["hq"] + c["hkv"]]  # the q and k heads of the qkv layer's output
        at = _positions(c["T"], len(sections), rs.randint(0, 2000))
        s["pos"] = _ints(at, dev)
        s["table"] = _table(c["T"] + 2064, sections, dev)
        s["sections"] = tuple(sections)
        return s
    _cache(s, gen, dev)
    if c["op"] == "compact":
        table, lens = _compact_tables(c, int(seed))
    else:
        ctx, more = _step_lens(c)[:2] if c["op"] == "step" else _fork_lens(c)
        lens = ctx
        table = np.full((c["B"], c["width"]), -1, np.int64)
        order, at = rs.permutation(c["pages"]), 0
        for b in range(c["B"]):
            n = -(-int(ctx[b]) // c["page"])
            table[b, :n] = order[at:at + n]
            at += n
        new = more if c["op"] == "step" else np.ones(c["B"], np.int64)
        s["cu"] = _ints(np.concatenate([[0], np.cumsum(new)]), dev)
        s["tokens"] = int(new.sum())
        s["ctx"] = _ints(ctx, dev)
        if c["op"] == "step":
            kept = _step_lens(c)[2]
            s["kept"] = _ints(kept, dev)
            s["accepted"] = _ints(ctx + (kept >= 0).sum(1), dev)
        else:
            s["parents"] = _ints(more, dev)
    s["table"], s["lens"] = _ints(table, dev), _ints(lens, dev)
    s["refs"] = _ints(np.bincount(table[table >= 0], minlength=c["pages"]), dev)
    if c["op"] == "compact":
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    return _handles(s)


# ---------------------------------------------------------------- plain forms
def _plain_int8(s):
    x = s["x"].float()
    if s["clamp"]:
        x = x.clamp(-s["clamp"], s["clamp"])
    scale = x.abs().amax(-1, keepdim=True) * (1.0 / 127.0)
    codes = (x * torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))).round().clamp(-127, 127)
    y = torch.matmul(codes, s["w"].float().t()) * scale * s["sw"]
    return (y + s["b"] if s["bias"] else y).to(DT[s["dst"]])


def _axis_of_pairs(sections, order):
    """The axis of each pair."""
    n, axes = sum(sections), len(sections)
    if order == "blocks":
        return np.repeat(np.arange(axes), sections)
    i = np.arange(n)
    return np.where(i // axes < np.asarray(sections)[i % axes], i % axes, 0)


def _plain_axes(s):
    axis = torch.from_numpy(_axis_of_pairs(s["sections"], s["order"])).to(s["x"].device)
    n, x = axis.numel(), s["x"].float()
    cs = s["table"][s["pos"].long()[axis].t(), torch.arange(n, device=x.device)][:, None]  # [T, 1, n, 2]
    cos, sin = cs[..., 0], cs[..., 1]
    if s["layout"] == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1).to(DT[s["dst"]])


def _count(refs, pages, by):
    """refs changed by `by` for every page in `pages` (int32, -1: none)."""
    refs.scatter_add_(0, pages.clamp(min=0).flatten().long(), ((pages >= 0).int() * by).flatten())


def _plain_truncate(s, lens):
    """Sequences shortened to `lens`, the pages past them given back."""
    cut = (lens >= 0) & (lens < s["lens"])
    s["lens"].copy_(torch.where(cut, lens, s["lens"]))
    held = (s["lens"] + s["page"] - 1) // s["page"]
    past = torch.arange(s["width"], device=lens.device)[None, :] >= held[:, None]
    _count(s["refs"], torch.where(past, s["table"], -1), -1)
    s["table"].masked_fill_(past, -1)


def _plain_fork(s, parents):
    """Each sequence becomes a copy of its parent, which shares the pages; -1 ends it."""
    there = parents >= 0
    at = parents.clamp(min=0).long()
    table = torch.where(there[:, None], s["table"][at], -1)
    _count(s["refs"], s["table"], -1)
    _count(s["refs"], table, 1)
    s["lens"].copy_(torch.where(there, s["lens"][at], 0))
    s["table"].copy_(table)


def _plain_extend(s, cu, tokens):
    """Pages for new tokens: their slots, and the pages to copy because others share them (source, destination)."""
    dev, page, B, W = cu.device, s["page"], s["B"], s["width"]
    new = cu[1:] - cu[:-1]
    total = s["lens"] + new
    go = (new > 0) & (total <= W * page)
    held, want = (s["lens"] + page - 1) // page, (total + page - 1) // page
    last = torch.gather(s["table"], 1, (held - 1).clamp(min=0).long()[:, None])[:, 0]
    part = go & (s["lens"] % page != 0)
    earlier = torch.ones(B, B, device=dev).tril(-1) > 0
    rank = (earlier & part[None, :] & (last[:, None] == last[None, :])).sum(1)
    shared = part & (s["refs"][last.clamp(min=0).long()] - rank > 1)
    need = torch.where(go, want - held + shared.int(), 0)
    end = need.cumsum(0)
    number = torch.arange(s["pages"], device=dev)
    free = torch.sort(torch.where(s["refs"] == 0, number, s["pages"] + number)).values
    go = go & (end <= (s["refs"] == 0).sum())
    shared = shared & go
    place = torch.arange(W, device=dev)[None, :]
    mine = go[:, None] & (place >= (held - shared.int())[:, None]) & (place < want[:, None])
    at = (end - need)[:, None] + place - (held - shared.int())[:, None]
    given = free[at.clamp(0, s["pages"] - 1)].int()
    src = torch.where(shared, last, -1)
    dst = torch.where(shared, free[(end - need).clamp(0, s["pages"] - 1)].int(), -1)
    s["table"].copy_(torch.where(mine, given, s["table"]))
    _count(s["refs"], src, -1)
    _count(s["refs"], torch.where(mine, given, -1), 1)
    t = torch.arange(tokens, device=dev, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    to = (s["lens"][b] + t - cu[b]).long()
    slot = torch.gather(s["table"][b], 1, (to // page).clamp(max=W - 1)[:, None])[:, 0] * page + (to % page).int()
    slots = torch.where(go[b], slot, -1)
    s["lens"].copy_(torch.where(go, total, s["lens"]))
    return slots, src, dst


def _plain_copy(s, src, dst):
    """Pages src copied to dst; an empty entry (-1) repeats the first that is none, or copies page 0 to itself."""
    first = (src >= 0).int().argmax()
    at, to = (torch.where(src >= 0, v, v[first].clamp(min=0)).long() for v in (src, dst))
    for name in ("k", "v", "ks", "vs"):
        s[name][to] = s[name][at]


def _plain_keep(s):
    """Accepted drafts moved to the places after their sequence's older tokens."""
    B, most, page = *s["kept"].shape, s["page"]
    to = s["ctx"][:, None] + torch.arange(most, device=s["kept"].device)[None, :]
    at = torch.where(s["kept"] >= 0, s["ctx"][:, None] + s["kept"], to)
    pt, pa = (torch.gather(s["table"], 1, (v // page).long()).long() for v in (to, at))
    for name in ("k", "v", "ks", "vs"):
        s[name][pt, :, (to % page).long()] = s[name][pa, :, (at % page).long()]


def _plain_compact(s, most):
    """The highest live pages moved to the lowest free ones: sources and destinations [most], -1 past the last."""
    dev, P = s["refs"].device, s["pages"]
    live = s["refs"] > 0
    number = torch.arange(P, device=dev)
    n = min(most, P)
    high = torch.sort(torch.where(live, number, -1), descending=True).values[:n]
    low = torch.sort(torch.where(live, P, number)).values[:n]
    go = low < high
    map_ = number.clone().scatter_(0, high.clamp(min=0), torch.where(go, low, high.clamp(min=0)))  # page 0 never moves
    s["table"].copy_(torch.where(s["table"] >= 0, map_[s["table"].clamp(min=0).long()].int(), -1))
    held = torch.where(go, s["refs"][high.clamp(min=0)], 0)
    s["refs"].scatter_add_(0, high.clamp(min=0), -held)
    s["refs"].scatter_add_(0, low.clamp(max=P - 1), held)
    out = torch.full((2, most), -1, dtype=torch.int32, device=dev)
    out[0, :n], out[1, :n] = torch.where(go, high, -1).int(), torch.where(go, low, -1).int()
    return out[0], out[1]


def _back(s):
    """The compaction's pool as it was, so that a pass can be run again (its sources' entries are still there)."""
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])


def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "int8":
            return _plain_int8(s)
        if op == "axes":
            return _plain_axes(s)
        if op == "step":
            _plain_truncate(s, s["ctx"])
            out = _plain_extend(s, s["cu"], s["tokens"])
            _plain_keep(s)
            _plain_truncate(s, s["accepted"])
        elif op == "fork":
            _plain_truncate(s, s["ctx"])
            _plain_fork(s, s["parents"])
            out = _plain_extend(s, s["cu"], s["tokens"])
            _plain_copy(s, out[1], out[2])
        else:
            _back(s)
            out = _plain_compact(s, s["n"])
            _plain_copy(s, *out)
        return (*out, s["table"], s["lens"], s["refs"], s["k"], s["ks"], s["v"], s["vs"])
    import compressed_linear_amd as cla
    if op == "int8":
        return s["layer"](s["x"], out_dtype=DT[s["dst"]])
    if op == "axes":
        return cla.rope(s["x"], s["pos"], s["table"], layout=s["layout"], out_dtype=DT[s["dst"]], sections=s["sections"],
                        order=s["order"])
    pool, cache = s["pool"], s["cache"]
    if op == "step":  # an answer is taken back and drafted anew; between the calls lie the layers, append and attention
        pool.truncate(s["ctx"])
        out = pool.extend(s["cu"], s["tokens"])
        cache.keep(pool.block_table, s["ctx"], s["kept"])
        pool.truncate(s["accepted"])
    elif op == "fork":  # the last continuations end, and their prompts get new ones with a token each
        pool.truncate(s["ctx"])
        pool.fork(s["parents"])
        out = pool.extend(s["cu"], s["tokens"])
        cache.copy_pages(out[1], out[2])
    else:
        _back(s)
        out = pool.compact(s["n"])
        cache.copy_pages(*out)
    return (*out, pool.block_table, pool.lens, pool.refs, cache.k, cache.k_scale, cache.v, cache.v_scale)


# ------------------------------------------------------------------- 64 bits
def _exact_pool(s):
    """The pool's operations one sequence and page at a time: (slots, src, dst), table, lens, refs, moved entries
    as (from page, from place, to page, to place)."""
    page, op = s["page"], s["op"]
    table, lens, refs = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "lens", "refs"))
    moved = []

    def shorten(b, n):
        held = -(-int(n) // page)
        for w in range(held, s["width"]):
            if table[b, w] >= 0:
                refs[table[b, w]] -= 1
                table[b, w] = -1
        lens[b] = n

    if op == "compact":
        src, dst = np.full(s["n"], -1, np.int64), np.full(s["n"], -1, np.int64)
        low, high, to = 0, s["pages"] - 1, {}
        for i in range(s["n"]):
            while low < s["pages"] and refs[low] != 0:
                low += 1
            while high >= 0 and refs[high] == 0:
                high -= 1
            if low >= high:
                break
            src[i], dst[i] = high, low
            to[high] = low
            refs[low], refs[high] = refs[high], 0
            moved.append((high, None, low, None))
        for b in range(s["B"]):
            for w in range(s["width"]):
                table[b, w] = to.get(int(table[b, w]), table[b, w])
        return (src, dst), table, lens, refs, moved
    ctx, cu = s["ctx"].tolist(), s["cu"].tolist()
    for b in range(s["B"]):
        shorten(b, ctx[b])
    if op == "fork":
        old, long, parents = table.copy(), lens.copy(), s["parents"].tolist()
        for b in range(s["B"]):
            shorten(b, 0)
        for b, p in enumerate(parents):
            table[b], lens[b] = old[p], long[p]
            for w in table[b][table[b] >= 0]:
                refs[w] += 1
    free = iter(np.flatnonzero(refs == 0).tolist())
    slots, src, dst = np.full(s["tokens"], -1, np.int64), np.full(s["B"], -1, np.int64), np.full(s["B"], -1, np.int64)
    for b in range(s["B"]):
        n = int(lens[b])
        for t in range(cu[b], cu[b + 1]):
            at = n + t - cu[b]
            if at % page and t == cu[b] and refs[table[b, at // page]] > 1:
                src[b], dst[b] = table[b, at // page], next(free)
                refs[src[b]] -= 1
                refs[dst[b]] = 1
                table[b, at // page] = dst[b]
                moved.append((src[b], None, dst[b], None))
            if at % page == 0:
                table[b, at // page] = next(free)
                refs[table[b, at // page]] = 1
            slots[t] = table[b, at // page] * page + at % page
        lens[b] = n + cu[b + 1] - cu[b]
    if op == "step":
        for b, row in enumerate(s["kept"].tolist()):
            for j, i in enumerate(row):
                if i >= 0:
                    f, g = ctx[b] + i, ctx[b] + j
                    moved.append((table[b, f // page], f % page, table[b, g // page], g % page))
            shorten(b, ctx[b] + sum(i >= 0 for i in row))
    return (slots, src, dst), table, lens, refs, moved


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "int8":
        x = s["x"].double()
        if s["clamp"]:
            x = torch.minimum(torch.maximum(x, torch.tensor(-s["clamp"], device=x.device)), torch.tensor(s["clamp"], device=x.device))
        # codes are defined down to each rounding: the scale, its reciprocal and the product with it are fp32 values
        rounded = lambda v: v.float().double()  # noqa: E731
        scale = rounded(x.abs().max(-1).values * rounded(torch.tensor(1 / 127, dtype=torch.float64)).item())
        inverse = torch.where(scale > 0, rounded(1 / scale), torch.zeros_like(scale))
        codes = torch.round(rounded(x * inverse[:, None]))
        y = torch.mm(codes, s["w"].double().t()) * torch.outer(scale, s["sw"].double())
        return y if s["b"] is None else y + s["b"].double()
    if s["op"] == "axes":
        x = s["x"].double()
        y, sections, n = x.clone(), s["sections"], sum(s["sections"])
        axis, left = [], list(sections)
        for i in range(n):  # blocks: the first axis that has pairs left; turns: the next one that has, or the first axis
            a = next(a for a in range(len(left)) if left[a]) if s["order"] == "blocks" else i % len(left)
            a = a if left[a] and (s["order"] == "blocks" or i // len(left) < sections[a]) else 0
            left[a] -= 1
            axis.append(a)
        for i, a in enumerate(axis):
            c, sn = (s["table"][s["pos"][a].long(), i, j].double()[:, None] for j in (0, 1))
            p, q = (i, i + n) if s["layout"] == "half" else (2 * i, 2 * i + 1)
            y[..., p] = x[..., p] * c - x[..., q] * sn
            y[..., q] = x[..., q] * c + x[..., p] * sn
        return y
    out, table, lens, refs, moved = _exact_pool(s)
    tensors = []
    for name in ("k", "ks", "v", "vs"):
        new = s[name].clone()
        if moved and moved[0][1] is None:
            f, _, g, _ = (torch.tensor([m[i] for m in moved] if i % 2 == 0 else [0]) for i in range(4))
            new[g.to(new.device)] = s[name][f.to(new.device)]
        elif moved:
            f, i, g, j = (torch.tensor([int(m[n]) for m in moved], device=new.device) for n in range(4))
            new[g, :, j] = s[name][f, :, i]
        tensors.append(new)
    dev = s["refs"].device
    return (*(_ints(v, dev) for v in out), _ints(table, dev), _ints(lens, dev), _ints(refs, dev), *tensors)
