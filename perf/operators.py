"""Cases and plain forms of the serving operators around the compressed linear
layers: rotary positions, the quantised K/V cache (append, read back), attention
of drafted tokens over that cache, and log probabilities of given tokens.

`run(state)` computes an operator in elementary torch operations in 32 bits
(`own` false) or through the package's entry points (`own` true).  The head
layouts are those of this repository's layer sets: 32 + 2 x 32 heads of 128
(LLaMA-7B, 4096), 52 heads (6656) and 64 + 2 x 8 heads (LLaMA-70B, qkv 8192 -> 10240).

Cache layout (both forms work on the same tensors): k and v are uint8
[pages, kv heads, page size, D] holding code + 128 with one fp16 scale per
(token, head), or, for int4, uint8 [pages, kv heads, page size, D / 2] holding two
nibbles code + 8 (channel 2i in the low one) with one fp16 scale per 32 channels.
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
        # the q and k heads of one new token of one sequence, as the qkv layer leaves them (fp32)
        dict(name="rope 1 token", op="rope", T=1, hq=64, hkv=8, D=128, rot=128, layout="half", src="f32", dst="bf16",
             P=8192, factor=1.0),
        # a prompt of 8192 tokens; interleaved pairs on half of the head, positions past the trained length
        dict(name="rope prompt", op="rope", T=8192, hq=64, hkv=8, D=128, rot=64, layout="interleaved", src="bf16",
             dst="bf16", P=32768, factor=4.0),
        # one decode step of 64 sequences: every new key rotated, both quantised; then those entries read back
        dict(name="cache step int8", op="cache", write=64, read=64, pages=4096, page=64, hq=64, hkv=8, D=128,
             kind="int8", rot=128, layout="half", src="f32", dst="bf16", P=8192),
        # a prompt of 8000 tokens written to an int4 cache, keys already rotated; read back for a second pass
        dict(name="cache prompt int4", op="cache", write=8000, read=8000, pages=600, page=16, hq=0, hkv=8, D=128,
             kind="int4", rot=0, layout="half", src="bf16", dst="f16", P=0),
        # a chunk of 512 tokens joins a long prefix, which is then read back whole (32 heads)
        dict(name="cache read long", op="cache", write=512, read=40000, pages=400, page=128, hq=32, hkv=32, D=128,
             kind="int8", rot=128, layout="interleaved", src="bf16", dst="f16", P=65536),
        # one token of one short sequence, 32 heads: latency
        dict(name="attn 1 token short", op="attention", B=1, T=1, L=511, hq=32, hkv=32, D=128, kind="int8", page=16,
             io="f16", tree=False),
        # a decode step of 64 sequences of up to 8192 tokens, 8 query heads to a kv head
        dict(name="attn decode batch", op="attention", B=64, T=1, L=8192, hq=64, hkv=8, D=128, kind="int8", page=64,
             io="bf16", tree=False),
        # one token of one very long sequence, int4
        dict(name="attn 1 token long", op="attention", B=1, T=1, L=131001, hq=64, hkv=8, D=128, kind="int4", page=128,
             io="bf16", tree=False),
        # trees of up to 16 drafted tokens of 8 sequences, one query head to a kv head
        dict(name="attn trees", op="attention", B=8, T=16, L=4000, hq=52, hkv=52, D=128, kind="int8", page=32,
             io="f16", tree=True),
        # a tree of 64 drafted tokens over a long sequence: 512 query rows to a kv head, bound by arithmetic
        dict(name="attn tree long", op="attention", B=1, T=64, L=61441, hq=64, hkv=8, D=128, kind="int8", page=64,
             io="bf16", tree=True),
        # the token that follows one sequence, with 8 alternatives
        dict(name="logprobs 1 row", op="logprobs", T=1, V=32000, C=1, k=8, src="f32"),
        # scoring a batch of drafts or a prompt: 4096 rows, 4 candidates each
        dict(name="logprobs scoring", op="logprobs", T=4096, V=32000, C=4, k=5, src="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attention", "attention", "logprobs"])
    if op == "rope":
        hq, hkv = rng.choice([(32, 32), (64, 8), (52, 52), (16, 2)])
        D = rng.choice([64, 128])
        return dict(op=op, T=_log(rng, 1, 8192), hq=hq, hkv=hkv, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    layout=rng.choice(["half", "interleaved"]), src=rng.choice(["f32", "f16", "bf16"]),
                    dst=rng.choice(["f16", "bf16"]), P=_log(rng, 8192, 131072), factor=rng.choice([1.0, 2.0, 8.0]))
    if op == "cache":
        hq, hkv = rng.choice([(32, 32), (64, 8), (52, 52), (16, 2)])
        D = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        write = _log(rng, 1, 8192)
        read = rng.choice([write, write, _log(rng, write, 16384)])
        rot = rng.choice([0, D, D // 2])
        return dict(op=op, write=write, read=read, pages=-(-read // page) + rng.randrange(1, 100), page=page, hq=hq,
                    hkv=hkv, D=D, kind=rng.choice(["int8", "int4"]), rot=rot,
                    layout=rng.choice(["half", "interleaved"]), src=rng.choice(["f32", "f16", "bf16"]),
                    dst=rng.choice(["f16", "bf16"]), P=32768 if rot else 0)
    if op == "attention":
        hq, hkv = rng.choice([(32, 32), (64, 8), (52, 52), (16, 2), (12, 4)])
        D = rng.choice([64, 128])
        T = rng.choice([1, _log(rng, 2, 16), _log(rng, 2, 128)])
        B = _log(rng, 1, 64)
        L = _log(rng, 1, 131072)
        L = max(1, min(L, int(4e9 / (2 * B * hkv * D)) // 4, int(1e11 / (4.0 * B * T * hq * D))))
        return dict(op=op, B=B, T=T, L=L, hq=hq, hkv=hkv, D=D, kind=rng.choice(["int8", "int4"]),
                    page=rng.choice([16, 32, 64, 128]), io=rng.choice(["f16", "bf16"]), tree=T > 1)
    V = _log(rng, 1000, 150000)
    return dict(op=op, T=min(_log(rng, 1, 4096), int(1.3e8 / V)), V=V, C=rng.choice([1, 2, 7]),
                k=rng.choice([0, 1, 5, 16, 32]), src=rng.choice(["f32", "f16", "bf16"]))


def _row_bytes(c):
    """Bytes of one cached (token, head): codes and scales of K and V."""
    return 2 * (c["D"] + 2) if c["kind"] == "int8" else 2 * (c["D"] // 2 + 2 * (c["D"] // 32))


def _lens(case):
    """Context lengths and drafted tokens of each sequence; the longest of each is the case's own."""
    B, T, L = case["B"], case["T"], case["L"]
    r = np.random.default_rng(1000003 * B + 1009 * T + L)
    ctx = r.integers(L // 8, L + 1, B)
    new = r.integers(max(1, T // 2), T + 1, B)
    ctx[r.integers(B)] = L
    new[r.integers(B)] = T
    return ctx, new


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * (c["hq"] + c["hkv"]) * c["D"]
        return {"bytes": n * (SIZE[c["src"]] + SIZE[c["dst"]]) + c["T"] * (4 * c["rot"] + 4),
                "flops": 3.0 * c["T"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "cache":
        w, r, vals = c["write"] * c["hkv"], c["read"] * c["hkv"], 2 * c["D"]
        return {"bytes": w * (vals * SIZE[c["src"]] + _row_bytes(c)) + c["write"] * (4 + (4 * c["rot"] + 4 if c["rot"] else 0))
                + r * (_row_bytes(c) + vals * SIZE[c["dst"]]) + 4 * c["read"],
                "flops": 4.0 * w * vals + 1.0 * r * vals}
    if c["op"] == "attention":
        ctx, new = _lens(c)
        rows = int(new.sum()) * c["hq"] * c["D"]
        return {"bytes": float((ctx + new).sum()) * c["hkv"] * _row_bytes(c) + 2 * rows * SIZE[c["io"]],
                "flops": 4.0 * float((new * (ctx + new)).sum()) * c["hq"] * c["D"]}
    return {"bytes": c["T"] * (c["V"] * SIZE[c["src"]] + 4.0 * (2 * c["C"] + 1 + 2 * c["k"])),
            "flops": 4.0 * c["T"] * c["V"]}


# -------------------------------------------------------------------- inputs
def _table(P, rot, factor, dev):
    """cos and sin of every position and pair [P, rot / 2, 2] (fp32 from 64 bits), positions divided by `factor`."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(P, dtype=torch.float64, device=dev)[:, None] / factor * inv[None, :]
    return torch.stack([a.cos(), a.sin()], -1).to(torch.float32).contiguous()


def _quant(v, kind):
    """Codes and scales of fp32 values [..., D] in the cache's format."""
    if kind == "int8":
        s = (v.abs().amax(-1, keepdim=True) / 127.0).clamp(max=65504.0).half()
        r = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(s, dtype=torch.float32))
        return ((v * r).round().clamp(-127, 127) + 128).to(torch.uint8), s.squeeze(-1)
    g = v.unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1, keepdim=True) / 7.0).clamp(max=8192.0).bfloat16().half()
    r = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(s, dtype=torch.float32))
    n = ((g * r).round().clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), s.squeeze(-1)


def _values(codes, scales, kind):
    """The fp32 values that codes and scales stand for [..., D]."""
    if kind == "int8":
        return (codes.float() - 128.0) * scales.float()[..., None]
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
    return (n.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _fill(shape_tokens, hkv, page, D, kind, gen, dev):
    """A cache of random keys or values, quantised page by page: (codes, scales).  A few channels of
    each head carry larger values, as keys do."""
    gain = 1.0 + 4.0 * (torch.rand(hkv, 1, D, generator=gen, device=dev) < 0.03)
    codes, scales = [], []
    for at in range(0, shape_tokens, 512):
        n = min(512, shape_tokens - at)
        v = torch.randn(n, hkv, page, D, generator=gen, device=dev) * gain
        a, b = _quant(v, kind)
        codes.append(a)
        scales.append(b)
    return torch.cat(codes), torch.cat(scales)


def _tree_masks(new, words, rs):
    """Each drafted token's ancestors and itself, as bits over its sequence's drafted tokens [sum, words] int64."""
    out = np.zeros((int(new.sum()), words), np.uint64)
    at = 0
    for t_b in new:
        rows = []
        for t in range(int(t_b)):
            up = rs.randint(-1, t) if t else -1
            rows.append((rows[up] if up >= 0 else 0) | (1 << t))
        for t, m in enumerate(rows):
            for w in range(words):
                out[at + t, w] = (m >> (64 * w)) & 0xFFFFFFFFFFFFFFFF
        at += int(t_b)
    return out.view(np.int64)


def _handle(state):
    """The cache object that a program keeps around its tensors (the plain form works on the tensors)."""
    if own:
        import compressed_linear_amd as cla
        state["cache"] = cla.KVCache(kind=state["kind"], k=state["k"], v=state["v"], k_scale=state["ks"],
                                     v_scale=state["vs"])
    return state


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    s = dict(c)
    if c["op"] == "rope":
        qkv = torch.randn(c["T"], c["hq"] + 2 * c["hkv"], c["D"], generator=gen, device=dev).to(DT[c["src"]])
        s["x"] = qkv[:, :c["hq"] + c["hkv"]]  # the q and k heads of the qkv layer's output
        first = rs.randint(0, c["P"] - c["T"] + 1)
        s["pos"] = torch.arange(first, first + c["T"], dtype=torch.int32, device=dev)
        s["table"] = _table(c["P"], c["rot"], c["factor"], dev)
        return s
    if c["op"] == "cache":
        H = c["hq"] + 2 * c["hkv"]
        qkv = torch.randn(c["write"], H, c["D"], generator=gen, device=dev).to(DT[c["src"]])
        s["knew"], s["vnew"] = qkv[:, c["hq"]:c["hq"] + c["hkv"]], qkv[:, c["hq"] + c["hkv"]:]
        s["k"], s["ks"] = _fill(c["pages"], c["hkv"], c["page"], c["D"], c["kind"], gen, dev)
        s["v"], s["vs"] = _fill(c["pages"], c["hkv"], c["page"], c["D"], c["kind"], gen, dev)
        if c["write"] == 64:  # a step of many sequences: places apart
            slots = torch.randperm(c["pages"] * c["page"], generator=gen, device=dev)[:c["read"]]
        else:  # the sequence's pages lie anywhere; its last tokens are the new ones
            pages = torch.randperm(c["pages"], generator=gen, device=dev)[:, None] * c["page"]
            slots = (pages + torch.arange(c["page"], device=dev)).flatten()[:c["read"]]
        s["rslots"] = slots.to(torch.int32)
        s["wslots"] = s["rslots"][c["read"] - c["write"]:].clone()
        s["pos"] = s["table"] = None
        if c["rot"]:
            first = rs.randint(0, c["P"] - c["write"] + 1)
            s["pos"] = torch.arange(first, first + c["write"], dtype=torch.int32, device=dev)
            s["table"] = _table(c["P"], c["rot"], 1.0, dev)
        return _handle(s)
    if c["op"] == "attention":
        ctx, new = _lens(c)
        width = int(-(-(ctx + new).max() // c["page"]))
        need = int((-(-(ctx + new) // c["page"])).sum())
        s["k"], s["ks"] = _fill(need + 3, c["hkv"], c["page"], c["D"], c["kind"], gen, dev)
        s["v"], s["vs"] = _fill(need + 3, c["hkv"], c["page"], c["D"], c["kind"], gen, dev)
        order = torch.randperm(need + 3, generator=gen, device=dev).to(torch.int32).cpu().numpy()
        table, at = np.zeros((c["B"], width), np.int32), 0
        for b in range(c["B"]):
            n = int(-(-(ctx[b] + new[b]) // c["page"]))
            table[b, :n] = order[at:at + n]
            at += n
        s["block_table"] = torch.from_numpy(table).to(dev)
        s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).to(dev)
        s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
        s["max_q"], s["max_ctx"] = int(new.max()), int(ctx.max())
        s["q"] = torch.randn(int(new.sum()), c["hq"], c["D"], generator=gen, device=dev).to(DT[c["io"]])
        s["mask"] = torch.from_numpy(_tree_masks(new, -(-int(new.max()) // 64), rs)).to(dev) if c["tree"] else None
        return _handle(s)
    # logits as a model leaves them: a spread of a few units, some tokens far above the rest
    x = torch.randn(c["T"], c["V"], generator=gen, device=dev) * 2.5
    hot = torch.randint(0, c["V"], (c["T"], 12), generator=gen, device=dev)
    x.scatter_add_(1, hot, 8.0 * torch.rand(c["T"], 12, generator=gen, device=dev))
    s["x"] = x.to(DT[c["src"]])
    ids = torch.randint(0, c["V"], (c["T"], c["C"]), generator=gen, device=dev)
    ids[:, 0] = hot[:, 0]
    s["ids"] = ids.to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms
def _rotated(x, pos, table, layout):
    """fp32 x [T, H, D] with its first 2 * table.shape[1] channels rotated."""
    n = table.shape[1]
    cs = table[pos.long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_cache(s):
    page = s["page"]
    k, v = s["knew"].float(), s["vnew"].float()
    if s["rot"]:
        k = _rotated(k, s["pos"], s["table"], s["layout"])
    p, o = s["wslots"].long() // page, s["wslots"].long() % page
    for_k, for_v = _quant(k, s["kind"]), _quant(v, s["kind"])
    s["k"][p, :, o], s["ks"][p, :, o] = for_k
    s["v"][p, :, o], s["vs"][p, :, o] = for_v
    p, o = s["rslots"].long() // page, s["rslots"].long() % page
    return (_values(s["k"][p, :, o], s["ks"][p, :, o], s["kind"]).to(DT[s["dst"]]),
            _values(s["v"][p, :, o], s["vs"][p, :, o], s["kind"]).to(DT[s["dst"]]))


def _plain_attention(s):
    B, hq, hkv, D, page = s["B"], s["hq"], s["hkv"], s["D"], s["page"]
    bt = s["block_table"].long()
    n = bt.shape[1] * page
    k = _values(s["k"][bt], s["ks"][bt], s["kind"]).permute(0, 2, 1, 3, 4).reshape(B * hkv, n, D)
    v = _values(s["v"][bt], s["vs"][bt], s["kind"]).permute(0, 2, 1, 3, 4).reshape(B * hkv, n, D)
    cu, ctx, T = s["cu"].long(), s["ctx"].long(), s["max_q"]
    t = torch.arange(T, device=bt.device)
    there = t[None, :] < (cu[1:] - cu[:-1])[:, None]  # [B, T]: rows of the padded batch that exist
    at = torch.where(there, cu[:-1, None] + t[None, :], 0)
    q = s["q"].float()[at].reshape(B, T, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B * hkv, -1, D)
    sc = torch.matmul(q, k.transpose(1, 2).contiguous()) * (1.0 / math.sqrt(D))
    i = torch.arange(n, device=bt.device)[None, :] - ctx[:, None]  # place among the drafted tokens
    if s["mask"] is None:
        tree = i[:, None, :] <= t[None, :, None]
    else:
        j = i.clamp(0, 64 * s["mask"].shape[1] - 1)
        bits = torch.gather(s["mask"][at], 2, (j // 64)[:, None, :].expand(B, T, n))
        tree = ((bits >> (j % 64)[:, None, :]) & 1).bool() & (i < T)[:, None, :]
    see = (i < 0)[:, None, :] | tree  # [B, T, n]
    sc = sc.reshape(B, hkv, hq // hkv, T, n).masked_fill(~see[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(sc - m)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = torch.matmul(p.reshape(B * hkv, -1, n), v).reshape(B, hkv, hq // hkv, T, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, D)[there].to(DT[s["io"]])


def _plain_logprobs(s):
    x, V = s["x"].float(), s["V"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total)
    entropy = (lse - ((x - m) * e).sum(-1, keepdim=True) / total).squeeze(-1)
    logp = torch.gather(x, 1, s["ids"].long()) - m - lse
    if not s["k"]:
        return logp, entropy
    # by value, then by lower index: one whole number per logit
    i = (x + 0.0).view(torch.int32)
    i = (i ^ ((i >> 31) & 0x7FFFFFFF)).long()
    key = i * (1 << 32) + (V - 1 - torch.arange(V, device=x.device))[None, :]
    top = torch.topk(key, s["k"], dim=-1).values
    ids = V - 1 - (top & 0xFFFFFFFF)
    return logp, entropy, ids.to(torch.int32), torch.gather(x, 1, ids) - m - lse


def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "rope":
            return _rotated(s["x"].float(), s["pos"], s["table"], s["layout"]).to(DT[s["dst"]])
        if op == "cache":
            return _plain_cache(s)
        return _plain_attention(s) if op == "attention" else _plain_logprobs(s)
    import compressed_linear_amd as cla
    if op == "rope":
        return cla.rope(s["x"], s["pos"], s["table"], layout=s["layout"], out_dtype=DT[s["dst"]])
    if op == "cache":
        s["cache"].append(s["knew"], s["vnew"], s["wslots"], positions=s["pos"], table=s["table"], layout=s["layout"])
        return s["cache"].read(s["rslots"], dtype=DT[s["dst"]])
    if op == "attention":
        return cla.tree_attention(s["q"], s["cache"], s["block_table"], s["ctx"], s["cu"], max_q=s["max_q"],
                                  max_ctx=s["max_ctx"], tree_mask=s["mask"])
    return cla.token_logprobs(s["x"], s["ids"], top_k=s["k"])


# ------------------------------------------------------------------- 64 bits
def _exact_codes(v, kind):
    """Values that a quantised head stands for, from the format's definition, v float64 [..., D]."""
    D = v.shape[-1]
    width, most, big = (D, 127, 65504.0) if kind == "int8" else (32, 7, 8192.0)
    g = v.reshape(*v.shape[:-1], D // width, width)
    s = torch.clamp(g.abs().max(-1, keepdim=True).values / most, max=big)
    s = (s.half() if kind == "int8" else s.bfloat16().half()).double()
    q = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
    return (q.clamp(-most, most) * s).reshape(v.shape)


def _exact_rope(x, pos, table, layout):
    y, n = x.clone(), table.shape[1]
    first = torch.arange(n, device=x.device) * (1 if layout == "half" else 2)
    second = first + (n if layout == "half" else 1)
    c, sn = table.double()[pos.long(), :, 0].unsqueeze(1), table.double()[pos.long(), :, 1].unsqueeze(1)
    y[..., first] = x[..., first] * c - x[..., second] * sn
    y[..., second] = x[..., second] * c + x[..., first] * sn
    return y


def _exact_stored(codes, scales, kind):
    """float64 values of stored rows [..., D]."""
    if kind == "int8":
        return (codes.double() - 128) * scales.double().unsqueeze(-1)
    y = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    y[..., 0::2] = (codes % 16).double() - 8
    y[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double() - 8
    return y * scales.double().repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rope":
        return _exact_rope(s["x"].double(), s["pos"], s["table"], s["layout"])
    if op == "cache":
        kn, vn = s["knew"].double(), s["vnew"].double()
        if s["rot"]:
            kn = _exact_rope(kn, s["pos"], s["table"], s["layout"])
        out, r = [], s["rslots"].long()
        for codes, scales, new in ((s["k"], s["ks"], kn), (s["v"], s["vs"], vn)):
            at = (r // s["page"], r % s["page"])
            old = _exact_stored(codes.transpose(1, 2)[at], scales.transpose(1, 2)[at], s["kind"])
            old[s["read"] - s["write"]:] = _exact_codes(new, s["kind"])  # the new tokens are the last ones read
            out.append(old)
        return tuple(out)
    if op == "attention":
        cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
        group = s["hq"] // s["hkv"]
        outs = []
        for b in range(s["B"]):
            t, n = cu[b + 1] - cu[b], ctx[b] + cu[b + 1] - cu[b]
            pages = s["block_table"][b, :-(-n // s["page"])].long()
            keep = torch.ones(t, n, dtype=torch.bool, device=s["q"].device)
            if s["mask"] is None:
                keep[:, ctx[b]:] = torch.ones(t, t, device=keep.device).tril().bool()
            else:
                for i in range(t):
                    keep[:, ctx[b] + i] = ((s["mask"][cu[b]:cu[b + 1], i // 64] >> (i % 64)) & 1).bool()
            o = torch.empty(t, s["hq"], s["D"], dtype=torch.float64, device=s["q"].device)
            for h in range(s["hkv"]):
                kk = _exact_stored(s["k"][pages, h], s["ks"][pages, h], s["kind"]).reshape(-1, s["D"])[:n]
                vv = _exact_stored(s["v"][pages, h], s["vs"][pages, h], s["kind"]).reshape(-1, s["D"])[:n]
                qq = s["q"][cu[b]:cu[b + 1], h * group:(h + 1) * group].double()
                a = torch.mm(qq.reshape(t * group, -1), kk.t()).reshape(t, group, n) / s["D"] ** 0.5
                a = torch.softmax(a.masked_fill(~keep[:, None, :], -math.inf), -1)
                o[:, h * group:(h + 1) * group] = torch.mm(a.reshape(t * group, n), vv).reshape(t, group, -1)
            outs.append(o)
        return torch.cat(outs)
    x = s["x"].double()
    logp = torch.log_softmax(x, -1)
    p = logp.exp()
    entropy = -(p * logp).sum(-1)
    given = torch.stack([logp[torch.arange(s["T"], device=x.device), s["ids"][:, j].long()] for j in range(s["C"])], 1)
    if not s["k"]:
        return given, entropy
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :s["k"]]
    return given, entropy, order.to(torch.int32), torch.gather(logp, 1, order)
