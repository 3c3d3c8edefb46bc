"""Cases of the verify step's operators: writing the MXFP8 key/value cache, reading it back, attention of a
tree of drafted tokens over it, and the verification of the drafts against the target's logits.

`listed()` holds the named cases, `draw(rng)` gives further ones of the same ranges, `prepare(case, seed)`
makes what a program has in hand before the call, `run(state)` is one pass: in plain torch operations where
`own` is false, through block_scaled_fp8_skinny_amd where it is true. `work(case)` counts the bytes and
operations that a pass cannot do without and `exact(case, seed)` gives the outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32                # values that share one power-of-two scale
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _write(name, rows, hq, hkv, dim, page, norm=True, rot=None, interleaved=False):
    c = dict(op="write", rows=rows, hq=hq, hkv=hkv, dim=dim, page=page, norm=norm,
             rot=dim if rot is None else rot, interleaved=interleaved)
    return dict(c, name=name) if name else c


def _read(name, rows, hkv, dim, page):
    c = dict(op="read", rows=rows, hkv=hkv, dim=dim, page=page)
    return dict(c, name=name) if name else c


def _attn(name, batch, nodes, length, hq, hkv, dim, page, tree, ragged):
    c = dict(op="attention", batch=batch, nodes=nodes, length=length, hq=hq, hkv=hkv, dim=dim, page=page,
             tree=tree, ragged=ragged)
    return dict(c, name=name) if name else c


def _verify(name, tree, batch, nodes, vocab, bf16=False):
    c = dict(op="verify", tree=tree, batch=batch, nodes=nodes, vocab=vocab, bf16=bf16)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's verify step: the root and five drafted tokens, a fused q/k/v projection's output
        _write("write_verify6", 6, 64, 8, 128, 64),
        # a prompt's chunk of an odd number of tokens, half of each head rotated
        _write("write_prompt", 8191, 64, 8, 128, 64, rot=64),
        # a short shared prefix copied out for one rank's heads
        _read("read_prefix", 517, 2, 64, 16),
        # a long prefix copied out whole
        _read("read_long", 65536, 8, 128, 64),
        # plain decode of one sequence: one token, a short cache, one rank's heads
        _attn("decode_b1", 1, 1, 1023, 16, 2, 128, 16, False, False),
        # plain decode of a batch, 64-wide heads without sharing
        _attn("decode_b16_mha64", 16, 1, 4099, 16, 16, 64, 32, False, True),
        # verify of chains of five drafts for a batch, ragged lengths
        _attn("chain_b32", 32, 6, 8192, 64, 8, 128, 64, False, True),
        # a tree of 64 drafted nodes per sequence
        _attn("tree64_b4", 4, 64, 16384, 64, 8, 128, 64, True, False),
        # one long context under a chain of drafts
        _attn("chain_long", 1, 6, 131072, 64, 8, 128, 64, False, False),
        # one sequence's chain on one rank's share of the vocabulary (the draft head's 32768 columns)
        _verify("verify_chain_b1", False, 1, 6, 32768),
        # a batch of chains on four times that
        _verify("verify_chain_b32", False, 32, 6, 131072),
        # trees of drafts for a batch
        _verify("verify_tree_b16", True, 16, 32, 32768),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "verify", "verify"])
    page = rng.choice([16, 32, 48, 64, 128])
    dim = rng.choice([64, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "write":
        hq = hkv * rng.choice([1, 2, 3, 4, 8])
        rows = _log(rng, 1, max(1, (8191 * 80 * 128) // ((hq + 2 * hkv) * dim)))
        return _write(None, rows, hq, hkv, dim, page, rng.random() < 0.75, rng.choice([0, dim, dim // 2]), rng.random() < 0.3)
    if op == "read":
        return _read(None, _log(rng, 1, 65536 * 8 * 128 // (hkv * dim)), hkv, dim, page)
    if op == "attention":
        g = rng.choice([1, 2, 3, 4, 7, 8, 16])
        tree = rng.random() < 0.5
        nodes = _log(rng, 2, 64) if tree else _log(rng, 1, 8)
        batch = _log(rng, 1, 32)
        # no more cache bytes than the long context, no more products than the tree of 64 nodes
        most = min(131072 * 8 * 128 // (batch * hkv * dim), 4 * 16384 * 64 * 64 * 128 // (batch * nodes * g * hkv * dim))
        length = _log(rng, max(nodes, 64), max(nodes, 64, min(most, 131072)))
        return _attn(None, batch, nodes, length, g * hkv, hkv, dim, page, tree, rng.random() < 0.6)
    tree = rng.random() < 0.5
    vocab = _log(rng, 1000, 131072)
    nodes = _log(rng, 2, 64) if tree else rng.randint(2, 8)
    batch = _log(rng, 1, max(1, min(64, 32 * 11 * 131072 // ((nodes if tree else 2 * nodes - 1) * vocab))))
    return _verify(None, tree, batch, nodes, vocab, rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _quantize(x):
    """fp32 [..., D] -> (e4m3 codes [..., D], scale bytes [..., D/32]): 2^s with s = floor(log2 amax) - 8
    per 32 values, values rounded to nearest even and saturated at 448."""
    b = x.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 9, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    q = torch.ldexp(b, -s.unsqueeze(-1)).clamp(-448, 448).to(torch.float32).to(F8)
    return q.flatten(-2).view(torch.uint8), (s + 127).to(torch.uint8)


def _random_cache(g, pages, heads, page, dim):
    """A cache that has been in use: every slot holds some token's values."""
    out = []
    for scale in (1.0, 0.7):
        x = torch.randn(pages, heads, page, dim, generator=g, device=DEV, dtype=torch.bfloat16).float() * scale
        out += _quantize(x)
        del x
    return out


def _prepare_write(c, g):
    R, hq, hkv, D, page = c["rows"], c["hq"], c["hkv"], c["dim"], c["page"]
    x = torch.randn(R, (hq + 2 * hkv) * D, generator=g, device=DEV).to(torch.bfloat16)   # a fused projection's rows
    q, k, v = x.split([hq * D, hkv * D, hkv * D], 1)
    n = (R + R // 4) // page + 2
    slots = torch.randperm(n * page, generator=g, device=DEV)[:R]
    start = int(torch.randint(0, 4096, (1,), generator=g, device=DEV))
    pos = torch.arange(start, start + R, device=DEV)
    s = dict(q=q, k=k, v=v, slots=slots, positions=pos, cache=[
        torch.zeros(n, hkv, page, w, dtype=torch.uint8, device=DEV) for w in (D, D // BLOCK, D, D // BLOCK)])
    s["q_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
    s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None
    s["table"] = None
    if c["rot"]:
        half = c["rot"] // 2
        a = torch.arange(start + R, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["table"] = torch.cat([a.cos(), a.sin()], 1).float()
    s["q_out"] = torch.empty(R, hq, D, dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_read(c, g):
    R, page = c["rows"], c["page"]
    n = R // page + 2
    s = dict(cache=_random_cache(g, n, c["hkv"], page, c["dim"]))
    pages = torch.randperm(n, generator=g, device=DEV)          # a sequence's pages, in its order
    t = torch.arange(R, device=DEV)
    s["slots"] = pages[t // page] * page + t % page
    s["k_out"], s["v_out"] = (torch.empty(R, c["hkv"], c["dim"], dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return s


def _tree(g, batch, nodes):
    """Random trees, every node after its parent, and the mask of each node's ancestors and itself."""
    r = torch.rand(batch, nodes, generator=g, device=DEV).cpu().tolist()
    parents = [[-1] + [int(r[b][n] * n) for n in range(1, nodes)] for b in range(batch)]
    masks = []
    for p in parents:
        m = [1]
        for n in range(1, nodes):
            m.append(m[p[n]] | 1 << n)
        masks.append([v - (1 << 64) if v >= 1 << 63 else v for v in m])
    return (torch.tensor(parents, dtype=torch.int32, device=DEV), torch.tensor(masks, dtype=torch.int64, device=DEV))


def _prepare_attention(c, g):
    B, T, L, page = c["batch"], c["nodes"], c["length"], c["page"]
    if c["ragged"]:
        lens = torch.randint(min(L, max(T, L // 8)), L + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        lens[0] = L
        nodes = torch.randint(max(1, T - 2), T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    else:
        lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
        nodes = None
    width = (L + page - 1) // page
    n = B * width + 1
    s = dict(cache=_random_cache(g, n, c["hkv"], page, c["dim"]), lens=lens, nodes=nodes, max_len=L)
    s["pages"] = torch.randperm(n, generator=g, device=DEV)[: B * width].view(B, width).to(torch.int32)
    s["mask"] = _tree(g, B, T)[1] if c["tree"] else None
    s["scale"] = c["dim"] ** -0.5
    s["q"] = torch.randn(B, T, c["hq"], c["dim"], generator=g, device=DEV).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_verify(c, g):
    B, T, V = c["batch"], c["nodes"], c["vocab"]
    dt = torch.bfloat16 if c["bf16"] else torch.float32
    logits = (3 * torch.randn(B, T, V, generator=g, device=DEV)).to(dt)
    temperature = 0.6 + 0.6 * torch.rand(B, generator=g, device=DEV)
    temperature[1::4] = 0                                        # some requests decode greedily
    s = dict(logits=logits, temperature=temperature)
    if c["tree"]:
        s["parents"], s["mask"] = _tree(g, B, T)
        rank = [[sum(q == p for q in row[:n]) for n, p in enumerate(row)] for row in s["parents"].tolist()]
        rank = torch.tensor(rank, device=DEV)                    # the drafter takes its best guesses in order
        near = (logits.float() + 0.3 * torch.randn(B, T, V, generator=g, device=DEV)).topk(min(V, T), -1).indices
        at = s["parents"].long().clamp(min=0)
        s["tokens"] = near[torch.arange(B, device=DEV)[:, None], at, rank].to(torch.int32)
        s["u"] = torch.rand(B, T, generator=g, device=DEV)
    else:
        s["draft"] = (0.9 * logits[:, : T - 1].float() + torch.randn(B, T - 1, V, generator=g, device=DEV)).to(dt)
        t = temperature.clamp(min=0.01)[:, None, None]
        p = torch.softmax(s["draft"].float() / t, -1)
        s["tokens"] = torch.multinomial(p.flatten(0, 1), 1, generator=g).view(B, T - 1).to(torch.int32)
        s["u"] = torch.rand(B, T - 1, generator=g, device=DEV)
        s["u_sample"] = torch.rand(B, generator=g, device=DEV)
    s["out"] = [torch.empty(B, T, dtype=torch.int32, device=DEV), torch.empty(B, T, dtype=torch.int32, device=DEV),
                torch.empty(B, dtype=torch.int32, device=DEV)]
    return s


def prepare(case, seed):
    s = {"write": _prepare_write, "read": _prepare_read, "attention": _prepare_attention, "verify": _prepare_verify}[case["op"]](case, _gen(seed))
    s["case"] = case
    if own:   # the handle and the workspace that a program keeps beside its tensors
        import block_scaled_fp8_skinny_amd as L
        s["lib"] = L
        if "cache" in s:
            s["handle"] = L.KVCache(*s["cache"])
        if case["op"] == "attention":
            s["ws"] = L.workspace_attention(case["batch"], case["nodes"], case["hq"], case["hkv"], case["dim"], case["length"])
        elif case["op"] == "verify":
            s["ws"] = L.workspace_verify(case["batch"], case["nodes"], case["vocab"])
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _norm_rotate(x, weight, table, pos, rot, interleaved):
    """fp32 [R, H, D]: the root-mean-square norm over D, then the rotation of the first `rot` values."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    if rot:
        cos, sin = table[pos].unsqueeze(1).chunk(2, -1)
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
        y = [a * cos - b * sin, b * cos + a * sin]
        y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
        x = torch.cat([y, x[..., rot:]], -1)
    return x


def _cache_views(cache):
    return [t.view(F8 if i % 2 == 0 else E8) for i, t in enumerate(cache)]


def _run_write(s):
    c = s["case"]
    q, k, v = (s[n].unflatten(1, (-1, c["dim"])) for n in "qkv")
    if own:
        s["lib"].bsfp8_cache_write(s["handle"], s["slots"], k, v, q=q, q_out=s["q_out"], q_weight=s["q_weight"],
                                   k_weight=s["k_weight"], eps=1e-6, cos_sin=s["table"], positions=s["positions"],
                                   interleaved=c["interleaved"])
        return [s["q_out"]] + _cache_views(s["cache"])
    q = _norm_rotate(q, s["q_weight"], s["table"], s["positions"], c["rot"], c["interleaved"]).to(torch.bfloat16)
    k = _norm_rotate(k, s["k_weight"], s["table"], s["positions"], c["rot"], c["interleaved"])
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    for t, x in zip(s["cache"], (*_quantize(k), *_quantize(v.float()))):
        t[page, :, at] = x
    return [q] + _cache_views(s["cache"])


def _dequantize(codes, scales):
    f = torch.ldexp(torch.ones((), device=DEV), scales.to(torch.int32) - 127)
    return (codes.view(F8).float().unflatten(-1, (-1, BLOCK)) * f.unsqueeze(-1)).flatten(-2)


def _run_read(s):
    if own:
        return s["lib"].bsfp8_cache_read(s["handle"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    c = s["case"]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    kq, ks, vq, vs = (t[page, :, at] for t in s["cache"])
    return _dequantize(kq, ks).to(torch.bfloat16), _dequantize(vq, vs).to(torch.bfloat16)


def _run_attention(s):
    c = s["case"]
    if own:
        return s["lib"].bsfp8_tree_attention(s["q"], s["handle"], s["pages"], s["lens"], nodes=s["nodes"], mask=s["mask"],
                                             scale=s["scale"], max_len=s["max_len"], ws=s["ws"], out=s["out"])
    B, T, D, H = c["batch"], c["nodes"], c["dim"], c["hkv"]
    kq, ks, vq, vs = (t[s["pages"].long()].transpose(2, 3).flatten(1, 2).transpose(1, 2) for t in s["cache"])   # [B, H, L, *]
    at = torch.arange(kq.shape[2], device=DEV)
    here = s["nodes"].long() if s["nodes"] is not None else torch.full((B,), T, device=DEV)
    node = at[None] - (s["lens"].long() - here)[:, None]                       # [B, L], below 0: the prefix
    row = torch.arange(T, device=DEV)
    if s["mask"] is None:
        seen = node[:, None] <= row[None, :, None]
    else:
        seen = (node[:, None] < 0) | ((s["mask"][:, :, None] >> node[:, None].clamp(0, 63)) & 1).bool()
    seen = seen & (node[:, None] < here[:, None, None]) & (row[None, :, None] < here[:, None, None])   # [B, T, L]
    q = s["q"].float().view(B, T, H, -1, D).permute(0, 2, 3, 1, 4).flatten(2, 3)                        # [B, H, g*T, D]
    x = q @ _dequantize(kq, ks).transpose(2, 3) * s["scale"]
    x = x.unflatten(2, (-1, T)).masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = torch.where((node < here[:, None])[:, None, :, None], _dequantize(vq, vs), 0)
    o = (x.flatten(2, 3) @ v).unflatten(2, (-1, T)) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, -1, D).to(torch.bfloat16)


def _probabilities(logits, temperature):
    """In 64 bits, since the decisions below compare neighbouring sums; temperature 0 puts all on the largest."""
    x = logits.double()
    t = temperature.double()[:, None, None]
    e = torch.exp((x - x.amax(-1, keepdim=True)) / torch.where(t > 0, t, 1))
    best = x.argmax(-1, keepdim=True)
    hot = torch.zeros_like(x).scatter_(-1, best, 1.0)
    return torch.where(t > 0, e / e.sum(-1, keepdim=True), hot)


def _pick(w, u):
    """The first index whose running sum of the weights passes u times their sum."""
    total = w.cumsum(-1)
    at = torch.searchsorted(total, u.double()[..., None] * total[..., -1:], right=True)
    last = (w > 0).to(torch.int64).cumsum(-1).argmax(-1, keepdim=True)
    return torch.minimum(at, last).squeeze(-1)


def _run_verify(s):
    c = s["case"]
    T = c["nodes"]
    tokens, path, count = s["out"]
    if own and c["tree"]:
        return s["lib"].bsfp8_verify_tree(s["logits"], s["tokens"], s["parents"], s["temperature"], s["u"], ws=s["ws"],
                                          out_tokens=tokens, path=path, n_accepted=count)
    if own:
        return s["lib"].bsfp8_verify_chain(s["logits"], s["draft"], s["tokens"], s["temperature"], s["u"], s["u_sample"],
                                           ws=s["ws"], out_tokens=tokens, n_accepted=count)
    p = _probabilities(s["logits"], s["temperature"])
    place = torch.arange(T, device=DEV)
    if c["tree"]:
        mine = _pick(p, s["u"])                                               # each node's sampled next token
        up = s["parents"].long()
        ok = s["tokens"] == mine.gather(1, up.clamp(min=0))
        twin = (up[:, :, None] == up[:, None]) & (s["tokens"][:, :, None] == s["tokens"][:, None]) & (place[None, :] < place[:, None])
        ok = (ok & ~twin.any(-1)) | (place == 0)
        line = ((s["mask"][:, :, None] >> place) & 1).bool()                  # a node's ancestors and itself
        ok = (ok[:, None] | ~line).all(-1)
        n = ok.sum(-1)
        path = torch.where(ok, place, T).sort(-1).values                      # ancestors come first
        leaf = path.gather(1, n[:, None] - 1)
        path = torch.where(place < n[:, None], path, -1)
        inner = torch.cat([path[:, 1:], torch.full_like(path[:, :1], -1)], 1)
        out = torch.where(inner >= 0, s["tokens"].long().gather(1, inner.clamp(min=0)), -1)
        out = torch.where(place == n[:, None] - 1, mine.gather(1, leaf), out)
        return out.int(), path.int(), (n - 1).int()
    q = _probabilities(s["draft"], s["temperature"])
    x = s["tokens"].long()[..., None]
    ok = s["u"].double() * q.gather(-1, x).squeeze(-1) < p[:, :-1].gather(-1, x).squeeze(-1)
    greedy = s["temperature"][:, None] == 0
    ok = torch.where(greedy, p[:, :-1].gather(-1, x).squeeze(-1) > 0, ok)
    n = ok.long().cumprod(-1).sum(-1)
    at = n[:, None, None].expand(-1, 1, c["vocab"])
    mine = p.gather(1, at).squeeze(1)
    rest = (mine - q.gather(1, at.clamp(max=T - 2)).squeeze(1)).clamp(min=0)
    rest = torch.where(((n < T - 1) & (rest.sum(-1) > 0))[:, None] & ~greedy, rest, mine)
    out = torch.cat([s["tokens"].long(), torch.full_like(n[:, None], -1)], 1)
    out = torch.where(place < n[:, None], out, torch.where(place == n[:, None], _pick(rest, s["u_sample"])[:, None], -1))
    return out.int(), n.int()


def run(state):
    return {"write": _run_write, "read": _run_read, "attention": _run_attention, "verify": _run_verify}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "write":
        R, D = c["rows"], c["dim"]
        read = R * ((c["hq"] + 2 * c["hkv"]) * D * 2 + 16 + 4 * c["rot"])
        wrote = R * (c["hq"] * D * 2 + 2 * c["hkv"] * (D + D // BLOCK))
        return {"bytes": read + wrote, "flops": R * D * 10 * (c["hq"] + 2 * c["hkv"])}
    if c["op"] == "read":
        n = c["rows"] * c["hkv"] * c["dim"]
        return {"bytes": 2 * n * (1 + 1 / BLOCK + 2) + 8 * c["rows"], "flops": 2 * n}
    if c["op"] == "attention":
        # ragged lengths lie evenly between an eighth of the largest and the largest
        mean = c["length"] * (0.5625 if c["ragged"] and c["batch"] > 1 else 1.0)
        tokens, D = c["batch"] * mean, c["dim"]
        cache = tokens * c["hkv"] * 2 * (D + D // BLOCK) + 4 * tokens / c["page"]
        return {"bytes": cache + 4 * c["batch"] * c["nodes"] * c["hq"] * D, "flops": 4 * tokens * c["nodes"] * c["hq"] * D}
    rows = c["batch"] * (c["nodes"] if c["tree"] else 2 * c["nodes"] - 1)
    return {"bytes": rows * c["vocab"] * (2 if c["bf16"] else 4), "flops": 4 * rows * c["vocab"]}


# ------------------------------------------------------------------------------------------------
# the outputs in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------------
def _values(codes, scales):
    """e4m3 codes and scale bytes as 64-bit values, from the bit fields."""
    b = codes.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, (e - 10).double()))
    s = torch.pow(2.0, scales.double() - 127).repeat_interleave(BLOCK, -1)
    return torch.where(b >= 128, -mag, mag) * s


def _exact_heads(x, w, s, c):
    x = x.double().reshape(c["rows"], -1, c["dim"])
    if w is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * w.double()
    if c["rot"]:
        h = c["rot"] // 2
        i = torch.arange(h, device=DEV)
        ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + h)
        z = torch.complex(x[..., ia], x[..., ib])
        t = s["table"][s["positions"]].double()
        z = z * torch.complex(t[:, :h], t[:, h:])[:, None]
        x[..., ia], x[..., ib] = z.real, z.imag
    return x


def _exact_codes(x):
    """64-bit values -> the values of the nearest e4m3 codes and of the scale bytes."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, torch.floor(torch.log2(torch.where(top > 0, top, 1))) - 8, -127.0).clamp(-127, 127)
    y = b * torch.pow(2.0, -s)
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448).reshape(x.shape), torch.pow(2.0, s).squeeze(-1)


def exact(case, seed):
    c = case
    if c["op"] == "verify":
        return None                                   # tokens and counts: whole numbers
    s = prepare(case, seed)
    if c["op"] == "write":
        found = [_exact_heads(s["q"], s["q_weight"], s, c)]
        for x, w, t in ((s["k"], s["k_weight"], 0), (s["v"], None, 2)):
            x = _exact_heads(x, w, s, c) if t == 0 else x.double().reshape(c["rows"], -1, c["dim"])
            for values, old in zip(_exact_codes(x), s["cache"][t: t + 2]):
                full = torch.zeros(old.shape, dtype=torch.float64, device=DEV) if values.shape[-1] == c["dim"] else torch.full(
                    old.shape, 2.0 ** -127, dtype=torch.float64, device=DEV)
                view = full.permute(0, 2, 1, 3)
                view[s["slots"] // c["page"], s["slots"] % c["page"]] = values
                found.append(full)
        return found
    if c["op"] == "read":
        page, at = s["slots"] // c["page"], s["slots"] % c["page"]
        kq, ks, vq, vs = (t.permute(0, 2, 1, 3)[page, at] for t in s["cache"])
        return [_values(kq, ks), _values(vq, vs)]
    B, T, D, H = c["batch"], c["nodes"], c["dim"], c["hkv"]
    out = torch.zeros(B, T, c["hq"], D, dtype=torch.float64, device=DEV)
    kq, ks, vq, vs = s["cache"]
    for b in range(B):
        n = int(s["lens"][b])
        t = T if s["nodes"] is None else int(s["nodes"][b])
        pages = s["pages"][b, : -(-n // c["page"])].long()
        seen = torch.ones(t, n, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            seen[:, n - t:] = torch.ones(t, t, device=DEV).tril().bool()
        else:
            seen[:, n - t:] = ((s["mask"][b, :t, None] >> torch.arange(t, device=DEV)) & 1).bool()
        for h in range(H):
            k, v = (_values(x[pages, h].reshape(-1, D)[:n], y[pages, h].reshape(-1, D // BLOCK)[:n]) for x, y in ((kq, ks), (vq, vs)))
            g = c["hq"] // H
            q = s["q"][b, :t, h * g: h * g + g].double()                       # [t, g, D]
            z = (q.reshape(-1, D) @ k.T * s["scale"]).reshape(t, g, n).masked_fill(~seen[:, None], -math.inf)
            out[b, :t, h * g: h * g + g] = (torch.softmax(z, -1).reshape(-1, n) @ v).reshape(t, g, D)
    return out
