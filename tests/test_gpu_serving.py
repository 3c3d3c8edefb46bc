"""GPU parity of the verify step's operators with oracle/serving.py (float64): the MXFP8 cache written and read, attention
of drafted tokens over it, and the verification of the drafts, at the sizes, masks and values where they can go wrong.

Tolerances (u = the half step of a type: bf16 2^-8, fp32 2^-24), fixed before the first run:
  * q_out: the bf16 rounding, plus the fp32 arithmetic of the norm and rotation (dim + 16 roundings of |a| + |b|);
  * cached values: half a step of e4m3 at the stored scale plus the same fp32 arithmetic, saturation at 448 scales; the
    scale is the rule's on the exact maximum, or its neighbour's where the maximum lies within the arithmetic of a power
    of two; bit for bit where nothing is computed (values, and keys without norm and rotation);
  * attention: bf16 of the result, u_bf16 for the weights' rounding and twice the scores' fp32 error (dim + 8 roundings of
    sum |q k| scale) and the fp32 sums, all on sum w |v|;
  * read, verification: equal.
"""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
import oracle.formats as F
import oracle.mx as MX
import oracle.serving as SV

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24


def bf16(r, shape, scale=1.0):
    """Seeded bf16 normals on the GPU, and their float64 values."""
    t = torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def cache_of(r, pages, heads, page, dim, special=True):
    """A cache in use (random codes and scales), and its values [slots, heads, dim] for K and V."""
    kq, vq = (r.integers(0, 256, (pages, heads, page, dim), dtype=np.uint8) for _ in range(2))
    for q in (kq, vq):
        q[(q & 0x7F) == 0x7F] = 0x12
    ks, vs = (r.integers(118, 124, (pages, heads, page, dim // 32), dtype=np.uint8) for _ in range(2))
    c = B.KVCache(*(torch.from_numpy(a).cuda() for a in (kq, ks, vq, vs)))
    vals = [SV.cache_values(q, s).transpose(0, 2, 1, 3).reshape(-1, heads, dim) for q, s in ((kq, ks), (vq, vs))]
    return c, vals[0], vals[1]


# ------------------------------------------------------------------------------------------------
# write
# ------------------------------------------------------------------------------------------------
WRITES = [  # rows, hq, hkv, dim, page, norm, rot, interleaved
    (1, 1, 1, 64, 16, False, 0, False),
    (1, 8, 2, 128, 64, True, 128, False),
    (5, 6, 2, 64, 48, True, 32, False),
    (7, 3, 3, 192, 16, True, 96, True),
    (33, 4, 1, 192, 32, True, 192, False),
    (6, 64, 8, 128, 64, True, 64, True),
    (9, 10, 5, 256, 128, True, 256, False),
    (300, 2, 1, 256, 16, False, 16, True),
    (3000, 0, 2, 64, 32, False, 64, False),
]


@pytest.mark.parametrize("case", WRITES, ids=lambda c: "R%d_q%d_kv%d_D%d_p%d_n%d_r%d_i%d" % c)
def test_write(case):
    R, hq, hkv, D, page, norm, rot, inter = case
    print("write", case, flush=True)
    r = np.random.default_rng(100 + R + D)
    xt, x = bf16(r, (R, (hq + 2 * hkv) * D + 8))                 # a row stride wider than the heads
    qt, kt, vt = (xt[:, a: a + n * D] for a, n in ((0, hq), (hq * D, hkv), ((hq + hkv) * D, hkv)))
    q, k, v = (x[:, a: a + n * D].reshape(R, n, D) for a, n in ((0, hq), (hq * D, hkv), ((hq + hkv) * D, hkv)))
    n_pages = R // page + 3
    slots = r.permutation(n_pages * page)[:R].astype(np.int64)
    if R > 4:
        slots[1], slots[3] = -1, n_pages * page                  # stored nowhere
    qw, kw = (bf16(r, (D,)) for _ in range(2)) if norm else ((None, None),) * 2
    pos = r.integers(0, 50, R)
    ang = r.uniform(-3, 3, (50, max(rot, 2) // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    c, s = (table[pos, : rot // 2].astype(np.float64), table[pos, rot // 2:].astype(np.float64)) if rot else (None, None)
    cache = B.KVCache.empty(n_pages, hkv, page, D)
    for t in (cache.kq, cache.vq, cache.ks, cache.vs):
        t.fill_(0x55)
    out = B.bsfp8_cache_write(cache, torch.from_numpy(slots).cuda(), kt, vt, q=qt if hq else None,
                              q_weight=qw[0] if hq else None, k_weight=kw[0], eps=1e-6,
                              cos_sin=torch.from_numpy(table).cuda() if rot else None,
                              positions=torch.from_numpy(pos).cuda() if rot else None, interleaved=inter)
    torch.cuda.synchronize()
    err = (D + 16) * U32                                         # per unit of |a| + |b|
    if hq:
        want = SV.head_values(q, qw[1], 1e-6, c, s, inter)
        amp = np.abs(SV.head_values(q, qw[1], 1e-6))             # a rotated value's terms are at most its pair's
        amp = amp + amp.max(-1, keepdims=True) * (rot > 0)
        assert np.all(np.abs(f64(out) - want) <= U16 * np.abs(want) + (1 + U16) * err * amp)
    else:
        assert out is None
    want = SV.head_values(k, kw[1], 1e-6, c, s, inter)
    amp = np.abs(SV.head_values(k, kw[1], 1e-6)).max(-1, keepdims=True) * (2 if norm or rot else 0)
    live = (slots >= 0) & (slots < n_pages * page)
    pg, off = slots[live] // page, slots[live] % page
    got_q, got_s = cache.kq.cpu().numpy()[pg, :, off], cache.ks.cpu().numpy()[pg, :, off]
    wq, ws = MX.quantize_mx_values(want[live].reshape(-1, D))
    wq, ws = wq.reshape(got_q.shape), ws.reshape(got_s.shape)
    if not norm and not rot:
        assert np.array_equal(got_q, wq) and np.array_equal(got_s, ws)
    amax = np.abs(want[live]).reshape(*got_s.shape, 32).max(-1)
    lo, hi = (MX.mx_scale_exponent(np.maximum(amax + d * err * amp[live], 0)) + 127 for d in (-1, 1))
    assert np.all((got_s >= lo) & (got_s <= hi))
    sc = np.repeat(np.exp2(got_s.astype(np.float64) - 127), 32, -1)
    near = np.clip(want[live], -448 * sc, 448 * sc)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(near), 1e-300) / sc)), -6) - 3) * sc
    assert np.all(np.abs(SV.cache_values(got_q, got_s) - near) <= step / 2 * (1 + 1e-3) + err * amp[live])
    wq, ws = MX.quantize_mx_values(v[live].reshape(-1, D))
    assert np.array_equal(cache.vq.cpu().numpy()[pg, :, off].reshape(-1, D), wq)
    assert np.array_equal(cache.vs.cpu().numpy()[pg, :, off].reshape(-1, D // 32), ws)
    free = np.ones(n_pages * page, bool)                         # every other slot is as it was
    free[slots[live]] = False
    for t in (cache.kq, cache.vq, cache.ks, cache.vs):
        assert np.all(t.cpu().numpy().transpose(0, 2, 1, 3).reshape(n_pages * page, -1)[free] == 0x55)


def test_write_nonfinite_and_extreme_values():
    """Blocks of zeros, infinities, NaN, the largest and the smallest bf16 values, and a position outside the table."""
    D, R = 64, 6
    x = torch.ones(R, D, dtype=torch.bfloat16)
    x[0] = 0
    x[1, 3], x[1, 40] = float("inf"), -float("inf")
    x[2, 5] = float("nan")
    x[3] = torch.finfo(torch.bfloat16).max
    x[4] = 2.0 ** -133
    cache = B.KVCache.empty(1, 1, 16, D)
    B.bsfp8_cache_write(cache, torch.arange(R).cuda(), x.cuda(), x.cuda())
    wq, ws = MX.quantize_mx_values(x.double().numpy())
    for q, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)):
        assert np.array_equal(q[0, 0, :R].cpu().numpy(), wq) and np.array_equal(s[0, 0, :R].cpu().numpy(), ws)
    table = torch.ones(4, 32).cuda()
    q_out = B.bsfp8_cache_write(cache, torch.arange(2).cuda(), x[4:].cuda(), x[4:].cuda(), q=x[4:].cuda(), cos_sin=table,
                                positions=torch.tensor([4, -1]).cuda())
    assert q_out[..., :32].isnan().all() and not q_out[..., 32:].isnan().any()
    assert (cache.ks[0, 0, :2, 0] == 255).all() and (cache.ks[0, 0, :2, 1] != 255).all()


# ------------------------------------------------------------------------------------------------
# read
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("R,heads,dim,page", [(1, 1, 64, 16), (517, 2, 64, 16), (40, 3, 192, 48), (33, 5, 256, 32), (64, 8, 128, 64)])
def test_read(R, heads, dim, page):
    print("read", R, heads, dim, page, flush=True)
    r = np.random.default_rng(7)
    n = R // page + 2
    codes, scales = (r.integers(0, 256, (2, n, heads, page, w), dtype=np.uint8) for w in (dim, dim // 32))
    c = B.KVCache(*(torch.from_numpy(a).cuda() for a in (codes[0], scales[0], codes[1], scales[1])))
    slots = r.integers(0, n * page, R)
    slots[R // 2] = -1 if R > 1 else 0
    out = B.bsfp8_cache_read(c, torch.from_numpy(slots).cuda())
    for got, q, s in zip(out, codes, scales):
        with np.errstate(over="ignore"):
            want = SV.cache_values(q, s).transpose(0, 2, 1, 3).reshape(n * page, heads, dim)[slots]
            want[slots < 0] = 0
            want = F.round_bf16(want)
        assert np.array_equal(f64(got), want, equal_nan=True)


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def attend(seed, T, hq, hkv, dim, page, lens, nodes=None, tree=False, max_len=None, scale=None, wide=0, spoil=None, table=None,
           launch=None):
    """One call and its check against the oracle; returns the output."""
    r = np.random.default_rng(seed)
    Bn = len(lens)
    W = max(1, -(-max(max(lens), 1) // page))
    n_pages = Bn * W + 1
    cache, K, V = cache_of(r, n_pages, hkv, page, dim)
    pages = r.permutation(n_pages)[: Bn * W].reshape(Bn, W).astype(np.int32)
    if table:
        table(pages, n_pages)
    mask = None
    if tree:
        mask = np.zeros((Bn, T), np.int64)
        for b in range(Bn):
            for t in range(T):
                up = int(mask[b, r.integers(0, t)]) if t else 0
                mask[b, t] = np.int64(np.uint64((up & (2 ** 64 - 1)) | 1 << t))
        if T > 2:
            mask[0, T - 1] = 0
    if spoil:
        spoil(cache, K, V, pages)
    qt, q = bf16(r, (Bn, T, hq * dim + wide), 1.0)
    q = q[..., : hq * dim].reshape(Bn, T, hq, dim)
    qv = qt[..., : hq * dim].unflatten(-1, (hq, dim))
    dev = lambda a: torch.from_numpy(np.asarray(a)).cuda()
    ln = np.asarray(lens, np.int32)
    nd = None if nodes is None else np.asarray(nodes, np.int32)
    args = (qv, cache, dev(pages), dev(ln))
    kw = dict(nodes=None if nd is None else dev(nd), mask=None if mask is None else dev(mask), scale=scale, max_len=max_len)
    print("attention", seed, T, hq, hkv, dim, page, lens, nodes, tree, max_len, flush=True)
    out = launch(args, kw) if launch else B.bsfp8_tree_attention(*args, **kw)
    torch.cuda.synchronize()
    got = f64(out)
    scale = dim ** -0.5 if scale is None else scale
    for b in range(Bn):
        n = int(min(ln[b], W * page if max_len is None else min(max_len, W * page)))
        here = T if nd is None else int(min(max(nd[b], 0), T))
        slots = SV.gather(pages[b], page, n_pages, n)
        see = SV.visible(T, n, here, None if mask is None else mask[b]) & (slots >= 0)
        want, mag, big = SV.attention(q[b], K[slots], V[slots], see, scale)
        tol = U16 * np.abs(want) + (U16 + 2 * (dim + 8) * U32 * big + (n + 8) * U32) * mag + 1e-30
        ok = np.abs(got[b] - want) <= tol
        ok |= np.isnan(want) & np.isnan(got[b])
        assert ok.all(), (b, np.argwhere(~ok)[:4], got[b][~ok][:4], want[~ok][:4])
    return out


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_attention_decode_lengths(dim, page):
    attend(1, 1, 4, 2, dim, page, [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300])


@pytest.mark.parametrize("g,T", [(1, 1), (1, 6), (2, 6), (3, 5), (4, 4), (7, 5), (8, 6), (16, 3), (5, 13)])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_attention_chains(g, T, dim):
    attend(2 + g, T, 2 * g, 2, dim, 32, [T, T + 1, 200, 517], nodes=[T, T - 1, 0, max(1, T - 2)])


@pytest.mark.parametrize("g,T", [(1, 64), (8, 16), (3, 33), (16, 64), (2, 2)])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (192, 48), (256, 16)])
def test_attention_trees(g, T, dim, page):
    attend(20 + g, T, g, 1, dim, page, [T, 3 * T + 5, 450], nodes=[T, T, T - 1], tree=True)


def test_attention_more_nodes_than_tokens():
    """A sequence shorter than its node count: the first nodes lie before its start, rows without a position are zeros."""
    attend(40, 6, 4, 2, 64, 16, [3, 0, 6], tree=True)
    attend(41, 6, 4, 2, 128, 16, [3, 1, 6])


def test_attention_long_chain_without_mask():
    attend(42, 150, 2, 1, 64, 16, [150, 400], nodes=[150, 131])


def test_attention_split_over_workgroups():
    """One long sequence beside short ones: every head is shared by many workgroups, joined by the second kernel."""
    attend(43, 2, 2, 1, 64, 64, [9000, 1, 130, 0, 5000])
    attend(44, 6, 8, 1, 128, 16, [6000])
    attend(45, 3, 4, 2, 256, 128, [70, 4000])


def test_attention_many_short_sequences():
    attend(46, 1, 2, 2, 64, 16, list(range(150)))


def test_attention_large_and_small_scores():
    attend(47, 4, 4, 2, 128, 32, [333, 64], scale=4.0)
    attend(48, 4, 4, 2, 128, 32, [333, 64], scale=-0.3)
    attend(49, 2, 2, 2, 64, 32, [100], scale=0.0)


def test_attention_strided_queries_and_bounds():
    attend(50, 5, 4, 2, 64, 16, [100, 37], wide=24)
    attend(51, 2, 2, 1, 64, 16, [300, 100], max_len=160)         # lengths above the bound are cut


def test_attention_absent_pages():
    def table(pages, n):
        pages[0, 1], pages[1, 0], pages[2, :] = -1, n, 2 ** 30
    attend(52, 3, 4, 2, 128, 16, [100, 50, 40], table=table)
    attend(53, 3, 4, 2, 64, 48, [100, 50, 40], table=table, tree=True)


def test_attention_nonfinite_leftovers_stay_unseen():
    """NaN keys and values past the sequence's end, in other nodes and in absent pages reach no row that does not see
    them; a NaN that a row sees makes it NaN."""
    def spoil(cache, K, V, pages):
        for t in (cache.kq, cache.vq):
            t[int(pages[0, 2]), :, 8:] = 0x7F                    # positions 40.. of sequence 0 (41 long): node 5 and the rest
        cache.ks[int(pages[1, 0]), :, 14] = 255                  # position 14 of sequence 1: its node 2 of 4
        cache.vs[int(pages[1, 0]), :, 14] = 255
        for t, x in ((cache.kq, K), (cache.vq, V)):
            x[int(pages[0, 2]) * 16 + 8: int(pages[0, 2]) * 16 + 16] = np.nan
            x[int(pages[1, 0]) * 16 + 14] = np.nan
    for dim in (64, 128, 192, 256):
        out = attend(54, 6, 4, 2, dim, 16, [41, 16], nodes=[6, 4], spoil=spoil)
        assert out[0, 5].isnan().all() and not out[0, :5].isnan().any()
        assert out[1, 2:4].isnan().all() and not out[1, :2].isnan().any() and not out[1, 4:].any()


def test_attention_on_another_stream_and_in_a_graph():
    keep = {}

    def launch(args, kw):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = B.bsfp8_tree_attention(*args, **kw)
        torch.cuda.current_stream().wait_stream(side)
        keep.update(args=args, kw=kw, out=out)
        return out
    attend(60, 6, 16, 2, 128, 32, [500, 77, 1300], nodes=[6, 3, 5], launch=launch)
    args, kw, eager = keep["args"], keep["kw"], keep["out"].clone()
    q, cache = args[0], args[1]
    ws = B.workspace_attention(q.shape[0], q.shape[1], q.shape[2], cache.heads, cache.dim, args[2].shape[1] * cache.page)
    out = torch.empty_like(eager)
    B.bsfp8_tree_attention(*args, **kw, ws=ws, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.bsfp8_tree_attention(*args, **kw, ws=ws, out=out)
    for _ in range(3):
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))


# ------------------------------------------------------------------------------------------------
# verification
# ------------------------------------------------------------------------------------------------
def _logits(r, shape, dt, spread=2.0):
    return torch.from_numpy((spread * r.standard_normal(shape)).astype(np.float32)).to(dt).cuda()


def _check_chain(lg, dr, tok, t, u, us, ws=None):
    Bn, T, V = lg.shape
    print("chain", Bn, T, V, lg.dtype, flush=True)
    dev = lambda a, d: torch.from_numpy(np.ascontiguousarray(a, d)).cuda()
    out, n = B.bsfp8_verify_chain(lg, dr, dev(tok, np.int32), dev(t, np.float32), dev(u, np.float32), dev(us, np.float32), ws=ws)
    for b in range(Bn):
        wo, wn = SV.verify_chain(f64(lg[b]), f64(dr[b]), tok[b], float(np.float32(t[b])), np.float32(u[b]).astype(np.float64),
                                 float(np.float32(us[b])))
        assert int(n[b]) == wn and np.array_equal(out[b].cpu().numpy(), wo), (b, out[b], wo, n[b], wn)
    return out, n


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 5), (2, 1), (2, 7), (3, 1001), (6, 2048), (6, 2041), (8, 8197), (5, 50001), (64, 129)])
def test_verify_chain(T, V, dt):
    r = np.random.default_rng(T * V)
    Bn = 9
    lg = _logits(r, (Bn, T, V), dt)
    dr = (0.8 * lg[:, : T - 1].float() + 0.6 * _logits(r, (Bn, T - 1, V), torch.float32)).to(dt)
    t = r.uniform(0.5, 1.3, Bn)
    t[::4] = 0
    tok = np.zeros((Bn, T - 1), np.int64)
    for b in range(Bn):
        for i in range(T - 1):
            tok[b, i] = SV.pick(SV.probabilities(f64(dr[b, i]), t[b]), r.random())
    ws = B.workspace_verify(Bn, T, V)
    for rep in range(2):                                         # the workspace is left ready for the next call
        out, n = _check_chain(lg, dr, tok, t, r.random((Bn, T - 1)), r.random(Bn), ws)
    if T > 1 and V > 100:
        assert int(n.max()) > 0


def test_verify_chain_edges():
    r = np.random.default_rng(5)
    Bn, T, V = 8, 4, 300
    lg = _logits(r, (Bn, T, V), torch.float32)
    dr = lg[:, : T - 1].clone()                                  # the drafter is the target: every u < 1 accepts
    tok = np.full((Bn, T - 1), 17)
    t = np.ones(Bn)
    u, us = r.random((Bn, T - 1)), r.random(Bn)
    lg[1, 1] = -float("inf")                                     # nothing to choose from
    lg[2, 0, :] = -float("inf")
    lg[2, 0, 17], lg[2, 1, 20:] = 0.0, float("nan")
    tok[3, 0], tok[4, 1] = V, -1                                 # tokens outside the vocabulary
    lg[5, 0, 9] = lg[5, 0, 30] = 50.0                            # a tie, greedily: the lower index
    t[5], t[6], t[7] = 0, 0, 1e-30
    tok[5, 0], tok[6, 0] = 30, int(lg[6, 0].argmax())
    us[0] = np.nextafter(np.float32(1), np.float32(0))
    _check_chain(lg, dr, tok, t, u, us)
    tok[5, 0] = 9
    _, n = _check_chain(lg, dr, tok, t, u, us)
    assert int(n[5]) >= 1 and int(n[3]) == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 3), (2, 1001), (17, 4099), (64, 2050), (32, 32768)])
def test_verify_tree(T, V, dt):
    r = np.random.default_rng(T + V)
    Bn = 5
    print("tree", T, V, dt, flush=True)
    lg = _logits(r, (Bn, T, V), dt, 4.0)
    t = np.array([1.0, 0.0, 0.7, 0.3, 1.2], np.float32)
    u = r.random((Bn, T)).astype(np.float32)
    par = np.full((Bn, T), -1, np.int32)
    tok = np.zeros((Bn, T), np.int32)
    for b in range(Bn):
        for i in range(1, T):
            p = par[b, i] = r.integers(0, i)
            own = SV.pick(SV.probabilities(f64(lg[b, p]), float(t[b])), float(u[b, p]))
            tok[b, i] = own if r.random() < 0.5 else r.integers(0, V)
        if T > 16:
            par[b, 5], par[b, 9] = 5, 12                         # not above the node: cut off
    dev = lambda a: torch.from_numpy(a).cuda()
    out, path, n = B.bsfp8_verify_tree(lg, dev(tok), dev(par), dev(t), dev(u))
    for b in range(Bn):
        wo, wp, wn = SV.verify_tree(f64(lg[b]), tok[b], par[b], float(t[b]), u[b].astype(np.float64))
        assert int(n[b]) == wn and np.array_equal(path[b].cpu().numpy(), wp) and np.array_equal(out[b].cpu().numpy(), wo)
    if T > 16:
        assert int(n.max()) > 1


def test_verify_in_a_graph():
    r = np.random.default_rng(8)
    Bn, T, V = 4, 6, 40000
    lg, dr = _logits(r, (Bn, T, V), torch.float32), _logits(r, (Bn, T - 1, V), torch.float32)
    tok = torch.from_numpy(r.integers(0, V, (Bn, T - 1)).astype(np.int32)).cuda()
    t = torch.ones(Bn).cuda()
    u, us = torch.rand(Bn, T - 1).cuda(), torch.rand(Bn).cuda()
    ws = B.workspace_verify(Bn, T, V)
    out, n = B.bsfp8_verify_chain(lg, dr, tok, t, u, us, ws=ws)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.bsfp8_verify_chain(lg, dr, tok, t, u, us, ws=ws, out_tokens=out, n_accepted=n)
    for _ in range(3):
        out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        B.bsfp8_verify_chain(lg, dr, tok, t, u, us, ws=ws)
