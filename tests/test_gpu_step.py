"""GPU parity of a serving step's operators with oracle/step.py (float64): the gated residual norms, page tables, bounds of
keys, the pages that they select with the attention over them, at the sizes, masks and values where they can go wrong.

Tolerances (u = the half step of a type: bf16 2^-8, fp32 2^-24), fixed before the first run:
  * a mean of squares: a thread adds at most 32 of them, then 6 + 16 partial sums: 54 roundings of positive terms, and one
    each for the square, the mean, eps; its 1/sqrt half of that and two ulp of the instruction: 32 u32;
  * h': the products z * inv * post * gate * scale and the sum: 32 + 6 u32 of |h| + |scale gate z|, and the type's rounding;
  * x: 40 u32 of |x| for its own norm, h's error over the row's root mean square (times |weight|), and the same in the mean:
    the row's rms error over its rms; the type's rounding; MXFP8 as the cache's;
  * tables, bounds, selected pages: equal (scores of pages are sums of products of bf16 values with a common range in 64
    bits, exact on both sides here but where a test says otherwise); attention as tests/test_gpu_serving.py.
"""
import numpy as np
import pytest
import torch

import block_scaled_fp8_skinny_amd as B
import oracle.mx as MX
import oracle.serving as SV
import oracle.step as ST
from test_gpu_serving import U16, U32, bf16, cache_of, f64

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).cuda()


# ------------------------------------------------------------------------------------------------
# norms
# ------------------------------------------------------------------------------------------------
NORMS = [  # rows, width, fp32 residual, gate, post norm, MXFP8
    (1, 8, False, None, False, False),
    (3, 64, True, "channel", True, True),
    (5, 512, False, "row", True, True),
    (5, 520, True, "row", False, False),
    (7, 1024, False, None, True, True),
    (2, 1032, True, "channel", True, False),
    (2, 2048, False, "row", True, True),
    (130, 2056, False, "channel", False, False),
    (6, 5120, False, "channel", True, True),
    (1100, 5120, True, None, True, True),
    (9, 16384, True, "row", True, True),
    (3, 16392, False, "row", True, False),
    (2, 32768, True, "channel", True, True),
    (9000, 64, False, None, True, True),
]


def norm_inputs(case, seed=0):
    R, W, f32, gate, post, mx = case
    r = np.random.default_rng(seed + R + W)
    if f32:
        h = torch.from_numpy((4 * r.standard_normal((R, W + 4))).astype(np.float32)).cuda()[:, :W]
    else:
        h = bf16(r, (R, W + 8), 4.0)[0][:, :W]
    y = bf16(r, (R, W + 16))[0][:, 8: 8 + W]
    w, p = (bf16(r, (W,))[0] for _ in range(2))
    g = None if gate is None else bf16(r, (W,) if gate == "channel" else (R, W + 8), 0.5)[0][..., :W]
    return h, y, w, p if post else None, g


def check_norm(h, y, w, p, g, scale, got_h, got_x, got_mx, eps=1e-6):
    n = lambda t: None if t is None else f64(t)
    want_h, want_x, amp = ST.residual_norm(f64(h), n(y), n(w), n(p), n(g), scale, eps)
    err = 38 * U32 * amp if y is not None else 0 * amp
    if got_h is not None:
        u = U32 if got_h.dtype is torch.float32 else U16
        assert np.all(np.abs(f64(got_h) - want_h) <= u * np.abs(want_h) + (1 + u) * err)
    rms = np.sqrt((want_h ** 2).mean(-1, keepdims=True) + eps)
    aw = 1 if w is None else np.abs(f64(w))
    off = np.abs(want_x) * (40 * U32 + np.sqrt((err ** 2).mean(-1, keepdims=True)) / rms) + err / rms * aw
    if got_x is not None:
        assert np.all(np.abs(f64(got_x) - want_x) <= U16 * np.abs(want_x) + (1 + U16) * off)
    if got_mx is not None:
        q, s = (t.cpu().numpy() for t in got_mx)
        top = lambda v: MX.mx_scale_exponent(np.maximum(v, 0).reshape(*s.shape, 32).max(-1)) + 127
        assert np.all((s >= top(np.abs(want_x) - off)) & (s <= top(np.abs(want_x) + off)))
        sc = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, -1)
        near = np.clip(want_x, -448 * sc, 448 * sc)
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(near), 1e-300) / sc)), -6) - 3) * sc
        assert np.all(np.abs(SV.cache_values(q, s) - near) <= step / 2 * (1 + 1e-3) + off)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "R%d_W%d_f%d_%s_p%d_m%d" % c)
def test_norm(case):
    print("norm", case, flush=True)
    h, y, w, p, g = norm_inputs(case)
    R, W, f32, _, _, mx = case
    kw = dict(weight=w, post_weight=p, gate=g, scale=0.3)
    both = dict(x_out=torch.empty(R, W, dtype=torch.bfloat16, device="cuda"))
    if mx:
        both["mx_out"] = tuple(torch.empty(R, n, dtype=torch.uint8, device="cuda") for n in (W, W // 32))
    out, x = B.bsfp8_residual_norm(h, y, **kw, **both)
    x, q = x if mx else (x, None)
    check_norm(h, y, w, p, g, 0.3, out, x, q)
    assert out.dtype is h.dtype
    # one output alone, and in place: the same bits
    out2, x2 = B.bsfp8_residual_norm(h, y, **kw)
    assert torch.equal(out, out2) and torch.equal(x, x2)
    if mx:
        _, q2 = B.bsfp8_residual_norm(h, y, mx=True, **kw)
        assert torch.equal(q[0], q2[0]) and torch.equal(q[1], q2[1])
    wide = torch.full((R, W + 8), 7.0, dtype=h.dtype, device="cuda")
    mine = wide[:, :W]
    mine.copy_(h)
    out3, x3 = B.bsfp8_residual_norm(mine, y, h_out=mine, **kw)
    assert torch.equal(mine, out) and torch.equal(x3, x) and (wide[:, W:] == 7).all()


@pytest.mark.parametrize("W", [8, 72, 96, 128, 136, 256, 264, 288, 8192, 8200, 24000])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_every_layout(W, f32):
    """Several rows in a wave, rows of a workgroup of one, two and four groups a thread; more rows than fit at once."""
    case = (33 if W > 512 else 9001, W, f32, "row", True, W % 32 == 0)
    h, y, w, p, g = norm_inputs(case)
    out, x = B.bsfp8_residual_norm(h, y, weight=w, post_weight=p, gate=g, scale=-0.7)
    check_norm(h, y, w, p, g, -0.7, out, x, None)
    out, x = B.bsfp8_residual_norm(h, y, weight=w, scale=2.0, mx=case[5])
    check_norm(h, y, w, None, None, 2.0, out, None if case[5] else x, x if case[5] else None)


@pytest.mark.parametrize("W", [64, 2560])
def test_norm_without_a_block(W):
    h = norm_inputs((6, W, True, None, False, False))[0]
    out, x = B.bsfp8_residual_norm(h)
    assert out is h
    check_norm(h, None, None, None, None, 1.0, None, x, None)
    h = norm_inputs((6, W, False, None, False, False))[0]
    w = bf16(np.random.default_rng(3), (W,))[0]
    copy = torch.empty(6, W, dtype=torch.bfloat16, device="cuda")
    out, (q, s) = B.bsfp8_residual_norm(h, weight=w, h_out=copy, mx=True, eps=0.5)
    assert torch.equal(copy, h)
    check_norm(h, None, w, None, None, 1.0, out, None, (q, s), eps=0.5)


def test_norm_of_zeros_infinities_and_nan():
    h = torch.ones(5, 256, dtype=torch.bfloat16, device="cuda")
    y = torch.ones(5, 256, dtype=torch.bfloat16, device="cuda")
    h[0], y[0] = 0, 0
    y[1, 7] = float("nan")
    h[2, 9] = float("inf")
    y[3] = 0
    out, (x, (q, s)) = B.bsfp8_residual_norm(h, y, post_weight=y[4].clone(), x_out=torch.empty_like(h), mx_out=(
        torch.empty(5, 256, dtype=torch.uint8, device="cuda"), torch.empty(5, 8, dtype=torch.uint8, device="cuda")))
    assert (out[0] == 0).all() and (x[0] == 0).all() and (q[0] == 0).all() and (s[0] == 0).all()
    assert out[1].isnan().all() and x[1].isnan().all() and (s[1] == 255).all()
    assert torch.isinf(out[2, 9]) and x[2, 9].isnan() and (x[2, :9] == 0).all()   # inf / inf, and 1 / inf
    assert (out[3] == 1).all() and torch.allclose(x[3:].float(), torch.ones(2, 256, device="cuda"))


# ------------------------------------------------------------------------------------------------
# tables
# ------------------------------------------------------------------------------------------------
class Tables:
    """A table and a stack on the GPU beside the oracle's, whose pages are all different."""

    def __init__(self, seed, Bn, W, page, spare, capacity=None):
        self.r = np.random.default_rng(seed)
        self.Bn, self.W, self.page = Bn, W, page
        n = Bn * W + spare
        self.capacity = n if capacity is None else capacity
        ids = self.r.permutation(n)
        self.pages = [[-7] * W for _ in range(Bn)]
        self.stack = ids.tolist()[: self.capacity]
        self.lens = [0] * Bn
        self.t = torch.full((Bn, W), -7, dtype=torch.int32, device="cuda")
        self.free = torch.full((self.capacity,), -9, dtype=torch.int32, device="cuda")
        self.free[: len(self.stack)] = dev(np.array(self.stack, np.int32)) if self.stack else 0
        self.n = torch.tensor([len(self.stack)], dtype=torch.int32, device="cuda")

    def step(self, new, rows, per_seq=0, out=None, lens=None):
        lens = self.lens if lens is None else lens
        i32 = lambda x: dev(np.array(x, np.int32).reshape(-1))
        want = ST.step_tables(self.pages, lens, new, self.stack, self.page, rows, per_seq, self.capacity)
        got = B.bsfp8_step_tables(self.t, i32(lens), i32(new), self.free, self.n, self.page, rows, per_seq, n_free_out=out)
        for name, w, g in zip(got._fields, want, got):
            assert g.cpu().tolist() == list(w), name
        if self.Bn and self.W:
            assert self.t.cpu().tolist() == self.pages
        n = (self.n if out is None else out).item()
        assert n == len(self.stack) and self.free[:n].cpu().tolist() == self.stack
        self.lens = want[4]
        if out is not None:
            self.n = out
        return got


@pytest.mark.parametrize("Bn,W,page", [(1, 4, 16), (5, 9, 1), (37, 20, 48), (700, 6, 16), (1500, 3, 64)])
@pytest.mark.parametrize("per_seq", [0, 5])
def test_tables_over_many_steps(Bn, W, page, per_seq):
    """Requests that come, grow, shrink and end, with the library's own lengths from step to step."""
    print("tables", Bn, W, page, per_seq, flush=True)
    t = Tables(Bn, Bn, W, page, 3)
    for step in range(6):
        kind = t.r.random(Bn)
        grow = t.r.integers(1, 6, Bn)
        fresh = t.r.integers(0, W * page + 1, Bn)
        new = [0 if k < 0.15 else max(0, n - 3) if k < 0.3 else int(f) if n == 0 and step < 4 else min(W * page, n + int(g))
               for k, g, f, n in zip(kind, grow, fresh, t.lens)]
        rows = Bn * 5 if per_seq else sum(max(0, a - b) for a, b in zip(new, t.lens)) + 7 * (step % 2)
        out = torch.zeros(1, dtype=torch.int32, device="cuda") if step % 2 else None
        t.step(new, rows, per_seq, out)


@pytest.mark.parametrize("Bn", [3, 1100])
def test_tables_when_pages_run_out(Bn):
    t = Tables(1, Bn, 8, 16, -7 * Bn)                            # one page a request
    t.step([int(x) for x in t.r.integers(0, 129, Bn)], Bn * 128)
    t.step([n // 2 for n in t.lens], 5)                          # gives some back
    t.step([n + 40 for n in t.lens], Bn * 40 + 1)
    t.step([0] * Bn, 0)
    assert t.n.item() == Bn


def test_tables_past_their_width_and_rows():
    t = Tables(2, 4, 3, 16, 5)
    t.step([60, 48, 10, 0], 100)                                 # 60 positions need a page too many; 118 tokens, 100 rows
    assert t.lens == [48, 48, 10, 0]
    t.step([50, 49, 11, -5], 9, per_seq=2)
    t.step([-1, 0, 0, 0], 3, lens=[48, 48, 11, -3])


def test_tables_with_a_short_stack_and_none():
    t = Tables(3, 5, 4, 16, 0, capacity=6)                       # more pages come back than the stack holds: dropped
    t.step([16, 16, 16, 16, 16], 80)
    t.t.copy_(dev(np.arange(100, 120, dtype=np.int32).reshape(5, 4)))
    t.pages[:] = t.t.cpu().tolist()
    t.step([0, 0, 0, 0, 5], 4, lens=[64, 64, 64, 64, 64])
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    got = B.bsfp8_step_tables(z(0, 4), z(0), z(0), z(0), z(1), 16, 3)
    assert got.slots.tolist() == [-1] * 3 and got.starts.tolist() == [0] and got.counts.tolist() == [0] * 4
    got = B.bsfp8_step_tables(z(2, 0), z(2), z(2) + 3, z(0), z(1), 16, 3)
    assert got.slots.tolist() == [-1] * 3 and got.positions.tolist() == [0, 1, 2] and got.held.tolist() == [0, 0]
    assert got.counts.tolist() == [6, 0, 0, 2]


def test_rows_behind_the_last_are_left():
    t = Tables(4, 2, 4, 16, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    big = [torch.full((40,), 77, dtype=d, device="cuda") for d in (torch.int64, torch.int64, torch.int32)]
    B.bsfp8_step_tables(t.t, i32([0, 0]), i32([5, 4]), t.free, t.n, 16, 6, slots=big[0][:6], positions=big[1][:6], seqs=big[2][:6])
    for x in big:
        assert (x[6:] == 77).all() and (x[:6] != 77).all()


def test_a_long_request_among_many():
    """Lengths near the ends of 32 bits: positions and slots are 64-bit, a table entry far along its row."""
    W, page = 1 << 20, 2048
    t = torch.full((1, W), 3, dtype=torch.int32, device="cuda")
    t[0, -1] = 5
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    end = (1 << 31) - 1
    got = B.bsfp8_step_tables(t, i32(end - 3), i32(end), torch.zeros(4, dtype=torch.int32, device="cuda"), i32(0), page, 5)
    assert got.positions.tolist() == [end - 3, end - 2, end - 1, 0, 0] and got.held.tolist() == [end]
    assert got.slots.tolist() == [5 * page + (p % page) for p in (end - 3, end - 2, end - 1)] + [-1, -1]
    t = torch.full((3, 4), 9, dtype=torch.int32, device="cuda")
    three = torch.tensor([0, 5, 0], dtype=torch.int32, device="cuda")
    got = B.bsfp8_step_tables(t, three, three + end - 5, torch.zeros(4, dtype=torch.int32, device="cuda"), i32(0), 16, 4)
    assert got.starts.tolist() == [0, end - 5, end, end] and got.counts.tolist()[0] == end   # (they end there)
    assert got.counts[3].item() == 3 * 2 ** 27 - 1


# ------------------------------------------------------------------------------------------------
# bounds
# ------------------------------------------------------------------------------------------------
def bounds_case(seed, heads, dim, page, lens, first=None, max_new=None, spoil=None, table=None):
    r = np.random.default_rng(seed)
    W = max(1, -(-max(lens) // page))
    n = len(lens) * W + 2
    cache, K, _ = cache_of(r, n, heads, page, dim)
    pages = r.permutation(n)[: len(lens) * W].reshape(len(lens), W).astype(np.int32)
    if table:
        table(pages, n)
    if spoil:
        spoil(cache, K)
    print("bounds", seed, heads, dim, page, lens, first, max_new, flush=True)
    got = torch.full((n, heads, 2, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    B.bsfp8_cache_bounds(cache, dev(pages), dev(np.array(lens, np.int32)), got, max_new=max_new,
                         first=None if first is None else dev(np.array(first, np.int32)))
    want = np.full(got.shape, 3.0)
    for b, ln in enumerate(lens):
        ln = min(ln, W * page)
        f = min(max(0, first[b]), ln) if first is not None else 0
        f = max(f, ln - max_new) if max_new is not None else f
        for j in range(f // page, -(-ln // page)):
            if f < ln and 0 <= pages[b, j] < n:
                at = int(pages[b, j]) * page
                want[pages[b, j]] = ST.key_bounds(K[at: at + min(page, ln - j * page)])
    assert np.array_equal(f64(got), want, equal_nan=True)
    return got


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 48, 64, 272])
def test_bounds(dim, page):
    bounds_case(1, 3, dim, page, [0, 1, 15, page, page + 1, 3 * page - 5])
    bounds_case(2, 1, dim, page, [5, 200, 310], first=[4, 0, 305], max_new=200)
    bounds_case(3, 2, dim, page, [300, 290], first=[-4, 400], max_new=7)


def test_bounds_of_special_keys():
    def spoil(cache, K):
        cache.kq[:, 0, 3, 5] = 0x7F                              # NaN codes, NaN scales, and values past bf16's largest
        K[3::16, 0, 5] = np.nan
        cache.ks[:, 1, 7, 1] = 255
        K[7::16, 1, 32:] = np.nan
        cache.ks[:, 1, 9, 0], cache.kq[:, 1, 9, :4] = 254, 0x78   # 256 * 2^127
        K[9::16, 1, :32] = SV.cache_values(cache.kq[:, 1, 9, :32].cpu().numpy(), np.full((cache.pages, 1), 254, np.uint8))
        K[9::16, 1, :32] = np.where(np.abs(K[9::16, 1, :32]) > 2.0 ** 127 * 1.998, np.sign(K[9::16, 1, :32]) * np.inf, K[9::16, 1, :32])
    got = bounds_case(4, 2, 64, 16, [40, 16, 9], spoil=spoil)
    assert got.isnan().any() and got.isinf().any()


def test_bounds_of_absent_pages():
    def table(pages, n):
        pages[0, 1], pages[1, 0] = -1, n
    bounds_case(5, 2, 128, 16, [60, 40], table=table)


# ------------------------------------------------------------------------------------------------
# selection and attention
# ------------------------------------------------------------------------------------------------
def choose(seed, T, hq, hkv, dim, page, lens, count, sinks=1, recent=2, nodes=None, max_len=None, wide=0, change=None, attend=True,
           scale=None, extra=0):
    """One selection and the attention over it, against the oracle."""
    r = np.random.default_rng(seed)
    Bn = len(lens)
    W = max(1, -(-max(max(lens), 1) // page)) + extra
    n_pages = Bn * W + 1
    cache, K, V = cache_of(r, n_pages, hkv, page, dim)
    pages = r.permutation(n_pages)[: Bn * W].reshape(Bn, W).astype(np.int32)
    qt, q = bf16(r, (Bn, T, hq * dim + wide))
    bounds = B.bsfp8_cache_bounds(cache, dev(pages), dev(np.full(Bn, W * page, np.int32)))
    if change:
        change(qt, q, bounds, pages, n_pages)
    q = q[..., : hq * dim].reshape(Bn, T, hq, dim)
    qv = qt[..., : hq * dim].unflatten(-1, (hq, dim))
    i32 = lambda x: None if x is None else dev(np.array(x, np.int32))
    print("select", seed, T, hq, hkv, dim, page, lens, count, sinks, recent, nodes, flush=True)
    sel, held = B.bsfp8_select_pages(qv, bounds, i32(pages), i32(lens), count, page, nodes=i32(nodes), sinks=sinks, recent=recent,
                                     max_len=max_len)
    out = B.bsfp8_sparse_attention(qv.flatten(0, 1), cache, sel, held, scale=scale) if attend else None
    torch.cuda.synchronize()
    bd, g = f64(bounds), hq // hkv
    got_sel, got_held = sel.cpu().numpy(), held.cpu().numpy()
    for b in range(Bn):
        ln = min(lens[b], W * page if max_len is None else min(max_len, W * page))
        here = T if nodes is None else min(max(nodes[b], 0), T)
        for t in range(T):
            n = max(0, ln - here + t + 1) if t < here else 0
            N, row = -(-n // page), b * T + t
            there = (pages[b, :N] >= 0) & (pages[b, :N] < n_pages)
            ids = np.where(there, pages[b, :N], 0)
            m = min(N, count)
            assert got_held[row] == ((m - 1) * page + n - (N - 1) * page if N else 0), (b, t)
            for h in range(hkv):
                want = np.full(count, -1)
                s = ST.page_scores(q[b, t, h * g: h * g + g], bd[ids, h]) if N > count else np.zeros(N)
                at = ST.select(s, there, N, count, sinks, recent)
                want[:m] = np.where(there, pages[b, :N], -1)[at]
                assert got_sel[row, h].tolist() == want.tolist(), (b, t, h)
            if not attend:
                continue
            for h in range(hkv):
                w = got_sel[row, h, :m]
                slots = np.where(w[:, None] >= 0, w[:, None] * page + np.arange(page), -1).reshape(-1)[: int(got_held[row])]
                see = (slots >= 0)[None]
                sc = dim ** -0.5 if scale is None else scale
                want, mag, big = SV.attention(q[b, t: t + 1, h * g: h * g + g], K[slots, h: h + 1], V[slots, h: h + 1], see, sc)
                tol = U16 * np.abs(want) + (U16 + 2 * (dim + 8) * U32 * big + (len(slots) + 8) * U32) * mag + 1e-30
                got = f64(out[row, h * g: h * g + g])
                assert np.all(np.abs(got - want[0]) <= tol[0]), (b, t, h)
    return sel, held, out


@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8, 16, 20, 64])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (192, 48), (256, 16)])
def test_selection(g, dim, page):
    choose(g, 1, 2 * g, 2, dim, page, [0, 1, page, 3 * page, 3 * page + 1, 20 * page - 3], 4)
    choose(100 + g, 5, g, 1, dim, page, [5, 9 * page + 2, 17 * page], 6, nodes=[5, 3, 0])


def test_selection_bounds_and_strides():
    choose(200, 3, 4, 2, 64, 16, [400, 333], 5, max_len=200, wide=24)
    choose(201, 2, 4, 2, 128, 16, [400, 333], 7, sinks=0, recent=1, extra=3)
    choose(202, 2, 4, 2, 128, 16, [400, 333], 7, sinks=4, recent=3)        # nothing left to choose
    choose(203, 2, 4, 2, 64, 16, [400, 333], 1, sinks=0, recent=1)         # its own page alone
    choose(204, 17, 2, 2, 64, 16, [400, 3], 5)                             # more tokens than the sequence holds
    choose(205, 2, 6, 2, 64, 16, [260], 9, scale=-0.3)


@pytest.mark.parametrize("pages", [257, 2048, 2049, 5000])
def test_selection_of_many_pages(pages):
    choose(210, 2, 3, 1, 64, 16, [pages * 16 - 9, 40 * 16], 33, attend=False)
    choose(211, 1, 8, 1, 128, 16, [pages * 16], pages - 1, attend=False)
    choose(212, 1, 1, 1, 64, 16, [pages * 16], pages // 2, sinks=0, recent=1, attend=False)


@pytest.mark.parametrize("pages", [40, 600, 3000])
def test_equal_scores_go_to_the_first_pages(pages):
    def zero(qt, q, bounds, table, n):
        qt[:], q[:] = 0, 0
    choose(220, 1, 2, 1, 64, 16, [pages * 16 - 1], 20, change=zero, attend=False)

    def same(qt, q, bounds, table, n):                           # half of the pages alike, and the best
        bounds[dev(table[0, 5::2].astype(np.int64))] = 100.0
        bounds[dev(table[0, 6::2].astype(np.int64))] = -100.0
        qt[:], q[:] = 1, 1
    choose(221, 1, 2, 1, 64, 16, [pages * 16 - 1], 12, change=same, attend=False)
    choose(222, 1, 2, 1, 64, 16, [pages * 16 - 1], pages // 2 + 9, change=same, attend=False)


def test_scores_of_every_size():
    """Bounds from 2^-100 to 2^100, of either sign: one histogram after another until the border is found."""
    def spread(qt, q, bounds, table, n):
        r = np.random.default_rng(9)
        e = torch.from_numpy(np.exp2(r.integers(-100, 100, n)) * r.choice([-1.0, 1.0], n))
        x = torch.zeros(bounds.shape, dtype=torch.bfloat16)
        x[:, :, :, 0] = e.to(torch.bfloat16)[:, None, None]
        bounds.copy_(x.cuda())
        qt[..., 1:], q[..., 1:] = 0, 0
        qt[..., 0], q[..., 0] = 1, 1
    for count in (5, 300, 700, 1190):
        choose(230, 1, 1, 1, 64, 16, [1200 * 16], count, change=spread, attend=False)


def test_absent_pages_and_values_that_are_not_finite():
    def change(qt, q, bounds, table, n):
        table[0, 3], table[0, 7], table[1, 2] = -1, n, 2 ** 30
        bounds[int(table[0, 9]), 0, 0, 3] = float("nan")
        bounds[int(table[0, 11]), 1, 1, 40] = float("inf")
        bounds[int(table[1, 4]), 0, 0, 7] = -float("inf")
    for count in (6, 25, 38):
        choose(240, 1, 4, 2, 64, 16, [640, 600], count, change=change, attend=False)

    def queries(qt, q, bounds, table, n):
        qt[0, 0, 5], q[0, 0, 5] = float("nan"), np.nan
        qt[1, 0, 70], q[1, 0, 70] = float("inf"), np.inf
    choose(241, 1, 2, 2, 64, 16, [640, 600], 9, change=queries, attend=False)


def test_absent_pages_reach_no_row():
    def change(qt, q, bounds, table, n):
        table[0, 3], table[0, 0], table[1, :] = -1, n, -1
    sel, held, out = choose(242, 1, 4, 2, 64, 16, [300, 200], 8, change=change)
    assert (out[1] == 0).all() and (sel[1] == -1).all()


def test_one_token_is_dense_attention_where_all_pages_are_taken():
    """With room for every page the list is the table, and the attention bit for bit the dense one's."""
    r = np.random.default_rng(250)
    cache, _, _ = cache_of(r, 60, 2, 16, 128)
    pages, lens = dev(r.permutation(60)[:60].reshape(3, 20), np.int32), dev([320, 57, 0], np.int32)
    q = bf16(r, (3, 1, 8, 128))[0]
    bounds = B.bsfp8_cache_bounds(cache, pages, lens)
    sel, held = B.bsfp8_select_pages(q, bounds, pages, lens, 20, 16)
    assert held.tolist() == [320, 57, 0] and torch.equal(sel[0, 0], pages[0]) and torch.equal(sel[0, 1], pages[0])
    out = B.bsfp8_sparse_attention(q[:, 0], cache, sel, held)
    assert torch.equal(out, B.bsfp8_tree_attention(q, cache, pages, lens)[:, 0])


def test_lists_of_a_callers_own():
    """Pages in any order, twice in a list, other lists for other heads, lengths past the list."""
    r = np.random.default_rng(251)
    cache, K, V = cache_of(r, 12, 3, 16, 64)
    sel = r.integers(0, 12, (4, 3, 5)).astype(np.int32)
    sel[1, 0] = 7
    sel[2, 1, 2] = 99
    held = np.array([80, 33, 500, -4], np.int32)
    qt, q = bf16(r, (4, 6, 64))
    out = f64(B.bsfp8_sparse_attention(qt, cache, dev(sel), dev(held)))
    for i in range(4):
        n = min(max(int(held[i]), 0), 80)
        for h in range(3):
            w = sel[i, h]
            slots = np.where((w >= 0) & (w < 12), w, -99)[:, None] * 16 + np.arange(16)
            slots = np.where(slots >= 0, slots, -1).reshape(-1)[:n]
            want, mag, big = SV.attention(q[i: i + 1, 2 * h: 2 * h + 2], K[slots, h: h + 1], V[slots, h: h + 1], (slots >= 0)[None], 0.125)
            tol = U16 * np.abs(want) + (U16 + 2 * 72 * U32 * big + 88 * U32) * mag + 1e-30
            assert np.all(np.abs(out[i, 2 * h: 2 * h + 2] - want[0]) <= tol[0]), (i, h)


# ------------------------------------------------------------------------------------------------
# together: another stream, a captured step, workspaces that serve many sizes
# ------------------------------------------------------------------------------------------------
def step_of(seed, Bn=5, page=16, dim=64):
    """A decode step's calls on buffers of its own: tables, cache write, bounds, selection, attention, norm."""
    r = np.random.default_rng(seed)
    W, hkv, hq, width = 30, 2, 8, 8 * dim
    n = Bn * W
    i32 = torch.int32
    s = dict(cache=B.KVCache.empty(n, hkv, page, dim), pages=torch.full((Bn, W), -1, dtype=i32, device="cuda"),
             free=torch.arange(n, dtype=i32, device="cuda"), n_free=torch.full((1,), n, dtype=i32, device="cuda"),
             lens=torch.zeros(Bn, dtype=i32, device="cuda"), bounds=torch.zeros(n, hkv, 2, dim, dtype=torch.bfloat16, device="cuda"))
    s["h"] = bf16(r, (Bn, width))[0]
    s["x"] = bf16(r, (Bn, (hq + 2 * hkv) * dim))[0]
    s["ws"], s["wa"] = B.workspace_select(Bn, 1, hkv, W), B.workspace_attention(Bn, 1, hq, hkv, dim, 6 * page)
    s["weight"] = bf16(r, (width,))[0]

    def run():
        new = s["lens"] + 1
        t = B.bsfp8_step_tables(s["pages"], s["lens"], new, s["free"], s["n_free"], page, Bn, 1)
        x = s["x"] * (1 + s["lens"][:, None] % 7).to(torch.bfloat16)
        q, k, v = x.split([hq * dim, hkv * dim, hkv * dim], 1)
        B.bsfp8_cache_write(s["cache"], t.slots, k, v)
        B.bsfp8_cache_bounds(s["cache"], s["pages"], t.held, s["bounds"], first=s["lens"], max_new=1)
        q = q.unflatten(1, (hq, dim)).unsqueeze(1)
        sel, held = B.bsfp8_select_pages(q, s["bounds"], s["pages"], t.held, 6, page, ws=s["ws"])
        y = B.bsfp8_sparse_attention(q[:, 0], s["cache"], sel, held, ws=s["wa"])
        out, x = B.bsfp8_residual_norm(s["h"], y.flatten(1), weight=s["weight"], post_weight=s["weight"], h_out=s["h"])
        s["lens"].copy_(t.held)
        return sel, held, y, x
    return s, run


def test_steps_on_another_stream_and_in_a_graph():
    """150 decode steps: eagerly, on another stream, and replayed from a graph with eager work between, agree bit for bit."""
    eager, run = step_of(7)
    side_s, side_run = step_of(7)
    graph_s, graph_run = step_of(7)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    first = [t.clone() for t in run()]
    graph_run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = graph_run()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = side_run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    for step in range(1, 150):
        want = run()
        g.replay()
        with torch.cuda.stream(side):
            got = side_run()
        if step % 10 == 9 or step < 4:
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), step
            assert all(torch.equal(a, b) for a, b in zip(want, held)), step
    torch.cuda.synchronize()
    assert eager["lens"].tolist() == [150] * 5 and eager["n_free"].item() == 150 - 50
    for k in ("pages", "n_free", "lens", "bounds", "h"):
        assert torch.equal(eager[k], side_s[k]) and torch.equal(eager[k], graph_s[k]), k


def test_a_selection_workspace_serves_smaller_calls():
    ws = B.workspace_select(6, 4, 2, 700)
    ws.fill_(0xFF)
    r = np.random.default_rng(260)
    for Bn, T, W in ((6, 4, 700), (1, 1, 30), (6, 1, 90), (2, 3, 699), (6, 4, 700)):
        n = Bn * W
        bounds = bf16(r, (n, 2, 2, 64))[0]
        pages, lens = dev(r.permutation(n).reshape(Bn, W), np.int32), dev(np.full(Bn, W * 16), np.int32)
        q = bf16(r, (Bn, T, 4, 64))[0]
        a = B.bsfp8_select_pages(q, bounds, pages, lens, 20, 16, ws=ws)
        b = B.bsfp8_select_pages(q, bounds, pages, lens, 20, 16)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("pages", [8192, 8193, 20000])
def test_selection_of_very_many_pages(pages):
    """Keys that are held and keys that are read again in every round; equal ones among them."""
    choose(270, 1, 2, 1, 64, 16, [pages * 16 - 3], 50, attend=False)

    def few(qt, q, bounds, table, n):
        bounds.copy_(torch.randint(-2, 3, (n, 1, 1, 1), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).expand_as(bounds))
        qt[:], q[:] = 1, 1
    for count in (7, pages // 5, pages - 9):
        choose(271, 1, 2, 1, 64, 16, [pages * 16 - 3], count, change=few, attend=False)


@pytest.mark.parametrize("left", [63, 64, 65, 66, 67, 68])
def test_selection_about_the_ranked_number(left):
    for count in (4, 33, left - 1):
        choose(280 + left, 1, 2, 1, 64, 16, [(left + 3) * 16], count, attend=False)


@pytest.mark.parametrize("pages", [40, 100, 900, 3000, 17000])
def test_scores_closer_than_fp32_tells(pages):
    """Scores of 256 and more that differ by 2^-20: the border lies among many that fp32 cannot tell apart."""
    def near(qt, q, bounds, table, n):
        r = np.random.default_rng(12)
        x = np.zeros((n, 64))
        x[:, 0], x[:, 7] = 256, r.integers(-60, 60, n) * 2.0 ** -20
        x[::5, 3] = r.choice([-1.0, 1.0], len(x[::5]))
        bounds.copy_(torch.from_numpy(x).to(torch.bfloat16).cuda()[:, None, None, :].expand_as(bounds))
        qt[:], q[:] = 1, 1
    for count in (4, pages // 3, pages // 2, pages - 5):
        choose(290, 1, 3, 1, 64, 16, [pages * 16 - 3], count, change=near, attend=False)
