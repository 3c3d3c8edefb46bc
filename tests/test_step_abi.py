"""CPU checks of the serving step's entry points: every refusal of sizes, strides, alignment, missing or overlapping buffers
returns its status before any GPU work, and the binding refuses what the library cannot see. No kernel is launched."""
import ctypes

import pytest
import torch

import block_scaled_fp8_skinny_amd as B
from test_serving_abi import NULL, P, cache, lib  # noqa: F401

INF, NAN = float("inf"), float("nan")


def norm(lib, h=P(1), ldh=64, dt=0, y=P(2), ldy=64, gate=P(3), ldg=64, post=P(4), w=P(5), scale=1.0, eps=1e-6, R=5, W=64, ho=P(6),
         ldo=64, x=P(7), xq=P(8), xs=P(9)):
    return lib.bsfp8_residual_norm(h, ldh, dt, y, ldy, gate, ldg, post, w, scale, eps, R, W, ho, ldo, x, xq, xs, NULL)


def test_norm_refusals(lib):
    assert norm(lib, R=0) == B.OK
    for bad in (dict(R=-1), dict(R=1 << 31), dict(W=0), dict(W=4), dict(W=68), dict(W=32776, ldh=1 << 20, ldy=1 << 20, ldo=1 << 20),
                dict(W=72, ldh=72, ldy=72, ldg=72, ldo=72)):
        assert norm(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(dt=2), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(scale=INF), dict(scale=NAN), dict(h=NULL),
                dict(y=NULL), dict(xq=NULL), dict(xs=NULL), dict(ho=NULL, x=NULL, xq=NULL, xs=NULL), dict(ho=P(2, 64)), dict(x=P(1, 64)),
                dict(ho=P(1), ldo=72), dict(ho=P(1, 128)), dict(xq=P(7, 16)), dict(xs=P(5)), dict(x=P(3, 512)), dict(xq=P(4, 16)),
                dict(ho=P(6), x=P(6, 128))):
        assert norm(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ldh=56), dict(ldh=68), dict(ldy=60), dict(ldg=8), dict(ldg=-8), dict(ldg=68), dict(ldo=63), dict(h=P(1, 8)),
                dict(y=P(2, 2)), dict(gate=P(3, 8)), dict(post=P(4, 4)), dict(w=P(5, 8)), dict(ho=P(6, 8)), dict(x=P(7, 2)), dict(xq=P(8, 1)),
                dict(dt=1, ldh=66), dict(dt=1, ldo=70)):
        assert norm(lib, **bad) == B.ESTRIDE, bad


def tables(lib, lens=P(1), new=P(2), Bn=3, page=16, pages=P(3), ld=4, free=P(4), cap=9, n=P(5), n_out=P(6), R=7, per=0, slots=P(7),
           pos=P(8), seqs=P(9), starts=P(10), held=P(11), counts=P(12)):
    return lib.bsfp8_step_tables(lens, new, Bn, page, pages, ld, free, cap, n, n_out, R, per, slots, pos, seqs, starts, held, counts,
                                 NULL)


def test_tables_refusals(lib):
    for bad in (dict(Bn=-1), dict(Bn=(1 << 20) + 1), dict(page=0), dict(page=1 << 31), dict(ld=-1), dict(ld=1 << 31), dict(cap=-1),
                dict(cap=1 << 31), dict(R=-1), dict(R=(1 << 31) - 4096), dict(per=-1), dict(per=1 << 31), dict(Bn=1 << 16, ld=1 << 15)):
        assert tables(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(lens=NULL), dict(new=NULL), dict(pages=NULL), dict(free=NULL), dict(n=NULL), dict(slots=NULL), dict(pos=NULL),
                dict(seqs=NULL), dict(starts=NULL), dict(held=NULL), dict(counts=NULL), dict(held=P(1)), dict(held=P(2, 8)),
                dict(slots=P(8)), dict(starts=P(11)), dict(counts=P(5)), dict(n=P(1)), dict(n_out=P(3, 44)), dict(pages=P(4, 32))):
        assert tables(lib, **bad) == B.EINVAL, bad


def bounds(lib, c=None, pages=P(5), ld=4, lens=P(6), first=P(7), Bn=3, most=9, out=P(8)):
    return lib.bsfp8_cache_bounds(c if c is not None else cache(), pages, ld, lens, first, Bn, most, out, NULL)


def test_bounds_refusals(lib):
    assert bounds(lib, Bn=0) == B.OK and bounds(lib, most=0) == B.OK and bounds(lib, c=cache(pages=0)) == B.OK
    for bad in (dict(c=cache(dim=96)), dict(c=cache(page=8)), dict(Bn=-1), dict(ld=-1), dict(ld=1 << 31), dict(most=-1), dict(most=1 << 31),
                dict(Bn=1 << 25), dict(Bn=1 << 20, ld=1 << 10, most=1 << 14)):
        assert bounds(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(pages=NULL), dict(lens=NULL), dict(out=NULL), dict(out=P(1, 32)), dict(out=P(5)), dict(out=P(7)),
                dict(c=ctypes.c_void_p(0))):
        assert bounds(lib, **bad) == B.EINVAL, bad
    assert bounds(lib, out=P(8, 8)) == B.ESTRIDE


def select(lib, q=P(1), ldq=256, Bn=3, T=2, hq=4, bd=P(2), n=9, heads=2, page=16, dim=64, pages=P(3), ld=8, lens=P(4), nodes=P(5),
           most=128, count=4, sinks=1, recent=1, ws=P(6), wsb=1 << 30, sel=P(7), held=P(8)):
    return lib.bsfp8_select_pages(q, ldq, Bn, T, hq, bd, n, heads, page, dim, pages, ld, lens, nodes, most, count, sinks, recent, ws, wsb,
                                  sel, held, NULL)


def test_select_refusals(lib):
    assert select(lib, Bn=0) == B.OK
    for bad in (dict(dim=96), dict(page=8), dict(page=24), dict(n=-1), dict(n=1 << 28), dict(heads=0), dict(hq=3), dict(hq=130, ldq=130 * 64),
                dict(ld=-1), dict(most=-1), dict(most=(1 << 31) - (1 << 14) + 1), dict(count=0), dict(sinks=-1), dict(recent=0),
                dict(sinks=2, recent=3), dict(sinks=(1 << 62), recent=(1 << 62)), dict(T=0), dict(Bn=-1), dict(Bn=1 << 21), dict(count=1 << 27),
                dict(ld=1 << 30, most=(1 << 31) - (1 << 14))):
        assert select(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(q=NULL), dict(bd=NULL), dict(pages=NULL), dict(lens=NULL), dict(sel=NULL), dict(held=NULL), dict(sel=P(1)),
                dict(held=P(4)), dict(ws=P(2)), dict(sel=P(8)), dict(held=P(3, 16)), dict(ws=P(7))):
        assert select(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ldq=248), dict(ldq=260), dict(q=P(1, 8)), dict(bd=P(2, 8))):
        assert select(lib, **bad) == B.ESTRIDE, bad
    need = B.bsfp8_select_workspace_bytes(3, 2, 2, 8)
    assert need > 0
    for bad in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P(6, 8))):
        assert select(lib, **bad) == B.EWORKSPACE, bad
    for a in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, -1), (1, 1, 1, 65535 * 64 + 1), (1 << 22, 1, 1, 1)):
        assert B.bsfp8_select_workspace_bytes(*a) == 0
    for a in ((1, 1, 1, 0), (7, 3, 2, 90)):
        for d in range(4):
            more = [x + (i == d) for i, x in enumerate(a)]
            assert 0 < B.bsfp8_select_workspace_bytes(*a) <= B.bsfp8_select_workspace_bytes(*more)


def sparse(lib, q=P(5), ldq=256, R=6, hq=4, c=None, sel=P(6), count=4, held=P(7), scale=0.1, ws=P(8), wsb=1 << 30, out=P(9)):
    return lib.bsfp8_sparse_attention(q, ldq, R, hq, c if c is not None else cache(), sel, count, held, scale, ws, wsb, out, NULL)


def test_sparse_refusals(lib):
    assert sparse(lib, R=0) == B.OK
    for bad in (dict(R=-1), dict(hq=3), dict(hq=130, ldq=130 * 64), dict(count=0), dict(count=1 << 27), dict(count=1 << 40), dict(c=cache(dim=96)),
                dict(R=1 << 30)):
        assert sparse(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(q=NULL), dict(out=NULL), dict(held=NULL), dict(sel=NULL), dict(scale=INF), dict(out=P(5)), dict(ws=P(9)), dict(out=P(3)),
                dict(out=P(6, 32)), dict(ws=P(7))):
        assert sparse(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ldq=248), dict(q=P(5, 8)), dict(out=P(9, 8))):
        assert sparse(lib, **bad) == B.ESTRIDE, bad
    need = B.bsfp8_attention_workspace_bytes(6, 1, 4, 2, 64, 64)
    for bad in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P(8, 4))):
        assert sparse(lib, **bad) == B.EWORKSPACE, bad


def sample(lib, lg=P(1), ld=1000, dt=1, R=3, V=1000, t=P(2), k=P(3), p=P(4), m=P(5), u=P(6), ws=P(7), wsb=1 << 30, tok=P(8), f=P(9),
           ldf=1000):
    return lib.bsfp8_sample(lg, ld, dt, R, V, t, k, p, m, u, ws, wsb, tok, f, ldf, NULL)


def test_sample_refusals(lib):
    assert sample(lib, R=0) == B.OK
    for bad in (dict(R=-1), dict(R=1 << 24), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25, ldf=1 << 25)):
        assert sample(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(dt=2), dict(lg=NULL), dict(t=NULL), dict(u=NULL), dict(tok=NULL), dict(tok=P(1)), dict(ws=P(1)), dict(f=P(1, 16)),
                dict(f=P(1), ldf=1004), dict(tok=P(9)), dict(ws=P(9)), dict(tok=P(2)), dict(f=P(6)), dict(ws=P(8))):
        assert sample(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ld=999), dict(ldf=998), dict(lg=P(1, 4)), dict(f=P(9, 8)), dict(ld=1 << 41)):
        assert sample(lib, **bad) == B.ESTRIDE, bad
    need = B.bsfp8_sample_workspace_bytes(3, 1000)
    assert need > 0
    for bad in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P(7, 8))):
        assert sample(lib, **bad) == B.EWORKSPACE, bad
    for a in ((0, 9), (1 << 24, 9), (3, 0), (3, (1 << 24) + 1)):
        assert B.bsfp8_sample_workspace_bytes(*a) == 0
    sizes = [(1, 1), (1, 1024), (1, 1025), (1, 131072), (7, 131072), (7, 131073), (64, 1 << 20), (64, 1 << 24)]
    for a, b in zip(sizes, sizes[1:]):
        assert 0 < B.bsfp8_sample_workspace_bytes(*a) <= B.bsfp8_sample_workspace_bytes(*b)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    z = torch.zeros
    bf = torch.bfloat16
    for bad in (z(2, 64), z(64, dtype=bf), z(2, 64, dtype=bf)):
        with pytest.raises(ValueError):
            B.bsfp8_residual_norm(bad)
    with pytest.raises(TypeError):
        B.bsfp8_residual_norm(z(2, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        B.bsfp8_residual_norm("h")
    i = torch.int32
    with pytest.raises(ValueError):
        B.bsfp8_step_tables(z(2, 3, dtype=i), z(2, dtype=i), z(2, dtype=i), z(4, dtype=i), z(1, dtype=i), 16, 4)
    with pytest.raises(ValueError):
        B.bsfp8_select_pages(z(1, 1, 4, 64, dtype=bf), z(3, 2, 2, 64, dtype=bf), z(1, 2, dtype=i), z(1, dtype=i), 2, 16)
    with pytest.raises(TypeError):
        B.bsfp8_cache_bounds("cache", z(1, 2, dtype=i), z(1, dtype=i))
    with pytest.raises(TypeError):
        B.bsfp8_sparse_attention(z(1, 4, 64, dtype=bf), None, z(1, 2, 3, dtype=i), z(1, dtype=i))
    for bad in (z(8), z(2, 8)):
        with pytest.raises(ValueError):
            B.bsfp8_sample(bad, None, None)
    with pytest.raises(TypeError):
        B.bsfp8_sample(z(2, 8, dtype=torch.float16), None, None)
