"""CPU checks of the verify step's entry points: every refusal of sizes, strides, alignment, missing or overlapping buffers
returns its status before any GPU work, and the binding refuses what the library cannot see. No kernel is launched."""
import ctypes

import pytest
import torch

import block_scaled_fp8_skinny_amd as B

NULL = ctypes.c_void_p(0)


def P(i, off=0):
    return ctypes.c_void_p((i << 36) + off)                      # far apart: nothing overlaps


def cache(pages=8, heads=2, page=16, dim=64, at=(1, 2, 3, 4)):
    s = B._KVCacheStruct(*(p if isinstance(p, int) and p > 64 else p << 36 for p in at), pages, heads, page, dim)
    return ctypes.byref(s)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from block_scaled_fp8_skinny_amd import build
        build.build()
    return B.lib()


def write(lib, c=None, R=4, slots=P(5), k=P(6), ldk=128, v=P(7), ldv=128, q=P(8), ldq=256, hq=4, qo=P(9), qw=NULL, kw=NULL,
          eps=1e-6, cs=P(10), npos=9, rot=64, pos=P(11), inter=0):
    return lib.bsfp8_cache_write(c if c is not None else cache(), slots, R, k, ldk, v, ldv, q, ldq, hq, qo, qw, kw, eps, cs,
                                 npos, rot, pos, inter, NULL)


def test_cache_shapes(lib):
    for bad in (dict(dim=32), dict(dim=96), dict(dim=512), dict(page=8), dict(page=24), dict(page=0), dict(heads=0),
                dict(pages=-1), dict(pages=1 << 27), dict(page=1 << 40)):
        assert write(lib, cache(**bad)) == B.ESHAPE
        assert lib.bsfp8_cache_read(cache(**bad), P(5), 1, P(6), P(7), NULL) == B.ESHAPE
    assert write(lib, ctypes.c_void_p(0)) == B.EINVAL
    assert write(lib, cache(at=(1, 0, 3, 4))) == B.EINVAL
    assert write(lib, cache(at=((1 << 36) + 8, 2, 3, 4))) == B.ESTRIDE


def test_write_refusals(lib):
    assert write(lib, R=0) == B.OK
    for bad in (dict(R=-1), dict(hq=-1), dict(rot=8), dict(rot=80), dict(rot=-16), dict(npos=-1), dict(npos=0)):
        assert write(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(slots=NULL), dict(k=NULL), dict(v=NULL), dict(q=NULL), dict(qo=NULL), dict(cs=NULL), dict(pos=NULL),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inter=2), dict(qo=P(8, 64)),
                dict(qo=P(1, 32)), dict(k=P(1, 32)), dict(v=P(4, 16)), dict(cs=P(9, 16)), dict(slots=P(3))):
        assert write(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ldk=120), dict(ldk=132), dict(ldv=64), dict(ldq=248), dict(k=P(6, 8)), dict(q=P(8, 2)), dict(qo=P(9, 4)),
                dict(qw=P(12, 2)), dict(kw=P(12, 8)), dict(cs=P(10, 4))):
        assert write(lib, **bad) == B.ESTRIDE, bad


def test_read_refusals(lib):
    rd = lib.bsfp8_cache_read
    assert rd(cache(), NULL, 0, NULL, NULL, NULL) == B.OK
    assert rd(cache(), P(5), -1, P(6), P(7), NULL) == B.ESHAPE
    assert rd(cache(), P(5), 1 << 30, P(6), P(7), NULL) == B.ESHAPE
    for a in ((NULL, P(6), P(7)), (P(5), NULL, P(7)), (P(5), P(6), NULL), (P(5), P(6), P(6, 64)), (P(5), P(1), P(7))):
        assert rd(cache(), a[0], 4, a[1], a[2], NULL) == B.EINVAL
    assert rd(cache(), P(5), 4, P(6, 8), P(7), NULL) == B.ESTRIDE


def test_grid_limits(lib):
    """More workgroups than a launch can count (2^24 of 256 threads) are refused, not handed to the launch."""
    assert write(lib, R=1 << 24, k=P(1 << 10), v=P(2 << 10), q=P(3 << 10), qo=P(4 << 10), slots=P(5 << 10),
                 pos=P(6 << 10)) == B.ESHAPE
    assert lib.bsfp8_cache_read(cache(dim=256), P(5), 1 << 27, P(1 << 10), P(2 << 10), NULL) == B.ESHAPE
    assert B.bsfp8_attention_workspace_bytes(1 << 20, 1, 16, 16, 64, 64) == 0
    assert B.bsfp8_attention_workspace_bytes((1 << 20) - 1, 1, 16, 16, 64, 64) > 0
    assert B.bsfp8_verify_workspace_bytes(1 << 18, 64, 8) == 0
    assert B.bsfp8_verify_workspace_bytes(1 << 18, 32, 8) > 0


def attn(lib, c=None, q=P(5), ldq=256, Bn=3, T=2, hq=4, pages=P(6), ld=4, lens=P(7), nodes=NULL, mask=P(8), max_len=64,
         ws=P(9), wsb=1 << 30, out=P(10)):
    return lib.bsfp8_tree_attention(q, ldq, Bn, T, hq, c if c is not None else cache(), pages, ld, lens, nodes, mask, 0.1,
                                    max_len, ws, wsb, out, NULL)


def test_attention_refusals(lib):
    assert attn(lib, Bn=0) == B.OK
    for bad in (dict(T=0), dict(T=65), dict(hq=3), dict(hq=0), dict(hq=130, ldq=130 * 64), dict(Bn=-1), dict(max_len=-1),
                dict(ld=-1), dict(max_len=1 << 31), dict(T=1 << 20, Bn=1 << 12, mask=NULL), dict(c=cache(dim=96))):
        assert attn(lib, **bad) == B.ESHAPE, bad
    for bad in (dict(q=NULL), dict(out=NULL), dict(lens=NULL), dict(pages=NULL), dict(out=P(5, 256)), dict(ws=P(10)),
                dict(out=P(3)), dict(ws=P(8))):
        assert attn(lib, **bad) == B.EINVAL, bad
    for bad in (dict(ldq=248), dict(ldq=260), dict(q=P(5, 8)), dict(out=P(10, 8))):
        assert attn(lib, **bad) == B.ESTRIDE, bad
    need = B.bsfp8_attention_workspace_bytes(3, 2, 4, 2, 64, 64)
    assert need > 0
    for bad in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P(9, 8))):
        assert attn(lib, **bad) == B.EWORKSPACE, bad
    for a in ((3, 2, 5, 2, 64, 64), (3, 2, 4, 2, 96, 64), (0, 2, 4, 2, 64, 64), (3, 0, 4, 2, 64, 64), (3, 2, 4, 2, 64, -1)):
        assert B.bsfp8_attention_workspace_bytes(*a) == 0


def chain(lib, lg=P(1), dr=P(2), dt=1, Bn=3, T=4, V=100, tok=P(3), t=P(4), u=P(5), us=P(6), ws=P(7), wsb=1 << 30, out=P(8),
          n=P(9)):
    return lib.bsfp8_verify_chain(lg, dr, dt, Bn, T, V, tok, t, u, us, ws, wsb, out, n, NULL)


def tree(lib, lg=P(1), dt=1, Bn=3, T=4, V=100, tok=P(3), par=P(2), t=P(4), u=P(5), ws=P(7), wsb=1 << 30, out=P(8), path=P(6),
         n=P(9)):
    return lib.bsfp8_verify_tree(lg, dt, Bn, T, V, tok, par, t, u, ws, wsb, out, path, n, NULL)


def test_verify_refusals(lib):
    need = B.bsfp8_verify_workspace_bytes(3, 4, 100)
    assert need > 0
    for f in (chain, tree):
        assert f(lib, Bn=0) == B.OK
        for bad in (dict(T=0), dict(T=65), dict(V=0), dict(V=(1 << 24) + 1), dict(Bn=-1)):
            assert f(lib, **bad) == B.ESHAPE, bad
        for bad in (dict(dt=2), dict(lg=NULL), dict(tok=NULL), dict(t=NULL), dict(u=NULL), dict(out=NULL), dict(n=NULL),
                    dict(out=P(1, 64)), dict(n=P(8, 4)), dict(ws=P(1)), dict(out=P(3)), dict(n=P(5))):
            assert f(lib, **bad) == B.EINVAL, (f.__name__, bad)
        assert f(lib, lg=P(1, 4)) == B.ESTRIDE
        for bad in (dict(ws=NULL), dict(wsb=need - 1), dict(ws=P(7, 8))):
            assert f(lib, **bad) == B.EWORKSPACE, bad
    for bad in (dict(dr=NULL), dict(us=NULL)):
        assert chain(lib, **bad) == B.EINVAL
    for bad in (dict(par=NULL), dict(path=NULL), dict(path=P(8, 16))):
        assert tree(lib, **bad) == B.EINVAL
    for a in ((0, 4, 100), (3, 65, 100), (3, 4, 0)):
        assert B.bsfp8_verify_workspace_bytes(*a) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    z = torch.zeros
    with pytest.raises(ValueError):
        B.KVCache(z(2, 1, 16, 64, dtype=torch.uint8), z(2, 1, 16, 2, dtype=torch.uint8), z(2, 1, 16, 64, dtype=torch.uint8),
                  z(2, 1, 16, 2, dtype=torch.uint8))             # not on a GPU
    for shape in ((2, 1, 16, 96), (2, 1, 20, 64), (2, 16, 64)):
        with pytest.raises(ValueError):
            B.KVCache(*(z(*shape, dtype=torch.uint8) for _ in range(4)))
    with pytest.raises(TypeError):
        B.KVCache(*(z(2, 1, 16, 64) for _ in range(4)))
    with pytest.raises(TypeError):
        B.bsfp8_cache_read("cache", z(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        B.bsfp8_verify_chain(z(1, 2, 8, dtype=torch.float16), None, None, None, None, None)
    with pytest.raises(ValueError):
        B.bsfp8_verify_tree(z(1, 2, 8), None, None, None, None)  # not on a GPU
