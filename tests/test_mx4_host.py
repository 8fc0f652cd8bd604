"""The 4-bit and table operators' checks of their arguments, without a GPU: every call below
is refused on the host, or has nothing to do. Also the host reference used by the GPU tests,
on values worked by hand."""
import ctypes

import numpy as np
import pytest

from tests import mx4_ref as ref

P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10004)  # never dereferenced


@pytest.fixture(scope="module")
def ne():
    import hashed_gram_embedding_horner_b200 as m
    return m


def test_reference_on_hand_worked_blocks():
    x = np.zeros((1, 64))
    x[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]  # ties go to the even code
    x[0, 32:36] = [-7.9, 1024 * 0, 0.3, 0.2]
    codes, scales = ref.quantise(x)
    assert scales.tolist() == [[127, 127]]
    assert codes[0, :8].tolist() == [7, 6, 6, 4, 4, 2, 2, 0]
    assert codes[0, 32:36].tolist() == [15, 0, 1, 0]  # -6 (saturated), 0, 0.5, 0
    assert ref.values(codes, scales)[0, 32:36].tolist() == [-6, 0, 0.5, 0]
    assert ref.quantise(np.full((1, 32), 2.0 ** -140))[1][0, 0] == 0
    assert ref.quantise(np.full((1, 32), 1.5 * 2.0 ** 20))[1][0, 0] == 127 + 18
    t = ref.tile_bytes(np.arange(130 * 5, dtype=np.int64).reshape(130, 5).astype(np.uint8))
    assert len(t) == 2 * 2 * 512
    assert t[(33 % 32) * 16 + 1 * 4 + 2] == (33 * 5 + 2) % 256 and t[512 + 0] == 4 and t[512 + 1] == 0
    assert t[2 * 512 + 1 * 16] == (129 * 5) % 256
    rows, grads, mags, cnt = ref.grad_rows(np.array([4, 1, 4, 2]), np.array([[1.0], [2.0], [-3.0], [5.0]]), 2.0, 2)
    assert rows.tolist() == [1, 4] and grads.tolist() == [[4.0], [-4.0]] and mags.tolist() == [[4.0], [8.0]]
    assert cnt.tolist() == [1, 2]


def test_scale_bytes(ne):
    f = ne._lib.ngram_mx4_scale_bytes
    assert f(10, 64, 0) == 20 and f(10, 64, 1) == 512 and f(129, 160, 1) == 2 * 2 * 512 and f(0, 32, 0) == 0
    assert f(-1, 64, 0) == 0 and f(4, 33, 0) == 0 and f(4, 64, 2) == 0 and f(4, 0, 0) == 0


def test_quantize_refusals(ne):
    q = lambda src=FAKE, dt=0, r=4, c=64, st=64, co=FAKE, sc=FAKE, lay=0: ne._lib.ngram_mx4_quantize(
        src, dt, r, c, st, co, sc, lay, None)
    assert q(r=-1) == -1 and q(c=0) == -1 and q(dt=2) == -1 and q(lay=2) == -1 and q(st=63) == -1
    assert q(src=None) == -1 and q(co=None) == -1 and q(sc=None) == -1 and q(r=1 << 31) == -1
    assert q(c=48, st=48) == -2
    assert q(co=ODD) == -3 and q(sc=ODD) == -3 and q(src=P(0x10001)) == -3 and q(src=P(0x10002), dt=1) == -3
    assert q(r=0, src=None, co=None, sc=None) == 0


def test_product_refusals(ne):
    lib = ne._lib
    mx = lambda c=0x10000, s=0x20000: ctypes.byref(ne._Mx4(c, s))
    need = lib.ngram_mx4_product_workspace_bytes(8, 8, 64)
    assert need > 0 and lib.ngram_mx4_product_workspace_bytes(-1, 8, 64) == 0
    f = lambda a=mx(), b=mx(), M=8, N=8, K=64, al=1.0, out=FAKE, dt=0, ld=8, ws=FAKE, wb=need: lib.ngram_mx4_product(
        a, b, M, N, K, al, out, dt, ld, ws, wb, None)
    assert f(a=None) == -1 and f(b=None) == -1 and f(M=-1) == -1 and f(N=-1) == -1 and f(K=0) == -1
    assert f(al=float("nan")) == -1 and f(al=float("inf")) == -1 and f(dt=2) == -1 and f(ld=7) == -1
    assert f(ws=None) == -1 and f(ws=ODD) == -3 and f(wb=need - 1) == -4 and f(K=65) == -2
    assert f(a=mx(None)) == -1 and f(b=mx(0x10000, None)) == -1 and f(out=None) == -1
    assert f(a=mx(0x10008)) == -3 and f(b=mx(0x10000, 0x20008)) == -3 and f(out=P(0x10001)) == -3
    assert f(M=0) == 0 and f(N=0, ld=0) == 0


@pytest.mark.parametrize("M,N,K,sms,form", [
    (32768, 2048, 2048, 148, 256), (65536, 4096, 4096, 148, 256), (2300, 2048, 2048, 148, 256),  # 72 of 74 pairs' tiles
    (1280, 4096, 4096, 148, 320), (1280, 4096, 1024, 148, 192), (28600, 318, 1056, 148, 320), (1280, 2048, 2048, 148, 192), (512, 4096, 4096, 148, 128), (333, 1111, 2080, 148, 64),
    (5, 4096, 4096, 148, 64), (4, 4096, 4096, 148, 0), (1, 16384, 16384, 148, 128), (1, 1, 32, 2, 0), (5, 1, 32, 2, 64), (1280, 4096, 4096, 40, 256),
])
def test_product_tiles_for_a_device_size(ne, M, N, K, sms, form):
    assert ne.ngram_mx4_product_form(M, N, K, sms) == form


def test_product_form_refusals(ne):
    for bad in ((0, 1, 32, 148), (1, 0, 32, 148), (1, 1, 0, 148), (1, 1, 32, 1), (1 << 31, 1, 32, 148)):
        assert ne._lib.ngram_mx4_product_form(*bad) == -1
        with pytest.raises(ne.NgramError):
            ne.ngram_mx4_product_form(*bad)


def _plan(ne, V0=1000, D=128, N=3, K=2, V=(11, 13, 17, 19), dtype=0):
    return ne.ngram_embed_plan_create(V0, D, N, K, V, dtype)


def test_layer_refusals(ne):
    lib = ne._lib
    plan = _plan(ne)
    tabs = (ne._Mx4 * 4)(*[ne._Mx4(0x30000, 0x40000)] * 4)
    need = lib.ngram_embed_mx4_workspace_bytes(plan.handle, 100)
    # head, codes of 100 rows of 128, one row block of one scale tile
    assert need == 33024 + 100 * 64 + 512
    assert lib.ngram_embed_mx4_workspace_bytes(plan.handle, -1) == 0
    assert lib.ngram_embed_mx4_workspace_bytes(None, 10) == 0
    W = ctypes.byref(ne._Mx4(0x50000, 0x60000))
    fwd = lambda h=plan.handle, tok=FAKE, off=FAKE, B=2, T=100, e0=FAKE, tb=tabs, w=W, cache=None, out=FAKE, ws=FAKE, wb=need: \
        lib.ngram_embed_fwd_mx4(h, tok, off, B, T, e0, tb, w, cache, None, out, ws, wb, None)
    prj = lambda h=plan.handle, tok=FAKE, idx=FAKE, T=100, e0=FAKE, tb=tabs, w=W, out=FAKE, ws=FAKE, wb=need: \
        lib.ngram_embed_project_mx4(h, tok, idx, T, e0, tb, w, out, ws, wb, None)
    for f in (fwd, prj):
        assert f(h=None) == -1 and f(tok=None) == -1 and f(T=-1) == -1 and f(e0=None) == -1 and f(tb=None) == -1
        assert f(w=None) == -1 and f(out=None) == -1 and f(ws=None) == -1 and f(wb=need - 1) == -4
        assert f(ws=ODD) == -3 and f(out=ODD) == -3 and f(e0=ODD) == -3
        assert f(w=ctypes.byref(ne._Mx4(0x50008, 0x60000))) == -3 and f(w=ctypes.byref(ne._Mx4(0x50000, None))) == -1
        bad = (ne._Mx4 * 4)(*[ne._Mx4(0x30000, 0x40000)] * 3, ne._Mx4(0x30004, 0x40000))
        assert f(tb=bad) == -3
        assert f(T=0) == 0
    assert fwd(off=None) == -1 and fwd(B=0) == -1 and fwd(B=-1) == -1 and prj(idx=None) == -1
    assert fwd(cache=ctypes.byref(ne._Cache(0x1000, 0x2000, 0x3000, 1, 8))) == -1  # capacity < N - 1
    for kw in (dict(D=64, N=3, K=2), dict(N=1, K=1, V=())):  # d = 16; no sub-tables
        p = _plan(ne, **kw)
        assert lib.ngram_embed_mx4_workspace_bytes(p.handle, 100) == 0
        assert fwd(h=p.handle, wb=1 << 30) == -2 and prj(h=p.handle, wb=1 << 30) == -2
        with pytest.raises(ne.NgramError):
            ne.new_embed_mx4_workspace(p, 10, device="cpu")


def test_embedding_refusals(ne):
    lib = ne._lib
    head = lib.ngram_embedding_workspace_bytes(0, 64)
    assert head >= 33024 and lib.ngram_embedding_workspace_bytes(-1, 64) == 0
    assert lib.ngram_embedding_workspace_bytes(10, 0) == 0
    fw = lambda tab=FAKE, sc=None, dt=0, V=50, D=64, ids=FAKE, n=9, s=1.0, pad=-1, out=FAKE, od=0, ld=64, ws=FAKE, wb=head: \
        lib.ngram_embedding_fwd(tab, sc, dt, V, D, ids, n, s, pad, out, od, ld, ws, wb, None)
    assert fw(tab=None) == -1 and fw(dt=3) == -1 and fw(dt=2) == -1 and fw(V=0) == -1 and fw(V=1 << 31) == -1
    assert fw(D=0) == -1 and fw(n=-1) == -1 and fw(s=float("nan")) == -1 and fw(out=None) == -1 and fw(od=2) == -1
    assert fw(ld=63) == -1 and fw(ws=None) == -1 and fw(ids=None, n=51) == -1
    assert fw(D=20, ld=24) == -2 and fw(dt=2, sc=FAKE, D=40) == -2
    assert fw(tab=ODD) == -3 and fw(out=ODD) == -3 and fw(ws=ODD) == -3 and fw(ld=65) == -3 and fw(wb=100) == -4
    assert fw(n=0, tab=None, out=None) == 0
    need = lib.ngram_embedding_workspace_bytes(9, 64)
    assert need > head
    bw = lambda ids=FAKE, n=9, g=FAKE, gd=0, gs=64, V=50, D=64, s=1.0, dt=FAKE, ws=FAKE, wb=need: lib.ngram_embedding_bwd(
        ids, n, g, gd, gs, V, D, s, -1, dt, ws, wb, None)
    rw = lambda ids=FAKE, n=9, g=FAKE, gd=0, gs=64, V=50, D=64, s=1.0, dt=FAKE, ws=FAKE, wb=need, rows=FAKE, cnt=FAKE: \
        lib.ngram_embedding_bwd_rows(ids, n, g, gd, gs, V, D, s, -1, rows, cnt, dt, ws, wb, None)
    for f in (bw, rw):
        assert f(ids=None) == -1 and f(n=-1) == -1 and f(g=None) == -1 and f(gd=2) == -1 and f(gs=63) == -1
        assert f(V=0) == -1 and f(D=0) == -1 and f(s=float("inf")) == -1 and f(dt=None) == -1 and f(ws=None) == -1
        assert f(D=20, gs=24) == -2 and f(g=ODD) == -3 and f(dt=ODD) == -3 and f(ws=ODD) == -3 and f(gs=65) == -3
        assert f(wb=need - 1) == -4
    assert rw(rows=None) == -1 and rw(cnt=None) == -1


def test_binding_refuses_host_tensors_and_wrong_shapes(ne):
    import torch
    cpu = torch.zeros((4, 64))
    with pytest.raises(ne.NgramError):
        ne.Mx4(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8), 4, 64)
    with pytest.raises(ne.NgramError):
        ne.Mx4.empty(4, 40, device="cpu")
    with pytest.raises(ne.NgramError):
        ne.ngram_embedding_fwd(cpu, torch.zeros(4, dtype=torch.int32), cpu, cpu)
    with pytest.raises(ne.NgramError):
        ne.ngram_embedding_bwd(torch.zeros(4, dtype=torch.int32), cpu, cpu, cpu)
    with pytest.raises(ne.NgramError):
        ne.ngram_embedding_bwd_rows(torch.zeros(4, dtype=torch.int32), cpu, 4, torch.zeros(4, dtype=torch.int32),
                                    torch.zeros(1, dtype=torch.int32), cpu, cpu)
    for none in (None, torch.zeros(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ne.NgramError):
            ne._space(none, -1)


@pytest.mark.parametrize("limit,most", [(16, 65536), (15, 32768), (8, 32768), (4, 16384), (1, 4096), (0, 0), (32, 65536)])
def test_gradient_sort_fits_the_clusters_that_a_device_places(ne, limit, most):
    """Never more CTAs than the device places, room for every id (4096 a CTA), and the sort in
    tiles for what does not fit."""
    for n in (1, 1024, 1025, 4096, 4097, 8192, 8193, 16384, 16385, 32768, 32769, 65536, 65537, 1 << 30):
        ctas = ne.ngram_embedding_sort_ctas(n, limit)
        assert ctas <= limit and (ctas == 0) == (n > most)
        assert ctas == 0 or (n <= 4096 * ctas and ctas & (ctas - 1) == 0)
    for n, ctas in ((1000, 1), (16384, 16), (16385, 16), (32769, 16)):  # a whole device: few ids a thread
        assert limit < 16 or ne.ngram_embedding_sort_ctas(n, limit) == ctas
    for bad in ((0, 16), (-1, 16), (1 << 31, 16), (5, -1)):
        with pytest.raises(ne.NgramError):
            ne.ngram_embedding_sort_ctas(*bad)


def test_three_rows_take_a_warp_a_column_where_four_do(ne):
    """The kernel of few rows computes three rows as four: as long, so the same choice."""
    form = ne.ngram_mx4_product_form
    for N in range(32, 20000, 96):
        for K in (512, 1024, 2080, 4096, 8192, 16384):
            assert form(3, N, K) == form(4, N, K), (N, K)


def test_plan_tells_its_device(ne):
    import torch
    plan = _plan(ne)
    assert plan.device == (torch.cuda.current_device() if torch.cuda.is_available() else -1)
    assert ne._lib.ngram_embed_plan_device(None) == -1


def test_gradient_pieces(ne):
    """The longest pieces that leave 4096 warps (1024 for the middle ones) of 256 columns."""
    for n in (1, 8, 641, 4096, 32767, 32768, 65536, 131072, 524161, 524160, 1 << 30):
        for D in (8, 136, 256, 264, 2048, 4096, 7176):
            warps = lambda p: -(-n // p) * -(-D // 256)
            want = 128 if warps(128) >= 4096 else (32 if warps(32) >= 1024 else 8)
            assert ne.ngram_embedding_piece(n, D) == want
    for bad in ((0, 8), (1 << 31, 8), (5, 0), (5, 1 << 31)):
        with pytest.raises(ne.NgramError):
            ne.ngram_embedding_piece(*bad)


def test_strides_of_arrays_that_are_read(ne):
    """0, or at least the columns; the refusal that follows (a misaligned array) shows that the
    stride was let through."""
    q = lambda st: ne._lib.ngram_mx4_quantize(FAKE, 0, 4, 64, st, ODD, FAKE, 0, None)
    assert [q(st) for st in (-64, -1, 1, 63)] == [-1] * 4 and [q(st) for st in (0, 64, 65)] == [-3] * 3
    need = ne._lib.ngram_embedding_workspace_bytes(9, 64)
    dense = lambda st: ne._lib.ngram_embedding_bwd(FAKE, 9, FAKE, 1, st, 50, 64, 1.0, -1, ODD, FAKE, need, None)
    rows = lambda st: ne._lib.ngram_embedding_bwd_rows(FAKE, 9, FAKE, 1, st, 50, 64, 1.0, -1, FAKE, FAKE, ODD, FAKE, need, None)
    for f in (dense, rows):
        assert [f(st) for st in (-64, -1, 8, 63)] == [-1] * 4 and [f(st) for st in (0, 64, 68)] == [-3] * 3
