"""4-bit tables on the GPU: quantisation bit-exact, the product and the layer within the bound
of their fp32 sums and one output rounding, against plain 64-bit definitions on the host."""
import numpy as np
import pytest
import torch

import oracle
from synth import gen
from tests import mx4_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: ref.BF16_HALF, F32: ref.F32_HALF}


@pytest.fixture(scope="module")
def ne():
    import hashed_gram_embedding_horner_b200 as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def device_mx4(ne, codes, scales, layout):
    s = ref.tile_bytes(scales, fill=255) if layout == ne.MX4_TILES else scales  # rows past the last: NaN bytes
    return ne.Mx4(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(s).cuda(), codes.shape[0], codes.shape[1],
                  layout)


def special_rows(cols):
    """Blocks of every special kind, tiled over a row of `cols`."""
    z = np.zeros(32)
    one = np.zeros(32)
    one[5] = -1.0
    ties = np.resize(np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0]), 32)
    sat = np.resize(np.array([7.9375, 6.5, -7.0, 0.1]), 32)
    tiny = np.resize(np.array([2.0 ** -126, -2.0 ** -130, 2.0 ** -133, 0.0]), 32)
    huge = np.resize(np.array([3.3e38, -1e38, 1e30]), 32)
    inf = one.copy()
    inf[0] = np.inf
    nan = one.copy()
    nan[31] = np.nan
    neg0 = -z
    rows = [np.resize(np.concatenate([b, one]), cols) for b in (z, one, ties, sat, tiny, huge, inf, nan, neg0)]
    return np.stack(rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (130, 96), (257, 160), (9, 512)])
def test_quantize_is_the_definition(ne, dtype, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, 1)))).to(dtype)
    if rows == 9:
        x = torch.from_numpy(special_rows(cols)).to(dtype)
    codes, scales = ref.quantise(f64(x))
    for layout in (ne.MX4_ROWS, ne.MX4_TILES):
        q = ne.Mx4.empty(rows, cols, layout)
        q.scales.fill_(77)  # rows past the last keep what was there
        ne.ngram_mx4_quantize(x.cuda(), q)
        assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes))
        want = scales if layout == ne.MX4_ROWS else ref.tile_bytes(scales, fill=77)
        assert np.array_equal(q.scales.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_reads_strided_and_unaligned_rows(ne, dtype):
    rng = np.random.default_rng(5)
    buf = torch.from_numpy(rng.standard_normal((40, 331))).to(dtype).cuda()
    for view in (buf[:, 8:72], buf[3:, 5:133], buf[::2, 1:33], buf[7:8, 3:35]):
        codes, scales = ref.quantise(f64(view))
        q = ne.Mx4.empty(view.shape[0], view.shape[1], ne.MX4_ROWS)
        ne.ngram_mx4_quantize(view, q)
        assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes)) and np.array_equal(q.scales.cpu().numpy(), scales)


def test_quantising_what_a_quantised_row_stands_for_changes_nothing(ne):
    x = torch.randn((70, 256), device="cuda")
    q, r = ne.Mx4.empty(70, 256), ne.Mx4.empty(70, 256)
    back = torch.empty((70, 256), device="cuda")
    ne.ngram_mx4_quantize(x, q)
    ne.ngram_embedding_fwd(q, None, back, ne.new_embedding_workspace(0, 256))
    ne.ngram_mx4_quantize(back, r)
    assert torch.equal(q.codes, r.codes) and torch.equal(q.scales, r.scales)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 16, 64), (5, 7, 96), (2, 64, 128), (128, 128, 256), (129, 257, 288), (127, 65, 320), (64, 192, 512),
    (33, 4096, 1024), (300, 1000, 2080), (640, 512, 4096), (1, 2048, 4096), (2000, 1536, 544),
    (600, 2048, 1056), (2300, 2048, 320), (2200, 2100, 96), (1290, 2047, 544), (700, 2500, 64), (3024, 5774, 64),
    (6864, 2528, 96), (2290, 2048, 1056), (2300, 2041, 2048),
    (1279, 4095, 2080), (1100, 4352, 2304), (28600, 318, 1056),
    (1, 4096, 4096), (2, 2041, 64), (3, 1000, 4128), (4, 130, 8224), (2, 129, 4096), (4, 512, 512),
])
def test_product_within_the_bound_of_its_sums(ne, M, N, K, out_dtype):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, b = ref.random_mx4(rng, M, K), ref.random_mx4(rng, N, K)
    av, bv = ref.values(*a), ref.values(*b)
    out = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    ws = ne.new_mx4_workspace(M, N, K)
    ne.ngram_mx4_product(device_mx4(ne, *a, ne.MX4_TILES), device_mx4(ne, *b, ne.MX4_TILES), out, ws, alpha=0.5)
    assert ne.ngram_embed_get_status(ws) == 0
    want = av @ bv.T * 0.5
    assert (np.abs(f64(out) - want) <= ref.product_bound(av, bv * 0.5, HALF[out_dtype], want)).all()


def test_products_above_take_every_form_of_tiles(ne):
    sizes = [m.args[1] for m in test_product_within_the_bound_of_its_sums.pytestmark
             if m.name == "parametrize" and m.args[0] == "M,N,K"][0]
    assert {ne.ngram_mx4_product_form(*s) for s in sizes} == {0, 64, 128, 192, 256, 320}


@pytest.mark.parametrize("rows", [37, 3])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_product_writes_only_its_own_columns(ne, out_dtype, rows):
    rng = np.random.default_rng(3)
    a, b = ref.random_mx4(rng, rows, 96), ref.random_mx4(rng, 41, 96)
    av, bv = ref.values(*a), ref.values(*b)
    want = av @ bv.T
    for lo, width in ((0, 64), (3, 57), (8, 72)):
        buf = torch.full((rows + 2, width), 7.0, dtype=out_dtype, device="cuda")
        out = buf[1:rows + 1, lo:lo + 41]
        ne.ngram_mx4_product(device_mx4(ne, *a, ne.MX4_TILES), device_mx4(ne, *b, ne.MX4_TILES), out,
                             ne.new_mx4_workspace(rows, 41, 96))
        assert (np.abs(f64(out) - want) <= ref.product_bound(av, bv, HALF[out_dtype], want)).all()
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("rows", [130, 4, 1])
def test_product_carries_nan_blocks_and_wide_scales(ne, rows):
    """A NaN block makes its row (of A) or column (of B) NaN and nothing else; scales at the
    ends of the range multiply as powers of two."""
    rng = np.random.default_rng(9)
    a, b = ref.random_mx4(rng, rows, 256), ref.random_mx4(rng, 70, 256)
    a[1][rows - 1, 3] = 255
    b[1][5, 0] = 255
    out = torch.empty((rows, 70), device="cuda")
    ws = ne.new_mx4_workspace(rows, 70, 256)
    ne.ngram_mx4_product(device_mx4(ne, *a, ne.MX4_TILES), device_mx4(ne, *b, ne.MX4_TILES), out, ws)
    av, bv = ref.values(*a), ref.values(*b)
    got, want = f64(out), av @ bv.T
    assert np.isnan(got[rows - 1]).all() and np.isnan(got[:, 5]).all()
    ok = ~np.isnan(want)
    assert ok.sum() == (rows - 1) * 69
    assert (np.abs(got - want)[ok] <= ref.product_bound(np.nan_to_num(av), np.nan_to_num(bv), ref.F32_HALF,
                                                        np.nan_to_num(want))[ok]).all()
    a[1][:], b[1][:] = 0, 254  # 2^-127 and 2^127: the product's scales cancel
    ne.ngram_mx4_product(device_mx4(ne, *a, ne.MX4_TILES), device_mx4(ne, *b, ne.MX4_TILES), out, ws)
    av, bv = ref.values(*a), ref.values(*b)
    want = av @ bv.T
    assert (np.abs(f64(out) - want) <= ref.product_bound(av, bv, ref.F32_HALF, want)).all()


def make_layer(ne, seed, V0, D, N, K, V, dtype):
    rng = np.random.default_rng(seed)
    S = (N - 1) * K
    d = D // S
    E = [ref.random_mx4(rng, v, d, spread=2) for v in V]
    for e in E:
        e[1][:] -= 5
    W = ref.random_mx4(rng, D, D, spread=1)
    W[1][:] -= 3
    E0 = torch.from_numpy(rng.standard_normal((V0, D))).to(dtype).cuda()
    plan = ne.ngram_embed_plan_create(V0, D, N, K, V, ne.NGRAM_BF16 if dtype == BF16 else ne.NGRAM_F32)
    return dict(plan=plan, E0=E0, E=[device_mx4(ne, *e, ne.MX4_ROWS) for e in E], W=device_mx4(ne, *W, ne.MX4_TILES),
                E_vals=[ref.values(*e) for e in E], W_vals=ref.values(*W))


LAYERS = [  # V0, D, N, K, V, dtype
    (50, 32, 2, 1, (61,), BF16),
    (97, 96, 2, 3, (101, 103, 107), F32),
    (1000, 512, 3, 2, (997, 1009, 1013, 1019), BF16),
    (300, 1280, 5, 2, (211, 223, 227, 229, 233, 239, 241, 251), BF16),
    (131, 288, 4, 1, (400, 401, 402), F32),
    (131072, 1024, 3, 1, (3001, 3011), BF16),
]


@pytest.mark.parametrize("lengths", [[1], [1, 2], [5, 0, 1, 3], [127, 2], [100, 300, 0, 41], [1300]])
@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer_from_4bit_tables(ne, case, lengths):
    V0, D, N, K, V, dtype = LAYERS[case]
    L = make_layer(ne, case, V0, D, N, K, V, dtype)
    off = gen.offsets_from_lengths(lengths)
    T = int(off[-1])
    tokens = np.random.default_rng(T).integers(0, V0, T).astype(np.int32)
    out = torch.full((T, D), 3.0, dtype=dtype, device="cuda")
    ws = ne.new_embed_mx4_workspace(L["plan"], T)
    ne.ngram_embed_plan_set_output_scale(L["plan"], 1.5)
    ne.ngram_embed_fwd_mx4(L["plan"], torch.from_numpy(tokens).cuda(), torch.from_numpy(off).cuda(), L["E0"], L["E"],
                           L["W"], out, ws)
    assert ne.ngram_embed_get_status(ws) == 0
    want, acc, _ = ref.layer(V0, N, K, V, tokens, off, f64(L["E0"]), L["E_vals"], L["W_vals"], out_scale=1.5)
    assert (np.abs(f64(out) - want) <= acc + HALF[dtype] * (np.abs(want) + acc)).all()


@pytest.mark.parametrize("dtype,D,N,K,lengths", [
    (BF16, 1024, 3, 1, [3000, 0, 1, 700, 299]), (F32, 1024, 3, 1, [3999]), (BF16, 1056, 4, 1, [2049, 2048]),
    (BF16, 1280, 5, 2, [1] * 3000), (BF16, 2048, 3, 2, [2300]), (F32, 2048, 3, 2, [1, 2299]), (BF16, 2080, 2, 1, [1200, 101]),
    (BF16, 2240, 3, 1, [2500]), (F32, 2240, 3, 1, [1, 0, 2449]),
])
def test_layer_of_many_tokens(ne, dtype, D, N, K, lengths):
    """Several tiles a CTA, in every form of them; twice on one workspace, then with ids out of
    range, then with bad offsets."""
    S = (N - 1) * K
    V0, V = 5000, [3001 + 10 * s for s in range(S)]
    L = make_layer(ne, D, V0, D, N, K, V, dtype)
    off = gen.offsets_from_lengths(lengths)
    T = int(off[-1])
    rng = np.random.default_rng(T)
    ws = ne.new_embed_mx4_workspace(L["plan"], T)
    off_d = torch.from_numpy(off).cuda()
    for bad in (False, False, True):
        tokens = rng.integers(0, V0, T).astype(np.int32)
        good = tokens.copy()
        if bad:
            tokens[::501], good[::501] = np.where(np.arange(len(tokens[::501])) % 2, V0, -3), 0
        out = torch.full((T, D), 3.0, dtype=dtype, device="cuda")
        ne.ngram_embed_fwd_mx4(L["plan"], torch.from_numpy(tokens).cuda(), off_d, L["E0"], L["E"], L["W"], out, ws)
        assert ne.ngram_embed_get_status(ws) == (0x1 if bad else 0)
        want, acc, idx = ref.layer(V0, N, K, V, good, off, f64(L["E0"]), L["E_vals"], L["W_vals"])
        assert (np.abs(f64(out) - want) <= acc + HALF[dtype] * (np.abs(want) + acc)).all()
    assert not bool(ws[256:33024].any())  # the counters of other calls stay zero
    ne.ngram_embed_clear_status(ws)
    again = torch.empty_like(out)
    ne.ngram_embed_project_mx4(L["plan"], torch.from_numpy(good).cuda(), torch.from_numpy(idx.astype(np.int32)).cuda(),
                               L["E0"], L["E"], L["W"], again, ws)
    assert torch.equal(again, out) and ne.ngram_embed_get_status(ws) == 0
    off_d[-1] -= 1  # tokens past the last sequence's end
    ne.ngram_embed_fwd_mx4(L["plan"], torch.from_numpy(good).cuda(), off_d, L["E0"], L["E"], L["W"], again, ws)
    assert ne.ngram_embed_get_status(ws) == 0x2


def test_layer_through_the_ring(ne):
    """Decode: windows continue into each slot's committed history, also through other slots."""
    V0, D, N, K, V, dtype = LAYERS[2]
    L = make_layer(ne, 11, V0, D, N, K, V, dtype)
    rng = np.random.default_rng(12)
    B, C, P = 37, 8, 5
    slots = rng.permutation(64)[:B].astype(np.int32)
    hist = [rng.integers(0, V0, int(rng.integers(0, 9))).astype(np.int32) for _ in range(B)]
    cache = ne.Cache.empty(64, C)
    ws = ne.new_embed_mx4_workspace(L["plan"], B * P)
    slots_d = torch.from_numpy(slots).cuda()
    off_h = gen.offsets_from_lengths([len(h) for h in hist])
    ne.ngram_cache_append(L["plan"], cache, torch.from_numpy(np.concatenate(hist).astype(np.int32)).cuda(),
                          torch.from_numpy(off_h).cuda(), ws, slots=slots_d)
    off = gen.offsets_from_lengths([P] * B)
    tokens = rng.integers(0, V0, B * P).astype(np.int32)
    out = torch.empty((B * P, D), dtype=dtype, device="cuda")
    ne.ngram_embed_fwd_mx4(L["plan"], torch.from_numpy(tokens).cuda(), torch.from_numpy(off).cuda(), L["E0"], L["E"],
                           L["W"], out, ws, cache=cache, cache_slots=slots_d)
    assert ne.ngram_embed_get_status(ws) == 0
    want, acc, _ = ref.layer(V0, N, K, V, tokens, off, f64(L["E0"]), L["E_vals"], L["W_vals"], histories=hist)
    assert (np.abs(f64(out) - want) <= acc + HALF[dtype] * (np.abs(want) + acc)).all()


def test_project_is_the_layer_given_its_indices_and_its_parts(ne):
    """The same rows by the stand-alone operators: hash, lookup of each sub-table, requantise
    (exact: the values are 4-bit already), product; then E_0 and the scale in 64 bits."""
    V0, D, N, K, V, dtype = LAYERS[3]
    S, d = 8, D // 8
    L = make_layer(ne, 21, V0, D, N, K, V, dtype)
    off = gen.offsets_from_lengths([150, 61])
    T = 211
    tokens = torch.from_numpy(np.random.default_rng(1).integers(0, V0, T).astype(np.int32)).cuda()
    off_d = torch.from_numpy(off).cuda()
    ws = ne.new_embed_mx4_workspace(L["plan"], T)
    whole, parts = (torch.empty((T, D), dtype=dtype, device="cuda") for _ in range(2))
    ne.ngram_embed_fwd_mx4(L["plan"], tokens, off_d, L["E0"], L["E"], L["W"], whole, ws)
    idx = torch.empty((T, S), dtype=torch.int32, device="cuda")
    ne.ngram_hash_indices(L["plan"], tokens, off_d, idx, ws)
    ne.ngram_embed_project_mx4(L["plan"], tokens, idx, L["E0"], L["E"], L["W"], parts, ws)
    assert torch.equal(whole, parts)
    G = torch.empty((T, D), dtype=F32, device="cuda")
    ews = ne.new_embedding_workspace(0, d)
    for s in range(S):
        ne.ngram_embedding_fwd(L["E"][s], idx[:, s].contiguous(), G[:, s * d:(s + 1) * d], ews)
    q = ne.Mx4.empty(T, D, ne.MX4_TILES)
    y = torch.empty((T, D), dtype=F32, device="cuda")
    ne.ngram_mx4_quantize(G, q)
    ne.ngram_mx4_product(q, L["W"], y, ne.new_mx4_workspace(T, D, D))
    want = (L["E0"].double()[tokens.long()] + y.double()) / (S + 1)
    mag = (G.double().abs() @ torch.from_numpy(np.abs(L["W_vals"])).cuda().T).cpu().numpy() / (S + 1)
    bound = 2 * D * 2.0 ** -23 * mag + ref.BF16_HALF * np.abs(f64(want)) * 1.001 + 1e-30
    assert (np.abs(f64(whole) - f64(want)) <= bound + 4 * ref.F32_HALF * np.abs(f64(want))).all()


def test_bad_ids_set_the_status_and_read_row_0(ne):
    V0, D, N, K, V, dtype = LAYERS[2]
    L = make_layer(ne, 31, V0, D, N, K, V, dtype)
    tokens = np.array([3, 4, 5], np.int32)
    idx = np.array([[1, 2, 3, 4], [5, 6, 7, 8], [9, 10, 11, 12]], np.int32)
    ws = ne.new_embed_mx4_workspace(L["plan"], 3)
    run = lambda t, i: (lambda o: (ne.ngram_embed_project_mx4(L["plan"], torch.from_numpy(t).cuda(),
                                                              torch.from_numpy(i).cuda(), L["E0"], L["E"], L["W"], o, ws),
                                   o)[1])(torch.empty((3, D), dtype=dtype, device="cuda"))
    for bad_t, bad_i in ((V0, 6), (-1, 6), (4, V[1]), (4, -7)):
        t, i, t0, i0 = tokens.copy(), idx.copy(), tokens.copy(), idx.copy()
        t[1], i[1, 1] = bad_t, bad_i
        t0[1], i0[1, 1] = (bad_t if 0 <= bad_t < V0 else 0), (bad_i if 0 <= bad_i < V[1] else 0)
        got = run(t, i)
        assert ne.ngram_embed_get_status(ws) == 0x1
        ne.ngram_embed_clear_status(ws)
        assert torch.equal(got, run(t0, i0)) and ne.ngram_embed_get_status(ws) == 0


def test_captured_replayed_and_on_another_stream(ne):
    """Quantise and product captured once and replayed on new inputs, beside an eager call with
    its own workspace on another stream."""
    rng = np.random.default_rng(4)
    w = ref.random_mx4(rng, 384, 512)
    W = device_mx4(ne, *w, ne.MX4_TILES)
    x = torch.randn((200, 512), device="cuda")
    q, out, ws = ne.Mx4.empty(200, 512, ne.MX4_TILES), torch.empty((200, 384), device="cuda"), ne.new_mx4_workspace(200, 384, 512)

    def step():
        ne.ngram_mx4_quantize(x, q)
        ne.ngram_mx4_product(q, W, out, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    q2, out2, ws2 = ne.Mx4.empty(200, 512, ne.MX4_TILES), torch.empty((200, 384), device="cuda"), ne.new_mx4_workspace(200, 384, 512)
    for k in range(3):
        x.copy_(torch.randn((200, 512), device="cuda") * (k + 1))
        torch.cuda.synchronize()
        graph.replay()
        ne.ngram_mx4_quantize(x, q2, stream=side)
        ne.ngram_mx4_product(q2, W, out2, ws2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
        av, bv = ref.values(*ref.quantise(f64(x))), ref.values(*w)
        want = av @ bv.T
        assert (np.abs(f64(out) - want) <= ref.product_bound(av, bv, ref.F32_HALF, want)).all()


def test_captured_behind_copies_and_across_two_streams(ne):
    """One graph: inputs copied and outputs cleared by copy and memset nodes, W and x quantised on
    two streams, joined in front of the product, which a lookup of the quantised rows follows."""
    M, N, K = 70, 160, 96
    xs, ws_ = torch.empty((M, K)).pin_memory(), torch.empty((N, K)).pin_memory()
    x, w = torch.empty((M, K), device="cuda"), torch.empty((N, K), device="cuda")
    a, b, rows = ne.Mx4.empty(M, K, ne.MX4_TILES), ne.Mx4.empty(N, K, ne.MX4_TILES), ne.Mx4.empty(M, K)
    out, back = torch.empty((M, N), device="cuda"), torch.empty((M, K), device="cuda")
    ws, ws2 = ne.new_mx4_workspace(M, N, K), ne.new_embedding_workspace(0, K)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        x.copy_(xs, non_blocking=True)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            w.copy_(ws_, non_blocking=True)
            ne.ngram_mx4_quantize(w, b)
        ne.ngram_mx4_quantize(x, a)
        ne.ngram_mx4_quantize(x, rows)
        out.zero_()
        main.wait_stream(side)
        ne.ngram_mx4_product(a, b, out, ws)
        back.zero_()
        ne.ngram_embedding_fwd(rows, None, back, ws2)

    with torch.cuda.stream(torch.cuda.Stream()):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(40)
    for k in range(3):
        xs.copy_(torch.from_numpy(rng.standard_normal((M, K)) * (k + 1)))
        ws_.copy_(torch.from_numpy(rng.standard_normal((N, K))))
        graph.replay()
        torch.cuda.synchronize()
        av, bv = (ref.values(*ref.quantise(f64(t))) for t in (xs, ws_))
        want = av @ bv.T
        assert (np.abs(f64(out) - want) <= ref.product_bound(av, bv, ref.F32_HALF, want)).all()
        assert np.array_equal(f64(back), av)


def test_products_of_every_form_at_once_on_two_streams(ne):
    """Two streams run products of different forms beside one another, with their own
    workspaces: each result has the bits of its call alone."""
    rng = np.random.default_rng(41)
    calls = []
    for M, N, K in ((2000, 1536, 256), (1280, 1024, 256), (700, 520, 320), (20, 640, 96), (1, 640, 4128)):
        a, b = (device_mx4(ne, *ref.random_mx4(rng, r, K), ne.MX4_TILES) for r in (M, N))
        out, ws = torch.empty((M, N), dtype=BF16, device="cuda"), ne.new_mx4_workspace(M, N, K)
        ne.ngram_mx4_product(a, b, out, ws)
        calls.append((a, b, out.clone(), [(torch.empty_like(out), ne.new_mx4_workspace(M, N, K)) for _ in range(2)]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for k in range(len(calls)):
            for i, st in enumerate(streams):
                a, b, _, own = calls[(k + i * 2) % len(calls)]
                ne.ngram_mx4_product(a, b, *own[i], stream=st)
    torch.cuda.synchronize()
    for _, _, want, own in calls:
        for out, ws in own:
            assert torch.equal(out, want) and ne.ngram_embed_get_status(ws) == 0


def tile_rows(tiles, rows, cols):
    """Scale bytes of some rows of an array of `cols`, from its tiles."""
    kt = -(-cols // 128)
    b = np.arange(cols // 32)
    at = [(r // 128 * kt + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4 for r in rows]
    return np.stack([tiles[torch.from_numpy(a).cuda()].cpu().numpy() for a in at])


def test_product_that_takes_seconds(ne):
    """A product of more than two seconds, the limit of the kernel's waits for one another, on
    CTA pairs (a square array by itself): no wait runs out. Some of its rows and columns."""
    R, K = 131072, 262144
    assert ne.ngram_mx4_product_form(R, R, K) in (256, 320)
    gen_d = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device="cuda", generator=gen_d)
    scales = torch.randint(120, 128, (R // 128 * (K // 128) * 512,), dtype=torch.uint8, device="cuda", generator=gen_d)
    a = ne.Mx4(codes, scales, R, K, ne.MX4_TILES)
    out, ws = torch.empty((R, R), dtype=BF16, device="cuda"), ne.new_mx4_workspace(R, R, K)
    ne.ngram_mx4_product(a, a, out, ws)
    assert ne.ngram_embed_get_status(ws) == 0
    rows, cols = [0, 129, 70000, R - 1], [0, 63, 64, 255, 256, 40001, R - 2, R - 1]
    av, bv = (ref.values(ref.unpack(codes[r].cpu().numpy()), tile_rows(scales, r, K)) for r in (rows, cols))
    got, want = f64(out[rows][:, cols]), av @ bv.T
    del codes, scales, out, a
    torch.cuda.empty_cache()
    assert (np.abs(got - want) <= ref.product_bound(av, bv, ref.BF16_HALF, want)).all()


@pytest.mark.parametrize("M", [5, 4])
def test_product_of_the_longest_rows(ne, M):
    """K near 2^31: rows of 1 GB, whose one tile takes more than two seconds; offsets past 32
    bits. Small integers under scales of 1 at a few places, zeros elsewhere: exact."""
    K = (1 << 31) - 288
    rng = np.random.default_rng(M)
    kt = -(-K // 128)
    parts = []
    at = [0, 1, 5000, K // 64, K // 32 - 7, K // 32 - 1]  # blocks that are not zero
    vals = []
    for rows in (M, 1):
        codes = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(kt * 512, dtype=torch.uint8, device="cuda")
        v = np.zeros((rows, len(at) * 32))
        for r in range(rows):
            for j, b in enumerate(at):
                c = rng.integers(0, 16, (1, 32), dtype=np.uint8)
                codes[r, b * 16:b * 16 + 16] = torch.from_numpy(ref.pack(c)[0]).cuda()
                scales[b // 4 * 512 + r * 16 + b % 4] = 127
                v[r, j * 32:j * 32 + 32] = ref.values(c, np.array([[127]], np.uint8))
        parts.append(ne.Mx4(codes, scales, rows, K, ne.MX4_TILES))
        vals.append(v)
    assert (ne.ngram_mx4_product_form(M, 1, K) == 0) == (M <= 4)
    out, ws = torch.empty((M, 1), device="cuda"), ne.new_mx4_workspace(M, 1, K)
    ne.ngram_mx4_product(parts[0], parts[1], out, ws)
    assert ne.ngram_embed_get_status(ws) == 0
    assert np.array_equal(f64(out), vals[0] @ vals[1].T)
    del codes, scales, parts
    torch.cuda.empty_cache()


def test_layer_of_another_device_s_plan_or_cache_is_refused(ne):
    """Before anything is launched: kernels of one device would read another's memory, or the
    host's."""
    V0, D, N, K, V, dtype = LAYERS[2]
    L = make_layer(ne, 51, V0, D, N, K, V, dtype)
    tokens, off = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    idx = torch.zeros((4, L["plan"].S), dtype=torch.int32, device="cuda")
    ws = ne.new_embed_mx4_workspace(L["plan"], 4)
    out = torch.full((4, D), 3.0, dtype=dtype, device="cuda")
    fwd = lambda **kw: ne.ngram_embed_fwd_mx4(L["plan"], tokens, off, L["E0"], L["E"], L["W"], out, ws, **kw)
    ring = ne.Cache.empty(1, 8)
    host = ne.Cache.empty(1, 8, device="cpu")
    for cache in (host, ne.Cache(ring.ring, host.len, ring.valid_from), ne.Cache(ring.ring, ring.len, host.valid_from)):
        with pytest.raises(ne.NgramError):
            fwd(cache=cache)
    here = L["plan"].device
    assert here == out.get_device()
    L["plan"].device = here + 1
    with pytest.raises(ne.NgramError):
        fwd()
    with pytest.raises(ne.NgramError):
        ne.ngram_embed_project_mx4(L["plan"], tokens, idx, L["E0"], L["E"], L["W"], out, ws)
    assert bool((out == 3.0).all())
    L["plan"].device = here
    fwd(cache=ring)
    assert ne.ngram_embed_get_status(ws) == 0


MANY_TILES = [  # M, N, K: three tiles and more for some CTA or pair of every form
    (60000, 60, 64), (60000, 60, 1056), (16384, 1000, 512), (130, 30000, 64), (9000, 1500, 1024), (60000, 190, 64),
    (16384, 1000, 1024), (34215, 423, 32), (56000, 320, 1056), (54669, 274, 32),
]
TILE_ROWS = {320: 256, 256: 256, 192: 128, 128: 128, 64: 128}


def tiles_a_worker(ne, M, N, K):
    """The form of a product and the most tiles that one CTA or pair of it takes."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    w = ne.ngram_mx4_product_form(M, N, K, sms)
    tiles = -(-M // TILE_ROWS[w]) * -(-N // w)
    return w, -(-tiles // (sms * 128 // TILE_ROWS[w]))


def gpu_bound(a, b, half, want):
    """mx4_ref.product_bound on 64-bit tensors of the GPU."""
    acc = a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().T)
    return acc + half * (want.abs() + acc)


@pytest.mark.parametrize("M,N,K", MANY_TILES)
def test_product_of_several_tiles_a_worker(ne, M, N, K):
    """Accumulators used again, stages that run on from tile to tile, ragged last tiles."""
    assert tiles_a_worker(ne, M, N, K)[1] >= 3
    rng = np.random.default_rng(M + N)
    a, b = ref.random_mx4(rng, M, K), ref.random_mx4(rng, N, K)
    A, B = device_mx4(ne, *a, ne.MX4_TILES), device_mx4(ne, *b, ne.MX4_TILES)
    av, bv = (torch.from_numpy(ref.values(*t)).cuda() for t in (a, b))
    want = av @ bv.T * 0.5
    ws = ne.new_mx4_workspace(M, N, K)
    for dtype in (BF16, F32):
        out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
        ne.ngram_mx4_product(A, B, out, ws, alpha=0.5)
        assert bool(((out.double() - want).abs() <= gpu_bound(av, bv * 0.5, HALF[dtype], want)).all())
    assert ne.ngram_embed_get_status(ws) == 0


MANY_TILES_LAYERS = [(64, 3, 1, 60000), (512, 3, 2, 14336), (1024, 3, 1, 14336), (320, 3, 1, 56500), (2048, 5, 2, 8192)]  # D, N, K, T


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,N,K,T", MANY_TILES_LAYERS)
def test_layer_of_several_tiles_a_worker(ne, D, N, K, T, dtype):
    assert tiles_a_worker(ne, T, D, D)[1] >= 3
    V0, S = 3000, (N - 1) * K
    V = [1001 + 10 * s for s in range(S)]
    L = make_layer(ne, D + T, V0, D, N, K, V, dtype)
    off = gen.offsets_from_lengths([T - 1001, 0, 1, 1000])
    tokens = np.random.default_rng(T).integers(0, V0, T).astype(np.int32)
    idx = torch.from_numpy(oracle.hash_indices(V0, N, K, V, oracle.context_windows(N, tokens, off)).astype(np.int64)).cuda()
    G = torch.cat([torch.from_numpy(e).cuda()[idx[:, s]] for s, e in enumerate(L["E_vals"])], dim=1)
    W, e0 = torch.from_numpy(L["W_vals"]).cuda(), L["E0"].double()[torch.from_numpy(tokens).cuda().long()]
    mag = G.abs() @ W.abs().T
    want = (e0 + G @ W.T) / (S + 1)
    # as mx4_ref.layer: the sums, the E_0 add, the scale and its product
    acc = (D * 2.0 ** -23 * mag + 3 * ref.F32_HALF * (mag + e0.abs())) / (S + 1)
    ws = ne.new_embed_mx4_workspace(L["plan"], T)
    out = torch.full((T, D), 3.0, dtype=dtype, device="cuda")
    ne.ngram_embed_fwd_mx4(L["plan"], torch.from_numpy(tokens).cuda(), torch.from_numpy(off).cuda(), L["E0"], L["E"],
                           L["W"], out, ws)
    assert ne.ngram_embed_get_status(ws) == 0
    assert bool(((out.double() - want).abs() <= acc + HALF[dtype] * (want.abs() + acc)).all())


def test_sizes_above_give_every_form_three_tiles_a_worker(ne):
    for sizes in (MANY_TILES, [(T, D, D) for D, _, _, T in MANY_TILES_LAYERS]):
        took = dict(tiles_a_worker(ne, *s) for s in sizes)
        assert set(took) == set(TILE_ROWS) and min(took.values()) >= 3


def test_products_of_all_forms_in_flight_on_two_streams(ne):
    """Pairs, single CTAs and the form of few rows beside one another, nothing waited for between
    the calls: each result has the bits of its call alone."""
    sizes = [(2300, 2048, 2048), (1280, 4096, 4096), (16384, 1000, 1024), (9000, 1500, 1024), (16384, 1000, 512),
             (333, 1111, 2080), (1, 4096, 4096), (28600, 318, 1056)]
    assert {ne.ngram_mx4_product_form(*s) for s in sizes} == {0, *TILE_ROWS}
    gen_d = torch.Generator(device="cuda").manual_seed(6)
    calls = []
    for M, N, K in sizes:
        a, b = (ne.Mx4(torch.randint(0, 256, (r, K // 2), dtype=torch.uint8, device="cuda", generator=gen_d),
                       torch.randint(120, 130, (ne._lib.ngram_mx4_scale_bytes(r, K, ne.MX4_TILES),), dtype=torch.uint8,
                                     device="cuda", generator=gen_d), r, K, ne.MX4_TILES) for r in (M, N))
        own = [(torch.empty((M, N), dtype=BF16, device="cuda"), ne.new_mx4_workspace(M, N, K)) for _ in range(3)]
        ne.ngram_mx4_product(a, b, *own[2])
        calls.append((a, b, own))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(30):
        for k in range(len(calls)):
            for i, st in enumerate(streams):
                a, b, own = calls[(k * (1 + 2 * i) + rep) % len(calls)]  # each stream in an order of its own
                ne.ngram_mx4_product(a, b, *own[i], stream=st)
    torch.cuda.synchronize()
    for _, _, own in calls:
        for out, ws in own[:2]:
            assert torch.equal(out, own[2][0]) and ne.ngram_embed_get_status(ws) == 0
