"""The lookup of one table and its gradient by sorted ids, on the GPU, against plain 64-bit
definitions on the host."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

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


def ids_of(rng, n, V, kind):
    if kind == "same":
        return np.full(n, V // 2, np.int32)
    if kind == "zipf":
        return np.minimum(rng.zipf(1.3, n) - 1, V - 1).astype(np.int32)
    if kind == "distinct":
        return rng.permutation(max(V, n))[:n].astype(np.int32) % V
    return rng.integers(0, V, n).astype(np.int32)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("kind,V,D,n", [
    ("bf16", 1, 8, 1), ("bf16", 100, 136, 33), ("f32", 50, 8, 7), ("f32", 313, 264, 1000), ("mx4", 9, 32, 5),
    ("mx4", 1000, 96, 700), ("mx4", 77, 2080, 130), ("bf16", 3000, 1024, 2049),
])
def test_lookup(ne, kind, V, D, n, out_dtype):
    rng = np.random.default_rng(V + D + n)
    if kind == "mx4":
        codes, scales = ref.random_mx4(rng, V, D, spread=20)
        scales[0, 0], scales[V - 1, D // 32 - 1] = 0, 254
        vals = ref.values(codes, scales)
        table = ne.Mx4(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda(), V, D, ne.MX4_ROWS)
    else:
        table = torch.from_numpy(rng.standard_normal((V, D))).to(BF16 if kind == "bf16" else F32).cuda()
        vals = f64(table)
    ids = rng.integers(0, V, n).astype(np.int32)
    ids[0], ids[-1] = 0, V - 1
    ws = ne.new_embedding_workspace(0, D)
    for scale, pad in ((1.0, -1), (0.37, V - 1), (-2.5, 0)):
        out = torch.full((n, D), 9.0, dtype=out_dtype, device="cuda")
        ne.ngram_embedding_fwd(table, torch.from_numpy(ids).cuda(), out, ws, scale=scale, pad_id=pad)
        want = ref.lookup(vals, ids, scale, pad)
        # one fp32 product, one rounding to the output type; f32 subnormals: half of 2^-149
        bound = (ref.F32_HALF + (HALF[out_dtype] if out_dtype == BF16 else 0)) * np.abs(want) * 1.01 + 2.0 ** -149
        if out_dtype == BF16:
            bound = np.maximum(bound, 2.0 ** -134)  # half of bf16's smallest subnormal
        # half a step above the largest number and more is an infinity
        over = np.abs(want) >= (2 - 2.0 ** (-8 if out_dtype == BF16 else -24)) * 2.0 ** 127
        got = f64(out)
        assert (got[over] == np.sign(want[over]) * np.inf).all()
        assert (np.abs(got[~over] - want[~over]) <= bound[~over]).all()
    assert ne.ngram_embed_get_status(ws) == 0


def test_lookup_into_strided_rows_whole_tables_and_bad_ids(ne):
    rng = np.random.default_rng(2)
    table = torch.from_numpy(rng.standard_normal((60, 64))).float().cuda()
    ws = ne.new_embedding_workspace(0, 64)
    buf = torch.full((50, 200), 5.0, device="cuda")
    ne.ngram_embedding_fwd(table, None, buf[:, 64:128], ws)  # ids None: rows 0 .. 49
    assert torch.equal(buf[:, 64:128], table[:50])
    assert bool((buf[:, :64] == 5.0).all()) and bool((buf[:, 128:] == 5.0).all())
    out = torch.empty((4, 64), device="cuda")
    ne.ngram_embedding_fwd(table, torch.tensor([3, 60, -1, 59], dtype=torch.int32, device="cuda"), out, ws)
    assert torch.equal(out, table[[3, 0, 0, 59]]) and ne.ngram_embed_get_status(ws) == 0x1
    ne.ngram_embed_clear_status(ws)
    assert ne.ngram_embed_get_status(ws) == 0


def check_rows(ne, ids, g, V, scale, pad, ws=None):
    n, D = g.shape
    ws = ne.new_embedding_workspace(n, D) if ws is None else ws
    rows = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    count = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    grads = torch.full((n, D), 4.0, dtype=F32, device="cuda")
    ids_d = torch.from_numpy(ids).cuda()
    ne.ngram_embedding_bwd_rows(ids_d, g, V, rows, count, grads, ws, scale=scale, pad_id=pad)
    want_rows, want, mags, cnt = ref.grad_rows(ids, f64(g), scale, pad)
    U = int(count)
    assert U == len(want_rows) and np.array_equal(rows[:U].cpu().numpy(), want_rows)
    assert (np.abs(f64(grads[:U]) - want) <= ref.grad_bound(mags, cnt)).all()
    assert bool((rows[U:] == -5).all()) and bool((grads[U:] == 4.0).all())  # left as they were
    dense = torch.ones((V, D), dtype=F32, device="cuda")
    ne.ngram_embedding_bwd(ids_d, g, dense, ws, scale=scale, pad_id=pad)
    full = torch.ones((V, D), dtype=F32, device="cuda")
    full[rows[:U].long()] += grads[:U]
    assert torch.equal(dense, full)
    return rows, grads, U


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,D,kind", [
    (1, 1, 8, "same"), (2, 5, 16, "same"), (31, 7, 8, "uniform"), (32, 1000, 40, "distinct"), (33, 3, 264, "uniform"),
    (64, 40, 256, "same"), (65, 40, 256, "same"), (257, 255, 136, "uniform"), (1024, 256, 24, "zipf"),
    (1025, 257, 8, "zipf"), (1500, 100000, 512, "distinct"), (3000, 70000, 72, "zipf"), (5000, 1 << 24, 8, "uniform"),
    (7001, 50, 32, "uniform"), (20000, 131072, 16, "zipf"),
    (4096, 300, 8, "zipf"), (4097, 2000, 8, "uniform"), (65536, 131072, 8, "zipf"),  # one cluster sorts up to 65536
    (65537, 131071, 8, "zipf"), (70001, 1 << 22, 8, "uniform"), (100003, 200, 16, "uniform"),
])
def test_gradient_rows_and_dense(ne, n, V, D, kind, dtype):
    rng = np.random.default_rng(n + V)
    ids = ids_of(rng, n, V, kind)
    g = torch.from_numpy(rng.standard_normal((n, D))).to(dtype).cuda()
    if V <= 131072:
        check_rows(ne, ids, g, V, 1.0, -1)
        check_rows(ne, ids, g, V, 0.3, int(ids[n // 2]))
    else:  # a dense table of this many rows is left out
        ws = ne.new_embedding_workspace(n, D)
        rows, count = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        grads = torch.zeros((n, D), device="cuda")
        ne.ngram_embedding_bwd_rows(torch.from_numpy(ids).cuda(), g, V, rows, count, grads, ws)
        want_rows, want, mags, cnt = ref.grad_rows(ids, f64(g), 1.0)
        U = int(count)
        assert np.array_equal(rows[:U].cpu().numpy(), want_rows)
        assert (np.abs(f64(grads[:U]) - want) <= ref.grad_bound(mags, cnt)).all()


def test_all_padded_none_and_values_at_padded_positions(ne):
    """No row left: count 0, nothing written. NaN and infinities at padded positions are not
    read into any sum."""
    n, D = 300, 64
    ws = ne.new_embedding_workspace(n, D)
    rows, count = torch.full((n,), 8, dtype=torch.int32, device="cuda"), torch.full((1,), 8, dtype=torch.int32, device="cuda")
    grads = torch.full((n, D), 8.0, device="cuda")
    g = torch.full((n, D), float("nan"), device="cuda")
    pads = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    ne.ngram_embedding_bwd_rows(pads, g, 10, rows, count, grads, ws, pad_id=3)
    assert int(count) == 0 and bool((rows == 8).all()) and bool((grads == 8.0).all())
    count.fill_(8)
    ne.ngram_embedding_bwd_rows(pads[:0], g[:0], 10, rows[:0], count, grads[:0], ws)
    assert int(count) == 0
    rng = np.random.default_rng(0)
    ids = rng.integers(0, 10, n).astype(np.int32)
    gh = rng.standard_normal((n, D)).astype(np.float32)
    gh[ids == 3] = np.inf
    ok = gh.copy()
    ok[ids == 3] = 0
    out = []
    for x in (gh, ok):
        dense = torch.zeros((10, D), device="cuda")
        ne.ngram_embedding_bwd(torch.from_numpy(ids).cuda(), torch.from_numpy(x).cuda(), dense, ws, pad_id=3)
        out.append(dense)
    assert torch.equal(out[0], out[1]) and bool((out[0][3] == 0).all())


def test_gradient_bits_repeat_and_bad_ids_count_as_row_0(ne):
    rng = np.random.default_rng(8)
    n, V, D = 4000, 500, 264
    ids = ids_of(rng, n, V, "zipf")
    g = torch.from_numpy(rng.standard_normal((n, D))).to(BF16).cuda()
    ws = ne.new_embedding_workspace(n, D)
    first = check_rows(ne, ids, g, V, 1.0, -1, ws)
    for _ in range(3):
        again = check_rows(ne, ids, g, V, 1.0, -1, ws)
        assert again[2] == first[2] and torch.equal(again[1], first[1])
    bad, good = ids.copy(), ids.copy()
    bad[::97], good[::97] = np.where(np.arange(len(bad[::97])) % 2, V, -4), 0
    a, b = torch.zeros((V, D), device="cuda"), torch.zeros((V, D), device="cuda")
    ne.ngram_embedding_bwd(torch.from_numpy(bad).cuda(), g, a, ws)
    assert ne.ngram_embed_get_status(ws) == 0x1
    ne.ngram_embed_clear_status(ws)
    ne.ngram_embedding_bwd(torch.from_numpy(good).cuda(), g, b, ws)
    assert torch.equal(a, b) and ne.ngram_embed_get_status(ws) == 0


def test_gradient_of_strided_rows(ne):
    rng = np.random.default_rng(6)
    ids = ids_of(rng, 90, 20, "uniform")
    for dtype, lo, width in ((BF16, 8, 160), (F32, 4, 148)):
        buf = torch.from_numpy(rng.standard_normal((90, width))).to(dtype).cuda()
        check_rows(ne, ids, buf[:, lo:lo + 136], 20, 1.25, -1)


def test_gradient_is_the_lookup_s_by_differences(ne):
    """Linear: (L(table + h E) - L(table)) / h = <dTable, E> for L = <lookup, g>, in 64 bits on
    what the library returns for tables whose values fp32 holds exactly."""
    rng = np.random.default_rng(13)
    V, D, n = 30, 40, 200
    ids = ids_of(rng, n, V, "zipf")
    ids_d = torch.from_numpy(ids).cuda()
    ws = ne.new_embedding_workspace(n, D)
    base = rng.integers(-64, 65, (V, D)).astype(np.float32)
    direction = rng.integers(-8, 9, (V, D)).astype(np.float32)
    g = rng.integers(-16, 17, (n, D)).astype(np.float32)

    def L(table):
        out = torch.empty((n, D), device="cuda")
        ne.ngram_embedding_fwd(torch.from_numpy(table).cuda(), ids_d, out, ws, scale=0.5, pad_id=2)
        return float((f64(out) * g).sum())

    d = torch.zeros((V, D), device="cuda")
    ne.ngram_embedding_bwd(ids_d, torch.from_numpy(g).cuda(), d, ws, scale=0.5, pad_id=2)
    assert L(base + direction) - L(base) == float((f64(d) * direction).sum())  # small integers and halves: exact


def test_train_a_4bit_table_through_its_master(ne):
    """Quantise a master, look it up, take the gradient as rows, update the touched master
    rows, requantise: each step against the definitions on the values of the step before."""
    rng = np.random.default_rng(77)
    V, D, n = 200, 96, 500
    master = torch.from_numpy(rng.standard_normal((V, D)) * 0.05).float().cuda()
    q = ne.Mx4.empty(V, D)
    ws = ne.new_embedding_workspace(n, D)
    rows, count = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = torch.zeros((n, D), device="cuda")
    for step in range(3):
        before = master.clone()
        ne.ngram_mx4_quantize(master, q)
        codes, scales = ref.quantise(f64(master))
        assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes)) and np.array_equal(q.scales.cpu().numpy(), scales)
        ids = ids_of(rng, n, V, "zipf")
        ids_d = torch.from_numpy(ids).cuda()
        out = torch.empty((n, D), dtype=BF16, device="cuda")
        ne.ngram_embedding_fwd(q, ids_d, out, ws, scale=2.0)
        assert np.array_equal(f64(out), ref.values(codes, scales)[ids] * 2.0)  # 4 bits times 2: exact in bf16
        g = out - 1.0
        ne.ngram_embedding_bwd_rows(ids_d, g, V, rows, count, grads, ws, scale=2.0)
        want_rows, want, mags, cnt = ref.grad_rows(ids, f64(g), 2.0)
        U = int(count)
        assert np.array_equal(rows[:U].cpu().numpy(), want_rows)
        assert (np.abs(f64(grads[:U]) - want) <= ref.grad_bound(mags, cnt)).all()
        master[rows[:U].long()] -= 0.01 * grads[:U]
        untouched = np.setdiff1d(np.arange(V), want_rows)
        assert torch.equal(master[untouched], before[untouched])


def test_gradient_captured_and_replayed(ne):
    rng = np.random.default_rng(21)
    n, V, D = 700, 300, 72
    ids, g = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros((n, D), device="cuda")
    ws = ne.new_embedding_workspace(n, D)
    rows, count, grads = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((n, D), device="cuda")
    call = lambda: ne.ngram_embedding_bwd_rows(ids, g, V, rows, count, grads, ws, scale=1.5, pad_id=0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        h = ids_of(rng, n, V, ("zipf", "uniform", "same")[k])
        ids.copy_(torch.from_numpy(h).cuda())
        g.copy_(torch.from_numpy(rng.standard_normal((n, D))).float().cuda())
        graph.replay()
        want_rows, want, mags, cnt = ref.grad_rows(h, f64(g), 1.5, 0)
        U = int(count)
        assert np.array_equal(rows[:U].cpu().numpy(), want_rows)
        assert (np.abs(f64(grads[:U]) - want) <= ref.grad_bound(mags, cnt)).all()


def test_on_other_streams_at_once(ne):
    """The current stream of a `with` block and a given one, each with its own workspace: lookups
    and gradients, sorted in one cluster and in tiles, beside one another give the bits of a call
    alone."""
    rng = np.random.default_rng(31)
    V, D = 4000, 72
    sizes = (3000, 70000)
    table = torch.from_numpy(rng.standard_normal((V, D))).float().cuda()
    ins = []
    for n in sizes:
        ids = torch.from_numpy(ids_of(rng, n, V, "zipf")).cuda()
        ins.append((ids, torch.from_numpy(rng.standard_normal((n, D))).float().cuda()))

    def call(k, st=None):
        ids, g = ins[k]
        out, d, ws = torch.empty_like(g), torch.zeros((V, D), device="cuda"), ne.new_embedding_workspace(sizes[k], D)
        torch.cuda.synchronize()  # allocated and cleared before another stream takes them
        ne.ngram_embedding_fwd(table, ids, out, ws, scale=1.5, pad_id=1, stream=st)
        ne.ngram_embedding_bwd(ids, g, d, ws, scale=1.5, pad_id=1, stream=st)
        return out, d

    alone = [call(k) for k in range(2)]
    for _ in range(3):
        given = torch.cuda.Stream()
        with torch.cuda.stream(torch.cuda.Stream()):
            both = [call(0, given), call(1)]
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("pad_id", [0, 49, 50, 1 << 40])
def test_padding_at_the_table_s_edges(ne, pad_id):
    """A pad id of the first, the last and no row; an id past the table that is the pad id is
    padding, any other reads row 0 (a row of its own even where 0 is the pad id)."""
    rng = np.random.default_rng(32)
    n, V, D = 600, 50, 40
    ids = rng.integers(0, V + 2, n).astype(np.int32)
    table = rng.integers(-64, 65, (V, D)).astype(np.float32)
    g = rng.integers(-16, 17, (n, D)).astype(np.float32)
    ws = ne.new_embedding_workspace(n, D)
    ids_d, out = torch.from_numpy(ids).cuda(), torch.full((n, D), 9.0, device="cuda")
    d = torch.zeros((V, D), device="cuda")
    ne.ngram_embedding_fwd(torch.from_numpy(table).cuda(), ids_d, out, ws, pad_id=pad_id)
    ne.ngram_embedding_bwd(ids_d, torch.from_numpy(g).cuda(), d, ws, pad_id=pad_id)
    assert ne.ngram_embed_get_status(ws) == 0x1
    pad = ids == pad_id
    row = np.where(ids < V, ids, 0)
    want = np.zeros((V, D))
    np.add.at(want, row[~pad], g[~pad].astype(np.float64))
    assert np.array_equal(f64(out), np.where(pad[:, None], 0.0, table[row]))
    assert np.array_equal(f64(d), want)  # sums of at most 600 integers below 17: exact


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx4"])
def test_whole_table_is_the_lookup_of_its_rows_in_order(ne, kind):
    """ids None stands for 0, 1, ..: the same bits as those ids given, padding included."""
    rng = np.random.default_rng(61)
    V, D, n = 90, 96, 83
    if kind == "mx4":
        codes, scales = ref.random_mx4(rng, V, D)
        table = ne.Mx4(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda(), V, D, ne.MX4_ROWS)
    else:
        table = torch.from_numpy(rng.standard_normal((V, D)) + 10).to(BF16 if kind == "bf16" else F32).cuda()
    ws = ne.new_embedding_workspace(0, D)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    for pad in (-1, 0, 3, n - 1, n, V - 1, V, 1 << 31, (1 << 32) + 3):
        got, want = (torch.full((n, D), 9.0, device="cuda") for _ in range(2))
        ne.ngram_embedding_fwd(table, None, got, ws, scale=0.7, pad_id=pad)
        ne.ngram_embedding_fwd(table, ids, want, ws, scale=0.7, pad_id=pad)
        assert torch.equal(got, want)
        assert bool((got[pad] == 0).all()) if 0 <= pad < n else bool((got != 0).any(dim=1).all())
    assert ne.ngram_embed_get_status(ws) == 0


@pytest.mark.parametrize("scale", [3e38, -3.4e38, 2.0 ** 127, 1.5, 0.37, 2.0 ** -126, 1.1754942e-38, 1.37 * 2.0 ** -140,
                                   -2.0 ** -149, 0.0])
def test_lookup_of_every_4bit_value_rounds_its_product_once(ne, scale):
    """All codes under all scale bytes times scales up to fp32's ends: the fp32 number nearest
    to the product, then the bf16 number nearest to that. A product of a 24-bit scale, a code
    of two bits and a power of two is exact in 64 bits."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    table = ne.Mx4(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda(), 256, 32, ne.MX4_ROWS)
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        want = torch.from_numpy((ref.values(codes, scales) * np.float64(np.float32(scale))).astype(np.float32))
    ws = ne.new_embedding_workspace(0, 32)
    for dtype in (F32, BF16):
        out = torch.full((256, 32), 9.0, dtype=dtype, device="cuda")
        ne.ngram_embedding_fwd(table, None, out, ws, scale=scale)
        assert torch.allclose(out.cpu(), want.to(dtype), rtol=0, atol=0, equal_nan=True)


FIRST_CALL = """
import torch, hashed_gram_embedding_horner_b200 as ne
n, D, V = 3000, 64, 500
ids, g = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda"), torch.ones((n, D), device="cuda")
d, ws = torch.zeros((V, D), device="cuda"), ne.new_embedding_workspace(n, D)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ne.ngram_embedding_bwd(ids, g, d, ws)
assert not bool(d.any())
graph.replay()
assert torch.equal(d, torch.bincount(ids, minlength=V).float()[:, None].expand(V, D))
"""


def test_gradient_captured_as_a_process_s_first_call():
    """What a device is asked and told once (shared memory, cluster sizes) may fall into a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def many_ids(rng, n, V, kind):
    """`one`: nearly all positions one id, among others before and behind it."""
    ids = ids_of(rng, n, V, "zipf" if kind == "one" else kind)
    if kind == "one":
        ids[rng.random(n) < 0.97] = V // 2
    return ids


PIECES = [  # n, V, D, kind: of all lengths of pieces, sorted in a cluster and in tiles, runs of over 1024 pieces
    (20000, 3000, 7176, "zipf"), (65536, 5000, 2056, "zipf"), (32768, 4000, 4096, "one"), (70001, 2500, 2040, "zipf"),
    (150000, 700, 1024, "one"), (600000, 900, 8, "same"), (100000, 300, 64, "one"), (64000, 99, 24, "same"),
    (9000, 50, 8, "same"), (9100, 50, 16, "one"),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,D,kind", PIECES)
def test_gradient_in_pieces_of_every_length(ne, n, V, D, kind, dtype):
    """Sums of small integers are exact in any order: equal to the plain sums in 64 bits. With
    and without padding, as rows and densely."""
    rng = np.random.default_rng(n + D)
    ids = torch.from_numpy(many_ids(rng, n, V, kind)).cuda()
    g = torch.randint(-8, 9, (n, D), dtype=torch.int8, device="cuda", generator=torch.Generator("cuda").manual_seed(n)).to(dtype)
    ws = ne.new_embedding_workspace(n, D)
    rows, count = (torch.full((k,), -5, dtype=torch.int32, device="cuda") for k in (n, 1))
    grads, dense = torch.full((n, D), 4.0, device="cuda"), torch.empty((V, D), device="cuda")
    for pad in (-1, int(ids[n // 3]), V // 2):
        keep = ids != pad
        want = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, ids[keep].long(), g[keep].double()) * 0.5
        used = torch.unique(ids[keep])
        ne.ngram_embedding_bwd_rows(ids, g, V, rows, count, grads, ws, scale=0.5, pad_id=pad)
        U = int(count)
        assert U == len(used) and torch.equal(rows[:U], used)
        assert torch.equal(grads[:U].double(), want[used.long()])
        dense.fill_(3.0)
        ne.ngram_embedding_bwd(ids, g, dense, ws, scale=0.5, pad_id=pad)
        assert torch.equal(dense.double(), want + 3.0)
    assert ne.ngram_embed_get_status(ws) == 0


def test_gradients_above_take_every_piece_and_sort(ne):
    forms = {(ne.ngram_embedding_piece(n, D), ne.ngram_embedding_sort_ctas(n) > 0) for n, _, D, _ in PIECES}
    assert {p for p, _ in forms} == {8, 32, 128} and {(32, False), (128, False), (128, True)} <= forms
    for kind in ("same", "one"):  # runs over more than 1024 pieces, of every length
        assert {ne.ngram_embedding_piece(n, D) for n, _, D, k in PIECES
                if k == kind and 0.97 * n > 1025 * ne.ngram_embedding_piece(n, D)} == {8, 32, 128}


def test_lookups_and_gradients_in_flight_at_once(ne):
    """Two streams, nothing waited for between the calls: lookups and gradients, one side sorted in
    a cluster and the other in tiles, give the bits of a call alone every time."""
    rng = np.random.default_rng(33)
    V, D = 4000, 136
    table = torch.from_numpy(rng.standard_normal((V, D))).float().cuda()
    sides = []
    for n in (60000, 90000):
        ids = torch.from_numpy(ids_of(rng, n, V, "zipf")).cuda()
        g = torch.from_numpy(rng.standard_normal((n, D))).float().cuda()
        own = [dict(out=torch.empty_like(g), rows=torch.zeros(n, dtype=torch.int32, device="cuda"), grads=torch.zeros_like(g),
                    count=torch.zeros(1, dtype=torch.int32, device="cuda"), dense=torch.zeros((V, D), device="cuda"),
                    ws=ne.new_embedding_workspace(n, D)) for _ in range(3)]
        sides.append((ids, g, own))

    def call(side, k, st=None):
        ids, g, own = sides[side]
        o = own[k]
        ne.ngram_embedding_fwd(table, ids, o["out"], o["ws"], scale=1.5, pad_id=1, stream=st)
        ne.ngram_embedding_bwd_rows(ids, g, V, o["rows"], o["count"], o["grads"], o["ws"], scale=1.5, pad_id=1, stream=st)
        ne.ngram_embedding_bwd(ids, g, o["dense"], o["ws"], scale=1.5, pad_id=1, stream=st)

    repeats = 10
    for side in range(2):
        for _ in range(repeats):
            call(side, 0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    begin, end = ([torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2))
    for r in range(repeats):
        for side, st in enumerate(streams):  # a given stream, and the current one
            if r == 0:
                begin[side].record(st)
            call(side, 1, st)
            with torch.cuda.stream(st):
                call(side, 2)
            if r == repeats - 1:
                end[side].record(st)
    torch.cuda.synchronize()
    assert begin[0].elapsed_time(end[1]) > 0 and begin[1].elapsed_time(end[0]) > 0  # beside one another
    for _, _, own in sides:
        U = int(own[0]["count"])
        for o in own[1:]:
            assert int(o["count"]) == U and torch.equal(o["rows"][:U], own[0]["rows"][:U])
            assert torch.equal(o["grads"][:U], own[0]["grads"][:U]) and torch.equal(o["out"], own[0]["out"])
            assert torch.equal(o["dense"], own[0]["dense"]) and ne.ngram_embed_get_status(o["ws"]) == 0


def test_lookup_and_quantisation_of_more_rows_than_a_launch(ne):
    """2^28 rows of 32 columns are a launch's most: the rows at its border and the last ones, a
    padding id behind it, an id as far as the table goes."""
    n, D = (1 << 28) + 70, 32
    q = ne.Mx4.empty(n, D)
    x = torch.randint(-6, 7, (n, D), dtype=torch.int8, device="cuda").to(BF16)
    ne.ngram_mx4_quantize(x, q)
    some = torch.cat([torch.arange(0, 70), torch.arange((1 << 28) - 70, n)]).cuda()
    codes, scales = ref.quantise(f64(x[some]))
    assert np.array_equal(q.codes[some].cpu().numpy(), ref.pack(codes)) and np.array_equal(q.scales[some].cpu().numpy(), scales)
    vals = torch.from_numpy(ref.values(codes, scales)).cuda()
    ws = ne.new_embedding_workspace(0, D)
    x.fill_(9.0)
    pad = (1 << 28) + 3
    ne.ngram_embedding_fwd(q, None, x, ws, scale=2.0, pad_id=pad)
    vals[some == pad] = 0
    assert torch.equal(x[some].double(), vals * 2.0)  # 4 bits times 2: exact in bf16
    ids = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    ne.ngram_embedding_fwd(q, ids, x, ws, scale=2.0, pad_id=pad)
    assert torch.equal(x[n - 1 - some].double(), vals * 2.0) and ne.ngram_embed_get_status(ws) == 0
    del q, x, ids
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_and_quantisation_of_one_row_for_all(ne, dtype):
    """A broadcast row (stride 0), as a mean's gradient is: the same bits as its copies."""
    rng = np.random.default_rng(71)
    n, V, D = 700, 40, 160
    row = torch.from_numpy(rng.standard_normal(D)).to(dtype).cuda()
    g = row.expand(n, D)
    ids = ids_of(rng, n, V, "zipf")
    got = check_rows(ne, ids, g, V, 0.5, -1)
    want = check_rows(ne, ids, g.contiguous(), V, 0.5, -1)
    assert got[2] == want[2] and torch.equal(got[1], want[1])
    for lo in (0, 5):
        view = torch.cat([row, row])[lo:lo + 128].expand(33, 128)
        a, b = ne.Mx4.empty(33, 128), ne.Mx4.empty(33, 128)
        ne.ngram_mx4_quantize(view, a)
        ne.ngram_mx4_quantize(view.contiguous(), b)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
