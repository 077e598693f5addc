"""The experts' products on the GPU against the 64-bit implementation, at
sizes, segments and layouts where they can go wrong.  Rows of no segment must
stay as they were."""
import numpy as np
import pytest

import moe_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _draw(rng, rows, E, K, wide, sigma=100.0):
    """Random rows and weights; every e4m3 value but NaN occurs."""
    def q(*shape):
        x = torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).clamp(-448, 448)
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    a, w = q(rows, K), q(E, wide, K)
    a_s = torch.from_numpy((rng.uniform(0.5, 2.0, (rows, K // 128)) / sigma).astype(np.float32))
    w_s = torch.from_numpy((rng.uniform(0.5, 2.0, (E, (wide + 127) // 128, K // 128))
                            / (sigma * np.sqrt(K))).astype(np.float32))
    return a, a_s, w, w_s


def _np(*ts):
    return [t.numpy() for t in ts]


def _check_product(ep, offset, a, a_s, w, w_s, R=1, M=0):
    off = torch.tensor(offset, dtype=torch.int32)
    y = torch.full((a.shape[0], w.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm(off.cuda(), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), y, R, M)
    ref, mag, valid = moe_ref.product(offset, *_np(a, a_s, w, w_s), R, M)
    err = moe_ref.sum_error_8bit(mag, a.shape[1])
    got = y.cpu().double().numpy()
    bad = np.abs(got - ref) > moe_ref.BF16_HALF * (np.abs(ref) + err) + err
    assert not bad[valid].any(), np.argwhere(bad & valid[:, None])[:5]
    # and as a whole: half a step of bf16, and a quarter of that for the sums
    # (on random blocks of 128 they are off by 1.5e-5, far below)
    off2 = np.linalg.norm((got - ref)[valid])
    assert off2 <= (moe_ref.BF16_HALF + moe_ref.BF16_HALF / 4) * np.linalg.norm(ref[valid])
    assert (got[~valid] == 7.0).all()
    return y


def _check_gated(ep, offset, a, a_s, w, w_s, R=1, M=0):
    off = torch.tensor(offset, dtype=torch.int32)
    N = w.shape[1] // 2
    q = torch.full((a.shape[0], N), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((a.shape[0], N // 128), 7.0, device="cuda")
    ep.ep_expert_gated(off.cuda(), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), q, s, R, M)
    h, err, valid = moe_ref.gated(offset, *_np(a, a_s, w, w_s), R, M)
    qn, sn = q.cpu().numpy(), s.cpu().numpy()
    moe_ref.check_quantised(qn, sn, h, err, valid)
    assert (qn[~valid] == 0x55).all() and (sn[~valid] == 7.0).all()
    return q, s


def _offsets(counts, first=0):
    return [first] + (first + np.cumsum(counts)).tolist()


# experts' row counts: none, one, ends at, before and after tile borders, long ones
COUNTS = [
    [1], [16], [0, 1], [3, 0, 5], [15, 16, 17], [31, 32, 33, 0, 1], [63, 64, 65], [127, 0, 128, 129], [300, 2, 0, 0, 1],
    [255, 257], [8] * 40, [0] * 20 + [5] + [0] * 20, [700],
]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:5])) + f"x{len(c)}")
@pytest.mark.parametrize("K,N", [(128, 8), (256, 136), (640, 256), (1152, 1000)])
def test_product_segments(ep, counts, K, N):
    rng = np.random.default_rng(K + N + len(counts))
    off = _offsets(counts)
    _check_product(ep, off, *_draw(rng, off[-1] + 9, len(counts), K, N))


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:5])) + f"x{len(c)}")
@pytest.mark.parametrize("K,N", [(128, 128), (384, 256), (1152, 384)])
def test_gated_segments(ep, counts, K, N):
    rng = np.random.default_rng(K + N + len(counts))
    off = _offsets(counts)
    _check_gated(ep, off, *_draw(rng, off[-1] + 9, len(counts), K, 2 * N))


@pytest.mark.parametrize("rows,E,K,N", [(5000, 3, 512, 520), (2600, 64, 256, 264), (4100, 1, 1024, 384),
                                        (1, 1, 7168, 2048), (8, 300, 256, 128), (2048, 4096, 128, 128),
                                        (1100, 2, 2048, 640)])
def test_random_segments(ep, rows, E, K, N):
    """Random segments of every mean length, some rows before the first and behind the last segment."""
    rng = np.random.default_rng(rows + E)
    cut = np.sort(rng.integers(rows // 50, rows - rows // 60 + 1, size=E + 1)).tolist()
    if E > 100:
        N = min(N, 128)
    a, a_s, w, w_s = _draw(rng, rows, E, K, N)
    _check_product(ep, cut, a, a_s, w, w_s)
    N = (N + 127) // 128 * 128
    _check_gated(ep, cut, *_draw(rng, rows, E, K, 2 * N if E <= 100 else 256))


@pytest.mark.parametrize("E,R,M,counts", [(4, 2, 40, [3, 20, 17, 9]), (6, 3, 16, [16, 0, 20, 5, 0, 0]),
                                          (8, 4, 130, [1, 200, 100, 30, 0, 0, 65, 65]), (2, 1, 33, [30, 30])])
def test_rank_major_rows(ep, E, R, M, counts):
    """RANK_MAJOR blocks, some with more rows than they hold."""
    rng = np.random.default_rng(M)
    off = _offsets(counts)
    _check_product(ep, off, *_draw(rng, R * M, E, 256, 200), R, M)
    _check_gated(ep, off, *_draw(rng, R * M, E, 256, 256), R, M)


def test_rank_major_far_more_pairs_than_rows(ep):
    """Blocks that drop most of their pairs: the segment starts lie far past the rows."""
    rng = np.random.default_rng(17)
    off = _offsets([70, 5, 0, 90, 300, 1, 20, 2, 0, 0, 50, 60, 8, 9, 10, 400])
    R, M = 4, 40
    _check_product(ep, off, *_draw(rng, R * M, 16, 256, 264), R, M)
    _check_gated(ep, off, *_draw(rng, R * M, 16, 256, 256), R, M)


def test_slice_of_the_offsets(ep):
    """One rank's experts: a slice of a dispatch's offsets with those experts' weights."""
    rng = np.random.default_rng(6)
    off = _offsets([30, 5, 0, 70, 12, 9])
    a, a_s, w, w_s = _draw(rng, off[-1], 6, 384, 256)
    whole = _check_product(ep, off, a, a_s, w, w_s)
    part = _check_product(ep, off[2:5], a, a_s, w[2:4], w_s[2:4])
    lo, hi = off[2], off[4]
    assert torch.equal(part[lo:hi], whole[lo:hi])


def test_offsets_out_of_range_are_clamped(ep):
    """Entries below 0, past the rows or descending reach no row outside the buffers."""
    rng = np.random.default_rng(7)
    a, a_s, w, w_s = _draw(rng, 50, 4, 256, 256)
    for bad in ([-5, 10, 20, 30, 90], [0, 60, 70, 80, 90], [40, 30, 20, 10, 0], [0, 10, 5, 60, 20]):
        y = torch.full((50 + 64, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_gemm(torch.tensor(bad, dtype=torch.int32, device="cuda"), a.cuda(), a_s.cuda(), w.cuda(),
                          w_s.cuda(), y[:50])
        assert (y[50:] == 7.0).all()
    y = torch.full((50, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gemm(torch.zeros(5, dtype=torch.int32, device="cuda"), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda(), y)
    assert (y == 7.0).all()
    none = torch.empty(0, 256, dtype=torch.uint8, device="cuda")
    assert ep.expert_gemm(torch.zeros(5, dtype=torch.int32, device="cuda"), none,
                          torch.empty(0, 2, device="cuda"), w.cuda(), w_s.cuda()).shape == (0, 256)


def test_nan_rows_stay_in_their_rows(ep):
    """NaN in a row, and in the rows around a segment, reaches that row only; inf and zero scales follow fp32."""
    rng = np.random.default_rng(9)
    off = [4, 20, 41]
    a, a_s, w, w_s = _draw(rng, 60, 2, 256, 256)
    ref = _check_product(ep, off, a, a_s, w, w_s)
    a[:4], a[41:] = 0x7F, 0x7F
    a_s[:4], a_s[41:] = float("nan"), float("inf")
    a[10, 3], a_s[30, 1] = 0x7F, float("nan")
    y = ep.expert_gemm(torch.tensor(off, dtype=torch.int32).cuda(), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda())
    q, s = ep.expert_gated(torch.tensor(off, dtype=torch.int32).cuda(), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda())
    keep = [r for r in range(4, 41) if r not in (10, 30)]
    assert torch.equal(y[keep], ref[keep])
    assert torch.isnan(y[[10, 30]]).all() and not torch.isnan(s[keep]).any()
    assert ((q[[10, 30]] & 0x7F) == 0x7F).all()


def test_all_zero_groups_and_saturation(ep):
    """Groups of zeros get the scale 1; gates at both ends of the exponential."""
    rng = np.random.default_rng(10)
    a, a_s, w, w_s = _draw(rng, 40, 1, 256, 512)
    a[7] = 0
    w[0, 256:384] = 0             # the up rows of the first group
    a_s[9] *= 1e6                 # gates of +- thousands: h = g u or 0
    a_s[11] *= 1e-6
    q, s = _check_gated(ep, [0, 40], a, a_s, w, w_s)
    assert (s[:, 0] == 1).all() and (q[:, :128] & 0x7F == 0).all() and (s[7] == 1).all()


def test_products_repeat_to_the_bit(ep):
    rng = np.random.default_rng(12)
    off = torch.tensor(_offsets([200, 3, 0, 90]), dtype=torch.int32).cuda()
    x = [t.cuda() for t in _draw(rng, 293, 4, 2048, 512)]
    y, (q, s) = ep.expert_gemm(off, *x), ep.expert_gated(off, *x)
    for _ in range(5):
        assert torch.equal(ep.expert_gemm(off, *x), y)
        q2, s2 = ep.expert_gated(off, *x)
        assert torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("counts,K,N", [([1] * 8, 2048, 7168), ([150, 90], 7168, 1024), ([40, 1, 200], 2048, 2048)])
def test_wide_layers(ep, counts, K, N):
    rng = np.random.default_rng(K)
    off = _offsets(counts)
    _check_product(ep, off, *_draw(rng, off[-1] + 3, len(counts), K, N))
    _check_gated(ep, off, *_draw(rng, off[-1] + 3, len(counts), K, 2 * (N // 4)))


def test_weights_past_two_gib(ep):
    """An expert whose weights start past 2^31 and 2^32 bytes."""
    E, N, K = 5, 32768, 32768     # 1 GiB an expert
    rng = np.random.default_rng(13)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    a, a_s, _, _ = _draw(rng, 6, 1, K, 8)
    last = torch.from_numpy((rng.standard_normal((256, K)) * 100).astype(np.float32)).clamp(-448, 448)
    last = last.to(torch.float8_e4m3fn).view(torch.uint8)
    w[E - 1, -256:] = last.cuda()
    w_s = torch.full((E, N // 128, K // 128), 1e-5, device="cuda")
    y = ep.expert_gemm(torch.tensor([0, 0, 0, 2, 2, 6], dtype=torch.int32).cuda(), a.cuda(), a_s.cuda(), w, w_s)
    ref, mag, _ = moe_ref.product([0, 6], a.numpy(), a_s.numpy(), last.numpy()[None],
                                  np.full((1, 2, K // 128), 1e-5, np.float32))
    err = moe_ref.sum_error_8bit(mag, K)
    got = y.cpu().double().numpy()
    assert (got[:, :-256] == 0).all() and (got[:2] == 0).all()
    assert (np.abs(got[2:, -256:] - ref[2:]) <= moe_ref.BF16_HALF * (np.abs(ref[2:]) + err[2:]) + err[2:]).all()


# enough rows to fill the chip: the forms with large tiles, at every short length of K, ragged segments and widths
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640])
@pytest.mark.parametrize("rows,E,N", [(20000, 6, 1000), (26000, 41, 520), (4000, 64, 2056)])
def test_many_rows_product(ep, rows, E, N, K):
    rng = np.random.default_rng(rows + K)
    cut = np.sort(rng.integers(5, rows - 3, size=E + 1)).tolist()
    cut[2] = cut[1]
    _check_product(ep, cut, *_draw(rng, rows, E, K, N))


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640])
@pytest.mark.parametrize("rows,E,N", [(20000, 6, 384), (19000, 41, 256)])
def test_many_rows_gated(ep, rows, E, N, K):
    rng = np.random.default_rng(rows + K)
    cut = np.sort(rng.integers(5, rows - 3, size=E + 1)).tolist()
    cut[2] = cut[1]
    _check_gated(ep, cut, *_draw(rng, rows, E, K, 2 * N))


def test_many_rows_rank_major_and_nan(ep):
    """Large tiles over RANK_MAJOR blocks that overflow; NaN rows around the segments stay there."""
    rng = np.random.default_rng(21)
    off = _offsets([9000, 0, 3500, 2500, 7000, 800])
    R, M = 3, 8000
    x = _draw(rng, R * M, 6, 256, 768)
    _check_product(ep, off, *x, R, M)
    _check_gated(ep, off, *x, R, M)
    a, a_s, w, w_s = x
    off = [100, 12000, 12000, 23000]
    ref = _check_product(ep, off, a, a_s, w[:3], w_s[:3])
    refq = _check_gated(ep, off, a, a_s, w[:3], w_s[:3])
    a[:100], a[23000:], a_s[23000:] = 0x7F, 0x7F, float("nan")
    a[500, 7] = 0x7F
    o = torch.tensor(off, dtype=torch.int32).cuda()
    y = ep.expert_gemm(o, a.cuda(), a_s.cuda(), w[:3].cuda(), w_s[:3].cuda())
    q, s = ep.expert_gated(o, a.cuda(), a_s.cuda(), w[:3].cuda(), w_s[:3].cuda())
    keep = torch.ones(R * M, dtype=torch.bool)
    keep[:100], keep[23000:], keep[500] = False, False, False
    assert torch.equal(y[keep.cuda()], ref[keep.cuda()]) and torch.isnan(y[500]).all()
    assert torch.equal(q[keep.cuda()], refq[0][keep.cuda()]) and torch.equal(s[keep.cuda()], refq[1][keep.cuda()])


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 768])
def test_few_rows_every_length(ep, K):
    """One row for a few experts (K split over two groups of waves), and tens of rows, at every short length of K."""
    rng = np.random.default_rng(K)
    for counts, N in (([1, 0, 1, 2], 264), ([20, 33, 1], 520)):
        off = _offsets(counts)
        _check_product(ep, off, *_draw(rng, off[-1] + 2, len(counts), K, N))
        _check_gated(ep, off, *_draw(rng, off[-1] + 2, len(counts), K, 512))


@pytest.mark.parametrize("K", [128, 256, 896, 1024, 1152, 2176])
def test_one_expert_few_rows(ep, K):
    """A dense layer's few rows: K split over eight groups of waves, lengths shorter and longer than the groups."""
    rng = np.random.default_rng(K + 1)
    for rows, N in ((1, 8), (3, 72), (17, 520), (70, 264)):
        x = _draw(rng, rows + 3, 1, K, N)
        _check_product(ep, [2, rows + 2], *x)
    _check_gated(ep, [1, 18], *_draw(rng, 20, 1, K, 512))


def test_one_ranks_block_of_rank_major_rows(ep):
    """One rank's share of RANK_MAJOR rows: its block alone, its experts' slice of the offsets, num_ranks 1."""
    rng = np.random.default_rng(23)
    off = _offsets([30, 5, 0, 70, 12, 9, 3, 25])
    R, M = 4, 48   # rank 1's 70 rows pass its block, rank 3's do not fill theirs
    a, a_s, w, w_s = _draw(rng, R * M, 8, 256, 256)
    for r in range(R):
        rows, mine = slice(r * M, (r + 1) * M), slice(2 * r, 2 * r + 2)
        args = (off[2 * r:2 * r + 3], a[rows], a_s[rows], w[mine], w_s[mine])
        _check_product(ep, *args, R=1, M=M)
        _check_gated(ep, *args, R=1, M=M)


@pytest.mark.parametrize("copies", [1, 900])   # few rows, and tiles of many
def test_gate_far_below_zero(ep, copies):
    """silu's lower tail, where e^-g leaves binary32: h keeps its precision down to the smallest values.

    Every sum is one product, exact, so g and u are.  All of a row's h are equal: the byte is 448 and the scale h / 448.
    Bounds: 4 steps of h and one each of the scale, the quotient and the product, twice; and where values fall
    below 2^-126 half the smallest step of e^g (times g u) and of the scale (times 448)."""
    depth = np.repeat(np.arange(80.0, 104.0, dtype=np.float32), copies)
    rows = depth.size
    a = torch.zeros((rows, 128), dtype=torch.uint8)
    a[:, 0] = 0x38                                   # 1
    w = torch.zeros((1, 256, 128), dtype=torch.uint8)
    w[0, :128, 0] = 0xB8                             # -1: the gate
    w[0, 128:, 0] = 0x38
    u = np.float32(2.0 ** 20)
    a_s = torch.from_numpy(depth)[:, None].contiguous()
    w_s = torch.tensor([1.0, float(u)]).reshape(1, 2, 1)
    off = torch.tensor([0, rows], dtype=torch.int32)
    q, s = ep.expert_gated(off.cuda(), a.cuda(), a_s.cuda(), w.cuda(), w_s.cuda())
    d = depth.astype(np.float64)
    h = -d * np.exp(-d) / (1 + np.exp(-d)) * d * float(u)
    got = moe_ref.e4m3_value(q.cpu().numpy()) * s.cpu().double().numpy()
    tol = 16 * 2.0 ** -23 * np.abs(h) + 2.0 ** -149 * (d * d * float(u) + 448)
    assert (np.abs(got - h[:, None]) <= tol[:, None]).all()


@pytest.mark.parametrize("K", [768, 896, 1024, 1664])
@pytest.mark.parametrize("rows,E", [(13000, 24), (2500, 40)])
def test_many_rows_product_every_buffer(ep, rows, E, K):
    """Blocks of K past a whole turn of the tiles' buffers, by one to six of them."""
    rng = np.random.default_rng(K + rows)
    cuts = np.sort(rng.integers(0, rows + 1, E - 1)).tolist()
    _check_product(ep, [0] + cuts + [rows], *_draw(rng, rows, E, K, 1032))
