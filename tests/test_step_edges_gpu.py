"""Edges of the operators between the GEMVs on the GPU: rows of logits over several blocks, masks and bounds at the ends of pages
and of the page table, kernels by their route.  Formulas and tolerances are those of test_step_gpu."""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")

from tests.test_step_gpu import ATTN, B16, H16, TINY, U, Step, f64, kernel, rnd, run_sample  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.build()
    qg.lib()
    qg.qgemv_device_error(reset=True)
    yield
    assert qg.qgemv_device_error() == 0


# -------------------------------------------------------------------------------------------------------- attention

def check_seen(s, sees):
    """The result of a step of one sequence against the formula in 64 bits, its tokens seeing the keys `sees` [tokens, context]."""
    out, lse, u = f64(s.out), f64(s.lse), U[s.dtype]
    q, k, v = f64(s.q), f64(s.k[0]), f64(s.v[0])
    for h in range(s.H):
        kh, vh, qh = k[:, h // (s.H // s.KH)], v[:, h // (s.H // s.KH)], q[:, h]
        some = sees.any(0)  # (what no token sees may be anything)
        kh, vh = np.where(some[:, None], kh, 0.0), np.where(some[:, None], vh, 0.0)
        x = np.where(sees, s.scale * (qh @ kh.T), -np.inf)
        top = x.max(1, initial=-np.inf, keepdims=True)
        top = np.where(np.isinf(top), 0.0, top)
        p = np.exp(x - top)
        l = p.sum(1, keepdims=True)
        p = p / np.where(l == 0, 1, l)
        ref, A = p @ vh, p @ np.abs(vh)
        off = 2.0 ** -20 * s.scale * (np.linalg.norm(qh, axis=1) * np.linalg.norm(kh, axis=1).max(initial=0.0))[:, None]
        err = np.abs(out[:, h] - ref)
        assert np.all(err <= u * np.abs(ref) + (u + 4 * off + 2.0 ** -18) * A + TINY[s.dtype]), (h, np.nanmax(err))
        empty = l[:, 0] == 0
        assert np.array_equal(np.isneginf(lse[:, h]), empty)
        got, want = lse[~empty, h], (top[:, 0] + np.log(np.where(empty, 1.0, l[:, 0])))[~empty]
        assert np.all(np.abs(got - want) <= off[~empty, 0] + 2.0 ** -20 * np.maximum(1, np.abs(want)))


def window_sees(n, kv_len, window, readable):
    pos, t = kv_len - n + np.arange(n, dtype=np.int64), np.arange(kv_len)
    return (t[None] <= pos[:, None]) & (t[None] > pos[:, None] - window) & (t[None] < readable)


# heads that fit, groups that do and do not divide 128 (queries by tensor map, row by row), pages of multiples of 8 tokens and others
# (keys by tensor map, row by row)
@pytest.mark.parametrize("shape", ATTN + [([130, 3], [500, 300], 6, 2, 128, 5, H16), ([70], [333], 10, 2, 64, 24, B16),
                                          ([20, 40], [90, 1100], 9, 1, 96, 33, B16), ([3, 3], [40, 200], 64, 1, 64, 12, H16),
                                          ([150], [2000], 130, 1, 64, 8, B16), ([60], [700], 3, 3, 72, 64, H16)], ids=str)
def test_the_forced_kernel_is_the_one_that_runs(shape, kernel):  # noqa: F811
    new, ctx, H, KH, D, page, dtype = shape
    s = Step(60, new, ctx, H, KH, D, page, dtype)
    qg.qgemv_route_reset()
    qg.qgemv_attn(s.args())
    counts = qg.qgemv_route_counts()
    assert (counts[qg.ROUTE_ATTN_ROWS], counts[qg.ROUTE_ATTN_TILES]) == ((1, 0) if kernel == "16-row" or D > 128 else (0, 1))
    s.check()


# context, window; a context of 1000 lies wholly past the 256 tokens that may be read, one of 700 starts among them
@pytest.mark.parametrize("new", [3, 100])
@pytest.mark.parametrize("kv_len,window", [(1000, 500), (1000, 130), (700, 500), (700, 440), (360, 1), (355, 99)])
@pytest.mark.parametrize("limit", ["table", "max_kv"])
def test_window_past_the_keys_that_may_be_read(new, kv_len, window, limit, kernel):  # noqa: F811
    """The row of the page table, or max_kv, ends at 256 tokens; what follows the row in memory is no page number, so an entry
    read there would show in the device error word."""
    s = Step(70 + new, [new], [kv_len], 8, 2, 64, 16, B16)
    cols = 16
    memory = torch.full((1 << 14,), 2 ** 30, dtype=torch.int32, device="cuda")
    memory[:cols] = s.table[0, :cols]
    s.table = memory[:cols].view(1, cols) if limit == "table" else memory[:kv_len // 16 + 1].view(1, -1)
    qg.qgemv_device_error(reset=True)
    qg.qgemv_attn(s.args(window=window, max_kv=kv_len if limit == "table" else 16 * cols))
    check_seen(s, window_sees(new, kv_len, window, 16 * cols))
    assert qg.qgemv_device_error() == 0
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("new,ctx", [([1, 1, 3], [900, 40, 500]), ([150, 20, 1], [900, 40, 700])])
def test_a_view_of_a_longer_page_table(new, ctx, kernel):  # noqa: F811
    s = Step(76, new, ctx, 8, 2, 128, 16, B16)
    whole = torch.full((3, 500), 2 ** 30, dtype=torch.int32, device="cuda")  # a fixed table; this step needs a few of its columns
    whole[:, 2:2 + s.table.shape[1]] = s.table
    s.table = whole[:, 2:2 + s.table.shape[1]]
    qg.qgemv_attn(s.args(max_kv=5000))
    s.check()


def test_a_page_table_without_columns(kernel):  # noqa: F811
    s = Step(77, [3, 150], [0, 0], 4, 2, 64, 16, B16)
    s.table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    qg.qgemv_attn(s.args())
    s.check()


@pytest.mark.parametrize("new", [2, 100])
def test_a_table_row_and_a_page_whose_product_leaves_64_bits(new, kernel):  # noqa: F811
    """One page of 2^24 tokens, and rows of the table 2^40 entries apart: a row reaches further than any context."""
    page, kv_len = 1 << 24, 1200
    s = Step(75, [new], [kv_len], 4, 1, 8, page, B16)
    a = s.args()
    a.pages_stride = 1 << 40
    qg.qgemv_attn(a)
    s.check()


@pytest.mark.parametrize("max_kv,window", [(72, 22), (70, 22), (64, 30), (79, 10)])
def test_a_window_past_the_keys_looks_no_page_up(max_kv, window, kernel):  # noqa: F811
    """The page that holds max_kv ends before the window begins: it is not the tokens' affair, and may be given back."""
    s = Step(78, [3], [96], 8, 8, 128, 16, B16)
    s.table[0, :max_kv // 16 + 1] = -1
    qg.qgemv_device_error(reset=True)
    qg.qgemv_attn(s.args(window=window, max_kv=max_kv))
    assert qg.qgemv_device_error(reset=True) == 0
    check_seen(s, window_sees(3, 96, window, max_kv))


@pytest.mark.parametrize("new,kv_len", [(3, 1), (20, 2), (20, 0), (200, 90), (300, 300), (5, 700)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 90, 91])
def test_window_of_any_size(new, kv_len, window, kernel):  # noqa: F811
    """A window longer than any context masks nothing, also where tokens sit at positions below 0."""
    s = Step(80 + new, [new], [kv_len], 8, 2, 64, 16, B16)
    qg.qgemv_attn(s.args(window=window))
    check_seen(s, window_sees(new, kv_len, window, kv_len))
    if window >= 2 ** 30:
        plain = (s.out.clone(), s.lse.clone())
        qg.qgemv_attn(s.args())
        assert torch.equal(plain[0], s.out) and torch.equal(plain[1], s.lse)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("new,kv_len,window", [(1, 1000, 100), (3, 999, 333), (40, 1000, 129), (150, 1500, 201), (300, 700, 37)])
def test_window_leaves_what_lies_before_it_alone(new, kv_len, window, page, kernel):  # noqa: F811
    """Keys and values before the first token's window may be anything, and their pages given back (a table entry of -1)."""
    s = Step(90 + page, [new], [kv_len], 8, 2, 128, page, B16)
    sees = window_sees(new, kv_len, window, kv_len)
    first = int(sees.any(0).argmax())
    t = torch.arange(first, device="cuda")
    for x in (s.kc, s.vc):
        x[s.table[0, t // page].long(), t % page] = float("nan")
    s.table[0, :first // page] = -1
    qg.qgemv_device_error(reset=True)
    qg.qgemv_attn(s.args(window=window))
    assert qg.qgemv_device_error(reset=True) == 0
    check_seen(s, sees)


@pytest.mark.parametrize("new,kv_len,window,route", [
    (24, 24000, 1024, "rows"), (100, 24000, 300, "rows"), (16, 24000, 4000, "rows"),  # few keys a token: without the window, all take the other
    (64, 24000, 15000, "tiles"), (500, 9000, 1024, "tiles"), (1300, 3000, 600, "tiles")])
def test_window_decides_the_kernel_and_the_parts(new, kv_len, window, route):
    s = Step(95, [new], [kv_len], 32, 8, 128, 64, B16)
    if route == "rows":
        qg.qgemv_route_reset()
        qg.qgemv_attn(s.args())
        assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_TILES] == 1
    qg.qgemv_route_reset()
    qg.qgemv_attn(s.args(window=window))
    assert qg.qgemv_route_counts()[{"rows": qg.ROUTE_ATTN_ROWS, "tiles": qg.ROUTE_ATTN_TILES}[route]] == 1
    s.check(window=window)


@pytest.mark.parametrize("H,KH", [(8, 8), (6, 2), (4, 1), (20, 1)])
@pytest.mark.parametrize("new", [40, 333])
@pytest.mark.parametrize("window", [900, 1900, 2047, 2500, 6000])
def test_windows_whose_keys_are_cut_into_parts(new, window, H, KH):
    """The 128-row kernel at windows around the lengths where a row tile's keys make one part more: tokens at every offset in a key tile."""
    qg.qgemv_tune_attn(2)
    try:
        s = Step(96, [new, new // 3, 1], [6300, 2090 + new, 3001], H, KH, 64, 16, B16)
        qg.qgemv_attn(s.args(window=window))
        s.check(window=window)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
    finally:
        qg.qgemv_tune_attn(0)


@pytest.mark.parametrize("new,ctx", [([3, 2], [700, 40]), ([150, 20], [900, 40]), ([40, 1], [9000, 9000])])
def test_a_query_of_nan_shows_in_its_own_row_only(new, ctx, kernel):  # noqa: F811
    s = Step(97, new, ctx, 8, 2, 128, 16, B16)
    qg.qgemv_attn(s.args())
    out, lse = s.out.clone(), s.lse.clone()
    s.q[1, 5, 100] = float("nan")
    qg.qgemv_attn(s.args())
    assert bool(torch.isnan(s.out[1, 5]).all()) and bool(torch.isnan(s.lse[1, 5]))
    s.out[1, 5], s.lse[1, 5] = out[1, 5], lse[1, 5]
    assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("gap", [6.0, 10.0, 12.0, 14.0, 16.0, 17.5])
@pytest.mark.parametrize("dtype", [B16, H16])
@pytest.mark.parametrize("new,ctx", [(1, 40000), (100, 3000), (100, 20000)])
def test_many_keys_far_below_one(new, ctx, dtype, gap, kernel):  # noqa: F811
    """A first token that takes nearly all of the attention and has no value, as trained models have it: the result is what many keys
    `gap` nats below it add up to, and their probabilities must not lose bits for being small."""
    rng = np.random.default_rng(98)
    s = Step(98, [new], [ctx], 4, 2, 64, 64, dtype, scale=1.0)
    q = torch.zeros(new, 4, 64, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    q[..., 1:] = rnd(rng, (new, 4, 63), dtype, 0.1)
    s.q = q
    k, v = rnd(rng, (ctx, 2, 64), dtype, 0.1), rnd(rng, (ctx, 2, 64), dtype, 0.25) + 1.0
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = gap
    v[0] = 0.0
    s.k[0], s.v[0] = k, v
    t = torch.arange(ctx, device="cuda")
    at = s.table[0, t // 64].long(), t % 64
    s.kc[at], s.vc[at] = k, v
    qg.qgemv_attn(s.args())
    s.check()


# --------------------------------------------------------------------------------------------------------- sampling

# rows of two, four and eight blocks, the last of them with and without an odd end
@pytest.mark.parametrize("dtype", [torch.float32, B16, H16])
@pytest.mark.parametrize("n", [20481, 65541, 151936, 163843])
def test_sampling_special_rows_over_several_blocks(n, dtype):
    rng = np.random.default_rng(n)
    x = rnd(rng, (13, n), dtype, 2.0)
    inf, end = float("inf"), n - 1
    x[0] = -inf
    x[1, end] = float("nan")   # in the last block; an infinity in the first
    x[1, 17] = inf
    x[2, end] = inf            # the first of two infinities, in different blocks
    x[2, n // 2] = inf
    x[3] = -inf
    x[3, end] = -3.0           # one token is left
    x[4, ::2] = -inf
    x[5] = 0.25                # one tie of the whole row
    x[6] = -0.0
    x[6, ::3] = 0.0            # both zeros are one value
    x[7, 100:n - 100] = x[7].max()
    x[8, end] = 3e38 if dtype is not H16 else 6e4
    x[9] *= 1e-4
    x[10, end] = float("nan")
    x[10, end - 1] = float("nan")
    x[11] = -6e4
    x[12, :n - 40] = -inf      # only the last block has tokens
    u = rng.random(13, dtype=np.float32)
    for kw in (dict(), dict(k=np.full(13, 7)), dict(p=np.full(13, 0.5)), dict(mp=np.full(13, 0.1)), dict(T=np.zeros(13)),
               dict(k=np.full(13, 1000), p=np.full(13, 0.9), mp=np.full(13, 0.05)), dict(k=np.ones(13)),
               dict(T=np.full(13, 1e-3)), dict(p=np.full(13, 0.999))):
        a = run_sample(x, u=u, **kw)
        b = run_sample(x, u=u, flags=qg.QGEMV_FLAG_PDL, check=False, **kw)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1], equal_nan=True)
    for edge in (0.0, np.float32(1 - 2.0 ** -24)):
        run_sample(x, u=np.full(13, edge), k=np.full(13, 50))
    # rank 0 alone: the first of the largest, whichever block it lies in
    token, prob = run_sample(x, u=u, check=False, T=np.full(13, -1.0))
    ok = [3, 4, 5, 6, 7, 8, 9, 11, 12]
    assert np.array_equal(token[ok], f64(x).argmax(1)[ok]) and np.all(prob[ok] == 1)


@pytest.mark.parametrize("dtype,n", [(torch.float32, 40963), (B16, 151931), (H16, 81925)])
def test_sampling_unaligned_rows_over_several_blocks(dtype, n):
    rng = np.random.default_rng(n)
    wide = rnd(rng, (5, n + 6), dtype, 2.0)
    x = wide[:, :n]
    assert x.stride(0) * x.element_size() % 16
    u = rng.random(5, dtype=np.float32)
    for kw in (dict(k=np.full(5, 50), p=np.full(5, 0.8)), dict(p=np.full(5, 0.9)), dict(), dict(k=np.full(5, 2000)), dict(T=np.zeros(5))):
        a = run_sample(x, u=u, **kw)
        b = run_sample(x.contiguous(), u=u, **kw)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.float32, B16])
@pytest.mark.parametrize("n", [2003, 30011])
def test_sampling_at_the_largest_temperatures(n, dtype):
    """So flat that the edges of the histogram's bins lie beyond fp32, with fewer tokens left by a mask than top-k asks for."""
    rng = np.random.default_rng(n)
    x = rnd(rng, (6, n), dtype, 3.0)
    for i, left in enumerate((n, 1500, 900, 300, 20, 1)):
        x[i, torch.from_numpy(rng.permutation(n)[left:]).cuda()] = -float("inf")
    u = rng.random(6, dtype=np.float32)
    for k in (5, 400, 600, 1600):
        for p in (1.0, 0.7):
            kw = dict(k=np.full(6, k), p=np.full(6, p), u=u)
            a = run_sample(x, T=np.full(6, 1e38), **kw)
            b = run_sample(x, T=np.full(6, np.inf), check=False, **kw)
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
            run_sample(x, T=np.full(6, 2e36), **kw)


# the last length whose slices (an eighth each) stay in shared memory beside the rest, and the next one, which is read again from L2
@pytest.mark.parametrize("dtype,n", [(torch.float32, 382528), (torch.float32, 382529), (B16, 765056), (B16, 765057), (H16, 765056), (H16, 765064)])
def test_sampling_around_the_longest_slices_in_shared_memory(dtype, n):
    rng = np.random.default_rng(n)
    x = rnd(rng, (3, n), dtype, 2.0)
    x[1, ::3] = -float("inf")
    u = rng.random(3, dtype=np.float32)
    for kw in (dict(), dict(k=np.full(3, 50), p=np.full(3, 0.9)), dict(k=np.full(3, 3000)), dict(p=np.full(3, 0.8)), dict(mp=np.full(3, 0.01)),
               dict(T=np.zeros(3))):
        run_sample(x, u=u, **kw)
