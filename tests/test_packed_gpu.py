"""The packed key/value cache on the GPU: what is written is the definition's bytes, what is read their exact values rounded once,
and attention over it is held to its formula in 64 bits on those values.

Tolerances, from the arithmetic:
 - a written row equals the definition's bytes; a value read back equals the exact d c + m rounded to fp32 and then to its type;
 - rotated keys are packed from fp32 values that are off by 16 * 2^-24 (|a| + |b|) (fp32 products and sines of an angle good to 2^-24 of a
   half turn); a code is then off by half a step, and 2^-12 of it for the fp32 of the code.
"""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from . import packedref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_step_gpu import turned  # noqa: E402

B16, H16, F32 = torch.bfloat16, torch.float16, torch.float32
BITS = {"Q4": 4, "Q8": 8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.build()
    qg.lib()
    qg.qgemv_device_error(reset=True)
    yield
    assert qg.qgemv_device_error() == 0


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows_of(kind, pages, page, heads, dim, order="token-head", fill=0xA5):
    """A cache tensor [pages, page, heads, row bytes], every byte `fill`, a page's tokens or heads first."""
    row = qg.qgemv_cache_row_bytes(kind, dim)
    if order == "token-head":
        return torch.full((pages, page, heads, row), fill, dtype=torch.uint8, device="cuda")
    return torch.full((pages, heads, page, row), fill, dtype=torch.uint8, device="cuda").transpose(1, 2)


def awkward(rng, tokens, heads, dim, dtype):
    """Values with equal ones, blocks of one value, large and tiny ones, far offsets."""
    x = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    x += np.where(rng.random((1, heads, dim)) < 0.1, 20.0, 0.0).astype(np.float32)
    kind = rng.integers(0, 8, (tokens, heads, dim // 32))
    b = x.reshape(tokens, heads, -1, 32)
    b[kind == 0] = b[kind == 0][:, :1]      # one value
    b[kind == 1] *= np.float32(1e-6)        # steps below fp16's normal range
    b[kind == 2] = 0
    b[kind == 3] *= np.float32(3e4)         # beyond fp16 in some places
    b[kind == 4] = np.round(b[kind == 4])   # halfway codes
    return torch.from_numpy(x).to(dtype).cuda()


def f32(t):
    return t.float().cpu().numpy()


def held(cache, kind, dim):
    """The part of a cache's rows that the definition fills."""
    n = dim * BITS[kind] // 8 + dim // 32 * 4
    return cache.cpu().numpy()[..., :n]


WRITE = [
    # tokens, heads, dim, page, type, order
    (1, 8, 128, 16, F32, "token-head"),
    (1, 1, 32, 1, B16, "token-head"),
    (61, 8, 128, 64, H16, "head-token"),
    (300, 3, 96, 7, B16, "token-head"),
    (37, 5, 64, 16, F32, "head-token"),
    (700, 2, 256, 33, H16, "token-head"),
    (5000, 4, 160, 32, B16, "token-head"),
    (9, 40, 224, 5, F32, "token-head"),
    (2500, 1, 32, 16, F32, "token-head"),
]


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("T,H,D,page,xt,order", WRITE)
def test_write_is_the_definition_bit_for_bit_and_reads_back(T, H, D, page, xt, order, kind):
    rng = np.random.default_rng(T + D)
    k, v = (awkward(rng, T, H, D, xt) for _ in range(2))
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2::5] = -1
    kc, vc = (rows_of(kind, pages, page, H, D, order) for _ in range(2))
    cache = qg.packed_cache(kind, kc, vc, D)
    qg.qgemv_route_reset()
    qg.qgemv_cache_write(qg.cache_write_args(k, v, cache, cuda(slots)))
    assert qg.qgemv_route_counts()[qg.ROUTE_CACHE_WRITE] == 1
    live = slots >= 0
    for x, c in ((k, kc), (v, vc)):
        want = ref.to_bytes(*ref.pack(f32(x), BITS[kind]), BITS[kind])
        n = D * BITS[kind] // 8 + D // 32 * 4
        got = c.cpu().numpy()
        rows = got[slots[live] // page, slots[live] % page]
        assert np.array_equal(rows[..., :n], want[live][..., :n])
        rest = np.setdiff1d(np.arange(pages * page), slots[live])
        assert np.all(got[rest // page, rest % page] == 0xA5)
    # every written token is read through a table of its own row, one sequence each
    order_ = rng.permutation(np.flatnonzero(live))
    table = cuda((slots[order_] // page).astype(np.int32)[:, None])
    first = cuda((slots[order_] % page).astype(np.int32))
    start = torch.arange(len(order_) + 1, dtype=torch.int32, device="cuda")
    for ot in (F32, B16, H16):
        ko, vo = (torch.full((len(order_) + 3, H, D), 9.0, dtype=ot, device="cuda") for _ in range(2))
        qg.qgemv_cache_read(qg.cache_read_args(cache, table, start, ko, vo, first=first))
        for c, o in ((kc, ko), (vc, vo)):
            exact = ref.values(c.cpu().numpy()[slots[order_] // page, slots[order_] % page], BITS[kind], D)
            want = torch.from_numpy(exact.astype(np.float32)).to(ot)
            assert torch.equal(o[:len(order_)].cpu(), want)
            assert bool((o[len(order_):] == 9.0).all())
    assert qg.qgemv_device_error() == 0


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_a_value_is_at_most_half_a_step_away(kind):
    rng = np.random.default_rng(3)
    x = awkward(rng, 400, 4, 128, F32).clamp(-65504, 65504)
    kc, vc = (rows_of(kind, 25, 16, 4, 128) for _ in range(2))
    qg.qgemv_cache_write(qg.cache_write_args(x, x, qg.packed_cache(kind, kc, vc, 128), torch.arange(400, device="cuda")))
    rows = kc.cpu().numpy().reshape(400, 4, -1)
    _, d, _ = ref.parts(rows, BITS[kind], 128)
    off = np.abs(ref.values(rows, BITS[kind], 128) - f32(x).astype(np.float64))
    assert np.all(off <= np.repeat(d.astype(np.float64), 32, -1) / 2 * (1 + 2.0 ** -12))


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_values_that_are_no_numbers(kind):
    x = torch.ones(3, 1, 64, device="cuda")
    x[0, 0, 5], x[1, 0, 40], x[1, 0, 41] = float("nan"), float("inf"), -float("inf")
    kc, vc = (rows_of(kind, 1, 4, 1, 64) for _ in range(2))
    cache = qg.packed_cache(kind, kc, vc, 64)
    qg.qgemv_cache_write(qg.cache_write_args(x, x, cache, torch.arange(3, device="cuda")))
    out = torch.empty(3, 1, 64, device="cuda")
    qg.qgemv_cache_read(qg.cache_read_args(cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                           torch.tensor([0, 3], dtype=torch.int32, device="cuda"), v_out=out))
    assert bool(out[0, 0, :32].isnan().all()) and bool((out[0, 0, 32:] == 1).all())       # the block with the NaN, no other
    want = ref.values(ref.to_bytes(*ref.pack(f32(x[1]), BITS[kind]), BITS[kind]), BITS[kind], 64).astype(np.float32)
    assert np.array_equal(out[1].cpu().numpy(), want) and float(out[1, 0, 41]) == -65504  # infinities as the largest fp16
    assert bool((out[2] == 1).all())


def test_write_slot_beyond_the_cache_is_skipped_and_reported():
    x = torch.randn(4, 2, 64, device="cuda")
    kc, vc = (rows_of("Q4", 2, 3, 2, 64) for _ in range(2))
    slots = torch.tensor([1, 6, 2 ** 40, -7], device="cuda")
    qg.qgemv_cache_write(qg.cache_write_args(x, x, qg.packed_cache("Q4", kc, vc, 64), slots))
    assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
    touched = (kc != 0xA5).any(-1).nonzero()
    assert touched.tolist() == [[0, 1, 0], [0, 1, 1]]


def test_read_of_ragged_sequences_bad_places_and_untouched_rows():
    rng = np.random.default_rng(8)
    H, D, page = 2, 96, 5
    kc, vc = (cuda(rng.integers(0, 120, (9, page, H, ref.row_bytes(8, D))).astype(np.uint8)) for _ in range(2))  # (finite scales)
    cache = qg.packed_cache("Q8", kc, vc, D)
    table = np.array([[3, 0, 8], [99, 1, 2], [-1, 4, 5], [6, 7, 6]], np.int32)
    start, first = np.array([2, 9, 9, 15, 16], np.int32), np.array([1, 0, 4, -1], np.int32)
    wide = torch.full((4, 7), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :3] = cuda(table)
    for t in (cuda(table), wide[:, :3]):  # whole rows, and a view of longer ones
        ko, vo = (torch.full((20, 3, D), 9.0, device="cuda")[:, :2] for _ in range(2))
        qg.qgemv_cache_read(qg.cache_read_args(cache, t, cuda(start), ko, vo, first=cuda(first)))
        assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
        for c, o in ((kc, ko), (vc, vo)):
            want = np.full((20, H, D), 9.0, np.float32)
            val = ref.values(c.cpu().numpy(), 8, D).astype(np.float32)
            for b in range(4):
                for r in range(start[b], start[b + 1]):
                    at = first[b] + r - start[b]
                    p = table[b, at // page] if 0 <= at < 15 else -1
                    want[r] = val[p, at % page] if 0 <= p < 9 else 0.0
            assert np.array_equal(o.cpu().numpy(), want)
    # one side only, and a table without columns: zeros
    ko = torch.full((4, H, D), 9.0, dtype=B16, device="cuda")
    qg.qgemv_cache_read(qg.cache_read_args(cache, cuda(table), cuda(np.array([0, 2, 2, 2, 2], np.int32)), k_out=ko))
    want = torch.from_numpy(ref.values(kc.cpu().numpy()[3, :2], 8, D).astype(np.float32)).to(B16)
    assert qg.qgemv_device_error(reset=True) == 0 and torch.equal(ko[:2].cpu(), want) and bool((ko[2:] == 9.0).all())
    qg.qgemv_cache_read(qg.cache_read_args(cache, cuda(table)[:1, :0], cuda(np.array([0, 3], np.int32)), k_out=ko))
    assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
    assert bool((ko[:3] == 0).all()) and bool((ko[3:] == 9.0).all())


ROPE = [
    # tokens, heads, kv heads, dim, rot, layout, input, output, page
    (1, 32, 8, 128, 128, "half", F32, B16, 16),
    (61, 16, 8, 128, 64, "interleaved", H16, H16, 64),
    (33, 3, 3, 96, 20, "half", F32, F32, 7),
    (33, 3, 3, 96, 20, "interleaved", B16, B16, 7),
    (300, 4, 2, 256, 256, "half", F32, H16, 5),
    (5, 0, 2, 64, 32, "half", B16, B16, 16),
    (700, 4, 1, 64, 64, "interleaved", B16, B16, 32),
]


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("keys_out", ["none", "out", "in place"])
@pytest.mark.parametrize("T,H,KH,D,rot,layout,xt,ot,page", ROPE)
def test_rope_into_a_packed_cache(T, H, KH, D, rot, layout, xt, ot, page, keys_out, kind):
    rng = np.random.default_rng(T + rot)
    bits = BITS[kind]
    qkv = torch.from_numpy(rng.standard_normal((T, (H + 2 * KH) * D), dtype=np.float32)).to(xt).cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, KH * D, KH * D], 1))
    k0 = k.double().cpu().numpy()
    pos = rng.integers(-5, 1 << 20, T).astype(np.int32)
    freqs, ms = qg.qgemv_rope_freqs(rot, 10000.0, "linear", 2.0)
    pages = -(-T // page) + 1
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2 + 1::5] = -1
    kc, vc = (rows_of(kind, pages, page, KH, D) for _ in range(2))
    qo = torch.empty(T, H, D, dtype=xt if keys_out == "in place" else ot, device="cuda") if H else None
    ko = {"none": None, "out": torch.empty(T, KH, D, dtype=ot, device="cuda"), "in place": k}[keys_out]
    v0 = v.clone()
    qg.qgemv_rope(qg.rope_args(q if H else None, k, v, cuda(pos), freqs.cuda(), qo, ko, qg.packed_cache(kind, kc, vc, D), cuda(slots),
                               rot, layout, ms))
    live = slots >= 0
    got_k, got_v = (c.cpu().numpy() for c in (kc, vc))
    at = slots[live] // page, slots[live] % page
    n = D * bits // 8 + D // 32 * 4
    assert np.array_equal(got_v[at][..., :n], ref.to_bytes(*ref.pack(f32(v0), bits), bits)[live][..., :n])
    table = [int(x) % 2 ** 64 for x in freqs.tolist()]
    want, mag = turned(k0, pos, table, rot, layout, ms)
    _, d, m = ref.parts(got_k[at], bits, D)
    slack = 16 * 2.0 ** -24 * mag[live]
    step = np.repeat(d.astype(np.float64), 32, -1)
    off = np.abs(ref.values(got_k[at], bits, D) - want[live])
    assert np.all(off <= step / 2 * (1 + 2.0 ** -12) + slack)
    # the step is no larger than the values ask for: the range, its fp32 and two roundings to fp16 on either side
    w = want[live].reshape(*want[live].shape[:-1], -1, 32)
    span = w.max(-1) - w.min(-1) + 2 * slack.reshape(w.shape).max(-1)
    unit = np.maximum(np.abs(w).max(-1) * 2.0 ** -10, 2.0 ** -24)
    assert np.all(d.astype(np.float64) <= (span + unit) / ((1 << bits) - 1) * (1 + 2.0 ** -9) + 2.0 ** -24)
    rest = np.setdiff1d(np.arange(pages * page), slots[live])
    assert np.all(got_k[rest // page, rest % page] == 0xA5) and np.all(got_v[rest // page, rest % page] == 0xA5)
    u = {B16: 2.0 ** -8, H16: 2.0 ** -11, F32: 2.0 ** -24}
    if ko is not None:
        err = np.abs(ko.double().cpu().numpy() - want)
        assert np.all(err <= u[ko.dtype] * np.abs(want) + 2.0 ** -25 + 16 * 2.0 ** -24 * mag)
    if H:
        qw, qm = turned(q.double().cpu().numpy(), pos, table, rot, layout, ms)
        assert np.all(np.abs(qo.double().cpu().numpy() - qw) <= u[qo.dtype] * np.abs(qw) + 2.0 ** -25 + 16 * 2.0 ** -24 * qm)
