"""The operators between the GEMVs, without a GPU: argument checks of rotary positions, attention and sampling, the rotary
frequencies against their formulas, the scratch sizes."""
import ctypes
import glob
import math
import os

import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")

HAS_GPU_NODE = bool(glob.glob("/dev/nvidia[0-9]*")) or os.path.exists("/dev/nvidiactl")
G = 1 << 30  # fake device addresses, far apart: validation never dereferences them
Q, K, V, QO, KO, KC, VC, POS, FREQ, SLOT, SCR, TAB, ST, LEN, LSE = (G * (i + 1) for i in range(15))
F32, BF16, F16 = qg.QGEMV_ACT_F32, qg.QGEMV_ACT_BF16, qg.QGEMV_ACT_F16


@pytest.fixture(scope="module")
def L():
    qg.build()
    return qg.lib()


def cache(**kw):
    c = dict(k=KC, v=VC, k_page=16 * 8 * 128, k_token=8 * 128, k_head=128, v_page=16 * 8 * 128, v_token=8 * 128,
             v_head=128, kind=BF16, num_pages=100, page_size=16, heads=8, dim=128)
    c.update(kw)
    return qg.QgemvCache(**c)


def rope(**kw):
    c = kw.pop("cache", cache())
    a = dict(q=Q, k=K, v=V, q_out=QO, k_out=KO, q_token=4096, q_head=128, k_token=1024, k_head=128, v_token=1024,
             v_head=128, q_out_token=4096, q_out_head=128, k_out_token=1024, k_out_head=128, positions=POS, freqs=FREQ,
             slots=SLOT, x_kind=F32, out_kind=BF16, tokens=5, heads=32, kv_heads=8, dim=128, rot_dim=128, layout=0,
             mscale=1.0)
    a.update(kw)
    s = qg.QgemvRopeArgs(**a)
    if c is not None:
        s.cache = ctypes.pointer(c)
    return s


ROPE_REFUSED = [
    (dict(x_kind=0), 1), (dict(out_kind=7), 1), (dict(layout=2), 1), (dict(tokens=-1), 1), (dict(heads=-1), 1),
    (dict(heads=0), 1),                                  # q without heads
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(cache=None), 1),                               # v and slots without a cache
    (dict(positions=None), 1), (dict(freqs=None), 1), (dict(rot_dim=3), 1), (dict(rot_dim=0), 1), (dict(rot_dim=130), 1),
    (dict(dim=124), 1), (dict(cache=cache(heads=4)), 1), (dict(cache=cache(dim=64)), 1), (dict(cache=cache(kind=F32)), 1),
    (dict(cache=cache(num_pages=0)), 1), (dict(cache=cache(page_size=0)), 1), (dict(cache=cache(k=None)), 1),
    (dict(cache=cache(k_page=-8)), 1), (dict(q_token=-128), 1),
    (dict(dim=264, rot_dim=128, cache=cache(dim=264)), 2), (dict(heads=70000), 2),
    (dict(q=Q + 8), 3), (dict(q_out=QO + 2), 3), (dict(q_token=4100), 3), (dict(k_out_head=129), 3), (dict(positions=POS + 2), 3),
    (dict(freqs=FREQ + 4), 3), (dict(slots=SLOT + 4), 3), (dict(cache=cache(k=KC + 8)), 3), (dict(cache=cache(v_head=4)), 3),
    (dict(q_out=Q), 6),                                  # in place with another type
    (dict(k_out=Q), 6), (dict(q_out=V), 6), (dict(k_out=QO), 6), (dict(cache=cache(k=Q)), 6), (dict(cache=cache(v=QO)), 6),
    (dict(q_out=POS - 64), 6), (dict(cache=cache(k=SLOT - 64)), 6),
    (dict(q=Q, q_out=Q, x_kind=BF16, q_token=4096, q_out_token=8192), 6),  # in place with other strides
]


@pytest.mark.parametrize("case,status", ROPE_REFUSED)
def test_rope_refuses_on_host(L, case, status):
    assert L.qgemv_rope(rope(**case), 0, None) == status


def test_rope_refuses_flags_and_null(L):
    assert L.qgemv_rope(rope(), 2, None) == 1 and L.qgemv_rope(rope(), 8, None) == 1
    assert L.qgemv_rope(None, 0, None) == 1


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
@pytest.mark.parametrize("case", [
    dict(),
    dict(cache=None, v=None, slots=None),                             # rotation only
    dict(k=None, k_out=None, kv_heads=0, cache=None, v=None, slots=None),  # queries only
    dict(q=None, q_out=None, heads=0, k_out=None),                    # keys into the cache only
    # three slices of one qkv row, rotated in place
    dict(q=Q, k=Q + 2 * 4096, v=Q + 2 * 5120, q_out=Q, k_out=Q + 2 * 4096, q_token=6144, k_token=6144, v_token=6144,
         q_out_token=6144, k_out_token=6144, x_kind=BF16, out_kind=BF16),
    dict(q=Q, k=Q + 4 * 4096, v=Q + 4 * 5120, q_token=6144, k_token=6144, v_token=6144),
])
def test_rope_accepts(L, case):
    assert L.qgemv_rope(rope(**case), 0, None) in (4, 5)  # every host check passed; no device here


def test_no_tokens_is_nothing_to_do(L):
    assert L.qgemv_rope(rope(tokens=0), 0, None) == 0
    assert L.qgemv_attn(attn(tokens=0), 0, None) == 0
    assert L.qgemv_attn(attn(seqs=0), 0, None) == 0
    assert L.qgemv_sample(F32, Q, 1000, 0, 1000, None, None, None, None, LEN, TAB, None, 0, None) == 0


def attn(**kw):
    c = kw.pop("cache", cache())
    a = dict(q=Q, out=QO, lse=None, q_token=4096, q_head=128, out_token=4096, out_head=128, pages=TAB, pages_stride=40,
             q_start=ST, kv_len=LEN, scratch=SCR, scratch_bytes=1 << 28, kind=BF16, tokens=6, heads=32, seqs=3, max_q=2,
             max_kv=600, scale=0.088, causal=1, window=0)
    a.update(kw)
    s = qg.QgemvAttnArgs(**a)
    if c is not None:
        s.cache = ctypes.pointer(c)
    return s


ATTN_REFUSED = [
    (dict(kind=F32), 1), (dict(kind=F16), 1), (dict(cache=None), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(pages=None), 1), (dict(q_start=None), 1), (dict(kv_len=None), 1), (dict(scratch=None), 1), (dict(tokens=-1), 1),
    (dict(seqs=-1), 1), (dict(heads=31), 1), (dict(heads=0), 1), (dict(max_q=-1), 1), (dict(max_kv=-1), 1),
    (dict(window=-1), 1), (dict(pages_stride=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=0.0), 1),
    (dict(scale=-0.1), 1),
    (dict(scratch_bytes=qg.QGEMV_ATTN_SCRATCH_HEAD - 1), 1), (dict(q_head=-128), 1),
    (dict(cache=cache(dim=264)), 2), (dict(heads=8 * 10000), 2),
    (dict(q=Q + 2), 3), (dict(out=QO + 8), 3), (dict(out_head=132), 3), (dict(scratch=SCR + 4), 3), (dict(pages=TAB + 2), 3),
    (dict(kv_len=LEN + 1), 3), (dict(lse=LSE + 2), 3), (dict(cache=cache(v=VC + 4)), 3),
    (dict(out=Q), 6), (dict(out=KC), 6), (dict(out=SCR), 6), (dict(lse=QO), 6), (dict(lse=SCR + 64), 6), (dict(scratch=Q - 256), 6),
    (dict(scratch=VC), 6), (dict(out=TAB), 6), (dict(lse=LEN), 6),
]


@pytest.mark.parametrize("case,status", ATTN_REFUSED)
def test_attn_refuses_on_host(L, case, status):
    assert L.qgemv_attn(attn(**case), 0, None) == status


def test_attn_refuses_flags_and_null(L):
    assert L.qgemv_attn(attn(), 2, None) == 1
    assert L.qgemv_attn(None, 0, None) == 1


def test_attn_wants_the_scratch_of_its_sizes(L):
    n = qg.qgemv_attn_scratch_bytes(1, 1, 32, 8, 128, 1, 100000)
    assert n > qg.QGEMV_ATTN_SCRATCH_HEAD
    one = dict(tokens=1, seqs=1, max_q=1, max_kv=100000, pages_stride=6250)
    assert L.qgemv_attn(attn(scratch_bytes=qg.QGEMV_ATTN_SCRATCH_HEAD, **one), 0, None) == 1
    if not HAS_GPU_NODE:
        assert L.qgemv_attn(attn(scratch_bytes=n, **one), 0, None) in (4, 5)


@pytest.mark.parametrize("sizes", [(-1, 1, 32, 8, 128, 1, 1), (1, 1, 32, 0, 128, 1, 1), (1, 1, 30, 8, 128, 1, 1),
                                   (1, 1, 32, 8, 12, 1, 1), (1, 1, 32, 8, 264, 1, 1), (1, 1, 32, 8, 128, 1, -1)])
def test_attn_scratch_of_invalid_sizes(L, sizes):
    assert qg.qgemv_attn_scratch_bytes(*sizes) == 0


def test_attn_scratch_stays_small(L):
    # parts are made only where there are few row tiles: the scratch does not grow with the batch or the prompt
    for seqs, new, ctx in ((1, 1, 1 << 20), (1, 1, 1 << 30), (64, 1, 32768), (4096, 1, 4096), (1, 8192, 8192), (8, 512, 65536),
                           (300, 7, 1 << 17)):
        assert 0 < qg.qgemv_attn_scratch_bytes(seqs, seqs * new, 32, 8, 128, new, ctx) <= 512 << 20


def test_tuning_hook_changes_the_plan_and_back(L):
    sizes = (4, 400, 8, 2, 128, 100, 300)
    plain = qg.qgemv_attn_scratch_bytes(*sizes)
    seen = set()
    for k in (1, 2):
        qg.qgemv_tune_attn(k)
        seen.add(qg.qgemv_attn_scratch_bytes(*sizes))
    qg.qgemv_tune_attn(0)
    assert plain in seen and len(seen) == 2 and qg.qgemv_attn_scratch_bytes(*sizes) == plain


def sample(L, **kw):
    a = dict(kind=F32, x=Q, stride=1000, m=4, n=1000, t=K, k=V, p=QO, mp=KO, u=LEN, token=TAB, prob=ST, flags=0)
    a.update(kw)
    return L.qgemv_sample(a["kind"], a["x"], a["stride"], a["m"], a["n"], a["t"], a["k"], a["p"], a["mp"], a["u"], a["token"],
                          a["prob"], a["flags"], None)


@pytest.mark.parametrize("case,status", [
    (dict(kind=0), 1), (dict(x=None), 1), (dict(u=None), 1), (dict(token=None), 1), (dict(m=-1), 1), (dict(n=0), 1),
    (dict(stride=999), 1), (dict(flags=2), 1), (dict(n=(1 << 20) + 1, stride=1 << 21), 2), (dict(x=Q + 4), 3),
    (dict(u=LEN + 2), 3), (dict(token=TAB + 1), 3), (dict(prob=ST + 2), 3), (dict(t=K + 1), 3), (dict(token=Q), 6),
    (dict(prob=Q + 15996), 6), (dict(token=LEN), 6), (dict(prob=K), 6), (dict(prob=TAB), 6), (dict(token=V + 8), 6),
])
def test_sample_refuses_on_host(L, case, status):
    assert sample(L, **case) == status


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
def test_valid_calls_without_a_gpu(L):
    assert sample(L) in (4, 5) and sample(L, t=None, k=None, p=None, mp=None, prob=None) in (4, 5)
    assert L.qgemv_attn(attn(), 0, None) in (4, 5) and L.qgemv_attn(attn(lse=LSE), qg.QGEMV_FLAG_PDL, None) in (4, 5)


def test_failure_injection_reaches_the_operators(L):
    qg.qgemv_debug_fail_next(4, 4)
    assert L.qgemv_rope(rope(), 0, None) == 4
    assert L.qgemv_attn(attn(), 0, None) == 4
    assert sample(L) == 4
    with pytest.raises(qg.QgemvError):
        qg.qgemv_rope_freqs(128)
    qg.qgemv_debug_fail_next(0, 0)


# ------------------------------------------------------------------------------------------- rotary frequencies

def turns(f):
    return f / (2 * math.pi)


def got(*a, **kw):
    f, ms = qg.qgemv_rope_freqs(*a, **kw)
    return [int(v) / 2.0 ** 64 for v in f], ms


# 64-bit arithmetic throughout (pow, log, one division by 2 pi): a few parts in 2^53, and the last place of 2^-64
def near(a, b):
    return abs(a - b) <= 64 * 2.0 ** -53 * abs(b) + 2.0 ** -63


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (96, 5e5), (128, 1e6), (256, 1.5)])
def test_freqs(rot, theta):
    f, ms = got(rot, theta)
    assert ms == 1.0 and len(f) == rot // 2
    assert all(near(v, turns(theta ** (-2.0 * i / rot))) for i, v in enumerate(f))


def test_freqs_scaled():
    rot, theta, base = 128, 1e6, [1e6 ** (-2.0 * i / 128) for i in range(64)]
    f, ms = got(rot, theta, "linear", 4.0)
    assert ms == 1.0 and all(near(v, turns(b / 4)) for v, b in zip(f, base))
    f, ms = got(rot, theta, "base", 4.0)  # the fastest pair is kept, the slowest is slowed by the factor
    assert ms == 1.0 and near(f[0], turns(1.0)) and near(f[-1], turns(base[-1] / 4))
    f, ms = got(rot, theta, "parts", 4.0, trained=32768.0, low=1.0, high=32.0)
    assert abs(ms - (0.1 * math.log(4.0) + 1)) < 1e-6
    for v, b in zip(f, base):
        n = 32768.0 * turns(b)  # turns over the trained positions
        assert turns(b / 4) * (1 - 1e-12) <= v <= turns(b) * (1 + 1e-12)
        if n > 40:
            assert near(v, turns(b))
        if n < 0.7:
            assert near(v, turns(b / 4))
    f, ms = got(rot, theta, "bands", 8.0, trained=8192.0, low=1.0, high=4.0)
    assert ms == 1.0
    for v, b in zip(f, base):
        n = 8192.0 * turns(b)
        g = min(1.0, max(0.0, (n - 1) / 3))
        assert near(v, turns(b * g + b / 8 * (1 - g)))


@pytest.mark.parametrize("a", [(0, 1e4, 0, 1, 1, 1, 2), (3, 1e4, 0, 1, 1, 1, 2), (258, 1e4, 0, 1, 1, 1, 2), (64, 1.0, 0, 1, 1, 1, 2),
                               (64, float("nan"), 0, 1, 1, 1, 2), (64, 1e4, 5, 1, 1, 1, 2), (64, 1e4, 1, 0.5, 1, 1, 2),
                               (2, 1e4, 2, 2, 1, 1, 2), (64, 1e4, 3, 2, 0, 1, 2), (64, 1e4, 3, 2, 1, 2, 2),
                               (64, 1e4, 4, 2, 1, 0, 2), (64, 1e4, 4, 2, 1, 3, 2)])
def test_freqs_refuses(L, a):
    out = (ctypes.c_ulonglong * 256)()
    assert L.qgemv_rope_freqs(*a, out, None) == 1
    assert L.qgemv_rope_freqs(64, 1e4, 0, 1, 1, 1, 2, None, None) == 1


def test_binding_refuses_unlike_tensors():
    x = torch.zeros(3, 4, 64)
    with pytest.raises(qg.QgemvError):
        qg.kv_cache(x, x)
    with pytest.raises(qg.QgemvError):
        qg.rope_args(x.transpose(1, 2), None, None, torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    with pytest.raises(qg.QgemvError):
        qg.rope_args(x, None, None, torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.int64), q_out=x)
    with pytest.raises(qg.QgemvError):
        qg.rope_args(x, None, None, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64), q_out=x)
    with pytest.raises(qg.QgemvError):
        qg.qgemv_sample(torch.zeros(2, 8, dtype=torch.float64), None, None, None, None, torch.zeros(2),
                        torch.zeros(2, dtype=torch.int32))
    with pytest.raises(qg.QgemvError):
        qg.qgemv_sample(torch.zeros(2, 8), None, None, None, None, torch.zeros(3), torch.zeros(2, dtype=torch.int32))
