"""Edges of the operators between the GEMVs without a GPU: sizes at the ends of the arithmetic, the scratch over all sizes, what
the binding takes."""
import itertools

import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")

from tests.test_step_host import HAS_GPU_NODE, KC, Q, QO, L, attn, cache, rope, sample  # noqa: E402,F401

HUGE, MANY = 1 << 40, 2 ** 31 - 1


# strides and sizes that are each allowed, but whose product leaves 64 bits: the memory a tensor spans cannot be told then, and
# an overlap went unseen
@pytest.mark.parametrize("case", [
    dict(q_token=HUGE, tokens=MANY), dict(q_out_token=HUGE, tokens=MANY), dict(k_token=HUGE, tokens=1 << 24),
    dict(v_token=HUGE, tokens=1 << 24), dict(cache=cache(k_page=HUGE, num_pages=1 << 24)), dict(cache=cache(v_page=HUGE, num_pages=MANY)),
    dict(cache=cache(k_token=HUGE, page_size=1 << 24)), dict(cache=cache(v_token=HUGE, page_size=MANY)),
])
def test_rope_refuses_spans_past_64_bits(L, case):  # noqa: F811
    assert L.qgemv_rope(rope(**case), 0, None) == 2


@pytest.mark.parametrize("case", [
    dict(q_token=HUGE, tokens=MANY), dict(out_token=HUGE, tokens=1 << 24), dict(seqs=MANY, pages_stride=HUGE),
    dict(pages_stride=HUGE + 1), dict(cache=cache(k_page=HUGE, num_pages=MANY)), dict(cache=cache(k_token=HUGE, page_size=MANY)),
    dict(cache=cache(v_token=HUGE, page_size=1 << 24)),
])
def test_attn_refuses_spans_past_64_bits(L, case):  # noqa: F811
    assert L.qgemv_attn(attn(**case), 0, None) == 2


def test_sample_refuses_spans_past_64_bits(L):  # noqa: F811
    assert sample(L, m=MANY, stride=HUGE) == 2
    assert sample(L, m=1 << 24, stride=HUGE) == 2


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
def test_large_strides_of_small_tensors_are_taken(L):  # noqa: F811
    assert L.qgemv_attn(attn(cache=cache(k=1 << 50, v=3 << 50, k_page=1 << 38, v_page=1 << 38)), 0, None) in (4, 5)
    # only what a row of the page table has to hold counts as read, not its whole stride
    assert L.qgemv_attn(attn(pages=KC + (1 << 29), pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) in (4, 5)
    assert L.qgemv_attn(attn(pages=QO - 256, pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) in (4, 5)
    assert L.qgemv_attn(attn(pages=QO - 148, pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) == 6


# ------------------------------------------------------------------------------------------------------- the scratch

SEQS, NEW, CONTEXT = (1, 2, 7, 48, 300), (1, 2, 8, 9, 16, 64, 250, 1056, 2000, 8192), (0, 1, 600, 4096, 24000, 32768, 131072, 1 << 20)


@pytest.fixture(params=[0, 1, 2], ids=["planned", "16-row", "128-row"])
def hook(request):
    qg.qgemv_tune_attn(request.param)
    yield
    qg.qgemv_tune_attn(0)


@pytest.mark.parametrize("heads,kv_heads,dim", [(32, 8, 128), (16, 8, 64), (8, 1, 96), (4, 4, 256)])
def test_scratch_never_falls_as_a_size_grows(L, hook, heads, kv_heads, dim):  # noqa: F811
    size = {(s, n, c): qg.qgemv_attn_scratch_bytes(s, s * n, heads, kv_heads, dim, n, c)
            for s, n, c in itertools.product(SEQS, NEW, CONTEXT)}
    assert min(size.values()) >= qg.QGEMV_ATTN_SCRATCH_HEAD
    for (s, n, c), v in size.items():
        for axis, steps in enumerate((SEQS, NEW, CONTEXT)):
            at = (s, n, c)[axis]
            if at != steps[-1]:
                up = [s, n, c]
                up[axis] = steps[steps.index(at) + 1]
                assert size[tuple(up)] >= v, (s, n, c, up)


def test_scratch_never_falls_from_one_length_to_the_next(L):  # noqa: F811
    for new in (9, 40, 64, 500, 1000, 1056, 1250, 2000):
        sizes = [qg.qgemv_attn_scratch_bytes(1, new, 32, 8, 128, new, c) for c in range(0, 1 << 19, 512)]
        assert sizes == sorted(sizes)
    for context in (3000, 24000, 131072):
        sizes = [qg.qgemv_attn_scratch_bytes(1, n, 32, 8, 128, n, context) for n in range(1, 3000)]
        assert sizes == sorted(sizes)
        sizes = [qg.qgemv_attn_scratch_bytes(b, b * 40, 32, 8, 128, 40, context) for b in range(1, 400)]
        assert sizes == sorted(sizes)


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
@pytest.mark.parametrize("dim", [64, 128])
def test_scratch_of_the_largest_call_serves_the_smaller_ones(L, hook, dim):  # noqa: F811
    one = cache(dim=dim, num_pages=1000)
    for seqs, new, context in ((4, 8192, 131072), (1, 4864, 32768), (48, 16, 16384), (1, 2000, 24000)):
        n = qg.qgemv_attn_scratch_bytes(seqs, seqs * new, 32, 8, dim, new, context)
        for s, q, c in itertools.product(SEQS, (1, 2, 9, 17, 100, 130, 257, 1024, 1056, 2048, 4864, 8192), (1, 300, 2048, 9999, 24000, 32768, 131072)):
            if s <= seqs and q <= new and c <= context:
                for tokens in {s * q, s + q - 1}:  # every sequence's, and one long one beside single tokens
                    call = attn(cache=one, tokens=tokens, seqs=s, max_q=q, max_kv=c, pages_stride=8192, scratch_bytes=n,
                                q_token=32 * dim, q_head=dim, out_token=32 * dim, out_head=dim, scratch=1 << 45)
                    assert L.qgemv_attn(call, 0, None) in (4, 5), (seqs, new, context, s, q, c)


# ------------------------------------------------------------------------------------------------------- the binding

def record(pages, max_kv, scratch=None):
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    kv = qg.kv_cache(*(torch.zeros(30, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))
    scratch = torch.zeros(1 << 20, dtype=torch.uint8) if scratch is None else scratch
    return qg.attn_args(q, kv, pages, torch.zeros(pages.shape[0] + 1, dtype=torch.int32), torch.zeros(pages.shape[0], dtype=torch.int32),
                        torch.empty_like(q), scratch, 1, max_kv, 0.1)


def test_binding_takes_a_view_of_a_longer_page_table():
    table = torch.zeros(5, 64, dtype=torch.int32)
    a = record(table[:, 3:13], 1000)
    assert (a.pages, a.pages_stride, a.seqs, a.max_kv) == (table.data_ptr() + 12, 64, 5, 160)
    assert record(table[:, :13], 100).max_kv == 100
    a = record(table, 2000)
    assert (a.pages_stride, a.max_kv) == (64, 1024)
    a = record(table[2:3, :7], 2000)  # a single row: no stride is needed
    assert (a.pages_stride, a.max_kv) == (7, 112)
    a = record(table[:, :0], 2000)
    assert (a.pages_stride, a.max_kv) == (0, 0)
    for bad in (table.t(), table[0].expand(5, 64), table.long(), table[0]):
        with pytest.raises(qg.QgemvError):
            record(bad, 100)


def test_binding_wants_a_contiguous_scratch():
    with pytest.raises(qg.QgemvError):
        record(torch.zeros(5, 64, dtype=torch.int32), 100, torch.zeros(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(qg.QgemvError):
        record(torch.zeros(5, 64, dtype=torch.int32), 100, torch.zeros(1 << 21, dtype=torch.uint8)[::2])


def test_binding_does_nothing_for_empty_tensors():
    """A step without tokens: empty tensors have no address."""
    none = lambda *n, dtype=torch.bfloat16: torch.empty(*n, dtype=dtype)  # noqa: E731
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    kv = qg.kv_cache(*(torch.zeros(30, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))
    q, k = none(0, 4, 64), none(0, 2, 64)
    assert q.data_ptr() == 0
    freqs = torch.zeros(32, dtype=torch.int64)
    qg.qgemv_rope(qg.rope_args(q, k, k, i32(0), freqs, none(0, 4, 64), none(0, 2, 64), kv, torch.zeros(0, dtype=torch.int64)), stream=0)
    qg.qgemv_rope(qg.rope_args(q, None, None, i32(0), freqs, none(0, 4, 64)), stream=0)
    scratch = torch.zeros(qg.qgemv_attn_scratch_bytes(3, 0, 4, 2, 64, 0, 100), dtype=torch.uint8)
    args = lambda table, starts, lens: qg.attn_args(q, kv, table, starts, lens, none(0, 4, 64), scratch, 0, 100, 0.1, lse=none(0, 4, dtype=torch.float32))  # noqa: E731
    qg.qgemv_attn(args(i32(3, 7), i32(4), i32(3)), stream=0)  # sequences, but no new tokens
    qg.qgemv_attn(args(i32(0, 7), i32(1), i32(0)), stream=0)  # no sequences
    f32 = none(0, dtype=torch.float32)
    qg.qgemv_sample(none(0, 1000), f32, i32(0), f32, f32, f32, i32(0), f32, stream=0)
    with pytest.raises(qg.QgemvError):
        qg.qgemv_sample(none(0, 0), f32, i32(0), f32, f32, f32, i32(0), f32, stream=0)


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
def test_a_page_table_without_columns_needs_no_address(L):  # noqa: F811
    assert L.qgemv_attn(attn(pages=None, pages_stride=0), 0, None) in (4, 5)  # tokens that see nothing
    assert L.qgemv_attn(attn(pages=None, pages_stride=0, tokens=0), 0, None) == 0


def test_empty_calls_are_checked_as_far_as_they_go(L):  # noqa: F811
    assert L.qgemv_rope(rope(tokens=0, q=None, k=None, v=None, q_out=None, k_out=None, positions=None, slots=None), 0, None) == 0
    assert L.qgemv_rope(rope(tokens=0, rot_dim=3), 0, None) == 1 and L.qgemv_rope(rope(tokens=0, layout=5), 0, None) == 1
    assert L.qgemv_attn(attn(tokens=0, scratch=None), 0, None) == 1 and L.qgemv_attn(attn(seqs=0, scale=0.0), 0, None) == 1
    assert L.qgemv_attn(attn(tokens=0, cache=None), 0, None) == 1
    assert sample(L, m=0, kind=0) == 1 and sample(L, m=0, x=None, u=None, token=None) == 0 and sample(L, m=0, stride=999) == 1
