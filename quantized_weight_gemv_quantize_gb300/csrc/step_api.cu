// C ABI of the operators between the GEMVs: rotary positions, attention over the paged cache, sampling.  Every check
// runs on the host before anything is enqueued.
#include <cuda.h>
#include <atomic>
#include <limits.h>
#include <math.h>
#include <mutex>
#include <stddef.h>

#include "../../include/qgemv.h"
#include "internal.h"
#include "step.h"

namespace qg {

static int elem_size(int kind) {
    return kind == QGEMV_ACT_F32 ? 4 : kind == QGEMV_ACT_BF16 || kind == QGEMV_ACT_F16 ? 2 : 0;
}

// Elements that a tensor may span: beyond any memory, and its bytes and addresses stay within 64 bits.
constexpr double SPAN_MAX = 9e15;

// A tensor [n0, n1, dim] with strides s0, s1 (elements of `size` bytes), as the memory it covers.
struct Region {
    const void* p;
    long long n0, s0, n1, s1, dim;
    int size;
    size_t bytes() const {
        if (n0 < 1 || n1 < 1) return 0;
        return static_cast<size_t>((n0 - 1) * s0 + (n1 - 1) * s1 + dim) * size;
    }
    // Strides in range (each up to 2^40, and the span that they and the sizes make), rows at multiples of 16 bytes and `step` elements.
    int check(int step) const {
        if (s0 < 0 || s1 < 0 || s0 > (1ll << 40) || s1 > (1ll << 40)) return QGEMV_ERR_INVALID_ARG;
        if ((s0 * size) % 16 || (s1 * size) % 16 || s0 % step || s1 % step || !api_aligned(p, 16)) return QGEMV_ERR_MISALIGNED;
        if (static_cast<double>(n0) * static_cast<double>(s0) + static_cast<double>(n1) * static_cast<double>(s1) > SPAN_MAX)
            return QGEMV_ERR_UNSUPPORTED;
        return QGEMV_OK;
    }
};

// Whether two tensors may share a byte.  Ranges that are apart do not; two that are slices of one buffer with the same
// outer stride do not when their spans within that stride are apart.  Anything else counts as an overlap.
static bool meet(const Region& a, const Region& b) {
    if (!a.p || !b.p || !a.bytes() || !b.bytes()) return false;
    if (!api_overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
    const long long stride = a.s0 * a.size;
    if (a.n0 > 1 && b.n0 > 1 && stride == b.s0 * b.size) {
        const long long wa = ((a.n1 - 1) * a.s1 + a.dim) * a.size, wb = ((b.n1 - 1) * b.s1 + b.dim) * b.size;
        if (wa <= stride && wb <= stride) {
            const long long d = static_cast<long long>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
            const long long at = ((d % stride) + stride) % stride;
            return !(at >= wa && at + wb <= stride);
        }
    }
    return true;
}

static bool same(const Region& a, const Region& b) {
    return a.p == b.p && a.s0 == b.s0 && a.s1 == b.s1 && a.size == b.size && a.n1 == b.n1;
}

// A cache as two regions of pages: [num_pages, the span of a page].
static size_t cache_bytes(const qgemv_cache& c, long long page, long long token, long long head) {
    return static_cast<size_t>((c.num_pages - 1) * page + (c.page_size - 1) * token + (c.heads - 1) * head + c.dim) * 2;
}

static int check_cache(const qgemv_cache* c) {
    if (!c->k || !c->v) return QGEMV_ERR_INVALID_ARG;
    if (c->kind != QGEMV_ACT_BF16 && c->kind != QGEMV_ACT_F16) return QGEMV_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->dim < 8 || c->dim % 8) return QGEMV_ERR_INVALID_ARG;
    if (c->dim > 256) return QGEMV_ERR_UNSUPPORTED;
    const long long s[6] = {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head};
    for (long long v : s) {
        if (v < 0 || v > (1ll << 40)) return QGEMV_ERR_INVALID_ARG;
        if (v % 8) return QGEMV_ERR_MISALIGNED;
    }
    for (int i = 0; i < 6; i += 3)  // no offset of the kernels' arithmetic leaves 64 bits
        if (static_cast<double>(c->num_pages) * static_cast<double>(s[i]) + static_cast<double>(c->page_size) * static_cast<double>(s[i + 1]) +
                static_cast<double>(c->heads) * static_cast<double>(s[i + 2]) > SPAN_MAX)
            return QGEMV_ERR_UNSUPPORTED;
    if (!api_aligned(c->k, 16) || !api_aligned(c->v, 16)) return QGEMV_ERR_MISALIGNED;
    return QGEMV_OK;
}

// ---------------------------------------------------------------------------------------------- rotary positions

static int run_rope(const qgemv_rope_args* a, unsigned flags, void* stream) {
    if (!a || (flags & ~QGEMV_FLAG_PDL)) return QGEMV_ERR_INVALID_ARG;
    const int xs = elem_size(a->x_kind), os = elem_size(a->out_kind);
    if (!xs || !os) return QGEMV_ERR_INVALID_ARG;
    if (a->layout != QGEMV_ROPE_HALF && a->layout != QGEMV_ROPE_INTERLEAVED) return QGEMV_ERR_INVALID_ARG;
    if (a->tokens < 0 || a->heads < 0 || a->kv_heads < 0 || a->heads + static_cast<long long>(a->kv_heads) < 1)
        return QGEMV_ERR_INVALID_ARG;
    if (a->dim < 8 || a->dim % 8 || a->rot_dim < 2 || a->rot_dim % 2 || a->rot_dim > a->dim) return QGEMV_ERR_INVALID_ARG;
    if (a->dim > 256 || a->heads > 65536 || a->kv_heads > 65536) return QGEMV_ERR_UNSUPPORTED;
    if (a->tokens == 0) return QGEMV_OK;  // (empty tensors may have no address)
    if (!a->positions || !a->freqs) return QGEMV_ERR_INVALID_ARG;
    const bool has_q = a->heads > 0, has_k = a->kv_heads > 0, has_c = a->cache != nullptr;
    if (has_q != (a->q != nullptr) || has_q != (a->q_out != nullptr) || has_k != (a->k != nullptr)) return QGEMV_ERR_INVALID_ARG;
    if (has_c != (a->v != nullptr) || has_c != (a->slots != nullptr)) return QGEMV_ERR_INVALID_ARG;
    if ((has_k && !a->k_out && !has_c) || (!has_k && (a->k_out || has_c))) return QGEMV_ERR_INVALID_ARG;
    int st;
    if (has_c) {
        if ((st = check_cache(a->cache))) return st;
        if (a->cache->heads != a->kv_heads || a->cache->dim != a->dim) return QGEMV_ERR_INVALID_ARG;
    }
    const long long T = a->tokens;
    const Region q = {a->q, T, a->q_token, a->heads, a->q_head, a->dim, xs};
    const Region k = {a->k, T, a->k_token, a->kv_heads, a->k_head, a->dim, xs};
    const Region v = {a->v, T, a->v_token, a->kv_heads, a->v_head, a->dim, xs};
    const Region qo = {a->q_out, T, a->q_out_token, a->heads, a->q_out_head, a->dim, os};
    const Region ko = {a->k_out, T, a->k_out_token, a->kv_heads, a->k_out_head, a->dim, os};
    const Region* all[5] = {&q, &k, &v, &qo, &ko};
    for (const Region* r : all) {
        if (!r->p) continue;
        if ((st = r->check(8))) return st;
    }
    if (!api_aligned(a->positions, 4) || !api_aligned(a->freqs, 8) || (a->slots && !api_aligned(a->slots, 8)))
        return QGEMV_ERR_MISALIGNED;
    const size_t nf = static_cast<size_t>(a->rot_dim / 2) * 8, np = static_cast<size_t>(T) * 4, ns = static_cast<size_t>(T) * 8;
    const Region* outs[2] = {&qo, &ko};
    for (const Region* o : outs) {
        if (!o->p) continue;
        const Region* own = o == &qo ? &q : &k;
        for (const Region* in : {&q, &k, &v})
            if (meet(*o, *in) && !(in == own && same(*o, *in) && a->x_kind == a->out_kind)) return QGEMV_ERR_OVERLAP;
        if (api_overlaps(o->p, o->bytes(), a->positions, np) || api_overlaps(o->p, o->bytes(), a->freqs, nf) ||
            (a->slots && api_overlaps(o->p, o->bytes(), a->slots, ns)))
            return QGEMV_ERR_OVERLAP;
    }
    if (meet(qo, ko)) return QGEMV_ERR_OVERLAP;
    if (has_c) {
        const qgemv_cache& c = *a->cache;
        const size_t kb = cache_bytes(c, c.k_page, c.k_token, c.k_head), vb = cache_bytes(c, c.v_page, c.v_token, c.v_head);
        for (const Region* r : all)
            if (r->p && (api_overlaps(c.k, kb, r->p, r->bytes()) || api_overlaps(c.v, vb, r->p, r->bytes())))
                return QGEMV_ERR_OVERLAP;
        const void* side[3] = {a->positions, a->freqs, a->slots};
        const size_t size[3] = {np, nf, ns};
        for (int i = 0; i < 3; ++i)
            if (api_overlaps(c.k, kb, side[i], size[i]) || api_overlaps(c.v, vb, side[i], size[i])) return QGEMV_ERR_OVERLAP;
    }
    int sms;
    unsigned* err;
    if ((st = api_device(&sms, &err))) return st;
    RopeArgs r = {};
    r.q = a->q, r.k = a->k, r.v = a->v, r.q_out = a->q_out, r.k_out = a->k_out;
    r.q_token = a->q_token, r.q_head = a->q_head, r.k_token = a->k_token, r.k_head = a->k_head;
    r.v_token = a->v_token, r.v_head = a->v_head;
    r.q_out_token = a->q_out_token, r.q_out_head = a->q_out_head, r.k_out_token = a->k_out_token, r.k_out_head = a->k_out_head;
    r.positions = a->positions, r.freqs = a->freqs, r.slots = a->slots, r.err = err;
    r.out_kind = a->out_kind, r.tokens = a->tokens, r.heads = a->heads, r.kv_heads = a->kv_heads;
    r.dim = a->dim, r.rot = a->rot_dim, r.mscale = a->mscale, r.page_size = 1;
    if (has_c) {
        const qgemv_cache& c = *a->cache;
        r.k_cache = c.k, r.v_cache = c.v, r.cache_kind = c.kind;
        r.kc_page = c.k_page, r.kc_token = c.k_token, r.kc_head = c.k_head;
        r.vc_page = c.v_page, r.vc_token = c.v_token, r.vc_head = c.v_head;
        r.page_size = c.page_size, r.num_slots = static_cast<long long>(c.num_pages) * c.page_size;
    }
    const bool half = a->layout == QGEMV_ROPE_HALF, vec = a->rot_dim % (half ? 16 : 8) == 0;
    // Blocks of a token: as many as its pieces fill once, until the tokens alone fill the GPU.
    const int w = vec ? 8 : 1;
    const long long per_token = static_cast<long long>(a->heads + 2 * a->kv_heads) * a->dim / w;
    long long y = (per_token + ROPE_THREADS - 1) / ROPE_THREADS;
    const long long enough = (32ll * sms + T - 1) / T;
    if (y > enough) y = enough;
    const bool pdl = (flags & QGEMV_FLAG_PDL) != 0;
    cudaError_t e = launch_step(rope_kernel_ptr(a->x_kind, half, vec), dim3(static_cast<unsigned>(T), static_cast<unsigned>(y)),
                                ROPE_THREADS, 0, 1, pdl, static_cast<cudaStream_t>(stream), r);
    if (e != cudaSuccess) return api_cuda_fail(e);
    api_route(QGEMV_ROUTE_ROPE, pdl);
    return QGEMV_OK;
}

// ---------------------------------------------------------------------------------------------------- attention

static std::atomic<int> g_attn_kernel{0};

static size_t round32(size_t n) { return (n + 31) / 32 * 32; }

constexpr int SMS = 152;

// Parts that row tiles may be cut into, all together: as many waves of blocks as half the square root of the context's key tiles, at most
// 16.  A wave costs its start and end, some 3 key tiles, so that more of them win nothing by the estimate below (the limit moves
// nothing by more than 0.01 us, for 1 to 4000 row tiles over 8 to 2^23 key tiles); it bounds the scratch.
static long long parts_max(long long blocks) {
    const long long waves = static_cast<long long>(ceil(sqrt(static_cast<double>(blocks)) / 2));
    return (waves < 16 ? waves : 16) * SMS;
}
// Blocks of the 16-row kernel: one wave, two an SM (one with the larger shared memory of long heads); each has records of 16 rows for two
// parts of split row tiles.
static int rows_grid(int dim) { return dim <= 128 ? 2 * SMS : SMS; }
static size_t scratch_of(size_t records, int dim) {
    return QGEMV_ATTN_SCRATCH_HEAD + round32(records * sizeof(float2)) + records * dim * sizeof(float);
}

static int attn_plan(int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv, int window,
                     AttnPlan* p) {
    if (seqs < 0 || tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || dim < 8 || dim % 8 || max_q < 0 ||
        max_kv < 0)
        return QGEMV_ERR_INVALID_ARG;
    if (dim > 256 || heads > 65536) return QGEMV_ERR_UNSUPPORTED;
    *p = AttnPlan{};
    p->scratch = p->scratch_most = QGEMV_ATTN_SCRATCH_HEAD;
    if (seqs == 0 || tokens == 0 || max_q == 0) return QGEMV_OK;
    if (max_q > tokens) max_q = tokens;
    const long long rows = static_cast<long long>(max_q) * (heads / kv_heads);
    if (max_kv > 1 << 30 || (rows + 15) / 16 * kv_heads > INT_MAX || rows > INT_MAX) return QGEMV_ERR_UNSUPPORTED;
    // Keys that a row tile goes over: the context, or with a window that of its first token to that of its last and what the rounding of the
    // range adds.  (The 128-row kernel's parts rely on it.)
    auto keys_of = [&](int tile, int step) {
        const int group = heads / kv_heads, later = (tile - 1) / group + 1, span = max_q - 1 < later ? max_q - 1 : later;
        const long long keys = static_cast<long long>(window) + span + step - 1;
        return window > 0 && keys < max_kv ? static_cast<int>(keys) : max_kv;
    };
    const int keys = keys_of(256, 128);
    // The 128-row kernel: 256 rows a block, one block an SM, the row tiles' contexts in n parts.  Its time in us: 9 for the launch, start and
    // end; waves of blocks, each as long as its part and about 3 key tiles for its start and end, at 1.4 a key tile; where parts are joined, 4
    // for the second kernel and their records, written and read at 5 TB/s.  Measured and by this rule: 32 and 8 heads of 128, 2000 tokens over 24000,
    // n = 1: 542 / 544, n = 2: 591 / 583, 4: 578 / 557, 8: 640 / 650; 1000 over 30000, n = 1: 346 / 342, 2: 375 / 365, 8: 405 / 390; 256 over 16000,
    // n = 1: 182 / 188, 4: 64 / 69, 8: 74 / 80; 64 over 4000, n = 1: 56 / 58, 4: 30 / 30.  At most 32 parts of at least 8 key tiles.
    const long long tiles = (rows + 255) / 256 * kv_heads * seqs, blocks = (static_cast<long long>(keys) + 127) / 128;
    // Or the row tiles that fill whole waves stay whole and only the rest is cut (1300 tokens over 30000: 492 us with all cut alike, 419;
    // 1500 over 20000: 368, 331; 2000 over 24000: no difference beyond that between GPUs).
    // All of these, and the choice of kernel below, were fitted at heads of 128 and 152 SMs; heads of 64 and 96 take much the same time in
    // the 128-row kernel (2000 over 8000: 164, 171 and 174 us at 64, 96 and 128), where the softmax sets the pace.
    const long long full = tiles / SMS * SMS;
    long long best = 1, best_whole = 0;
    double tiles_us = 0;
    for (long long n = 1; n <= 32 && (n == 1 || (n * 8 <= blocks && tiles <= INT_MAX)); ++n)
        for (const long long whole : {0ll, full}) {
            if (whole > 0 && (n == 1 || whole == tiles)) continue;
            if (n > 1 && (tiles - whole) * n > parts_max(blocks)) continue;
            const double part = static_cast<double>((blocks + n - 1) / n);
            const double waves = static_cast<double>(((tiles - whole) * n + SMS - 1) / SMS);
            const double records = n > 1 ? 8e-6 / 5 * static_cast<double>((tiles - whole) * n * (rows < 256 ? rows : 256) * dim) : 0;
            const double us = 9 + 1.4 * (waves * (part + 3) + static_cast<double>(whole / SMS * (blocks + 3))) + (n > 1 ? 4 + records : 0);
            if (n == 1 || us < tiles_us) best = n, best_whole = whole, tiles_us = us;
        }
    // Which kernel, for more than 32 rows (and heads of up to 128, which the 128-row kernel is built for): by what both would take, in us.  The
    // 16-row kernel goes over the keys once for 16 rows, 19 row tiles and keys a ns; over sequences of uneven length its time is their sum's, the
    // other's the longest's.  Measured, 8 key/value heads, 16-row against 128-row kernel in us: 64 rows over 4000 keys 18.5 / 26.7, 128 rows 24.6 / 27.9,
    // 256 rows 39.0 / 32.8; over 50000 keys 32 rows 51.2 / 52.4, 64 rows 84.5 / 53.0; 16 sequences of up to 8000: 32 rows 63.5 / 93.8, 48 rows
    // 78.7 / 94.4, 64 rows 141 / 94; 4 sequences of 300 with 64 tokens 18.5 / 18.5; 128 tokens alone 9.0 / 18.5, 256 over 1000 37.2 / 26.7.
    // With a window of 1024 over 24000 keys 24 tokens 11.7 / 22.6, 128 tokens 20.5 / 26.7, 500 tokens 65.2 / 31.0.
    const double keys16 = static_cast<double>((rows + 15) / 16) * kv_heads * seqs * keys_of(16, 16);
    const double rows_us = 8 + keys16 / 19000 * (seqs > 1 ? 0.75 : 1.0);
    const int forced = g_attn_kernel.load(std::memory_order_relaxed);
    p->tiles = dim <= 128 && (forced ? forced == 2 : rows > 32 && tiles_us < rows_us);
    size_t records = 0;
    if (!p->tiles) {
        p->grid = rows_grid(dim);
        records = static_cast<size_t>(p->grid) * 2 * 16;
        // Units of 64 keys, longer ones where the bounds alone would let the whole (twice over, for its rounding) pass 32 bits.
        const double row_tiles = static_cast<double>((rows + 15) / 16) * kv_heads * seqs;
        p->unit_shift = 6;
        while (p->unit_shift < 30 && row_tiles * (static_cast<double>(max_kv >> p->unit_shift) + 1) > 1e9) ++p->unit_shift;
        if (row_tiles > 1e9) return QGEMV_ERR_UNSUPPORTED;
    } else {
        if (tiles > INT_MAX) return QGEMV_ERR_UNSUPPORTED;
        p->row_tiles = static_cast<int>((rows + 255) / 256);
        p->rows_part = static_cast<int>(rows < 256 ? rows : 256);
        const long long chunk = ((keys + best - 1) / best + 127) / 128 * 128;
        p->chunk = static_cast<int>(chunk < 128 ? 128 : chunk);
        p->parts = keys > 0 ? static_cast<int>((static_cast<long long>(keys) + p->chunk - 1) / p->chunk) : 1;
        p->whole = p->parts > 1 ? static_cast<int>(best_whole) : 0;
        p->grid = p->whole + (tiles - p->whole) * p->parts;
        if (p->grid > INT_MAX) return QGEMV_ERR_UNSUPPORTED;
        if (p->parts > 1) records = static_cast<size_t>(p->grid - p->whole) * p->rows_part;
    }
    p->records = records;
    p->scratch = scratch_of(records, dim);
    // What every call of these sizes or smaller ones is content with: the choices above do not grow with the sizes, these bounds do.
    size_t most = dim <= 128 && forced == 2 ? 0 : static_cast<size_t>(rows_grid(dim)) * 2 * 16;
    if (dim <= 128 && (forced ? forced == 2 : rows > 32) && blocks >= 16) {
        const long long n = blocks / 8 < 32 ? blocks / 8 : 32, limit = parts_max(blocks);
        const long long parts = tiles < limit && tiles * n < limit ? tiles * n : limit;
        const size_t cut = static_cast<size_t>(parts) * (rows < 256 ? rows : 256);
        if (cut > most) most = cut;
    }
    p->scratch_most = scratch_of(most, dim);
    return QGEMV_OK;
}

// Dynamic shared memory of a kernel, set once per device.
static int allow_smem(const void* fn, unsigned smem) {
    static std::mutex mu;
    static const void* done[64][16];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return api_cuda_fail(e);
    if (dev < 0 || dev >= 64) return QGEMV_ERR_DEVICE;
    std::lock_guard<std::mutex> lk(mu);
    for (const void*& f : done[dev]) {
        if (f == fn) return QGEMV_OK;
        if (f) continue;
        if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) != cudaSuccess)
            return api_cuda_fail(e);
        f = fn;
        return QGEMV_OK;
    }
    return QGEMV_ERR_UNSUPPORTED;
}

// Tensor map of 16-bit elements with 64 of them to a row of a box, in the 128-byte swizzle; strides in elements.  False where the
// tensor cannot be described by one (then the kernel copies row by row).  Host arithmetic of the driver, about a microsecond.
static bool tensor_map(unsigned long long (&map)[16], const void* base, int kind, const long long (&size)[4], const long long (&stride)[3],
                       const int (&box)[4]) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    static_assert(sizeof(CUtensorMap) == sizeof(map), "");
    cuuint64_t dims[4], strides[3];
    cuuint32_t boxes[4];
    for (int i = 0; i < 4; ++i) dims[i] = static_cast<cuuint64_t>(size[i]), boxes[i] = static_cast<cuuint32_t>(box[i]);
    for (int i = 0; i < 3; ++i) {
        // (a dimension of one element is never stepped over: any valid stride will do)
        const long long s = size[i + 1] > 1 ? stride[i] : size[0];
        if (s <= 0 || s >= 1ll << 38 || s % 8) return false;
        strides[i] = static_cast<cuuint64_t>(s) * 2;
    }
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(reinterpret_cast<CUtensorMap*>(map),
                  kind == QGEMV_ACT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int run_attn(const qgemv_attn_args* a, unsigned flags, void* stream) {
    if (!a || (flags & ~QGEMV_FLAG_PDL)) return QGEMV_ERR_INVALID_ARG;
    if (a->kind != QGEMV_ACT_BF16 && a->kind != QGEMV_ACT_F16) return QGEMV_ERR_INVALID_ARG;
    if (!a->cache || !a->scratch) return QGEMV_ERR_INVALID_ARG;
    if (a->tokens != 0 && a->seqs != 0) {  // (empty tensors may have no address)
        if (!a->q || !a->out || !a->q_start || !a->kv_len) return QGEMV_ERR_INVALID_ARG;
        if (!a->pages && a->pages_stride != 0) return QGEMV_ERR_INVALID_ARG;
    }
    int st;
    if ((st = check_cache(a->cache))) return st;
    const qgemv_cache& c = *a->cache;
    if (c.kind != a->kind || a->tokens < 0 || a->seqs < 0 || a->pages_stride < 0 || a->window < 0) return QGEMV_ERR_INVALID_ARG;
    if (!(a->scale > 0.f && a->scale <= 1e30f)) return QGEMV_ERR_INVALID_ARG;  // NaN too
    AttnPlan p;
    if ((st = attn_plan(a->seqs, a->tokens, a->heads, c.heads, c.dim, a->max_q, a->max_kv, a->window, &p))) return st;
    if (a->pages_stride > (1ll << 40) || static_cast<double>(a->seqs) * static_cast<double>(a->pages_stride) > SPAN_MAX)
        return QGEMV_ERR_UNSUPPORTED;
    // The keys that a row of the page table reaches, and the entries of a row that may be read.
    const long long pages = (static_cast<long long>(a->max_kv) + c.page_size - 1) / c.page_size;
    const int reach = a->pages_stride < pages ? static_cast<int>(a->pages_stride * c.page_size) : a->max_kv;
    const long long entries = a->pages_stride < pages ? a->pages_stride : pages;
    if (a->scratch_bytes < p.scratch) return QGEMV_ERR_INVALID_ARG;
    const Region q = {a->q, a->tokens, a->q_token, a->heads, a->q_head, c.dim, 2};
    const Region o = {a->out, a->tokens, a->out_token, a->heads, a->out_head, c.dim, 2};
    for (const Region* r : {&q, &o})
        if ((st = r->check(1))) return st;
    if (!api_aligned(a->scratch, 16) || !api_aligned(a->pages, 4) || !api_aligned(a->q_start, 4) || !api_aligned(a->kv_len, 4) ||
        (a->lse && !api_aligned(a->lse, 4)))
        return QGEMV_ERR_MISALIGNED;
    if (a->tokens == 0 || a->seqs == 0 || p.grid == 0) return QGEMV_OK;
    // outputs: out, lse, scratch; inputs: q, the cache, the tables
    struct Span { const void* p; size_t n; };
    const Span in[] = {{c.k, cache_bytes(c, c.k_page, c.k_token, c.k_head)},
                       {c.v, cache_bytes(c, c.v_page, c.v_token, c.v_head)},
                       {a->pages, static_cast<size_t>((a->seqs - 1) * a->pages_stride + entries) * 4},
                       {a->q_start, (static_cast<size_t>(a->seqs) + 1) * 4},
                       {a->kv_len, static_cast<size_t>(a->seqs) * 4}};
    const size_t lse_bytes = a->lse ? static_cast<size_t>(a->tokens) * a->heads * 4 : 0;
    const Span out[] = {{a->out, o.bytes()}, {a->lse, lse_bytes}, {a->scratch, a->scratch_bytes}};
    for (int i = 0; i < 3; ++i) {
        if (!out[i].n) continue;
        for (const Span& s : in)
            if (s.n && api_overlaps(out[i].p, out[i].n, s.p, s.n)) return QGEMV_ERR_OVERLAP;
        if (i > 0 && api_overlaps(out[i].p, out[i].n, a->q, q.bytes())) return QGEMV_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (out[j].n && api_overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return QGEMV_ERR_OVERLAP;
    }
    if (meet(o, q)) return QGEMV_ERR_OVERLAP;
    int sms;
    unsigned* err;
    if ((st = api_device(&sms, &err))) return st;
    AttnArgs k = {};
    k.q = a->q, k.out = a->out, k.lse = a->lse;
    k.q_token = a->q_token, k.q_head = a->q_head, k.out_token = a->out_token, k.out_head = a->out_head;
    k.k = static_cast<const uint16_t*>(c.k), k.v = static_cast<const uint16_t*>(c.v);
    k.k_page = c.k_page, k.k_token = c.k_token, k.k_head = c.k_head;
    k.v_page = c.v_page, k.v_token = c.v_token, k.v_head = c.v_head;
    k.pages = a->pages, k.pages_stride = a->pages_stride, k.q_start = a->q_start, k.kv_len = a->kv_len;
    k.count = static_cast<unsigned*>(a->scratch);
    uint8_t* parts = static_cast<uint8_t*>(a->scratch) + QGEMV_ATTN_SCRATCH_HEAD;
    k.part_stat = reinterpret_cast<float2*>(parts);
    k.part_sum = reinterpret_cast<float*>(parts + round32(p.records * sizeof(float2)));
    k.err = err, k.num_pages = c.num_pages, k.page_size = c.page_size, k.kv_heads = c.heads, k.dim = c.dim;
    k.tokens = a->tokens, k.heads = a->heads, k.group = a->heads / c.heads, k.seqs = a->seqs;
    k.max_q = a->max_q, k.max_kv = reach;
    auto log2_of = [](int v) {
        int n = 0;
        while (1 << n < v) ++n;
        return 1 << n == v ? n : -1;
    };
    k.group_shift = log2_of(k.group), k.page_shift = log2_of(c.page_size);
    k.scale_log2 = a->scale * 1.44269504088896341f;
    k.window = a->window, k.causal = a->causal || a->window > 0;
    k.chunk = p.chunk, k.parts = p.parts, k.row_tiles = p.row_tiles, k.rows_part = p.rows_part, k.whole = p.whole;
    k.unit_shift = p.unit_shift;
    const bool pdl = (flags & QGEMV_FLAG_PDL) != 0;
    unsigned smem, threads;
    const void* fn = (p.tiles ? attn_tiles_kernel_ptr : attn_rows_kernel_ptr)(a->kind == QGEMV_ACT_BF16, c.dim, &smem, &threads);
    if ((st = allow_smem(fn, smem))) return st;
    cudaError_t e;
    if (p.tiles) {
        AttnTileArgs ta = {};
        // The tokens of one copy: the largest power of two that divides the page and a key tile; 8 is the swizzle's period.
        int box = 128;
        while (c.page_size % box) box /= 2;
        const long long cache[4] = {c.dim, c.page_size, c.num_pages, c.heads};
        if (box >= 8 && tensor_map(ta.k_map, c.k, c.kind, cache, {c.k_token, c.k_page, c.k_head}, {64, box, 1, 1}) &&
            tensor_map(ta.v_map, c.v, c.kind, cache, {c.v_token, c.v_page, c.v_head}, {64, box, 1, 1}))
            k.box = box;
        k.q_map = 128 % k.group == 0 && tensor_map(ta.q_map, a->q, c.kind, {c.dim, a->heads, a->tokens, 1},
                                                   {a->q_head, a->q_token, c.dim}, {64, k.group, 128 / k.group, 1});
        k.wide = api_aligned(a->out, 32) && api_aligned(k.part_sum, 32) && a->out_token % 16 == 0 && a->out_head % 16 == 0 && c.dim % 16 == 0;
        ta.a = k;
        e = launch_step(fn, dim3(static_cast<unsigned>(p.grid < sms ? p.grid : sms)), threads, smem, 1, pdl, static_cast<cudaStream_t>(stream), ta);
        if (e == cudaSuccess && p.parts > 1) {
            // starts with the tail of the kernel before it, and waits there
            const long long rows = (static_cast<long long>(p.row_tiles) * k.kv_heads * k.seqs - p.whole) * p.rows_part;
            e = launch_step(attn_join_kernel_ptr(a->kind == QGEMV_ACT_BF16),
                            dim3(static_cast<unsigned>((rows + JOIN_WARPS - 1) / JOIN_WARPS)), JOIN_WARPS * 32, 0, 1, true,
                            static_cast<cudaStream_t>(stream), k);
        }
    } else {
        e = launch_step(fn, dim3(static_cast<unsigned>(p.grid)), threads, smem, 1, pdl, static_cast<cudaStream_t>(stream), k);
    }
    if (e != cudaSuccess) return api_cuda_fail(e);
    api_route(p.tiles ? QGEMV_ROUTE_ATTN_TILES : QGEMV_ROUTE_ATTN_ROWS, pdl);
    return QGEMV_OK;
}

// ----------------------------------------------------------------------------------------------------- sampling

constexpr unsigned SAMPLE_SMEM_MAX = 220 * 1024;

static int run_sample(const SampleArgs& s, int kind, unsigned flags, void* stream) {
    const int size = elem_size(kind);
    if (!size || (flags & ~QGEMV_FLAG_PDL)) return QGEMV_ERR_INVALID_ARG;
    if (s.m < 0 || s.N < 1 || s.row_stride < s.N) return QGEMV_ERR_INVALID_ARG;
    if (s.m == 0) return QGEMV_OK;  // (empty tensors may have no address)
    if (!s.x || !s.u || !s.token) return QGEMV_ERR_INVALID_ARG;
    if (s.N > 1 << 20 || s.row_stride > (1ll << 40) || static_cast<double>(s.m) * static_cast<double>(s.row_stride) > SPAN_MAX)
        return QGEMV_ERR_UNSUPPORTED;
    if (!api_aligned(s.x, 16)) return QGEMV_ERR_MISALIGNED;
    const void* words[] = {s.temperature, s.top_k, s.top_p, s.min_p, s.u, s.token, s.prob};
    for (const void* w : words)
        if (w && !api_aligned(w, 4)) return QGEMV_ERR_MISALIGNED;
    const size_t n = static_cast<size_t>(s.m) * 4;
    const size_t xb = (static_cast<size_t>(s.m - 1) * s.row_stride + s.N) * size;
    const void* outs[] = {s.token, s.prob};
    for (const void* o : outs) {
        if (!o) continue;
        if (api_overlaps(o, n, s.x, xb)) return QGEMV_ERR_OVERLAP;
        for (int i = 0; i < 5; ++i)
            if (words[i] && api_overlaps(o, n, words[i], n)) return QGEMV_ERR_OVERLAP;
    }
    if (s.prob && api_overlaps(s.token, n, s.prob, n)) return QGEMV_ERR_OVERLAP;
    int sms, st;
    unsigned* err;
    if ((st = api_device(&sms, &err))) return st;
    // Blocks of a row: slices of at most 20480 tokens, up to the 8 blocks of a portable cluster.  Where the rows make more than two
    // waves of two blocks an SM, slices of twice that as long as two of them still fit (320 rows of 151936 bf16 logits: 273 -> 222 us;
    // 16 rows: 43 -> 54 us): each block's passes then carry fewer barriers.  A slice stays in shared memory where it fits
    // (up to 382528 fp32 or 765056 16-bit logits a row); longer ones are read again from L2.
    SampleArgs k = s;
    auto blocks_of = [&](int most) {
        int n = 1;
        while (n < 8 && (s.N + n - 1) / n > most) n *= 2;
        return n;
    };
    k.blocks = blocks_of(20480);
    if (static_cast<long long>(s.m) * k.blocks > 4ll * sms && size == 2) k.blocks = blocks_of(40960);
    k.slice = ((s.N + k.blocks - 1) / k.blocks + 7) / 8 * 8;
    const unsigned base = sample_smem_base(), room = SAMPLE_SMEM_MAX - base;  // 34016 of 225280 bytes
    k.staged = static_cast<unsigned>(k.slice) * size <= room;
    if (static_cast<long long>(s.m) * k.blocks > INT_MAX) return QGEMV_ERR_UNSUPPORTED;
    const void* fn = sample_kernel_ptr(kind);
    if ((st = allow_smem(fn, SAMPLE_SMEM_MAX))) return st;
    const bool pdl = (flags & QGEMV_FLAG_PDL) != 0;
    cudaError_t e = launch_step(fn, dim3(static_cast<unsigned>(s.m * k.blocks)), SAMPLE_THREADS,
                                base + (k.staged ? static_cast<unsigned>(k.slice) * size : 0u),
                                static_cast<unsigned>(k.blocks), pdl, static_cast<cudaStream_t>(stream), k);
    if (e != cudaSuccess) return api_cuda_fail(e);
    api_route(QGEMV_ROUTE_SAMPLE, pdl);
    return QGEMV_OK;
}

}  // namespace qg

using namespace qg;

extern "C" {

int qgemv_rope_freqs(int rot_dim, double theta, int scaling, double factor, double trained, double low, double high,
                     unsigned long long* out, float* mscale) {
    int st;
    if (api_injected(&st)) return st;
    if (!out || rot_dim < 2 || rot_dim % 2 || rot_dim > 256 || !(theta > 1.0) || !(theta < 1e300)) return QGEMV_ERR_INVALID_ARG;
    if (scaling < QGEMV_ROPE_SCALE_NONE || scaling > QGEMV_ROPE_SCALE_BANDS) return QGEMV_ERR_INVALID_ARG;
    if (scaling != QGEMV_ROPE_SCALE_NONE && !(factor >= 1.0 && factor < 1e9)) return QGEMV_ERR_INVALID_ARG;
    const bool windowed = scaling == QGEMV_ROPE_SCALE_PARTS || scaling == QGEMV_ROPE_SCALE_BANDS;
    if (windowed && !(trained >= 1.0 && trained < 1e18 && low > 0.0 && high > low && high < 1e18)) return QGEMV_ERR_INVALID_ARG;
    if (scaling == QGEMV_ROPE_SCALE_BASE && rot_dim < 4) return QGEMV_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    const int half = rot_dim / 2;
    if (scaling == QGEMV_ROPE_SCALE_BASE) theta *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    // PARTS: the (real) pair index that turns `turns` times over the trained positions, and the ramp between two of them
    auto pair = [&](double turns) { return rot_dim * log(trained / (turns * 2 * pi)) / (2 * log(theta)); };
    double first = 0, last = 0;
    if (scaling == QGEMV_ROPE_SCALE_PARTS) {
        first = floor(pair(high)), last = ceil(pair(low));
        if (first < 0) first = 0;
        if (last > rot_dim - 1) last = rot_dim - 1;
    }
    for (int i = 0; i < half; ++i) {
        double f = pow(theta, -2.0 * i / rot_dim);
        if (scaling == QGEMV_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == QGEMV_ROPE_SCALE_PARTS) {
            const double width = last - first > 1e-3 ? last - first : 1e-3;
            double g = (i - first) / width;
            g = g < 0 ? 0 : g > 1 ? 1 : g;
            f = f / factor * g + f * (1 - g);
        }
        if (scaling == QGEMV_ROPE_SCALE_BANDS) {
            const double turns = trained * f / (2 * pi);  // trained / wavelength
            double g = (turns - low) / (high - low);
            g = g < 0 ? 0 : g > 1 ? 1 : g;
            f = f / factor * (1 - g) + f * g;
        }
        out[i] = static_cast<unsigned long long>(f / (2 * pi) * 18446744073709551616.0 + 0.5);
    }
    if (mscale) *mscale = scaling == QGEMV_ROPE_SCALE_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
    return QGEMV_OK;
}

int qgemv_rope(const qgemv_rope_args* args, unsigned flags, void* stream) {
    int st;
    if (api_injected(&st)) return st;
    return run_rope(args, flags, stream);
}

void qgemv_tune_attn(int kernel) { g_attn_kernel.store(kernel == 1 || kernel == 2 ? kernel : 0); }

size_t qgemv_attn_scratch_bytes(int seqs, int tokens, int heads, int kv_heads, int dim, int max_q, int max_kv) {
    AttnPlan p;
    return attn_plan(seqs, tokens, heads, kv_heads, dim, max_q, max_kv, 0, &p) ? 0 : (p.scratch_most + 255) / 256 * 256;
}

int qgemv_attn(const qgemv_attn_args* args, unsigned flags, void* stream) {
    int st;
    if (api_injected(&st)) return st;
    return run_attn(args, flags, stream);
}

int qgemv_sample(int kind, const void* logits, long long row_stride, int m, int N, const float* temperature,
                 const int* top_k, const float* top_p, const float* min_p, const float* u, int* token_out,
                 float* prob_out, unsigned flags, void* stream) {
    int st;
    if (api_injected(&st)) return st;
    const SampleArgs s = {logits, row_stride, m, N, temperature, top_k, top_p, min_p, u, token_out, prob_out, 0, 0, 0};
    return run_sample(s, kind, flags, stream);
}

}  // extern "C"
