// Arguments of the kernels between the GEMVs (rotary positions, attention, sampling), shared by step_api.cu and the
// kernels' translation units.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qgemv.h"

namespace qg {

struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    void *k_cache, *v_cache;
    long long q_token, q_head, k_token, k_head, v_token, v_head;
    long long q_out_token, q_out_head, k_out_token, k_out_head;
    long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
    const int* positions;
    const unsigned long long* freqs;
    const long long* slots;
    unsigned* err;
    int out_kind, cache_kind;
    int tokens, heads, kv_heads, dim, rot;
    int page_size;
    long long num_slots;
    float mscale;
};

constexpr int ROPE_THREADS = 64;
// vec: heads are handled in 8-element pieces (the rotated part splits into whole pieces); half: the pairing.
const void* rope_kernel_ptr(int x_kind, bool half, bool vec);

struct AttnArgs {
    const void* q;
    void* out;
    float* lse;
    long long q_token, q_head, out_token, out_head;
    const uint16_t *k, *v;
    long long k_page, k_token, k_head, v_page, v_token, v_head;
    const int* pages;
    long long pages_stride;
    const int *q_start, *kv_len;
    unsigned* count;    // zero between calls: 16-row kernel, arrival counters, one a block; 128-row kernel, next part and blocks done
    float2* part_stat;  // records of the parts of split row tiles: maximum in use (base 2) and sum of each row,
    float* part_sum;    // and dim unnormalised sums of values
    unsigned* err;
    int num_pages, page_size, kv_heads, dim;
    int tokens, heads, group, seqs, max_q;
    int max_kv;  // bound of the keys that may be read: the caller's, or what a row of the page table reaches
    int group_shift, page_shift;  // log2 of group and page_size, -1 where they are no powers of two
    float scale_log2;   // scale * log2(e): the softmax runs in base 2
    int causal, window;
    int unit_shift;  // 16-row kernel: the work is divided in units of 2^unit_shift keys
    // 128-row kernel: keys of a part, parts of a row tile and row tiles of a sequence and key/value head in the grid, rows of a
    // part's records
    int chunk, parts, row_tiles, rows_part;
    int whole;       // the first row tiles, whole waves of blocks, that are not cut into parts
    int wide;        // out's and the records' rows begin at multiples of 32 bytes and are as long: the 128-row kernel writes 32 at a time
    int box;         // tokens of one tensor-map copy of the cache (128-row kernel), 0: no tensor map, every row is copied by itself
    int q_map;       // the queries too come by tensor map: a row tile is a box of 128 / group tokens by group heads
};

// The 128-row kernel's arguments: the cache's two tensor maps, [head, page, token, dim] with boxes of `box` tokens by 64
// elements in the 128-byte swizzle, and that of the queries, [1, token, head, dim].
struct AttnTileArgs {
    alignas(64) unsigned long long k_map[16], v_map[16], q_map[16];
    AttnArgs a;
};

struct AttnPlan {
    bool tiles;  // the 128-row tensor-memory kernel (else the 16-row one)
    int chunk, parts, row_tiles, rows_part, whole, unit_shift;
    long long grid;
    size_t records, scratch;  // rows of parts' records, bytes of scratch
    size_t scratch_most;      // scratch that serves every call of these sizes or smaller ones
};

const void* attn_rows_kernel_ptr(bool bf16, int dim, unsigned* smem, unsigned* threads);
const void* attn_tiles_kernel_ptr(bool bf16, int dim, unsigned* smem, unsigned* threads);
const void* attn_join_kernel_ptr(bool bf16);
constexpr int JOIN_WARPS = 8;  // rows of a block of the joining kernel

struct SampleArgs {
    const void* x;
    long long row_stride;
    int m, N;
    const float* temperature;
    const int* top_k;
    const float *top_p, *min_p, *u;
    int* token;
    float* prob;
    int blocks;  // blocks (one cluster) of a row
    int slice;   // tokens of a block, a multiple of 8
    int staged;  // the slice is kept in shared memory
};

constexpr int SAMPLE_THREADS = 512;  // (1024: one row 16.4 -> 20.5 us, 320 rows 224 -> 306 us)
unsigned sample_smem_base();         // shared memory beside the slice
const void* sample_kernel_ptr(int kind);

}  // namespace qg
