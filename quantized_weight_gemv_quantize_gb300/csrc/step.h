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
// vec: heads are handled in 8-element pieces (the rotated part splits into whole pieces); half: the pairing; packed: the cache's strides are
// in bytes and its rows packed.
const void* rope_kernel_ptr(int x_kind, bool half, bool vec, bool packed);

constexpr int UNPACK_QUERIES = 4;  // tokens of a block that takes queries

struct CacheWriteArgs {
    const void *k, *v;
    long long k_token, k_head, v_token, v_head;
    void *k_cache, *v_cache;
    long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;  // bytes
    const long long* slots;
    unsigned* err;
    long long num_slots;
    int tokens, heads, dim, page_size, page_shift;
    int block_tokens;  // tokens of a block, at most CACHE_TOKENS
};

struct CacheReadArgs {
    const uint8_t *k_cache, *v_cache;
    long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;  // bytes
    void *k_out, *v_out;
    long long k_token, k_head, v_token, v_head;
    const int *pages, *out_start, *first;
    long long pages_stride;
    unsigned* err;
    int out_kind, tokens, seqs, num_pages, heads, dim, page_size, page_shift;
    long long reach;   // context tokens that may be read
    int block_tokens;
};

constexpr int WRITE_THREADS = 128, READ_THREADS = 256, CACHE_TOKENS = 32;
const void* cache_write_kernel_ptr(int bits, int x_kind);
const void* cache_read_kernel_ptr(int bits);

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
    const float* units; // or that of each row (token-major), for queries that are scaled row by row
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

// How a block of the packed cache's kernel copies 16 keys of its heads.  On one page: by a tensor map of [token][all heads' rows], where they lie
// together; of [head][all tokens' rows], where those do; or of [head][token][row].  Where pages are no multiple of 16: the heads' rows of a token, where they
// lie together; a head's rows on a page, where those do; or every row by itself.
enum PackedCopies { COPY_ROWS, COPY_HEADS, COPY_BOXES, COPY_TOKENS, COPY_RUNS, COPY_EACH };

// The packed cache's kernel: the cache's two tensor maps, in units of 8 bytes.
struct AttnPackedArgs {
    alignas(64) unsigned long long k_map[16], v_map[16];
    AttnArgs a;            // k and v are not used; the cache's strides are in bytes
    const uint8_t *k, *v;
    int pitch, bf16;       // bytes of a row; type of q and out
    int copies;            // PackedCopies
    int hb_shift;          // log2 of the key/value heads that a block takes side by side
    unsigned few;          // keys that are not worth a block
};

// The copy in 16 bits that the 128-row kernel reads in place of a packed cache.
struct CacheUnpackArgs {
    AttnArgs a;              // the batch over the packed cache
    const uint8_t *k, *v;
    void *k_copy, *v_copy;
    int* table;
    long long per_seq;       // pages of a sequence in the copy
    int page_size, page_shift;  // of the copy: a power of two
    int key_blocks;          // blocks of a sequence that copy keys; those beyond them take its queries
    uint16_t* q_copy;        // bf16 queries in f16, times a power of two a row, and what the rows' scores are scaled by; null: they stay
    float* units;
};
const void* cache_unpack_kernel_ptr(int bits);

struct PackedLaunch {
    unsigned smem, threads, blocks;  // blocks an SM
    int rows, warps;                 // rows of a row tile and head, warps of a block
};
// rows: the most rows (new tokens by query heads of a key/value head) of a sequence
const void* attn_packed4_kernel_ptr(int dim, int rows, PackedLaunch* launch);
const void* attn_packed8_kernel_ptr(int dim, int rows, PackedLaunch* launch);
const void* attn_packed4f_kernel_ptr(int dim, int rows, PackedLaunch* launch);  // f16
const void* attn_packed8f_kernel_ptr(int dim, int rows, PackedLaunch* launch);

struct AttnPlan {
    bool tiles;  // the 128-row tensor-memory kernel (else that of few rows)
    bool forced; // by the tuning hook
    PackedLaunch packed;  // a packed cache's kernel of few rows, where it is taken
    int hb_shift;         // of it
    const void* packed_fn;
    int chunk, parts, row_tiles, rows_part, whole, unit_shift;
    long long grid;
    size_t records, scratch;  // rows of parts' records, bytes of scratch
    size_t copy;              // where in the scratch the copy of a packed cache begins
    size_t scratch_most;      // scratch that serves every call of these sizes or smaller ones
    size_t scratch_least;     // and that with which none of them is refused
};

const void* attn_rows_kernel_ptr(bool bf16, int dim, int seqs, unsigned* smem, unsigned* threads);
const void* attn_tiles_kernel_ptr(bool bf16, bool units, int dim, unsigned* smem, unsigned* threads);
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
