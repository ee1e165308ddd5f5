// kvc_kv4.h - the resident 4-bit cache: geometry and addressing shared by its kernels.
#pragma once

#include "kvc_common.h"

// A pool of pages as the kernels see it, passed by value.
struct Kv4Pool {
    uint8_t *codes;     // [n_pages][2][H] blocks of P * D/2 bytes
    uint32_t *params;   // [n_pages][2][H][D/G][P] of s | lo << 16 (fp16 bits)
    int64_t n_pages;
    int32_t H, D, G;
    int32_t pshift;     // log2 P
    int32_t *status;
};

// Block number of (page, K|V, head): 64 bits, since a long cache passes 2^31 bytes.
__host__ __device__ __forceinline__ int64_t kv4_block(const Kv4Pool &p, int64_t page, int kv, int head)
{
    return (page * 2 + kv) * p.H + head;
}

// One elementwise side of kvc_kv4_append / kvc_kv4_read.
struct Kv4Rows {
    const void *src;            // append: the rows read
    void *dst;                  // read: the rows written
    int64_t token_stride, head_stride;
    bool vec;                   // every 8-channel piece is 16-byte aligned
};

struct Kv4Attn {
    Kv4Pool pool;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *kv_len, *cu_q;
    int64_t n_q;
    int32_t B, Hq, R, max_pages, max_q;
    int32_t causal, window;
    float softcap, scale;
    bool q_vec;                 // every 8-channel piece of q is 16-byte aligned
    bool o_vec;                 // every 4-channel piece of out is 8-byte aligned
    int32_t ns;                 // splits of a row's keys
    int32_t tiles;              // tiles of query rows a (sequence, kv head)
    bool prompt;                // which kernel: tiles of 128 rows rather than 16
    float *part_o;              // [ns][n_q * Hq][D]
    float *part_ml;             // [ns][n_q * Hq][2]
    const int32_t *parents;     // of a tree's tokens (kvc_kv4_tree_attention), or NULL
    int32_t rows;               // of a tree's tile
};

// The rotation of a call of kvc_kv4_append_rotated, and its q.
struct Kv4Turn {
    const float *table;         // [n_positions][rot]: cosines, then sines
    const int64_t *positions;
    int64_t n_positions;
    int32_t rot;
    bool interleaved;
    Kv4Rows q;                  // src NULL: none; dst lies at the strides below
    int64_t out_token_stride, out_head_stride;
    bool out_vec;
    int32_t Hq;
};

hipError_t launch_kv4_append(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                             int dtype, const int64_t *slots, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                           int dtype, const int64_t *slots, hipStream_t stream);
hipError_t launch_kv4_append_rotated(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, const Kv4Turn &turn,
                                     int64_t n_tokens, int dtype, const int64_t *slots, hipStream_t stream);

// Pools that one launch of kvc_kv4_keep moves tokens in: their addresses are kernel arguments.
constexpr int kKeepPools = 64;

struct Kv4Keep {
    Kv4Pool pool;               // the geometry
    kvc_kv4_pool pools[kKeepPools];
    int32_t n_pools;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *base, *path, *n_keep;
    int64_t path_stride;
    int32_t B, max_path, max_pages;
};
hipError_t launch_kv4_keep(const Kv4Keep &a, hipStream_t stream);

// Tiles of query rows and splits of the keys for a call (the launch and the
// workspace size both follow them).
struct Kv4Plan {
    int32_t tiles, ns;
    int32_t most_ns;  // with window = 0: the most that any window makes it
    bool prompt;      // which kernel
    int32_t rows;     // of a tile of kvc_kv4_tree_attention, which goes by it
};
Kv4Plan kv4_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window);
hipError_t launch_kv4_attention(const Kv4Attn &a, bool bf16, hipStream_t stream);

// The same of kvc_kv4_tree_attention.
constexpr int32_t kTreeMost = 1024;  // tokens of a tree: a block holds their parents
Kv4Plan kv4_tree_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window);
hipError_t launch_kv4_tree(const Kv4Attn &a, bool bf16, hipStream_t stream);
