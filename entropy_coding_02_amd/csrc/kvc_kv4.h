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
};

hipError_t launch_kv4_append(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                             int dtype, const int64_t *slots, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4Pool &pool, const Kv4Rows &k, const Kv4Rows &v, int64_t n_tokens,
                           int dtype, const int64_t *slots, hipStream_t stream);

// Tiles of query rows and splits of the keys for a call (the launch and the
// workspace size both follow them).
struct Kv4Plan {
    int32_t tiles, ns;
    int32_t most_ns;  // with window = 0: the most that any window makes it
    bool prompt;      // which kernel
};
Kv4Plan kv4_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window);
hipError_t launch_kv4_attention(const Kv4Attn &a, bool bf16, hipStream_t stream);
