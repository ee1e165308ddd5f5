// kv4_tile.h - what the kernels of attention over the resident 4-bit cache share:
// addressing, loads, operands, the running softmax, the join of splits.
#pragma once

#include "kvc_kernels.h"
#include "kvc_kv4.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Arrays that no kernel here writes, read through the scalar cache: they
// neither occupy vector registers nor wait in line behind the codes.
typedef const int32_t __attribute__((address_space(4))) const_i32;
__device__ __forceinline__ int32_t scalar_load(const int32_t *p, int64_t i) { return ((const_i32 *)(uintptr_t)p)[i]; }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Nibble i of both halves of w as a pair of n 2^-9.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i)
{
    const uint32_t b = (i < 2 ? w : w >> 8) & (i & 1 ? 0x00F000F0u : 0x000F000Fu);
    const _Float16 f = i & 1 ? (_Float16)0x1p11f : (_Float16)0x1p15f;
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) * f16x2{f, f});
}
// The same less 7.5, exactly, for V.
__device__ __forceinline__ uint32_t centred_pair(uint32_t w, int i)
{
    const uint32_t b = (i < 2 ? w : w >> 8) & (i & 1 ? 0x00F000F0u : 0x000F000Fu);
    const _Float16 f = i & 1 ? (_Float16)0x1p11f : (_Float16)0x1p15f, c = (_Float16)(-7.5f * 0x1p-9f);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, b), f16x2{f, f}, f16x2{c, c}));
}
// A K dword (8 channels of a key) as 8 operands in the order 0,4,1,5,2,6,3,7.
__device__ __forceinline__ u32x4 code_octet(uint32_t w)
{
    return u32x4{code_pair(w, 0), code_pair(w, 1), code_pair(w, 2), code_pair(w, 3)};
}

__device__ __forceinline__ float s_of(uint32_t w) { return kvc_h2f(w & 0xFFFF); }
__device__ __forceinline__ float lo_of(uint32_t w) { return kvc_h2f(w >> 16); }
__device__ __forceinline__ float mid_of(uint32_t w) { return __builtin_fmaf(7.5f, s_of(w), lo_of(w)); }  // of a group's range

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ uint32_t f16_pair(float a, float b)
{
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Over the four lanes (16 apart) of a query row: swapping rows of 16, then
// halves, of a value with itself leaves both operands of the reduction.
__device__ __forceinline__ float row_max(float v)
{
    uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t x0 = x[0], x1 = x[1];
    b = __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1)));
    const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t y0 = y[0], y1 = y[1];
    return fmaxf(__builtin_bit_cast(float, y0), __builtin_bit_cast(float, y1));
}
__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// A barrier for LDS alone: __syncthreads also waits for every load on its way
// from memory, which here are the first codes.
__device__ __forceinline__ void lds_barrier() { __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// From a row's maximum and sum in powers of 2; a row without keys has L = 0, a
// row that met a NaN has L = NaN (its maximum may be -inf).
__device__ __forceinline__ float lse_of(float M, float L)
{
    return L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// What a wave loads for 32 keys: two tiles of 16.  A lane holds the codes it
// multiplies, but of the parameters only its share (a dword for each 64 of
// them): it works with those of four keys that 15 other lanes want too, so
// they pass through LDS rather than lie in 16 lanes' registers.
template <int D, int G>
struct Stage {
    static constexpr int NW = D / 32, NG = D / G, NP = (NG + 3) / 4;
    uint32_t k[2][NW], v[2][NW];
    uint32_t kp[2][NP], vp[2][NP];
};

template <int D, int G>
__device__ __forceinline__ void load_words(uint32_t *dst, const uint8_t *src)
{
    constexpr int NW = D / 32;
    if (NW == 2) {
        const u32x2 w = *(const u32x2 *)src;
        dst[0] = w[0], dst[1] = w[1];
    } else {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i) {
            const u32x4 w = *(const u32x4 *)(src + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[4 * i + j] = w[j];
        }
    }
}

// What a block works on: one (sequence, kv head), ROWS of its query rows (row =
// query * R + head within the group), one split of their keys.
struct Job {
    int b, h, split, tile;
    int nq, q0, len, pos0, rows, row0;
    int kbeg, kend;  // keys that some row of the tile sees
    int u0, u1;      // the split's units of 128 keys
};

// TREE: the queries are a tree's tokens.  Any of them may be its first.
template <int ROWS, bool TREE = false>
__device__ __forceinline__ bool make_job(const Kv4Attn &a, Job &j)
{
    uint32_t id = blockIdx.x;
    j.split = id % a.ns, id /= a.ns;
    j.h = id % a.pool.H, id /= a.pool.H;
    j.b = id % a.B;
    j.tile = a.tiles - 1 - id / a.B;  // under a causal mask the last tiles have the most keys: they go first
    bool bad = false;
    int64_t c0 = a.cu_q ? scalar_load(a.cu_q, j.b) : (int64_t)j.b * a.max_q;
    int64_t c1 = a.cu_q ? scalar_load(a.cu_q, j.b + 1) : c0 + a.max_q;
    if (c0 < 0 || c0 > a.n_q) bad = true, c0 = c0 < 0 ? 0 : a.n_q;
    if (c1 < c0 || c1 > a.n_q || c1 - c0 > a.max_q) {
        bad = true;
        c1 = c1 < c0 ? c0 : c1;
        c1 = c1 > a.n_q ? a.n_q : c1;
        c1 = c1 - c0 > a.max_q ? c0 + a.max_q : c1;
    }
    j.q0 = (int)c0;
    j.nq = (int)(c1 - c0);
    const int cap = a.max_pages << a.pool.pshift;
    j.len = scalar_load(a.kv_len, j.b);
    if (j.len > cap) bad = true, j.len = cap;
    if (j.len < 0) j.len = 0;
    if (bad && j.tile == a.tiles - 1 && threadIdx.x == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
    j.rows = j.nq * a.R;
    j.row0 = j.tile * ROWS;
    if (j.row0 >= j.rows) return false;
    j.pos0 = j.len - j.nq;
    const int last = min(j.row0 + ROWS, j.rows) - 1;
    const int i_lo = j.row0 / a.R, i_hi = last / a.R;
    j.kend = a.causal ? min(j.len, j.pos0 + i_hi + 1) : j.len;
    j.kbeg = a.window ? max(0, j.pos0 + (TREE ? 0 : i_lo) - a.window + 1) : 0;
    if (j.kend <= j.kbeg) {
        j.kbeg = j.kend = j.u0 = j.u1 = 0;
        return true;
    }
    // at most 2^23 units (2^30 keys) times 128 splits
    const uint32_t f = (uint32_t)j.kbeg / 128, n = (uint32_t)(j.kend + 127) / 128 - f, ns = (uint32_t)a.ns;
    j.u0 = (int)(f + n * (uint32_t)j.split / ns);
    j.u1 = (int)(f + n * ((uint32_t)j.split + 1) / ns);
    return true;
}

// Where a lane reads, in bytes from a tile's place in its page's K block or K
// parameters: V lies a fixed distance on.  (A page's codes are at most
// 2 * 1024 heads * 256 tokens * 128 bytes.)
template <int D, int G>
struct LaneAt {
    static constexpr int NG = D / G, NP = (NG + 3) / 4;
    uint32_t k, v, kp[NP], vp[NP];
    __device__ __forceinline__ LaneAt(int lane, const Kv4Pool &p)
    {
        const int r = lane & 15, h = lane >> 4;
        k = r * (D / 2) + h * (D / 8);
        v = h * (2 * D) + r * (D / 8) + ((uint32_t)p.H << p.pshift) * (D / 2);
        // group h (+ 4), key r; with fewer than four groups lanes repeat one
        for (int i = 0; i < NP; ++i) {
            kp[i] = (((uint32_t)((h + 4 * i) % NG) << p.pshift) + r) * 4;
            vp[i] = kp[i] + ((uint32_t)(p.H * NG) << p.pshift) * 4;
        }
    }
};

// The same for the whole wave, kept in scalar registers: this (sequence, head)
// and what a page number is multiplied by.
template <int D, int G>
struct WaveAt {
    const int32_t *table;
    const uint8_t *codes, *params;
    uint32_t page_codes, page_params;  // bytes of a page
    int t_lo, t_hi, shift, mask;       // tiles that some row sees; a tile's page and its place there
    uint32_t n_pages;
    __device__ __forceinline__ WaveAt(const Kv4Attn &a, const Job &j)
    {
        const int P = 1 << a.pool.pshift;
        table = a.table + j.b * a.table_stride;
        codes = a.pool.codes + (int64_t)j.h * (P * (D / 2));
        params = (const uint8_t *)a.pool.params + (int64_t)j.h * (D / G * P * 4);
        page_codes = (uint32_t)a.pool.H * P * D;
        page_params = (uint32_t)a.pool.H * P * (D / G) * 8;
        t_lo = j.kbeg >> 4;
        t_hi = (j.kend - 1) >> 4;
        shift = a.pool.pshift - 4;
        mask = (P >> 4) - 1;
        n_pages = (uint32_t)a.pool.n_pages;
    }
    // A tile that no row sees is read from one that some row does.
    __device__ __forceinline__ int tile(int blk, int t) const { return min(max(blk * 2 + t, t_lo), t_hi); }
};

// The table entries of a block's two tiles.
template <int D, int G>
__device__ __forceinline__ void load_pages(const WaveAt<D, G> &w, int blk, int32_t *page)
{
#pragma unroll
    for (int t = 0; t < 2; ++t) page[t] = w.table[w.tile(blk, t) >> w.shift];
}

template <int D, int G>
__device__ __forceinline__ void load_stage(const WaveAt<D, G> &w, int blk, const int32_t *pages, const LaneAt<D, G> &at,
                                           Stage<D, G> &st, bool &bad_page)
{
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t entry = (uint32_t)__builtin_amdgcn_readfirstlane(pages[t]);
        bad_page |= entry >= w.n_pages;
        const uint32_t page = entry < w.n_pages ? entry : 0;
        const uint32_t in = (uint32_t)(w.tile(blk, t) & w.mask);
        const uint8_t *codes = w.codes + (uint64_t)page * w.page_codes + in * (8 * D);
        const uint8_t *params = w.params + (uint64_t)page * w.page_params + in * 64;
        load_words<D, G>(st.k[t], codes + at.k);
#pragma unroll
        for (int i = 0; i < at.NP; ++i) st.kp[t][i] = *(const uint32_t *)(params + at.kp[i]);
        load_words<D, G>(st.v[t], codes + at.v);
#pragma unroll
        for (int i = 0; i < at.NP; ++i) st.vp[t][i] = *(const uint32_t *)(params + at.vp[i]);
    }
}

// Four channels of an output row.
template <bool BF>
__device__ __forceinline__ void store_out(const Kv4Attn &a, int64_t tok, int head, int c, f32x4 y)
{
    uint16_t *dst = a.out + tok * a.o_ts + head * a.o_hs + c;
    const u32x2 w = {BF ? bf16_pair(y[0], y[1]) : kvc_f2h2(y[0], y[1]), BF ? bf16_pair(y[2], y[3]) : kvc_f2h2(y[2], y[3])};
    if (a.o_vec) {
        *(u32x2 *)dst = w;
    } else {
        for (int i = 0; i < 4; ++i) dst[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// A lane's part of a query row: channels 8h .. 8h + 7 of every 32.
template <int D, bool BF>
__device__ __forceinline__ void load_query(const Kv4Attn &a, const Job &j, int row, int qi, int h, bool real, u32x4 *q)
{
    const uint16_t *src = a.q + (int64_t)(j.q0 + qi) * a.q_ts + (int64_t)(j.h * a.R + row % a.R) * a.q_hs + 8 * h;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        q[s] = u32x4{0, 0, 0, 0};
        if (!real) continue;
        if (a.q_vec)
            q[s] = *(const u32x4 *)(src + 32 * s);
        else
            for (int k = 0; k < 4; ++k) q[s][k] = src[32 * s + 2 * k] | (uint32_t)src[32 * s + 2 * k + 1] << 16;
    }
}

// The power of two (signed as the scale) that takes a row's largest to just
// under 2^15, and `up`, what its logits are then to be multiplied by.
template <int D, bool BF>
__device__ __forceinline__ float scale_query(const Kv4Attn &a, const u32x4 *q, float &up)
{
    uint32_t top = 0;  // the largest magnitude, by its bits
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(q[s][k] & 0x7FFFu, q[s][k] >> 16 & 0x7FFFu));
    const float big = row_max(BF ? __builtin_bit_cast(float, top << 16) : kvc_h2f(top));
    // 2^(14 - e) for a largest of 2^e; a row of zeros, or one with Inf or NaN, stays as it is
    const int e = big > 0.0f && big < __builtin_inff() ? max((int)(__builtin_bit_cast(uint32_t, big) >> 23) - 127, -100) : 14;
    // A scale of 0 is one too small to tell (0 times the -inf of a masked key
    // would be NaN).  2^9 undoes the codes' unit.
    up = fmaxf(__builtin_fabsf(a.scale), 1.0e-30f) * (a.softcap > 0.0f ? 1.0f : kLog2e);
    up = fmaxf(up * __builtin_bit_cast(float, (uint32_t)(127 + min(9 - 14 + e, 127)) << 23), 1.0e-37f);
    // a negative scale becomes a positive one of -q, so that the largest logit is found before scaling
    const float f = __builtin_bit_cast(float, (uint32_t)(127 + 14 - e) << 23);
    return a.scale < 0.0f ? -f : f;
}

// Eight channels of q, scaled, in the order of code_octet.
template <bool BF>
__device__ __forceinline__ u32x4 query_operand(u32x4 w, float f)
{
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = w[k / 2] >> (16 * (k & 1)) & 0xFFFFu;
        y[k] = (BF ? __builtin_bit_cast(float, b << 16) : kvc_h2f(b)) * f;
    }
    return u32x4{f16_pair(y[0], y[4]), f16_pair(y[1], y[5]), f16_pair(y[2], y[6]), f16_pair(y[3], y[7])};
}

// The term sum_g lo_g (sum_{c in g} q_c) of the logits as a matrix product of
// its own, which the codes' products start from: two multiply-adds fewer a
// logit.  A lane has key r's lo of group h (and h + 4) against that group's sum
// of q in three fp16 terms (33 bits, no coarser than 2^-25 of its 2^13 at most).
template <int NG>
__device__ __forceinline__ u32x4 lo_operand(const uint32_t *params, int h)
{
    u32x4 a = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < (NG + 3) / 4; ++i) {
        const uint32_t lo = params[i] >> 16;
        if (h + 4 * i < NG) a[2 * i] = lo | lo << 16, a[2 * i + 1] = lo;
    }
    return a;
}
template <int NG>
__device__ __forceinline__ u32x4 sum_operand(const float *qs, int h)
{
    u32x4 b = {0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const _Float16 t1 = (_Float16)qs[g];
        const float r1 = qs[g] - (float)t1;
        const _Float16 t2 = (_Float16)r1;
        const float r2 = r1 - (float)t2;
        if (h == g % 4) b[g / 4 * 2] = f16_pair(qs[g], r1), b[g / 4 * 2 + 1] = f16_pair(r2, 0.0f);
    }
    return b;
}

// log2 of the largest s of a key's groups, of which this lane holds `s`, and the
// lanes of the same key 16 apart the others; at least -24, the smallest s there
// is (what lies at a key that no row sees may be anything: NaN becomes -24).
template <int NG>
__device__ __forceinline__ float log2_top(float s)
{
    if (NG > 1) {
        const uint32_t b = __builtin_bit_cast(uint32_t, s);
        const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        const uint32_t x0 = x[0], x1 = x[1];
        s = fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
    }
    if (NG > 2) {
        const uint32_t b = __builtin_bit_cast(uint32_t, s);
        const auto x = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        const uint32_t x0 = x[0], x1 = x[1];
        s = fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
    }
    return fmaxf(__builtin_amdgcn_logf(s), -24.0f);
}

// Rows of which some p s passes the largest so far by 2^8 take the new one.
// top: the largest x + log2 s of the row's new keys, by lane; ref: what p is
// relative to (-inf: no key yet).  Returns what the sums are to be multiplied by.
__device__ __forceinline__ float rescale(float top, float &pass, float &ref, float &mu)
{
    top = row_max(top);
    const float to = top > pass ? top - 7.0f : ref;
    const float f = ref == -__builtin_inff() ? 1.0f : exp2_fast(ref - to);
    pass = top > pass ? top + 8.0f : pass;
    ref = to;
    mu = ref == -__builtin_inff() ? 0.0f : ref;
    return f;
}

// c tanh(u), u = x up / c, in powers of 2.  Its error has to be a share of the
// logit, whatever the cap: up to 5/8, u Q(u^2) with Q the minimax polynomial of
// tanh(u)/u there that is 1 at 0 (2^-27.8; fitted by weighted least squares), so
// that a cap far above the logits leaves them as they are; beyond,
// 1 - 2 / (exp(2u) + 1), which for small u would be a difference of near equals.
// Logits past 5/8 of their cap are few, and the branch is a wave's.
__device__ __forceinline__ void cap_logits(float cap, f32x4 (&x)[2], float &up)
{
    // or the compiler computes this for every call
#pragma unroll
    for (int t = 0; t < 2; ++t) __asm__ volatile("" : "+v"(x[t]));
    constexpr float kNear = 0.625f;
    const float in = fminf(up / cap, 1.0e30f), unit = up * kLog2e;  // 0 times infinity would be NaN
    float u[8], far = 0.0f;
    f32x4 y[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u[i] = x[i / 4][i % 4] * in;
        const float w = u[i] * u[i];
        float q = __builtin_fmaf(w, -0.00570498686f, 0.020639088f);
        q = __builtin_fmaf(w, q, -0.0537397154f);
        q = __builtin_fmaf(w, q, 0.133314416f);
        q = __builtin_fmaf(w, q, -0.333332807f);
        y[i / 4][i % 4] = x[i / 4][i % 4] * unit * __builtin_fmaf(w, q, 1.0f);
        far = fmaxf(far, __builtin_fabsf(u[i]));
    }
    if (__any(far > kNear)) {
        const float top = fminf(cap * kLog2e, 3.0e38f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = __builtin_amdgcn_rcpf(exp2_fast(u[i] * (2.0f * kLog2e)) + 1.0f);
            if (__builtin_fabsf(u[i]) > kNear) y[i / 4][i % 4] = top * __builtin_fmaf(-2.0f, r, 1.0f);
        }
    }
    x[0] = y[0], x[1] = y[1];
    up = 1.0f;
}

// Joins the splits of a row: D/4 lanes a split, as many splits at a time as
// fill the block, then their sums through LDS.  Rows that no sequence has were
// not written by any split, and are left alone here too.
template <int D, bool BF, int THREADS>
__global__ __launch_bounds__(THREADS) void k_kv4_join(Kv4Attn a)
{
    constexpr int LANES = D / 4, AT_ONCE = THREADS / LANES;
    __shared__ f32x4 lds_y[AT_ONCE][LANES];
    __shared__ float lds_l[AT_ONCE];
    const int64_t rows = a.n_q * a.Hq;
    const int64_t row = (a.cu_q ? (int64_t)max(scalar_load(a.cu_q, 0), 0) * a.Hq : 0) + blockIdx.x;
    if (row >= (a.cu_q ? min((int64_t)scalar_load(a.cu_q, a.B), a.n_q) * a.Hq : rows)) return;
    const int part = threadIdx.x % LANES, first = threadIdx.x / LANES;
    float M = -__builtin_inff();
    for (int s = threadIdx.x & 63; s < a.ns; s += 64) M = fmaxf(M, a.part_ml[(s * rows + row) * 2]);
    for (int off = 32; off; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    f32x4 y = {0, 0, 0, 0};
    float L = 0.0f;
#pragma unroll 4
    for (int s = first; s < a.ns; s += AT_ONCE) {
        const float ms = a.part_ml[(s * rows + row) * 2], ls = a.part_ml[(s * rows + row) * 2 + 1];
        const f32x4 ys = *(const f32x4 *)(a.part_o + (s * rows + row) * D + 4 * part);
        const float w = ls == 0.0f ? 0.0f : exp2_fast(ms - M);  // 0: no keys
        L += w * ls;
        y += w * ys;
    }
    lds_y[first][part] = y;
    if (part == 0) lds_l[first] = L;
    __syncthreads();
    if (first) return;
    L = lds_l[0];
    for (int i = 1; i < AT_ONCE; ++i) {
        y += lds_y[i][part];
        L += lds_l[i];
    }
    const int64_t tok = row / a.Hq;
    const int head = (int)(row % a.Hq);
    y *= L == 0.0f ? 0.0f : 1.0f / L;
    store_out<BF>(a, tok, head, 4 * part, y);
    if (a.lse && part == 0) a.lse[row] = lse_of(M, L);
}

}  // namespace
