// kvc_kv4_attn.hip - attention over the resident 4-bit cache.
//
// A cached value is y = lo + s n, n = 0..15.  A code within the mantissa of an
// fp16 whose exponent is zero is the subnormal n 2^-24 (or, four bits up,
// n 2^-20), exactly, and a packed multiplication makes it n 2^-9, two codes at
// a time; (s, lo) never touch the matrix operands:
//   logits   q.k = sum_g s_g (sum_{c in g} q_c n_c) + lo_g (sum_{c in g} q_c);
//            a query row is scaled by a power of two to just under 2^15 (an
//            fp16 then holds every bit of it that fp32 sums would), so the
//            products are exact;
// (The matrix instructions take the subnormals too, but align a sum's products
// by exponent, and a subnormal's leading bits lie up to ten places below its:
// outputs that average many keys then lost twice their last fp16 bit.)
//   output   o_c = sum_j (p_j s_jg) (n_jc - 7.5) + sum_j p_j mid_jg,  c in group g,
//            mid = lo + 7.5 s.  Sums of n itself are all positive and cancel
//            against lo; what they rounded off added up (2048 queries over 8192
//            keys of values of either sign: outputs off by 8e-5 in the mean,
//            centred by 8e-7, in the same time).
// p_j s_jg enters the matrix product as two fp16 terms (22 bits): one would
// be an error of the output's own size, since n s is up to twice the value it
// belongs to.  They keep those bits because p is taken relative not to the
// row's largest logit but to the largest p_j s_j, s_j the largest s of key j's
// groups, of which the product is 2^7: neither a token far larger than the others
// that the row hardly looks at, nor one far smaller that it looks at alone, takes
// the others' bits.  (Within a token a group whose s is 2^-k of the largest
// keeps 22 bits up to k = 10, and one fewer for each more.)  That maximum is let be
// until a p s passes it by 2^8: the sums are rescaled a few times a row rather
// than at every new maximum of any of a wave's rows, and p s stays below 2^15.
//
// Orientation: S^T = K q^T (16 keys x 16 query rows), so a lane holds one
// query row and four keys of a tile, which is just what P^T needs as the
// right operand of O^T = V^T P^T (keys 4h .. 4h+3 of two tiles are its eight
// k indices): probabilities never cross lanes, the terms with mid and the row
// sums are plain fp32 sums per lane, added over the four lanes of a row once
// at the end.
#include <algorithm>

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

template <int ROWS>
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
    j.kbeg = a.window ? max(0, j.pos0 + i_lo - a.window + 1) : 0;
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

template <int D, int G, bool BF>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : D == 128 ? (G == 32 ? 2 : 3) : 4) void k_kv4_attn(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = Stage<D, G>::NP, TILE = 64 * NP, NQ = (NW + kWaves - 1) / kWaves;
    // Each wave's results; while it runs, its parameters, [tile] K's s, then
    // [tile][s|mid] V's, each [group][16 keys], in fp32 (mixed-precision instructions run at half
    // rate), then [tile] log2 of each key's largest s of V.
    __shared__ __align__(16) float lds_o[kWaves][16][D];
    __shared__ float lds_ml[kWaves][2][16];
    // The query operands, which as registers would cost a wave a SIMD.
    __shared__ u32x4 lds_q[NW][64];
    Job j;
    if (!make_job<16>(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;  // this lane's query row, and its four keys of each tile
    float *const prm = &lds_o[wave][0][0];
    static_assert(6 * TILE + 32 <= 16 * D, "the parameters fit where the results go");
    const int row = j.row0 + col, qi = row / a.R;
    const int b_end = min(j.u1 * 4, (j.kend + 31) / 32);
    int blk = j.u0 * 4 + wave;
    const bool work = blk < b_end;
    const WaveAt<D, G> wat(a, j);

    // The pages of this wave's first two blocks, and its row of q (all of it,
    // for the row's largest; every wave then stores a part of the operands).
    int32_t first[2] = {0, 0}, pages[2] = {0, 0};
    float up;  // what the lane's row of logits is to be multiplied by
    {
        u32x4 qw[NW];
        load_query<D, BF>(a, j, row, qi, h, row < j.rows, qw);
        if (work) {
            load_pages(wat, blk, first);
            load_pages(wat, blk + kWaves, pages);
        }
        const float f = scale_query<D, BF>(a, qw, up);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            u32x4 w = qw[i * kWaves];
#pragma unroll
            for (int k = 1; k < kWaves; ++k)
                if (k < NW && wave == k) w = qw[(i * kWaves + k) % NW];
            if (wave + i * kWaves < NW) lds_q[wave + i * kWaves][lane] = query_operand<BF>(w, f);
        }
        lds_barrier();
    }

    f32x4 o[NT];
    // In powers of 2: pass, the p s at which the sums are rescaled, and ref, what p is relative to.
    float z[NG], pass = -__builtin_inff(), ref = -__builtin_inff(), mu = 0.0f, l = 0.0f;
#pragma unroll
    for (int c = 0; c < NT; ++c) o[c] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g] = 0.0f;
    if (work) {
        const LaneAt<D, G> at(lane, a.pool);
        Stage<D, G> cur, next;
        bool bad_page = false;
        load_stage<D, G>(wat, blk, first, at, cur, bad_page);

        // the group sums of q, in the codes' unit
        float qs[NG];
        {
            const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};  // 1
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c = {0, 0, 0, 0};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma(ones, lds_q[s][lane], c);
                qs[g] = c[0] * 0x1p-9f;
            }
        }
        const u32x4 sums = sum_operand<NG>(qs, h);
        const int pos = j.pos0 + qi;
        const int k_hi = a.causal ? min(j.len, pos + 1) : j.len;  // keys k_lo <= key < k_hi
        const int k_lo = a.window ? max(0, pos - a.window + 1) : 0;
        // keys that every row of the tile sees
        const int all_hi = a.causal ? min(j.len, j.pos0 + j.row0 / a.R + 1) : j.len;
        const int all_lo = a.window ? j.pos0 + min(j.row0 + 15, j.rows - 1) / a.R - a.window + 1 : 0;
        // A block's codes are on their way while the one before is worked on,
        // and its pages one block earlier still.  The last turns load the last
        // tile again rather than branch: where a load may or may not have been
        // issued, the wait for an older one is a wait for all.
        for (; blk < b_end; blk += kWaves) {
            int32_t after[2];  // loads return in order: before the codes, or they would wait for them
            load_pages(wat, blk + 2 * kWaves, after);
            load_stage<D, G>(wat, blk + kWaves, pages, at, next, bad_page);
            pages[0] = after[0], pages[1] = after[1];

#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    prm[t * TILE + 64 * i + lane] = s_of(cur.kp[t][i]);
                    prm[(2 * t + 2) * TILE + 64 * i + lane] = s_of(cur.vp[t][i]);
                    prm[(2 * t + 3) * TILE + 64 * i + lane] = mid_of(cur.vp[t][i]);
                }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float s = s_of(cur.vp[t][0]);
#pragma unroll
                for (int i = 1; i < NP; ++i) s = fmaxf(s, s_of(cur.vp[t][i]));
                prm[6 * TILE + 16 * t + col] = log2_top<NG>(s);
            }
            const int key0 = blk * 32;
            const bool partial = key0 + 32 > all_hi || key0 < all_lo;
            f32x4 x[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) x[t] = mfma(lo_operand<NG>(cur.kp[t], h), sums, f32x4{0, 0, 0, 0});
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                    const u32x4 q = lds_q[s][lane];
                    c[0] = mfma(code_octet(cur.k[0][s]), q, c[0]);
                    c[1] = mfma(code_octet(cur.k[1][s]), q, c[1]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 ks = *(const f32x4 *)&prm[t * TILE + 16 * g + 4 * h];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[t][i] = __builtin_fmaf(ks[i], c[t][i], x[t][i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            float mul = up;
            if (a.softcap > 0.0f) cap_logits(a.softcap, x, mul);
            if (partial)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = key0 + 16 * (i / 4) + 4 * h + i % 4;
                    if (key < k_lo || key >= k_hi) x[i / 4][i % 4] = -__builtin_inff();
                }
            float top = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 ls = *(const f32x4 *)&prm[6 * TILE + 16 * t + 4 * h];
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, __builtin_fmaf(x[t][i], mul, ls[i]));
            }
            if (__any(top > pass)) {
                const float f = rescale(top, pass, ref, mu);
                l *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) z[g] *= f;
#pragma unroll
                for (int c = 0; c < NT; ++c) o[c] *= f;
            }
            float p[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i / 4][i % 4] = exp2_fast(__builtin_fmaf(x[i / 4][i % 4], mul, -mu));
                l += p[i / 4][i % 4];
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                u32x4 hi, lo;
                f32x4 vs[2], vmid[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    vs[t] = *(const f32x4 *)&prm[(2 * t + 2) * TILE + 16 * g + 4 * h];
                    vmid[t] = *(const f32x4 *)&prm[(2 * t + 3) * TILE + 16 * g + 4 * h];
                }
                if (partial) {
                    // what lies at a key that the row does not see may be anything, NaN too
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (x[i / 4][i % 4] == -__builtin_inff()) vs[i / 4][i % 4] = vmid[i / 4][i % 4] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float s0 = vs[i / 4][i % 4], s1 = vs[i / 4][i % 4 + 1];
                    const float p0 = p[i / 4][i % 4], p1 = p[i / 4][i % 4 + 1];
                    z[g] = __builtin_fmaf(p0, vmid[i / 4][i % 4], z[g]);
                    z[g] = __builtin_fmaf(p1, vmid[i / 4][i % 4 + 1], z[g]);
                    const f32x2 a2 = {p0 * s0, p1 * s1};
                    const f16x2 t = __builtin_convertvector(a2, f16x2);
                    const f32x2 b2 = {a2[0] - (float)t[0], a2[1] - (float)t[1]};
                    hi[i / 2] = __builtin_bit_cast(uint32_t, t);
                    lo[i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b2, f16x2));
                }
// by pairs of tiles: the two terms of one would wait for each other
#pragma unroll
                for (int c = g * (G / 16); c < (g + 1) * (G / 16); c += 2) {
                    if (c % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                    const int w = 2 * (c / 4);
                    u32x4 va[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        va[k] = u32x4{centred_pair(cur.v[0][w], (c & 3) + k), centred_pair(cur.v[0][w + 1], (c & 3) + k),
                                      centred_pair(cur.v[1][w], (c & 3) + k), centred_pair(cur.v[1][w + 1], (c & 3) + k)};
                    o[c] = mfma(va[0], hi, o[c]);
                    o[c + 1] = mfma(va[1], hi, o[c + 1]);
                    o[c] = mfma(va[0], lo, o[c]);
                    o[c + 1] = mfma(va[1], lo, o[c + 1]);
                }
            }
            cur = next;
        }
        if (bad_page && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
    }

    __asm__ volatile("" ::: "memory");  // parameters are read, results may take their place
    // the four waves' parts: out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
    l = row_sum(l);
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g] = row_sum(z[g]);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(512.0f, o[c][i], z[16 * c / G]);
        *(f32x4 *)&lds_o[wave][col][16 * c + 4 * h] = y;
    }
    if (h == 0) {
        lds_ml[wave][0][col] = ref;
        lds_ml[wave][1][col] = l;
    }
    __syncthreads();
    // 16 threads a row
    const int mr = threadIdx.x / 16, part = threadIdx.x % 16;
    const int orow = j.row0 + mr;
    if (orow >= j.rows) return;
    float M = -__builtin_inff(), L = 0.0f, wgt[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[w][0][mr]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        wgt[w] = M == -__builtin_inff() ? 0.0f : exp2_fast(lds_ml[w][0][mr] - M);
        L += wgt[w] * lds_ml[w][1][mr];
    }
    const int head = j.h * a.R + orow % a.R;
    const int64_t tok = j.q0 + orow / a.R, grow = tok * a.Hq + head;
    const int64_t prow = (int64_t)j.split * a.n_q * a.Hq + grow;
    const float inv = a.ns > 1 ? 1.0f : (L == 0.0f ? 0.0f : 1.0f / L);
    for (int c = part * 4; c < D; c += 64) {
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) y += wgt[w] * *(const f32x4 *)&lds_o[w][mr][c];
        y *= inv;
        if (a.ns > 1) {
            *(f32x4 *)(a.part_o + prow * D + c) = y;
        } else {
            store_out<BF>(a, tok, head, c, y);
        }
    }
    if (part == 0) {
        if (a.ns > 1) {
            a.part_ml[prow * 2] = M;
            a.part_ml[prow * 2 + 1] = L;
        } else if (a.lse) {
            a.lse[grow] = lse_of(M, L);
        }
    }
}

// ------------------------------------------------------------ prompt pieces

constexpr int kRows = 128;   // query rows of a block, 32 a wave
constexpr int kKeys = 64;    // keys a turn

// Many query rows: a block's four waves have 32 rows each and share the keys.
// Each wave unpacks a tile of 16 of a turn's 64 keys into LDS, as the matrix
// operands that all of them read (in the order in which lanes read them: 16
// bytes a lane, no conflicts), while the codes of the next turn are on their
// way.  The terms are those of k_kv4_attn, with bf16 outputs too: one fp16 term of
// p s is off by 2^-12 of s n, which in a group with an outlier channel is many
// times its other channels' values (one channel in 32 offset by 30: outputs off
// by 5e-3, where the rounding to bf16 is 1.7e-3).  The second term costs a fifth
// of the time (2048 queries over 8192 keys, all else alike: 494 us, with one term
// 412); it is the residual of the exact product, by a mixed multiply-add (as a
// difference of fp32: 520).  That call takes 504 us, 475 TFLOP/s: the vector units
// are 60% busy, the matrix units 30%, LDS 42%, with two waves a SIMD.
template <int D, int G, bool BF>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv4_prompt(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = Stage<D, G>::NP, TILE = 64 * NP;
    constexpr int NK = 4 * NW * 64, NV = 2 * NT * 64;  // 16-byte operands of a turn
    // Groups whose p s are held at once: one, or the registers spill (in groups
    // of 32, 2 x 512 queries over 4096 keys 211 us, all at once 327); heads of 256 have the
    // accumulators' half of the file for it (512 over 4096 152 us, one by one 196).
    constexpr int GS = D == 256 ? NG : 1;
    struct Turn {
        u32x4 k[NK], v[NV];
        u32x4 klo[4 * 64];                  // lo_operand of K
        float ks[4 * TILE];                 // K's s, in fp32 once for all rows
        float vs[4 * TILE], vmid[4 * TILE];  // and V's
        float vtop[kKeys];                  // log2 of each key's largest s of V
    };
    extern __shared__ __align__(16) uint8_t lds_raw[];
    Turn *const turns = (Turn *)lds_raw;
    Job j;
    if (!make_job<kRows>(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;
    const int t_end = min(j.u1 * 2, (j.kend + kKeys - 1) / kKeys);
    int turn = j.u0 * 2;
    const WaveAt<D, G> wat(a, j);
    const LaneAt<D, G> at(lane, a.pool);

    // the wave's rows: two column tiles of 16
    const int row_w = j.row0 + 32 * wave;
    u32x4 q[2][NW];
    u32x4 sums[2];
    float up[2];
    int k_lo[2], k_hi[2];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int row = row_w + 16 * ct + col, qi = row / a.R;
        const bool real = row < j.rows;
        const int pos = j.pos0 + qi;
        k_hi[ct] = a.causal ? min(j.len, pos + 1) : j.len;
        k_lo[ct] = a.window ? max(0, pos - a.window + 1) : 0;
        load_query<D, BF>(a, j, row, qi, h, real, q[ct]);
        const float sign = scale_query<D, BF>(a, q[ct], up[ct]);
#pragma unroll
        for (int s = 0; s < NW; ++s) q[ct][s] = query_operand<BF>(q[ct][s], sign);
        const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};  // 1
        float qs[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f32x4 c = {0, 0, 0, 0};
#pragma unroll
            for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma(ones, q[ct][s], c);
            qs[g] = c[0] * 0x1p-9f;
        }
        sums[ct] = sum_operand<NG>(qs, h);
    }
    // keys that some row of the wave sees, and that every row does
    const int last = min(row_w + 32, j.rows) - 1;
    const int any_hi = row_w >= j.rows ? 0 : a.causal ? min(j.len, j.pos0 + last / a.R + 1) : j.len;
    const int any_lo = a.window ? j.pos0 + row_w / a.R - a.window + 1 : 0;
    const int all_hi = a.causal ? min(j.len, j.pos0 + row_w / a.R + 1) : j.len;
    const int all_lo = a.window ? j.pos0 + last / a.R - a.window + 1 : 0;

    f32x4 o[2][NT];
    float z[2][NG], pass[2], ref[2], mu[2], l[2];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
#pragma unroll
        for (int c = 0; c < NT; ++c) o[ct][c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < NG; ++g) z[ct][g] = 0.0f;
        pass[ct] = ref[ct] = -__builtin_inff();
        mu[ct] = l[ct] = 0.0f;
    }
    bool bad_page = false;

    // this wave's tile of a turn: loaded, then laid out in LDS
    uint32_t kw[NW], vw[NW], kp[NP], vp[NP];
    int32_t page = 0;
    const auto fetch = [&](int t) {
        const uint32_t entry = (uint32_t)__builtin_amdgcn_readfirstlane(page);
        bad_page |= entry >= wat.n_pages;
        const uint32_t pg = entry < wat.n_pages ? entry : 0;
        const uint32_t in = (uint32_t)(wat.tile(2 * t, wave) & wat.mask);
        const uint8_t *codes = wat.codes + (uint64_t)pg * wat.page_codes + in * (8 * D);
        const uint8_t *params = wat.params + (uint64_t)pg * wat.page_params + in * 64;
        load_words<D, G>(kw, codes + at.k);
        load_words<D, G>(vw, codes + at.v);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            kp[i] = *(const uint32_t *)(params + at.kp[i]);
            vp[i] = *(const uint32_t *)(params + at.vp[i]);
        }
    };
    const auto look_up = [&](int t) { page = wat.table[wat.tile(2 * t, wave) >> wat.shift]; };
    const auto lay_out = [&](int t, Turn &to) {
#pragma unroll
        for (int s = 0; s < NW; ++s) to.k[(wave * NW + s) * 64 + lane] = code_octet(kw[s]);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int w = 2 * (c / 4);
            const u32x2 d = {centred_pair(vw[w], c & 3), centred_pair(vw[w + 1], c & 3)};
            *(u32x2 *)((uint8_t *)&to.v[((wave >> 1) * NT + c) * 64 + lane] + 8 * (wave & 1)) = d;
        }
        // what lies at keys that no row sees may be anything
        const int key = t * kKeys + 16 * wave + col;
        const bool in = key >= j.kbeg && key < j.kend;
        float s_top = 0.0f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            to.ks[wave * TILE + 64 * i + lane] = in ? s_of(kp[i]) : 0.0f;
            kp[i] = in ? kp[i] : 0;
            const float s = in ? s_of(vp[i]) : 0.0f;
            s_top = fmaxf(s_top, s);
            to.vs[wave * TILE + 64 * i + lane] = s;
            to.vmid[wave * TILE + 64 * i + lane] = in ? mid_of(vp[i]) : 0.0f;
        }
        to.klo[wave * 64 + lane] = lo_operand<NG>(kp, h);
        to.vtop[16 * wave + col] = log2_top<NG>(s_top);
    };
    if (turn < t_end) {
        look_up(turn);
        fetch(turn);
        look_up(turn + 1);
        lay_out(turn, turns[0]);
    }
    for (int side = 0; turn < t_end; ++turn, side ^= 1) {
        lds_barrier();
        const Turn &now = turns[side];
        fetch(turn + 1);  // past the end: the last tile again
        look_up(turn + 2);
        if (turn * kKeys < any_hi && (turn + 1) * kKeys > any_lo) {
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int key0 = turn * kKeys + 32 * half;
                const bool partial = key0 + 32 > all_hi || key0 < all_lo;
                f32x4 x[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const u32x4 klo = now.klo[(2 * half + t) * 64 + lane];
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) x[ct][t] = mfma(klo, sums[ct], f32x4{0, 0, 0, 0});
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                        for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                            const u32x4 k = now.k[((2 * half + t) * NW + s) * 64 + lane];
                            c[0] = mfma(k, q[0][s], c[0]);
                            c[1] = mfma(k, q[1][s], c[1]);
                        }
                        const f32x4 ks = *(const f32x4 *)&now.ks[(2 * half + t) * TILE + 16 * g + 4 * h];
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[ct][t][i] = __builtin_fmaf(ks[i], c[ct][i], x[ct][t][i]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                float mul[2] = {up[0], up[1]}, top[2];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    if (a.softcap > 0.0f) cap_logits(a.softcap, x[ct], mul[ct]);
                    if (partial)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int key = key0 + 16 * (i / 4) + 4 * h + i % 4;
                            if (key < k_lo[ct] || key >= k_hi[ct]) x[ct][i / 4][i % 4] = -__builtin_inff();
                        }
                    top[ct] = x[ct][0][0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) top[ct] = fmaxf(top[ct], x[ct][i / 4][i % 4]);
                }
                const f32x4 ls[2] = {*(const f32x4 *)&now.vtop[32 * half + 4 * h], *(const f32x4 *)&now.vtop[32 * half + 16 + 4 * h]};
                float most = ls[0][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) most = fmaxf(most, ls[i / 4][i % 4]);
                // the largest logit with the largest s: a bound, and rarely past (2048 queries over
                // 8192 keys 504 us, with each logit's own s 512)
                if (__any(__builtin_fmaf(top[0], mul[0], most) > pass[0] || __builtin_fmaf(top[1], mul[1], most) > pass[1])) {
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) {
                        float t = -__builtin_inff();
#pragma unroll
                        for (int i = 0; i < 8; ++i) t = fmaxf(t, __builtin_fmaf(x[ct][i / 4][i % 4], mul[ct], ls[i / 4][i % 4]));
                        const float f = rescale(t, pass[ct], ref[ct], mu[ct]);
                        l[ct] *= f;
#pragma unroll
                        for (int g = 0; g < NG; ++g) z[ct][g] *= f;
#pragma unroll
                        for (int c = 0; c < NT; ++c) o[ct][c] *= f;
                    }
                }
                float p[2][8];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        p[ct][i] = exp2_fast(__builtin_fmaf(x[ct][i / 4][i % 4], mul[ct], -mu[ct]));
                        l[ct] += p[ct][i];
                    }
#pragma unroll
                for (int g0 = 0; g0 < NG; g0 += GS) {
                    u32x4 hi[GS][2], lo[GS][2];
#pragma unroll
                    for (int j = 0; j < 2 * GS; ++j) {
                        const int g = g0 + j % GS, ct = j / GS;
                        f32x4 vs[2], vmid[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            vs[t] = *(const f32x4 *)&now.vs[(2 * half + t) * TILE + 16 * g + 4 * h];
                            vmid[t] = *(const f32x4 *)&now.vmid[(2 * half + t) * TILE + 16 * g + 4 * h];
                        }
                        if (partial) {
                            // a NaN there must not reach a row that does not see it
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (x[ct][i / 4][i % 4] == -__builtin_inff()) vmid[i / 4][i % 4] = 0.0f;
                        }
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float s0 = vs[i / 4][i % 4], s1 = vs[i / 4][i % 4 + 1];
                            z[ct][g] = __builtin_fmaf(p[ct][i], vmid[i / 4][i % 4], z[ct][g]);
                            z[ct][g] = __builtin_fmaf(p[ct][i + 1], vmid[i / 4][i % 4 + 1], z[ct][g]);
                            const f32x2 a2 = {p[ct][i] * s0, p[ct][i + 1] * s1};
                            const f16x2 t = __builtin_convertvector(a2, f16x2);
                            const f16x2 r = {(_Float16)__builtin_fmaf(p[ct][i], s0, -(float)t[0]),
                                             (_Float16)__builtin_fmaf(p[ct][i + 1], s1, -(float)t[1])};
                            hi[g - g0][ct][i / 2] = __builtin_bit_cast(uint32_t, t);
                            lo[g - g0][ct][i / 2] = __builtin_bit_cast(uint32_t, r);
                        }
                    }
#pragma unroll
                    for (int c = g0 * (G / 16); c < (g0 + GS) * (G / 16); ++c) {
                        if (c % 2 == 0) __builtin_amdgcn_sched_barrier(0);
                        const u32x4 v = now.v[(half * NT + c) * 64 + lane];
                        const int g = 16 * c / G - g0;
                        o[0][c] = mfma(v, hi[g][0], o[0][c]);
                        o[1][c] = mfma(v, hi[g][1], o[1][c]);
                        o[0][c] = mfma(v, lo[g][0], o[0][c]);
                        o[1][c] = mfma(v, lo[g][1], o[1][c]);
                    }
                }
            }
        }
        lay_out(turn + 1, turns[side ^ 1]);  // nobody reads that side before the next barrier, nor since the last
    }
    if (bad_page && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);

#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        l[ct] = row_sum(l[ct]);
#pragma unroll
        for (int g = 0; g < NG; ++g) z[ct][g] = row_sum(z[ct][g]);
        const int row = row_w + 16 * ct + col;
        if (row >= j.rows) continue;
        const int head = j.h * a.R + row % a.R;
        const int64_t tok = j.q0 + row / a.R, grow = tok * a.Hq + head;
        const int64_t prow = (int64_t)j.split * a.n_q * a.Hq + grow;
        const float inv = a.ns > 1 ? 1.0f : (l[ct] == 0.0f ? 0.0f : 1.0f / l[ct]);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = __builtin_fmaf(512.0f, o[ct][c][i], z[ct][16 * c / G]) * inv;
            if (a.ns > 1)
                *(f32x4 *)(a.part_o + prow * D + 16 * c + 4 * h) = y;
            else
                store_out<BF>(a, tok, head, 16 * c + 4 * h, y);
        }
        if (h == 0) {
            if (a.ns > 1) {
                a.part_ml[prow * 2] = ref[ct];
                a.part_ml[prow * 2 + 1] = l[ct];
            } else if (a.lse) {
                a.lse[grow] = lse_of(ref[ct], l[ct]);
            }
        }
    }
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

// Heads of 256 in groups of 32 have no blocks of 128 rows: those spilled 226
// registers a lane (512 queries over 4096 keys, 4 heads: 254 us, tiles of 16 rows
// 246; 1024 over 8192, 8 heads: 1730 : 1361).
constexpr bool has_prompt(int D, int G) { return D != 256 || G != 32; }

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const int64_t blocks = (int64_t)a.ns * a.pool.H * a.B * a.tiles;
    hipError_t e;
    if (!a.prompt) {
        k_kv4_attn<D, G, BF><<<dim3((uint32_t)blocks), dim3(64 * kWaves), 0, s>>>(a);
    } else if constexpr (has_prompt(D, G)) {
        constexpr int lds = 2 * (4 * (D / 32) * 1024 + 2 * (D / 16) * 1024 + 4 * 1024 + 3 * 4 * 64 * Stage<D, G>::NP * 4 + kKeys * 4);
        // above 64 KB LDS has to be asked for; the attribute is per device, and cheap
        if (lds > 65536) {
            e = hipFuncSetAttribute((const void *)k_kv4_prompt<D, G, BF>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            if (e != hipSuccess) return e;
        }
        k_kv4_prompt<D, G, BF><<<dim3((uint32_t)blocks), dim3(256), lds, s>>>(a);
    }
    e = hipGetLastError();
    if (e == hipSuccess && a.ns > 1) {
        const dim3 rows((uint32_t)(std::min(a.n_q, (int64_t)a.B * a.max_q) * a.Hq));  // as many as sequences may have
        if (a.ns <= 8)
            k_kv4_join<D, BF, 64><<<rows, dim3(64), 0, s>>>(a);
        else
            k_kv4_join<D, BF, 512><<<rows, dim3(512), 0, s>>>(a);  // 64 splits of 64 rows: 4.7 us; 79 by 256 threads a third longer
        e = hipGetLastError();
    }
    return e;
}

template <int D, int G>
hipError_t attend_dt(const Kv4Attn &a, bool bf16, hipStream_t s)
{
    return bf16 ? attend<D, G, true>(a, s) : attend<D, G, false>(a, s);
}

}  // namespace

// Which kernel, and how many ways a row's keys are split.
//
// Blocks of 128 rows unpack a key once for all of them, but are few and long:
// they are taken where every sequence may fill one, the keys are 2048 or more
// and blocks and thousands of keys together occupy the chip (8 kv heads of
// 128, R = 4, us a call with its join, this kernel : tiles of 16 rows: 2048
// queries over 8192 keys 505 : 662, 2 x 512 over 4096 156 : 193, 8 x 32 over
// 4096 57 : 73, 128 over 16000 101 : 118, 512 over 4096 with 4 heads of 256
// 149 : 196; not for 1 x 64 over 4096 41 : 28, nor 1024 over 1024 55 : 43).
// Split: two blocks a compute unit (2 x up to 512 over up to 4096, fp16, in two
// 155, unsplit 212, in eight 187), 512 keys or more each.
//
// Tiles of 16 rows: a split costs a block's start and its part of the join, so
// 512 keys or fewer are not split (1 x 300 keys 9.2 us, in two 10.9), else it
// gets at least 256 keys while the blocks are fewer than the compute units,
// 512 up to two blocks a unit (D = 256: a unit holds one), 1024 beyond, up to
// eight a unit, which even out unequal sequences (us a call, this rule against
// its neighbours: 1 x 4000 keys 11.7, in 8 14.7, in 64 14.2; 1 x 16000 15.2, in
// 16 18.8, in 64 16.5; 64 x up to 8192 93, unsplit 106, in 8 99; 64 x up to
// 1000 20, in two 27).  Fewer than four blocks a unit are rounded down to as
// many on every unit where that takes no more than a quarter of them (on 8
// heads 1 x 80000, 79 ways 35, 64 ways 32; 1 x 100000, 98 ways 43, 96 ways 37;
// 2 x 40000, 40 ways 33, 32 ways 30).
namespace {

int64_t prompt_splits(const Kv4Pool &p, int64_t blocks, int64_t keys)
{
    const int64_t ns = std::min((p.D == 256 ? 256 : 512) / blocks, (keys + 511) / 512);
    return std::min<int64_t>(std::max<int64_t>(ns, 1), 128);
}

int64_t narrow_splits(const Kv4Pool &p, int64_t blocks, int64_t keys)
{
    const int64_t level[3][2] = {{256, 256}, {p.D == 256 ? 256 : 512, 512}, {2048, 1024}};  // blocks, keys
    int64_t ns = 1;
    if (keys > 512)
        for (int i = 0; i < 3; ++i) ns = std::max(ns, std::min(level[i][0] / blocks, (keys + level[i][1] - 1) / level[i][1]));
    ns = std::min<int64_t>(ns, 128);
    const int64_t even = ns * blocks / 256 * 256 / blocks;
    return ns * blocks < 1024 && even * 4 >= ns * 3 ? even : ns;
}

}  // namespace

Kv4Plan kv4_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window)
{
    Kv4Plan plan;
    // keys that a block of `rows` rows sees at most
    const auto keys_of = [&](int rows) { return window ? std::min(max_keys, window + rows / R + 1) : max_keys; };
    const int64_t wide_tiles = (max_q * R + kRows - 1) / kRows, tiles = (max_q * R + 15) / 16;
    const int64_t wide = std::max<int64_t>(n_seqs * p.H * wide_tiles, 1), narrow = std::max<int64_t>(n_seqs * p.H * tiles, 1);
    const int64_t keys = keys_of(kRows);
    plan.prompt = has_prompt(p.D, p.G) && max_q * R >= kRows && keys >= 2048 && wide * ((keys + 1023) / 1024) >= 256;
    plan.tiles = (int32_t)(plan.prompt ? wide_tiles : tiles);
    plan.ns = (int32_t)(plan.prompt ? prompt_splits(p, wide, keys) : narrow_splits(p, narrow, keys_of(16)));
    // either kernel's splits grow with the keys, so no window takes more than these
    plan.most_ns = (int32_t)std::max(narrow_splits(p, narrow, max_keys), plan.prompt ? prompt_splits(p, wide, max_keys) : 1);
    return plan;
}

hipError_t launch_kv4_attention(const Kv4Attn &a, bool bf16, hipStream_t stream)
{
    switch (a.pool.D * 1000 + a.pool.G) {
    case 64032: return attend_dt<64, 32>(a, bf16, stream);
    case 64064: return attend_dt<64, 64>(a, bf16, stream);
    case 128032: return attend_dt<128, 32>(a, bf16, stream);
    case 128064: return attend_dt<128, 64>(a, bf16, stream);
    case 128128: return attend_dt<128, 128>(a, bf16, stream);
    case 256032: return attend_dt<256, 32>(a, bf16, stream);
    case 256064: return attend_dt<256, 64>(a, bf16, stream);
    default: return attend_dt<256, 128>(a, bf16, stream);
    }
}
