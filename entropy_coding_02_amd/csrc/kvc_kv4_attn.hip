// kvc_kv4_attn.hip - attention over the resident 4-bit cache.
//
// With n a code (0..15) and m = 1 + n/16, a cached value is y = lo + 16 s (m - 1).
// m has at most 5 significant bits and its bits are the code's under a constant
// exponent, so one shift and one and-or turn two codes into two exact 16-bit
// matrix operands, and (s, lo) never touch them:
//   logits   q.k = sum_g s_g * 16 (sum_{c in g} q_c m_c - qs_g) + lo_g * qs_g,  qs_g = sum_{c in g} q_c;
//            the products are exact, -qs_g is the accumulator's start;
//   output   o_c = 16 sum_j (p_j s_jg) m_jc + sum_j p_j (lo_jg - 16 s_jg),  c in group g.
// p_j s_jg goes into the matrix product as two bf16 terms (17 bits; bf16
// because s spans the fp16 range), whatever the type of q: one rounding to 8
// or 11 bits would be an error of the output's own size, since m is up to
// four times the value it stands for.
//
// Orientation: S^T = K q^T (16 keys x 16 query rows), so a lane holds one
// query row and four keys of a tile, which is just what P^T needs as the
// right operand of O^T = V^T P^T (keys 4h .. 4h+3 of two tiles are its eight
// k indices): probabilities never cross lanes, the terms with lo and the row
// sums are plain fp32 sums per lane, added over the four lanes of a row once
// at the end.
#include "kvc_kernels.h"
#include "kvc_kv4.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;

template <bool BF>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Nibble I of both halves of w as a pair of 1 + n/16.
template <bool BF, int I>
__device__ __forceinline__ uint32_t unit_pair(uint32_t w)
{
    constexpr int at = BF ? 3 : 6;  // the code's place below the exponent
    constexpr uint32_t mask = 0x000F000Fu << at, one = BF ? 0x3F803F80u : 0x3C003C00u;
    const uint32_t x = 4 * I <= at ? w << (at - 4 * I) : w >> (4 * I - at);
    return (x & mask) | one;
}

// A K dword (8 channels of a key) as 8 operands in the order 0,4,1,5,2,6,3,7.
template <bool BF>
__device__ __forceinline__ u32x4 k_operand(uint32_t w)
{
    return u32x4{unit_pair<BF, 0>(w), unit_pair<BF, 1>(w), unit_pair<BF, 2>(w), unit_pair<BF, 3>(w)};
}

__device__ __forceinline__ float s_of(uint32_t w) { return kvc_h2f(w & 0xFFFF); }
__device__ __forceinline__ float lo_of(uint32_t w) { return kvc_h2f(w >> 16); }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Over the four lanes (16 apart) of a query row.
__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// From a row's maximum and sum in powers of 2; a row without keys has L = 0, a
// row that met a NaN has L = NaN (its maximum may be -inf).
__device__ __forceinline__ float lse_of(float M, float L)
{
    return L == 0.0f ? -__builtin_inff() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// What a wave loads for 32 keys: two tiles of 16.
template <int D, int G>
struct Stage {
    static constexpr int NW = D / 32, NG = D / G;
    uint32_t k[2][NW], v[2][NW];
    u32x4 kp[2][NG], vp[2][NG];
};

template <int D, int G>
__device__ __forceinline__ void load_words(uint32_t *dst, const uint8_t *src)
{
    constexpr int NW = D / 32;
    if (NW == 2) {
        const u32x2 w = *(const u32x2 *)src;
        dst[0] = w[0], dst[1] = w[1];
    } else {
        for (int i = 0; i < NW / 4; ++i) {
            const u32x4 w = *(const u32x4 *)(src + 16 * i);
            for (int j = 0; j < 4; ++j) dst[4 * i + j] = w[j];
        }
    }
}

// What a block works on: one (sequence, kv head), 16 of its query rows (row =
// query * R + head within the group), one split of their keys.
struct Job {
    int b, h, split, tile;
    int nq, q0, len, pos0, rows, row0;
    int kbeg, kend;  // keys that some row of the tile sees
    int u0, u1;      // the split's units of 128 keys
};

__device__ __forceinline__ bool make_job(const Kv4Attn &a, Job &j)
{
    uint32_t id = blockIdx.x;
    j.split = id % a.ns, id /= a.ns;
    j.h = id % a.pool.H, id /= a.pool.H;
    j.b = id % a.B;
    j.tile = id / a.B;
    bool bad = false;
    int64_t c0 = a.cu_q ? a.cu_q[j.b] : (int64_t)j.b * a.max_q;
    int64_t c1 = a.cu_q ? a.cu_q[j.b + 1] : c0 + a.max_q;
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
    j.len = a.kv_len[j.b];
    if (j.len > cap) bad = true, j.len = cap;
    if (j.len < 0) j.len = 0;
    if (bad && j.tile == 0 && threadIdx.x == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
    j.rows = j.nq * a.R;
    j.row0 = j.tile * 16;
    if (j.row0 >= j.rows) return false;
    j.pos0 = j.len - j.nq;
    const int last = j.row0 + 15 < j.rows ? j.row0 + 15 : j.rows - 1;
    const int i_lo = j.row0 / a.R, i_hi = last / a.R;
    j.kend = a.causal ? min(j.len, j.pos0 + i_hi + 1) : j.len;
    j.kbeg = a.window ? max(0, j.pos0 + i_lo - a.window + 1) : 0;
    if (j.kend <= j.kbeg) {
        j.kbeg = j.kend = j.u0 = j.u1 = 0;
        return true;
    }
    const int f = j.kbeg / 128, n = (j.kend + 127) / 128 - f;
    j.u0 = f + (int)((int64_t)n * j.split / a.ns);
    j.u1 = f + (int)((int64_t)n * (j.split + 1) / a.ns);
    return true;
}

template <int D, int G>
__device__ __forceinline__ void load_stage(const Kv4Attn &a, const Job &j, int blk, int lane, Stage<D, G> &st)
{
    constexpr int NG = D / G;
    const int r = lane & 15, h = lane >> 4;
    const int P = 1 << a.pool.pshift;
    const int t_lo = j.kbeg >> 4, t_hi = (j.kend - 1) >> 4;
    for (int t = 0; t < 2; ++t) {
        // a tile that no row sees is read from one that some row does
        const int kt = min(max(blk * 2 + t, t_lo), t_hi);
        int64_t page = a.table[j.b * a.table_stride + (kt >> (a.pool.pshift - 4))];
        if (page < 0 || page >= a.pool.n_pages) {
            if (lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
            page = 0;
        }
        const int off = (kt << 4) & (P - 1);
        const int64_t kb = kv4_block(a.pool, page, 0, j.h), vb = kb + a.pool.H;
        load_words<D, G>(st.k[t], a.pool.codes + kb * (P * (D / 2)) + (off + r) * (D / 2) + h * (D / 8));
        load_words<D, G>(st.v[t], a.pool.codes + vb * (P * (D / 2)) + (off / 4 + h) * (2 * D) + r * (D / 8));
        for (int g = 0; g < NG; ++g) {
            st.kp[t][g] = *(const u32x4 *)(a.pool.params + (kb * NG + g) * P + off + 4 * h);
            st.vp[t][g] = *(const u32x4 *)(a.pool.params + (vb * NG + g) * P + off + 4 * h);
        }
    }
}

template <int D, int G, bool BF>
__global__ __launch_bounds__(64 * kWaves) void k_kv4_attn(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16;
    __shared__ float lds_o[kWaves][16][D];
    __shared__ float lds_ml[kWaves][2][16];
    Job j;
    if (!make_job(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;
    const int row = j.row0 + col, qi = row / a.R;
    const bool real = row < j.rows;
    const int pos = j.pos0 + qi;
    const int k_hi = a.causal ? min(j.len, pos + 1) : j.len;      // keys k_lo <= key < k_hi
    const int k_lo = a.window ? max(0, pos - a.window + 1) : 0;
    // keys that every row of the tile sees
    const int all_hi = a.causal ? min(j.len, j.pos0 + j.row0 / a.R + 1) : j.len;
    const int all_lo = a.window ? j.pos0 + min(j.row0 + 15, j.rows - 1) / a.R - a.window + 1 : 0;

    // query operands in the codes' order, and the group sums of q as accumulators
    u32x4 q[NW];
    f32x4 neg_qs[NG];
    float qs16[NG];
    {
        const uint16_t *src = a.q + (int64_t)(j.q0 + qi) * a.q_ts + (int64_t)(j.h * a.R + row % a.R) * a.q_hs + 8 * h;
        for (int s = 0; s < NW; ++s) {
            u32x4 w = {0, 0, 0, 0};
            if (real) {
                if (a.q_vec)
                    w = *(const u32x4 *)(src + 32 * s);
                else
                    for (int i = 0; i < 4; ++i) w[i] = src[32 * s + 2 * i] | (uint32_t)src[32 * s + 2 * i + 1] << 16;
            }
            q[s] = u32x4{(w[0] & 0xFFFF) | w[2] << 16, w[0] >> 16 | (w[2] & 0xFFFF0000u),
                         (w[1] & 0xFFFF) | w[3] << 16, w[1] >> 16 | (w[3] & 0xFFFF0000u)};
        }
        constexpr uint32_t one = BF ? 0xBF80BF80u : 0xBC00BC00u;  // -1
        const u32x4 ones = {one, one, one, one};
        for (int g = 0; g < NG; ++g) {
            f32x4 c = {0, 0, 0, 0};
            for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma<BF>(ones, q[s], c);
            neg_qs[g] = c;
            qs16[g] = -c[0] * (1.0f / 16.0f);
        }
    }
    const float c2 = 16.0f * a.scale * (a.softcap > 0.0f ? 1.0f : kLog2e);

    f32x4 o[NT];
    float z[NG], m = -__builtin_inff(), l = 0.0f;
    for (int c = 0; c < NT; ++c) o[c] = f32x4{0, 0, 0, 0};
    for (int g = 0; g < NG; ++g) z[g] = 0.0f;

    const int b_end = min(j.u1 * 4, (j.kend + 31) / 32);
    Stage<D, G> cur, nxt;
    int blk = j.u0 * 4 + wave;
    if (blk < b_end) load_stage<D, G>(a, j, blk, lane, cur);
    for (; blk < b_end; blk += kWaves) {
        if (blk + kWaves < b_end) load_stage<D, G>(a, j, blk + kWaves, lane, nxt);
        const int key0 = blk * 32;
        float x[2][4];
        for (int t = 0; t < 2; ++t) {
            f32x4 s4 = {0, 0, 0, 0};
            for (int g = 0; g < NG; ++g) {
                f32x4 c = neg_qs[g];
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma<BF>(k_operand<BF>(cur.k[t][s]), q[s], c);
                for (int i = 0; i < 4; ++i)
                    s4[i] = __builtin_fmaf(lo_of(cur.kp[t][g][i]), qs16[g], __builtin_fmaf(s_of(cur.kp[t][g][i]), c[i], s4[i]));
            }
            for (int i = 0; i < 4; ++i) x[t][i] = s4[i] * c2;
        }
        if (a.softcap > 0.0f) {
            // tanh(y) = 1 - 2 / (exp(2y) + 1)
            const float c = 2.0f * kLog2e / a.softcap, top = a.softcap * kLog2e;
            for (int t = 0; t < 2; ++t)
                for (int i = 0; i < 4; ++i) x[t][i] = top - 2.0f * top * __builtin_amdgcn_rcpf(exp2_fast(x[t][i] * c) + 1.0f);
        }
        if (key0 + 32 > all_hi || key0 < all_lo) {
            for (int t = 0; t < 2; ++t)
                for (int i = 0; i < 4; ++i) {
                    const int key = key0 + 16 * t + 4 * h + i;
                    if (key < k_lo || key >= k_hi) {
                        x[t][i] = -__builtin_inff();
                        // what lies there may be anything, NaN too
                        for (int g = 0; g < NG; ++g) cur.vp[t][g][i] = 0;
                    }
                }
        }
        float mx = x[0][0];
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i / 4][i % 4]);
        mx = row_max(mx);
        if (__any(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -__builtin_inff() ? 1.0f : exp2_fast(m - mn);
            m = mn;
            l *= f;
            for (int g = 0; g < NG; ++g) z[g] *= f;
            for (int c = 0; c < NT; ++c) o[c] *= f;
        }
        const float mu = m == -__builtin_inff() ? 0.0f : m;
        float p[2][4];
        for (int t = 0; t < 2; ++t)
            for (int i = 0; i < 4; ++i) {
                p[t][i] = exp2_fast(x[t][i] - mu);
                l += p[t][i];
            }
        for (int g = 0; g < NG; ++g) {
            u32x4 hi, lo;
            for (int t = 0; t < 2; ++t)
                for (int i = 0; i < 4; i += 2) {
                    const uint32_t w0 = cur.vp[t][g][i], w1 = cur.vp[t][g][i + 1];
                    const float a0 = p[t][i] * s_of(w0), a1 = p[t][i + 1] * s_of(w1);
                    z[g] = __builtin_fmaf(p[t][i], lo_of(w0), z[g]);
                    z[g] = __builtin_fmaf(p[t][i + 1], lo_of(w1), z[g]);
                    z[g] = __builtin_fmaf(-16.0f, a0, z[g]);
                    z[g] = __builtin_fmaf(-16.0f, a1, z[g]);
                    const uint32_t hp = bf16_pair(a0, a1);
                    hi[2 * t + i / 2] = hp;
                    lo[2 * t + i / 2] = bf16_pair(a0 - __builtin_bit_cast(float, hp << 16),
                                                  a1 - __builtin_bit_cast(float, hp & 0xFFFF0000u));
                }
            for (int c = g * (G / 16); c < (g + 1) * (G / 16); ++c) {
                const int w = 2 * (c / 4);
                u32x4 va;
                for (int i = 0; i < 4; ++i) {
                    const uint32_t d = cur.v[i / 2][w + (i & 1)];
                    va[i] = (c & 3) == 0 ? unit_pair<true, 0>(d) : (c & 3) == 1 ? unit_pair<true, 1>(d)
                          : (c & 3) == 2 ? unit_pair<true, 2>(d) : unit_pair<true, 3>(d);
                }
                o[c] = mfma<true>(va, hi, o[c]);
                o[c] = mfma<true>(va, lo, o[c]);
            }
        }
        cur = nxt;
    }

    // the four waves' parts: out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
    l = row_sum(l);
    for (int g = 0; g < NG; ++g) z[g] = row_sum(z[g]);
    for (int c = 0; c < NT; ++c) {
        f32x4 y;
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(16.0f, o[c][i], z[16 * c / G]);
        *(f32x4 *)&lds_o[wave][col][16 * c + 4 * h] = y;
    }
    if (h == 0) {
        lds_ml[wave][0][col] = m;
        lds_ml[wave][1][col] = l;
    }
    __syncthreads();
    // 16 threads a row
    const int mr = threadIdx.x / 16, part = threadIdx.x % 16;
    const int orow = j.row0 + mr;
    if (orow >= j.rows) return;
    float M = -__builtin_inff(), L = 0.0f, wgt[kWaves];
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[w][0][mr]);
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
        for (int w = 0; w < kWaves; ++w) y += wgt[w] * *(const f32x4 *)&lds_o[w][mr][c];
        y *= inv;
        if (a.ns > 1) {
            *(f32x4 *)(a.part_o + prow * D + c) = y;
        } else {
            uint16_t *dst = a.out + tok * a.o_ts + head * a.o_hs + c;
            const u32x2 w = {BF ? bf16_pair(y[0], y[1]) : kvc_f2h2(y[0], y[1]), BF ? bf16_pair(y[2], y[3]) : kvc_f2h2(y[2], y[3])};
            if (a.o_vec) {
                *(u32x2 *)dst = w;
            } else {
                for (int i = 0; i < 4; ++i) dst[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            }
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

// Joins the splits of a row: one wave a row, D/64 channels a lane.
template <int D, bool BF>
__global__ __launch_bounds__(256) void k_kv4_join(Kv4Attn a)
{
    const int64_t rows = a.n_q * a.Hq, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= rows) return;
    float M = -__builtin_inff();
    for (int s = lane; s < a.ns; s += 64) M = fmaxf(M, a.part_ml[(s * rows + row) * 2]);
    for (int off = 32; off; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, 64));
    float y[D / 64] = {}, L = 0.0f;
    for (int s = 0; s < a.ns; ++s) {
        const float ms = a.part_ml[(s * rows + row) * 2], ls = a.part_ml[(s * rows + row) * 2 + 1];
        if (ls == 0.0f) continue;  // no keys
        const float w = exp2_fast(ms - M);
        L += w * ls;
        for (int i = 0; i < D / 64; ++i) y[i] += w * a.part_o[(s * rows + row) * D + lane + 64 * i];
    }
    const int64_t tok = row / a.Hq;
    const int head = (int)(row % a.Hq);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    for (int i = 0; i < D / 64; ++i) {
        const float v = y[i] * inv;
        a.out[tok * a.o_ts + head * a.o_hs + lane + 64 * i] =
            BF ? __builtin_bit_cast(uint16_t, (__bf16)v) : (uint16_t)kvc_f2h(v);
    }
    if (a.lse && lane == 0) a.lse[row] = lse_of(M, L);
}

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const int64_t blocks = (int64_t)a.ns * a.pool.H * a.B * a.tiles;
    k_kv4_attn<D, G, BF><<<dim3((uint32_t)blocks), dim3(64 * kWaves), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.ns > 1) {
        k_kv4_join<D, BF><<<dim3((uint32_t)((a.n_q * a.Hq + 3) / 4)), dim3(256), 0, s>>>(a);
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

Kv4Plan kv4_plan(int64_t n_seqs, int H, int R, int64_t max_q, int64_t max_keys)
{
    Kv4Plan p;
    p.tiles = (int32_t)((max_q * R + 15) / 16);
    const int64_t blocks = n_seqs * H * p.tiles;
    const int64_t units = (max_keys + 127) / 128;
    int64_t ns = blocks ? 1024 / blocks : 1;
    ns = ns < units ? ns : units;
    ns = ns < 128 ? ns : 128;
    p.ns = (int32_t)(ns < 1 ? 1 : ns);
    return p;
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
