// kvc_kv4_tree.hip - attention of a tree of drafted tokens over the resident
// 4-bit cache.
//
// The arithmetic is that of kvc_kv4_attn.hip (codes as matrix operands, s and lo
// outside of them, p s as two fp16 terms); what differs is which keys a row sees
// and how many rows there are: a tree's tokens times the heads of a group,
// typically 32 to 512, all over the same keys.  A wave therefore works on
// CT tiles of 16 rows at once and unpacks a block of 32 keys once for all of them.
//
// Of the drafted keys a row sees its own path.  A block that holds such keys
// walks the parents of its tokens once, in LDS, and keeps the path as bits, one word
// per token and block of 32 keys.
#include <algorithm>
#include <type_traits>

#include "kv4_tile.h"

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kWords = (kTreeMost + 62) / 32;  // blocks of 32 keys that a tree's may lie in

// The walk: bits[token of the tile][word] and the steps of each token's path.
// Word w is the block of keys 32 (first + w) .. + 31; bit k its key k.
struct Paths {
    uint32_t *bits;
    int first, words;  // of the blocks, and how many
    int base;          // keys before the tree
};

// Stages the parents of the sequence's tokens up to the tile's last; a bad one
// becomes -1, so that every walk ends.
__device__ __forceinline__ void stage_parents(const Kv4Attn &a, const Job &j, int last, int16_t *parent)
{
    bool bad = false;
    for (int i = threadIdx.x; i <= last; i += 64 * kWaves) {
        int p = a.parents[j.q0 + i];
        if (p < -1 || p >= i) bad = true, p = -1;
        parent[i] = (int16_t)p;
    }
    if (bad) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
}

// One thread a token of the tile (first_tok .. last_tok): its path's bits, and
// its length.  Keys below 0 do not exist.
__device__ __forceinline__ void walk(const Kv4Attn &a, const Paths &p, const int16_t *parent, int first_tok, int last_tok, int16_t *steps)
{
    const int i = threadIdx.x, tok = first_tok + i;
    if (tok > last_tok) return;
    uint32_t *const row = p.bits + i * p.words;
    for (int w = 0; w < p.words; ++w) row[w] = 0;
    int n = 0;
    for (int cur = tok; cur >= 0; cur = parent[cur], ++n) {
        const int key = p.base + cur;
        if (key >= 0 && (a.window == 0 || n < a.window)) row[(key >> 5) - p.first] |= 1u << (key & 31);
    }
    steps[i] = (int16_t)n;
}

// What an fp16 term of x leaves, as another.  A product by 1 so that it is one instruction.
__device__ __forceinline__ uint32_t rest_of(f32x2 x, f16x2 t)
{
    const f32x2 r = {__builtin_fmaf((float)t[0], -1.0f, x[0]), __builtin_fmaf((float)t[1], -1.0f, x[1])};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(r, f16x2));
}

template <int D, int G, bool BF, int CT>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void k_kv4_tree(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = Stage<D, G>::NP, TILE = 64 * NP, ROWS = 16 * CT;
    // Each wave's results, a tile of rows at a time; while it runs, its parameters (as in
    // k_kv4_attn).
    __shared__ __align__(16) float lds_o[kWaves][16][D];
    __shared__ float lds_ml[kWaves][2][ROWS];
    __shared__ u32x4 lds_q[CT][NW][64];
    __shared__ uint32_t lds_bits[ROWS * kWords];
    __shared__ int16_t lds_parent[kTreeMost], lds_steps[ROWS];
    Job j;
    if (!make_job<ROWS, true>(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;
    float *const prm = &lds_o[wave][0][0];
    static_assert(6 * TILE + 32 <= 16 * D, "the parameters fit where the results go");
    const int b_end = min(j.u1 * 4, (j.kend + 31) / 32);
    int blk = j.u0 * 4 + wave;
    const bool work = blk < b_end;
    const WaveAt<D, G> wat(a, j);

    const int last_row = min(j.row0 + ROWS, j.rows) - 1;
    const int tok0 = j.row0 / a.R, tok1 = last_row / a.R;  // the tile's tokens
    Paths paths;
    paths.bits = lds_bits;
    paths.base = j.pos0;
    paths.first = max(j.pos0, 0) >> 5;
    paths.words = max(((j.kend + 31) >> 5) - paths.first, 0);
    const bool walks = b_end > paths.first || a.window;  // the same for the whole block
    if (walks) stage_parents(a, j, tok1, lds_parent);

    int32_t first[2] = {0, 0}, pages[2] = {0, 0};
    float up[CT];
    if (work) {
        load_pages(wat, blk, first);
        load_pages(wat, blk + kWaves, pages);
    }
    // a tile's queries are laid out by every wave in turn, a part of the channels each
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = j.row0 + 16 * ct + col;
        u32x4 qw[NW];
        load_query<D, BF>(a, j, row, row / a.R, h, row < j.rows, qw);
        const float f = scale_query<D, BF>(a, qw, up[ct]);
#pragma unroll
        for (int s = 0; s < NW; ++s)
            if (wave == s % kWaves) lds_q[ct][s][lane] = query_operand<BF>(qw[s], f);
    }
    lds_barrier();
    if (walks) {
        walk(a, paths, lds_parent, tok0, tok1, lds_steps);
        lds_barrier();
    }

    f32x4 o[CT][NT];
    float z[CT][NG], pass[CT], ref[CT], mu[CT], l[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int c = 0; c < NT; ++c) o[ct][c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < NG; ++g) z[ct][g] = 0.0f;
        pass[ct] = ref[ct] = -__builtin_inff();
        mu[ct] = l[ct] = 0.0f;
    }
    if (work) {
        const LaneAt<D, G> at(lane, a.pool);
        Stage<D, G> cur, next;
        bool bad_page = false;
        load_stage<D, G>(wat, blk, first, at, cur, bad_page);

        u32x4 sums[CT];
        int k_lo[CT];  // the first key before the tree that the lane's row sees
        const uint32_t *bits[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};  // 1
            float qs[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c = {0, 0, 0, 0};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) c = mfma(ones, lds_q[ct][s][lane], c);
                qs[g] = c[0] * 0x1p-9f;
            }
            sums[ct] = sum_operand<NG>(qs, h);
            const int i = min(j.row0 + 16 * ct + col, last_row) / a.R - tok0;
            bits[ct] = lds_bits + i * paths.words;
            k_lo[ct] = a.window ? max(0, j.pos0 + lds_steps[i] - a.window) : 0;
        }
        // keys that every row of the tile sees: those before the tree, with a window those of its longest path
        const int all_lo = a.window ? j.pos0 + j.nq - a.window : 0;
        // a block of keys, and the next one's on their way; masks: some rows may not see some of its keys
        const auto step = [&](auto masks, Stage<D, G> &cur, Stage<D, G> &next) {
            int32_t after[2];
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
            f32x4 x[CT][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const u32x4 klo = lo_operand<NG>(cur.kp[t], h);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) x[ct][t] = mfma(klo, sums[ct], f32x4{0, 0, 0, 0});
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c[CT][2];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) c[ct][0] = c[ct][1] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                    const u32x4 k0 = code_octet(cur.k[0][s]), k1 = code_octet(cur.k[1][s]);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        const u32x4 q = lds_q[ct][s][lane];
                        c[ct][0] = mfma(k0, q, c[ct][0]);
                        c[ct][1] = mfma(k1, q, c[ct][1]);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 ks = *(const f32x4 *)&prm[t * TILE + 16 * g + 4 * h];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[ct][t][i] = __builtin_fmaf(ks[i], c[ct][t][i], x[ct][t][i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            float mul[CT], p[CT][8];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                mul[ct] = up[ct];
                if (a.softcap > 0.0f) cap_logits(a.softcap, x[ct], mul[ct]);
                if (masks) {
                    // keys before the tree from k_lo on, and the path's
                    const int n = min(max(j.pos0 - key0, 0), 32), m = min(max(k_lo[ct] - key0, 0), 32);
                    uint32_t see = (uint32_t)((1ull << n) - 1) & ~(uint32_t)((1ull << m) - 1);
                    if (blk >= paths.first) see |= bits[ct][blk - paths.first];
                    see >>= 4 * h;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!(see >> (16 * (i / 4) + i % 4) & 1)) x[ct][i / 4][i % 4] = -__builtin_inff();
                }
                float top = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 ls = *(const f32x4 *)&prm[6 * TILE + 16 * t + 4 * h];
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, __builtin_fmaf(x[ct][t][i], mul[ct], ls[i]));
                }
                if (__any(top > pass[ct])) {
                    const float f = rescale(top, pass[ct], ref[ct], mu[ct]);
                    l[ct] *= f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) z[ct][g] *= f;
#pragma unroll
                    for (int c = 0; c < NT; ++c) o[ct][c] *= f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[ct][i] = exp2_fast(__builtin_fmaf(x[ct][i / 4][i % 4], mul[ct], -mu[ct]));
                    l[ct] += p[ct][i];
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                u32x4 hi[CT], lo[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    f32x4 vs[2], vmid[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        vs[t] = *(const f32x4 *)&prm[(2 * t + 2) * TILE + 16 * g + 4 * h];
                        vmid[t] = *(const f32x4 *)&prm[(2 * t + 3) * TILE + 16 * g + 4 * h];
                    }
                    if (masks) {
                        // what lies at a key that the row does not see may be anything, NaN too
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (x[ct][i / 4][i % 4] == -__builtin_inff()) vs[i / 4][i % 4] = vmid[i / 4][i % 4] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float s0 = vs[i / 4][i % 4], s1 = vs[i / 4][i % 4 + 1];
                        const float p0 = p[ct][i], p1 = p[ct][i + 1];
                        z[ct][g] = __builtin_fmaf(p0, vmid[i / 4][i % 4], z[ct][g]);
                        z[ct][g] = __builtin_fmaf(p1, vmid[i / 4][i % 4 + 1], z[ct][g]);
                        const f32x2 a2 = {p0 * s0, p1 * s1};
                        const f16x2 t = __builtin_convertvector(a2, f16x2);
                        hi[ct][i / 2] = __builtin_bit_cast(uint32_t, t);
                        lo[ct][i / 2] = rest_of(a2, t);
                    }
                }
#pragma unroll
                for (int c = g * (G / 16); c < (g + 1) * (G / 16); c += 2) {
                    if (c % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                    const int w = 2 * (c / 4);
                    u32x4 va[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        va[k] = u32x4{centred_pair(cur.v[0][w], (c & 3) + k), centred_pair(cur.v[0][w + 1], (c & 3) + k),
                                      centred_pair(cur.v[1][w], (c & 3) + k), centred_pair(cur.v[1][w + 1], (c & 3) + k)};
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        o[ct][c] = mfma(va[0], hi[ct], o[ct][c]);
                        o[ct][c + 1] = mfma(va[1], hi[ct], o[ct][c + 1]);
                    }
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        o[ct][c] = mfma(va[0], lo[ct], o[ct][c]);
                        o[ct][c + 1] = mfma(va[1], lo[ct], o[ct][c + 1]);
                    }
                }
            }
            blk += kWaves;
        };
        // Blocks that every row sees whole in a loop of their own, two at a time: sums and keys then stay in their registers.
        // Where registers are short already the second loop costs more: 16 sequences of up to 8192 keys, 8 KV heads, trees of
        // 96 rows, D = 128 G = 64 119 us (without 123); of 128 rows G = 32 225 (215); 8 sequences with D = 256, G = 32 551 (399),
        // G = 64 236 (198); 64 sequences of 16 rows, which lose a third wave a SIMD, 141 (129).
        constexpr bool APART = CT > 1 && D <= 128 && 64 * D <= 128 * G;
        const int from = (max(all_lo, 0) + 31) / 32, until = min(b_end, max(j.pos0, 0) / 32);
        while (blk < b_end) {
            if (APART && blk >= from) {
                while (blk + kWaves < until) {
                    step(std::false_type(), cur, next);
                    step(std::false_type(), next, cur);
                }
                if (blk >= b_end) break;
            }
            if constexpr (APART)
                step(std::true_type(), cur, next);
            else
                step(blk < from || blk >= until, cur, next);
            cur = next;
        }
        if (bad_page && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);
    }

    // the four waves' parts, a tile of rows at a time: out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
    const int mr = threadIdx.x / 16, part = threadIdx.x % 16;  // 16 threads a row
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        __syncthreads();  // parameters, or the tile before, are read: results may take their place
        l[ct] = row_sum(l[ct]);
#pragma unroll
        for (int g = 0; g < NG; ++g) z[ct][g] = row_sum(z[ct][g]);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(512.0f, o[ct][c][i], z[ct][16 * c / G]);
            *(f32x4 *)&lds_o[wave][col][16 * c + 4 * h] = y;
        }
        if (h == 0) {
            lds_ml[wave][0][16 * ct + col] = ref[ct];
            lds_ml[wave][1][16 * ct + col] = l[ct];
        }
        __syncthreads();
        const int orow = j.row0 + 16 * ct + mr;
        if (orow >= j.rows) continue;
        float M = -__builtin_inff(), L = 0.0f, wgt[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[w][0][16 * ct + mr]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            wgt[w] = M == -__builtin_inff() ? 0.0f : exp2_fast(lds_ml[w][0][16 * ct + mr] - M);
            L += wgt[w] * lds_ml[w][1][16 * ct + mr];
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
            if (a.ns > 1)
                *(f32x4 *)(a.part_o + prow * D + c) = y;
            else
                store_out<BF>(a, tok, head, c, y);
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
}

// ------------------------------------------------------------- many rows

// Blocks of 128 rows where that many can be had (kv4_tree_plan): four waves of 32 rows share 32 keys a turn,
// which they unpack together, once, into matrix operands in LDS while they work on the turn before.
// Bound by the vector and matrix units' issue: with D = 128 G = 64 a wave's turn is some 300 vector, 54 matrix and 50 LDS
// instructions, of two waves a SIMD.  60 tokens of 8 heads a KV head, 80000 keys, 8 KV heads, bf16: 357 us, 0.44 PFLOP/s of
// products (tiles of 32 rows 403 us).  Tried and not better: blocks of 64 rows and two times 32 keys (210 us, these
// 125, of 16 sequences of up to 8192 keys), waves of 64 rows (130 to 380 registers spilled, 855 us).
//
// Here V's s is in its operand: v - mid = s (n - 7.5) is 15 bits, two fp16 terms, so that p is one operand
// for all groups instead of p s and a sum of p mid for each (4 vector instructions a probability and group):
//   o_c = sum_j p_j (hi + lo)_jc,   and one more product with the rows mid_g (two terms each) and
//   "1" gives sum_j p_j mid_jg and sum_j p_j.
// The rows of 16 keys are scaled by f, a power of two that takes their largest value to 2^8, and
// their p by 1 / f: the terms then keep what fp16 has below 2^9, 33 bits of those keys' largest value,
// whatever other keys' sizes.
// bf16 outputs: p in one fp16 term, the sum that divides included, so that they are exact
// averages whose weights are off by 2^-11 of themselves at most: 2^-11 sum_j p_j |v_j - out| / sum_j p_j,
// an eighth of a bf16 rounding of what is averaged, channel by channel (one term of p s would be off by a share
// of s, which one outlying channel makes large for its whole group).  fp16 outputs: two terms, 22 bits.
// lse is from unrounded p either way (two terms are as good).
constexpr int kTreeRows = 128;

// Over a row of 16 lanes: neighbours and pairs, then mirrored halves, whose quads already agree.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v)
{
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true)));
}
__device__ __forceinline__ float max16(float v) { return dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(v)))); }

// What a turn's 32 keys are to the matrix unit.
template <int D, int G>
struct Turn {
    static constexpr int NW = D / 32, NT = D / 16;
    u32x4 k[2][NW][64];
    u32x2 v[NT][2][2][64];     // V's hi and lo, of either tile of 16 keys
};
// What goes with them, known a turn earlier.
template <int D, int G>
struct Keys {
    static constexpr int NG = D / G, NP = (NG + 3) / 4, NZ = (2 * NG + 1 + 15) / 16;  // products of the rows mid and 1
    uint16_t z[NZ][64][8];     // an operand: row 2g, 2g + 1: mid_g's terms, then the scale f itself
    uint16_t nan[64][8];       // an operand: row g is 1 where a key's group is NaN
    u32x2 klo[NP][2][64];      // lo_operand of K: groups 0..3, 4..7; zero where there is none
    float ks[2][NG][16];       // K's s
    uint16_t s[2][NG][16];     // V's s, scaled
    float e[2], f[2];          // of the tiles: -log2 f, f
    uint32_t any_nan[2], pad[2];
};
constexpr int kAhead = 3;      // turns' Keys: one read, one read to unpack V by, one written

template <int D, int G, bool BF>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv4_tree_wide(Kv4Attn a)
{
    static_assert(D >= 128, "a wave unpacks whole pairs of V's dwords");
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = (NG + 3) / 4, ND = NW / 2;
    constexpr bool TWO = !BF;                          // terms of p
    typedef Turn<D, G> T;
    typedef Keys<D, G> K;
    constexpr int NZ = K::NZ;
    extern __shared__ __align__(16) uint8_t lds_raw[];
    T *const turns = (T *)lds_raw;
    K *const keys = (K *)(lds_raw + 2 * sizeof(T));
    // what the largest tree of the call takes
    int16_t *const lds_steps = (int16_t *)(lds_raw + 2 * sizeof(T) + kAhead * sizeof(K)), *const lds_parent = lds_steps + kTreeRows;
    uint32_t *const lds_bits = (uint32_t *)(lds_parent + (a.max_q + 1) / 2 * 2);
    __shared__ u32x4 lds_sums[kTreeRows / 16][64];     // sum_operand of the rows
    __shared__ uint32_t lds_nan[kTreeRows];            // a row's groups in which it met NaN
    Job j;
    if (!make_job<kTreeRows, true>(a, j)) return;
    int lane = threadIdx.x & 63, col = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // where a tile has fewer rows the same waves would idle in every block
    const int rg = (wave + (int)blockIdx.x) & 3;
    const int tile = wave & 1, d0 = (wave >> 1) * ND;  // this wave's part in unpacking: a tile's dwords d0 ..
    const int t_end = min(j.u1 * 4, (j.kend + 31) / 32);
    int turn = j.u0 * 4;
    const WaveAt<D, G> wat(a, j);

    const int last_row = min(j.row0 + kTreeRows, j.rows) - 1;
    const int tok0 = j.row0 / a.R, tok1 = last_row / a.R;
    Paths paths;
    paths.bits = lds_bits;
    paths.base = j.pos0;
    paths.first = max(j.pos0, 0) >> 5;
    paths.words = max(((j.kend + 31) >> 5) - paths.first, 0);
    const bool walks = t_end > paths.first || a.window;
    if (walks) {
        stage_parents(a, j, tok1, lds_parent);
        lds_barrier();
        walk(a, paths, lds_parent, tok0, tok1, lds_steps);
    }
    // rows of the operands that no group has
    for (int i = threadIdx.x; i < (int)(kAhead * sizeof(K)) / 16; i += 256) ((u32x4 *)keys)[i] = u32x4{0, 0, 0, 0};
    if (threadIdx.x < kTreeRows) lds_nan[threadIdx.x] = 0;
    lds_barrier();

    const int row_w = j.row0 + 32 * rg;
    u32x4 q[2][NW];
    float up[2];
    uint32_t toks = 0;  // which of the tile's tokens the lane's rows are
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int row = row_w + 16 * ct + col;
        load_query<D, BF>(a, j, row, row / a.R, h, row < j.rows, q[ct]);
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
        lds_sums[2 * rg + ct][lane] = sum_operand<NG>(qs, h);  // read by this wave alone
        toks |= (uint32_t)(min(row, last_row) / a.R - tok0) << (16 * ct);
    }
    // keys that some row of the wave sees, and that every row does
    const int any_hi = row_w >= j.rows ? 0 : j.pos0 + min(row_w + 31, last_row) / a.R + 1;
    const int any_lo = a.window ? j.pos0 - a.window + 1 : 0;
    const int all_lo = a.window ? j.pos0 + j.nq - a.window : 0;

    f32x4 o[2][NT], z[2][NZ];
    float ref[2], l[2];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
#pragma unroll
        for (int c = 0; c < NT; ++c) o[ct][c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NZ; ++i) z[ct][i] = f32x4{0, 0, 0, 0};
        ref[ct] = -__builtin_inff();
        l[ct] = 0.0f;
    }

    // ---- unpacking.  In turn t the operands of t + 1 are laid out, a part of a tile by each wave, by what the first of a
    // tile's waves found out about its keys in turn t - 1 (Keys).
    bool bad_page = false;
    uint32_t pages = 0;                    // of this wave's tiles of 64 turns, a lane each
    uint32_t kw[ND], vw[ND], kw2[ND], vw2[ND], kp[NP], vp[NP];  // codes of t + 1, and of t + 2 on their way with the parameters
    const auto tile_of = [&](int t) { return min(max(t * 2 + tile, wat.t_lo), wat.t_hi); };
    const auto look_up = [&](int t) {
        const uint32_t entry = (uint32_t)wat.table[tile_of(t + lane) >> wat.shift];
        bad_page |= entry >= wat.n_pages;
        pages = entry < wat.n_pages ? entry : 0;
    };
    // a lane has the parameters of key `col`, group g_l (and g_l + 4)
    const auto group_l = [&](int h) { return NG == 1 ? 0 : NG == 2 ? h & 1 : h; };
    const uint32_t k_at = col * (D / 2) + h * (D / 8) + 4 * d0;
    const uint32_t v_at = h * (2 * D) + col * (D / 8) + ((uint32_t)a.pool.H << a.pool.pshift) * (D / 2) + 4 * d0;
    const uint32_t p_at = (((uint32_t)group_l(h) << a.pool.pshift) + col) * 4, to_v = ((uint32_t)(a.pool.H * NG) << a.pool.pshift) * 4;
    const int turn0 = turn;
    const auto fetch = [&](int t) {
        const int i = t - turn0;
        if ((i & 63) == 0) look_up(t);
        const uint32_t page = (uint32_t)__builtin_amdgcn_readlane((int)pages, i & 63), in = (uint32_t)(tile_of(t) & wat.mask);
        const uint8_t *codes = wat.codes + (uint64_t)page * wat.page_codes + in * (8 * D);
        const uint8_t *params = wat.params + (uint64_t)page * wat.page_params + in * 64;
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            kw2[i] = ((const uint32_t *)(codes + k_at))[i];
            vw2[i] = ((const uint32_t *)(codes + v_at))[i];
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t g = p_at + ((uint32_t)(4 * i) << a.pool.pshift) * 4;
            kp[i] = *(const uint32_t *)(params + g);
            vp[i] = *(const uint32_t *)(params + (g + to_v));
        }
    };
    const auto fetched = [&]() {
#pragma unroll
        for (int i = 0; i < ND; ++i) kw[i] = kw2[i], vw[i] = vw2[i];
    };
    const auto lay_keys = [&](int t, K &to) {
        const int key = t * 32 + 16 * tile + col, at = 4 * tile + col % 4;
        const bool in = key >= j.kbeg && key < j.kend;  // what lies at keys that no row sees may be anything
        float mid[NP], s[NP], top = 0.0f;
        bool is_nan[NP], some = false;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int g = group_l(h) + 4 * i;
            const uint32_t w = in ? kp[i] : 0, lo = w >> 16;
            to.ks[tile][g][col] = s_of(w);
            to.klo[i][tile][col + 16 * group_l(h)] = u32x2{lo | lo << 16, lo};
            const uint32_t x = in ? vp[i] : 0;
            s[i] = s_of(x);
            mid[i] = mid_of(x);
            is_nan[i] = !(mid[i] == mid[i]);
            some |= is_nan[i];
            mid[i] = is_nan[i] ? 0.0f : mid[i];
            s[i] = is_nan[i] ? 0.0f : s[i];
            top = fmaxf(top, __builtin_fmaf(7.5f, s[i], __builtin_fabsf(mid[i])));
        }
        if (NG > 1) {
            const uint32_t b = __builtin_bit_cast(uint32_t, top);
            const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
            const uint32_t x0 = x[0], x1 = x[1];
            top = fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
        }
        if (NG > 2) {
            const uint32_t b = __builtin_bit_cast(uint32_t, top);
            const auto x = __builtin_amdgcn_permlane32_swap(b, b, false, false);
            const uint32_t x0 = x[0], x1 = x[1];
            top = fmaxf(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
        }
        top = max16(top);
        // f = 2^(8 - e) for a largest of 2^e (at most 2^17), and at most 2^15
        const int e = max((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127, -7);
        const float f = __builtin_bit_cast(float, (uint32_t)(127 + 8 - e) << 23);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int g = group_l(h) + 4 * i;
            to.s[tile][g][col] = (uint16_t)kvc_f2h(s[i] * f * 512.0f);
            const float m = mid[i] * f;
            const uint32_t hi = kvc_f2h(m);
            uint16_t *const row = &to.z[g / 8][2 * g % 16 + 16 * (col / 4)][at];
            row[0] = (uint16_t)hi;
            row[8] = (uint16_t)kvc_f2h(m - kvc_h2f(hi));
            to.nan[g + 16 * (col / 4)][at] = is_nan[i] ? 0x3C00 : 0;
        }
        // the same from every group
        to.z[NZ - 1][2 * NG % 16 + 16 * (col / 4)][at] = (uint16_t)kvc_f2h(f);
        to.e[tile] = (float)(e - 8);
        to.f[tile] = f;
        to.any_nan[tile] = __ballot(some) != 0;
    };
    // Part `part` of `parts` of the operands of turn t.
    constexpr int VN = 2, V_ITEMS = ND / VN * 4;  // dwords of V at once
    const auto lay_operands = [&](T &to, const K &by, int part, int parts) {
#pragma unroll
        for (int i = 0; i < ND; ++i)
            if (i * parts / ND == part) to.k[tile][d0 + i][lane] = code_octet(kw[i]);
        // V with s of this lane's four keys
#pragma unroll
        for (int item = 0; item < V_ITEMS; ++item) {
            if (item * parts / V_ITEMS != part) continue;
            const int i = item / 4 * VN, n = item % 4, c = (d0 + i) / 2 * 4 + n;
            u32x2 hi, lo;
#pragma unroll
            for (int k = 0; k < VN; ++k) {
                const u16x2 sp = *(const u16x2 *)&by.s[tile][16 * c / G][4 * h + 2 * ((d0 + i + k) & 1)];
                const f16x2 t2 = __builtin_bit_cast(f16x2, centred_pair(vw[i + k], n)), s2 = __builtin_bit_cast(f16x2, sp);
                const f16x2 first = t2 * s2;
                hi[k] = __builtin_bit_cast(uint32_t, first);
                lo[k] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(t2, s2, -first));
            }
            to.v[c][0][tile][lane] = hi;
            to.v[c][1][tile][lane] = lo;
        }
    };

    // ---- the work
    // which rows of a column tile see how many of which groups' NaN: a product of its own
    const auto meet_nan = [&](const K &by, int ct, uint32_t see) {
        const u32x4 is = *(const u32x4 *)&by.nan[lane][0];
        u32x4 sees;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const int at = 16 * (i / 4) + i % 4;
            sees[i / 2] = (see >> at & 1 ? 0x3C00u : 0) | (see >> (at + 1) & 1 ? 0x3C000000u : 0);
        }
        const f32x4 n = mfma(is, sees, f32x4{0, 0, 0, 0});
        uint32_t met = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) met |= n[i] > 0.0f ? 1u << i : 0;
        if (met) atomicOr(&lds_nan[16 * (2 * rg + ct) + col], met << (4 * h));
    };
    // rows of which some p passes the largest so far by 2^8: what their sums were multiplied by, and p is relative to now
    const auto pass_on = [&](int ct, float top) {
        float pass = ref[ct] + 15.0f, mu;  // as rescale leaves it
        const float by = rescale(top, pass, ref[ct], mu);
        l[ct] *= by;
#pragma unroll
        for (int i = 0; i < NZ; ++i) z[ct][i] *= by;
#pragma unroll
        for (int c = 0; c < NT; ++c) o[ct][c] *= by;
        return mu;
    };
    const auto load_v = [&](const T &now, int c, u32x4 *v) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const u32x2 a0 = now.v[c][k][0][lane], a1 = now.v[c][k][1][lane];
            v[k] = u32x4{a0[0], a0[1], a1[0], a1[1]};
        }
    };
    const auto load_klo = [&](const K &by, int tt) {
        const u32x2 a0 = by.klo[0][tt][lane], a1 = NP > 1 ? by.klo[NP - 1][tt][lane] : u32x2{0, 0};
        return u32x4{a0[0], a0[1], a1[0], a1[1]};
    };
    // p of a column tile as operands, and its sum; at[tile]: e less what p is relative to
    const auto weigh = [&](const f32x4 *x, float mul, const float *at, const float *f, int ct, u32x4 &hi, u32x4 &lo) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const f32x2 p = {exp2_fast(__builtin_fmaf(x[tt][i], mul, at[tt])), exp2_fast(__builtin_fmaf(x[tt][i + 1], mul, at[tt]))};
                const f16x2 t2 = __builtin_convertvector(p, f16x2);
                hi[2 * tt + i / 2] = __builtin_bit_cast(uint32_t, t2);
                if (TWO) {
                    lo[2 * tt + i / 2] = rest_of(p, t2);
                } else {
                    sum = i ? sum + p[0] : p[0];
                    sum += p[1];
                }
            }
            if (!TWO) l[ct] = __builtin_fmaf(sum, f[tt], l[ct]);
        }
    };
    const auto largest = [&](const f32x4 *x, float mul, const float *e) {
        float m[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) m[tt] = __builtin_fmaf(fmaxf(fmaxf(x[tt][0], x[tt][1]), fmaxf(x[tt][2], x[tt][3])), mul, e[tt]);
        return fmaxf(m[0], m[1]);
    };
    // A turn with masks, a cap, or the first.
    const auto work = [&](int t, const T &now, const K &by) {
        const int key0 = t * 32;
        if (key0 >= any_hi || key0 + 32 <= any_lo) return;
        const bool partial = key0 + 32 > j.pos0 || key0 < all_lo;
        f32x4 x[2][2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const u32x4 klo = load_klo(by, tt);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) x[ct][tt] = mfma(klo, lds_sums[2 * rg + ct][lane], f32x4{0, 0, 0, 0});
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                    const u32x4 k = now.k[tt][s][lane];
                    c[0] = mfma(k, q[0][s], c[0]);
                    c[1] = mfma(k, q[1][s], c[1]);
                }
                const f32x4 ks = *(const f32x4 *)&by.ks[tt][g][4 * h];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[ct][tt][i] = __builtin_fmaf(ks[i], c[ct][i], x[ct][tt][i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const float e[2] = {by.e[0], by.e[1]}, f[2] = {by.f[0], by.f[1]};
        u32x4 hi[2], lo[2];
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            float mul = up[ct];
            if (a.softcap > 0.0f) {
                float cap = a.softcap;
                __asm__ volatile("" : "+s"(cap), "+v"(mul));  // or what the cap makes of them is kept in registers
                cap_logits(cap, x[ct], mul);
            }
            uint32_t see = ~0u;  // the lane's keys that its row sees
            if (partial) {
                // keys before the tree from k_lo on, and the path's
                const int tok = toks >> (16 * ct) & 0xFFFF;
                const int k_lo = a.window ? max(0, j.pos0 + lds_steps[tok] - a.window) : 0;
                const int n = min(max(j.pos0 - key0, 0), 32), m = min(max(k_lo - key0, 0), 32);
                see = (uint32_t)((1ull << n) - 1) & ~(uint32_t)((1ull << m) - 1);
                if (t >= paths.first) see |= lds_bits[tok * paths.words + t - paths.first];
                see >>= 4 * h;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!(see >> (16 * (i / 4) + i % 4) & 1)) x[ct][i / 4][i % 4] = -__builtin_inff();
            }
            const float top = largest(x[ct], mul, e);
            float mu = ref[ct] == -__builtin_inff() ? 0.0f : ref[ct];
            if (__any(top > ref[ct] + 15.0f)) mu = pass_on(ct, top);
            const float at[2] = {e[0] - mu, e[1] - mu};
            weigh(x[ct], mul, at, f, ct, hi[ct], lo[ct]);
            if (by.any_nan[0] | by.any_nan[1]) meet_nan(by, ct, see);
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            const u32x4 zo = *(const u32x4 *)&by.z[i][lane][0];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                z[ct][i] = mfma(zo, hi[ct], z[ct][i]);
                if (TWO) z[ct][i] = mfma(zo, lo[ct], z[ct][i]);
            }
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            if (c % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            u32x4 v[2];
            load_v(now, c, v);
#pragma unroll
            for (int term = 0; term < (TWO ? 3 : 2); ++term)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) o[ct][c] = mfma(v[term == 1], term == 2 ? lo[ct] : hi[ct], o[ct][c]);
        }
    };
    // A turn that every row of the wave sees whole, after another and without a cap, and the next one's operands laid out
    // meanwhile: the matrix unit takes 16 cycles an instruction, of which a wave's vector instructions can have 12.
    const auto both = [&](const T &now, const K &by, T &to, const K &to_by) {
        u32x4 k[2][NW];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int s = 0; s < NW; ++s) k[tt][s] = now.k[tt][s][lane];
        const uint32_t some_nan = by.any_nan[0] | by.any_nan[1];
        const float e[2] = {by.e[0], by.e[1]}, f[2] = {by.f[0], by.f[1]};
        __builtin_amdgcn_sched_barrier(0);
        f32x4 x[2][2], c[2][NG], ks[NG];
        const auto products = [&](int tt) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) c[ct][g] = mfma(k[tt][s], q[ct][s], s == g * (G / 32) ? f32x4{0, 0, 0, 0} : c[ct][g]);
            const u32x4 klo = load_klo(by, tt);
#pragma unroll
            for (int g = 0; g < NG; ++g) ks[g] = *(const f32x4 *)&by.ks[tt][g][4 * h];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) x[ct][tt] = mfma(klo, lds_sums[2 * rg + ct][lane], f32x4{0, 0, 0, 0});
        };
        const auto scaled = [&](int tt) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int g = 0; g < NG; ++g) x[ct][tt][i] = __builtin_fmaf(ks[g][i], c[ct][g][i], x[ct][tt][i]);
        };
        products(0);
        __builtin_amdgcn_sched_barrier(0);
        scaled(0);
        products(1);
        __builtin_amdgcn_sched_barrier(0);
        scaled(1);
        const float top[2] = {largest(x[0], up[0], e), largest(x[1], up[1], e)};
        if (__any(top[0] > ref[0] + 15.0f || top[1] > ref[1] + 15.0f || some_nan)) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                pass_on(ct, top[ct]);
                if (some_nan) meet_nan(by, ct, ~0u);
            }
        }
        u32x4 va[2][2][2], zo[NZ], hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < NZ; ++i) zo[i] = *(const u32x4 *)&by.z[i][lane][0];
        load_v(now, 0, va[0][0]);
        load_v(now, 1, va[0][1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const float mu = ref[ct] == -__builtin_inff() ? 0.0f : ref[ct], at[2] = {e[0] - mu, e[1] - mu};
            weigh(x[ct], up[ct], at, f, ct, hi[ct], lo[ct]);
        }
        __builtin_amdgcn_sched_barrier(0);
        constexpr int PAIRS = NT / 2, EACH = TWO ? 6 : 4;  // of channel tiles, and a pair's products
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            // a pair's operands are on their way since the one before
            if (p + 1 < PAIRS) load_v(now, 2 * p + 2, va[(p + 1) & 1][0]), load_v(now, 2 * p + 3, va[(p + 1) & 1][1]);
            lay_operands(to, to_by, p, PAIRS);
            if (p == 0)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int i = 0; i < NZ; ++i) {
                        z[ct][i] = mfma(zo[i], hi[ct], z[ct][i]);
                        if (TWO) z[ct][i] = mfma(zo[i], lo[ct], z[ct][i]);
                    }
#pragma unroll
            for (int term = 0; term < (TWO ? 3 : 2); ++term)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
                        o[ct][2 * p + i] = mfma(va[p & 1][i][term == 1], term == 2 ? lo[ct] : hi[ct], o[ct][2 * p + i]);
#pragma unroll
            for (int i = 0; i < 2 * EACH; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
                __builtin_amdgcn_sched_group_barrier(0x2, 3, 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // where the turn's, the next one's and the one's after lie, passed on from turn to turn
    T *now = turns, *to = turns + 1;
    K *by = keys, *to_by = keys + 1, *ahead = keys + 2;
    if (turn < t_end) {
        // as if the two turns before had been worked on
        fetch(turn);
        lay_keys(turn, *by);
        fetched();
        fetch(turn + 1);
        lay_keys(turn + 1, *to_by);
        lds_barrier();
        lay_operands(*now, *by, 0, 1);
        fetched();
    }
    // What follows from the lane is worked out in each turn: kept, it takes the queries' registers.
    const auto begin = [&]() {
        __asm__ volatile("" : "+v"(lane));
        col = lane & 15, h = lane >> 4;
        lds_barrier();
        fetch(turn + 2);
    };
    const auto end = [&]() {
        fetched();
        ++turn;
        T *const t0 = now;
        now = to, to = t0;
        K *const k0 = by;
        by = to_by, to_by = ahead, ahead = k0;
    };
    // Turns that every row sees whole, without a cap: a loop of their own, in which the sums stay where they are.
    const int from = max(turn + 1, (max(all_lo, 0) + 31) / 32);
    const int until = a.softcap == 0.0f ? min(t_end, max(j.pos0, 0) / 32) : 0;
    while (turn < t_end) {
        if (turn >= from && turn < until) {
            // a wave without rows unpacks only
            if (row_w < j.rows) {
                while (turn < until) {
                    begin();
                    both(*now, *by, *to, *to_by);
                    if (d0 == 0) lay_keys(turn + 2, *ahead);
                    end();
                }
            } else {
                while (turn < until) {
                    begin();
                    lay_operands(*to, *to_by, 0, 1);
                    if (d0 == 0) lay_keys(turn + 2, *ahead);
                    end();
                }
            }
            continue;
        }
        begin();
        work(turn, *now, *by);
        // the other side: nobody reads it before the next barrier, nor since the last
        lay_operands(*to, *to_by, 0, 1);
        if (d0 == 0) lay_keys(turn + 2, *ahead);
        end();
    }
    if (bad_page) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);

#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        // a row's sums, in the lanes that hold its channels
        const int at_l = 2 * NG % 16;
        const float lhat = __shfl(z[ct][NZ - 1][at_l % 4], col + 16 * (at_l / 4), 64);
        const float L = TWO ? lhat : row_sum(l[ct]);
        const uint32_t met = lds_nan[16 * (2 * rg + ct) + col];  // by this wave alone
        const int row = row_w + 16 * ct + col;
        const int head = j.h * a.R + row % a.R;
        const int64_t tok = j.q0 + row / a.R, grow = tok * a.Hq + head;
        const int64_t prow = (int64_t)j.split * a.n_q * a.Hq + grow;
        // p's one term: an average with the weights as they were rounded; for a join, times the sum of those that were not
        const float inv = a.ns > 1 ? (TWO || lhat == 0.0f ? 1.0f : L / lhat) : (lhat == 0.0f ? 0.0f : 1.0f / lhat);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const f32x4 zg = z[ct][g / 8];
            float mid = __shfl(g & 1 ? zg[2] + zg[3] : zg[0] + zg[1], col + 16 * (g % 8 / 2), 64);
            if (met >> g & 1) mid = __builtin_nanf("");
#pragma unroll
            for (int c = g * (G / 16); c < (g + 1) * (G / 16); ++c) {
                f32x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = (o[ct][c][i] + mid) * inv;
                if (row >= j.rows) continue;
                if (a.ns > 1)
                    *(f32x4 *)(a.part_o + prow * D + 16 * c + 4 * h) = y;
                else
                    store_out<BF>(a, tok, head, 16 * c + 4 * h, y);
            }
        }
        if (h == 0 && row < j.rows) {
            if (a.ns > 1) {
                a.part_ml[prow * 2] = ref[ct];
                a.part_ml[prow * 2 + 1] = L;
            } else if (a.lse) {
                a.lse[grow] = lse_of(ref[ct], L);
            }
        }
    }
}

template <int D, int G, bool BF>
hipError_t attend_wide(const Kv4Attn &a, dim3 grid, hipStream_t s)
{
    const auto lds_of = [](int max_q) {
        return (int)(2 * sizeof(Turn<D, G>) + kAhead * sizeof(Keys<D, G>)) + 2 * kTreeRows + (max_q + 1) / 2 * 4 +
               4 * kTreeRows * ((max_q + 62) / 32);
    };
    const int lds = lds_of(a.max_q);
    // above 64 KB LDS has to be asked for; the attribute is per device, and cheap.  What the largest tree takes, always: calls of
    // several threads must not lower it for each other.
    const hipError_t e = hipFuncSetAttribute((const void *)k_kv4_tree_wide<D, G, BF>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             lds_of(kTreeMost));
    if (e != hipSuccess) return e;
    k_kv4_tree_wide<D, G, BF><<<grid, dim3(256), lds, s>>>(a);
    return hipGetLastError();
}

// Which shapes the wide blocks are faster for (16 sequences of up to 8192 keys, 8 KV heads, trees of 128 rows, bf16; 8
// sequences with D = 256): D = 128 G = 32, 64, 128: 133, 122, 118 us, tiles of 32 rows 215, 141, 121; D = 256 G = 32 335, 399.
// The others: D = 64 G = 32, 64: 97, 106 (trees of 96 rows 93, 86) and 93, 89; D = 256 G = 64: 228, 198.
constexpr bool has_wide(int D, int G) { return D == 128 || (D == 256 && G == 32); }

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const dim3 grid((uint32_t)((int64_t)a.ns * a.pool.H * a.B * a.tiles)), block(64 * kWaves);
    hipError_t e = hipErrorInvalidValue;
    if (a.rows == kTreeRows) {
        if constexpr (has_wide(D, G)) e = attend_wide<D, G, BF>(a, grid, s);
    } else {
        if (a.rows == 32)
            k_kv4_tree<D, G, BF, 2><<<grid, block, 0, s>>>(a);
        else
            k_kv4_tree<D, G, BF, 1><<<grid, block, 0, s>>>(a);
        e = hipGetLastError();
    }
    if (e == hipSuccess && a.ns > 1) {
        const dim3 rows((uint32_t)(std::min(a.n_q, (int64_t)a.B * a.max_q) * a.Hq));
        if (a.ns <= 8)
            k_kv4_join<D, BF, 64><<<rows, dim3(64), 0, s>>>(a);
        else
            k_kv4_join<D, BF, 512><<<rows, dim3(512), 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
}

template <int D, int G>
hipError_t attend_dt(const Kv4Attn &a, bool bf16, hipStream_t s)
{
    return bf16 ? attend<D, G, true>(a, s) : attend<D, G, false>(a, s);
}

// As many parts of the keys as fill the chip, for each level (blocks, keys of a part at the nearest): a part costs its share
// of the join and of what a block does once.
//   Tiles of up to 32 rows.  {256, 256}: 24 blocks of 2048 keys 22 us in 8 parts, 23 in 4, 28 in 2; 16 of 32768 40 in 32,
// 49 in 12.  {512, 512}: 64 of 8192 40 in 8, 61 in 2, 54 in 16.  {1536, 2048}, since blocks' lengths differ: 256 of 8192
// 79 in 4, 85 in 2, 108 in 8; 512 of 8192 128 in 3, 144 in 1, 178 in 8; 396 of a window of 2060 55 in 1, 60 in 2.
//   Blocks of 128 rows.  {512, 512}: 128 of 8192 121 in 4, 166 in 3, 132 in 8; 32 of 80000 358 in 16, 498 in 8.
// {1024, 2048} for sequences of several lengths: 128 of 16000 259 in 8, 312 in 4; of a single one 64 of 30000
// 267 in 8, 284 in 16.
int64_t splits(bool wide, bool several, int64_t blocks, int64_t keys)
{
    typedef std::pair<int64_t, int64_t> Level;
    const Level last = wide ? several ? Level{1024, 2048} : Level{512, 512} : Level{1536, 2048};
    int64_t ns = 1;
    if (keys > 512)
        for (const Level &l : {Level{256, 256}, Level{512, 512}, last})
            ns = std::max(ns, std::min(l.first / blocks, (keys + l.second / 2) / l.second));
    return std::min<int64_t>(ns, 128);
}

}  // namespace

Kv4Plan kv4_tree_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window)
{
    Kv4Plan plan = {};
    const int64_t most = std::max<int64_t>(max_q * R, 1), narrow = most > 16 ? 32 : 16, heads = std::max<int64_t>(n_seqs, 1) * p.H;
    const int64_t tiles = (most + narrow - 1) / narrow, wide_tiles = (most + kTreeRows - 1) / kTreeRows;
    // a window reaches back from the tree's first token, and its keys go on to the last
    const int64_t keys = window ? std::min(max_keys, window + max_q) : max_keys;
    // blocks of 128 rows where the longest tree gives at least 7/8 of their waves rows (three of four, trees of up to 96 rows:
    // 137 us for 124, since most are smaller; but with groups of 32 123 for 173) and the keys fill the chip (8 heads of 2
    // sequences of 2000 keys: 26 us for 23)
    const int64_t full = p.G == 32 ? 24 : 28;  // of 32
    const bool wide = has_wide(p.D, p.G) && tiles * 8 >= wide_tiles * full && heads * wide_tiles * ((keys + 511) / 512) >= 512;
    plan.rows = wide ? kTreeRows : (int32_t)narrow;
    plan.tiles = (int32_t)(wide ? wide_tiles : tiles);
    plan.ns = (int32_t)splits(wide, n_seqs > 1, heads * plan.tiles, keys);
    // a shorter window may make the blocks narrow
    plan.most_ns = (int32_t)splits(false, n_seqs > 1, heads * tiles, max_keys);
    if (wide) plan.most_ns = (int32_t)std::max<int64_t>(plan.most_ns, splits(true, n_seqs > 1, heads * wide_tiles, max_keys));
    return plan;
}

hipError_t launch_kv4_tree(const Kv4Attn &a, bool bf16, hipStream_t stream)
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
