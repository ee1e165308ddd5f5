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
        for (; blk < b_end; blk += kWaves) {
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
            const bool partial = key0 + 32 > j.pos0 || key0 < all_lo;
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
                if (partial) {
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
                    if (partial) {
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
                        const f32x2 b2 = {a2[0] - (float)t[0], a2[1] - (float)t[1]};
                        hi[ct][i / 2] = __builtin_bit_cast(uint32_t, t);
                        lo[ct][i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(b2, f16x2));
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

// Blocks of 32 RG rows for trees of more than 32.  A block's four waves are RG groups of 32
// rows times KG = 4/RG of keys; a turn of 32 KG keys is unpacked once, by all of them, into
// matrix operands in LDS.
//
// Here V's s is in its operand: v - mid = s (n - 7.5) is 15 bits, two fp16 terms, so that p
// is one operand for all groups instead of p s two for each (19 vector instructions a
// probability with two groups, here 11):
//   o_c = sum_j p_j (hi + lo)_jc,   and one more product with the rows mid_g (two terms each) and
//   "1" gives sum_j p_j mid_jg and sum_j p_j.
// A key's rows are scaled by f_j, a power of two that takes its largest value to 2^8, and p_j
// by 1 / f_j: its terms then keep what fp16 has below 2^9, 33 bits, whatever the others' sizes.
// bf16 outputs: p in one fp16 term, the sum that divides included, so that they are exact
// averages whose weights are off by 2^-11 of themselves at most: 2^-11 sum_j p_j |v_j - out| / sum_j p_j,
// an eighth of a bf16 rounding of what is averaged.  fp16 outputs: two terms, 22 bits.
// lse is from unrounded p either way (two terms are as good).
template <int D, int G, int KG>
struct Turn {
    static constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = (NG + 3) / 4;
    static constexpr int NZ = (2 * NG + 1 + 15) / 16;  // products of the rows mid and 1
    u32x4 k[KG][2][NW][64];
    u32x2 v[KG][NT][2][2][64];      // V's hi and lo, of either tile of 16 keys
    uint16_t z[KG][NZ][64][8];      // an operand: row 2g, 2g + 1: mid_g's terms, then the scale f itself
    uint16_t nan[KG][64][8];        // an operand: row g is 1 where a key's group is NaN; only where any_nan is its tile's
    float ks[KG][2][NG][16];        // K's s
    uint32_t kp[KG][2][NP][64];     // K's parameters as loaded, for lo_operand
    float e[KG][2][16], f[KG][2][16];  // -log2 f, f
    uint32_t any_nan[KG][2];
};

template <int D, int G, bool BF, int RG>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv4_tree_wide(Kv4Attn a)
{
    constexpr int NW = D / 32, NG = D / G, NT = D / 16, NP = (NG + 3) / 4, ROWS = 32 * RG, KG = 4 / RG;
    constexpr int BUFS = RG == 4 ? 2 : 1;
    constexpr bool TWO = !BF;                          // terms of p
    constexpr int SHARE = RG == 4 ? 2 : 1;             // waves that unpack one tile, a part of its dwords each
    constexpr int ND = NW / SHARE;
    typedef Turn<D, G, KG> T;
    constexpr int NZ = T::NZ;
    extern __shared__ __align__(16) uint8_t lds_raw[];
    T *const turns = (T *)lds_raw;
    // what the largest tree of the call takes
    int16_t *const lds_steps = (int16_t *)(lds_raw + BUFS * sizeof(T)), *const lds_parent = lds_steps + ROWS;
    uint32_t *const lds_bits = (uint32_t *)(lds_parent + (a.max_q + 1) / 2 * 2);
    __shared__ __align__(8) uint16_t lds_s[kWaves][NG][16];  // a tile's s of V, scaled, for the lanes that unpack it
    __shared__ u32x4 lds_sums[2 * RG][64];                   // sum_operand of the rows
    __shared__ uint32_t lds_nan[ROWS];                       // a row's groups in which it met NaN
    Job j;
    if (!make_job<ROWS, true>(a, j)) return;
    int lane = threadIdx.x & 63, col = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // where a tile has fewer rows than groups of them the same waves would idle in every block
    const int rg = (wave + (int)blockIdx.x) % RG, kg = RG == 4 ? 0 : (wave + (int)blockIdx.x) / RG % KG;
    const int tile = RG == 4 ? wave & 1 : wave;        // of a turn, unpacked by this wave: its dwords d0 ..
    const int d0 = RG == 4 ? (wave >> 1) * ND : 0;
    const int t_end = (min(j.u1 * 4, (j.kend + 31) / 32) + KG - 1) / KG;
    int turn = j.u0 * 4 / KG;
    const WaveAt<D, G> wat(a, j);

    const int last_row = min(j.row0 + ROWS, j.rows) - 1;
    const int tok0 = j.row0 / a.R, tok1 = last_row / a.R;
    Paths paths;
    paths.bits = lds_bits;
    paths.base = j.pos0;
    paths.first = max(j.pos0, 0) >> 5;
    paths.words = max(((j.kend + 31) >> 5) - paths.first, 0);
    const bool walks = t_end * KG > paths.first || a.window;
    if (walks) {
        stage_parents(a, j, tok1, lds_parent);
        lds_barrier();
        walk(a, paths, lds_parent, tok0, tok1, lds_steps);
    }
    // rows of the operands that no group has
    for (int i = threadIdx.x; i < BUFS * KG * (NZ + 1) * 64; i += 256) {
        const int buf = i / (KG * (NZ + 1) * 64), k = i / ((NZ + 1) * 64) % KG, z = i / 64 % (NZ + 1);
        u32x4 *const to = (u32x4 *)(z < NZ ? &turns[buf].z[k][z][i % 64][0] : &turns[buf].nan[k][i % 64][0]);
        *to = u32x4{0, 0, 0, 0};
    }
    if (threadIdx.x < ROWS) lds_nan[threadIdx.x] = 0;
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
        if (kg == 0) lds_sums[2 * rg + ct][lane] = sum_operand<NG>(qs, h);
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
    bool bad_page = false;

    // this wave's part of a turn: loaded, then laid out in LDS
    uint32_t kw[ND], vw[ND], kp[NP], vp[NP];
    int32_t page = 0;
    const auto tile_of = [&](int t) { return min(max(t * (2 * KG) + tile, wat.t_lo), wat.t_hi); };
    const auto look_up = [&](int t) { page = wat.table[tile_of(t) >> wat.shift]; };
    const auto fetch = [&](int t) {
        const uint32_t entry = (uint32_t)__builtin_amdgcn_readfirstlane(page);
        bad_page |= entry >= wat.n_pages;
        const uint32_t pg = entry < wat.n_pages ? entry : 0;
        const uint32_t in = (uint32_t)(tile_of(t) & wat.mask);
        const uint8_t *codes = wat.codes + (uint64_t)pg * wat.page_codes + in * (8 * D);
        const uint8_t *params = wat.params + (uint64_t)pg * wat.page_params + in * 64;
        const LaneAt<D, G> at(lane, a.pool);
        const uint32_t k_at = at.k + 4 * d0, v_at = at.v + 4 * d0;
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            kw[i] = ((const uint32_t *)(codes + k_at))[i];
            vw[i] = ((const uint32_t *)(codes + v_at))[i];
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            kp[i] = *(const uint32_t *)(params + at.kp[i]);
            vp[i] = *(const uint32_t *)(params + at.vp[i]);
        }
    };
    const auto lay_params = [&](int t, T &to) {
        const int kgt = tile >> 1, half = tile & 1;
        const int key = t * (32 * KG) + 16 * tile + col;
        const bool in = key >= j.kbeg && key < j.kend;  // what lies at keys that no row sees may be anything
        // of key `col`, groups h and h + 4
        float mid[NP], s[NP], top = 0.0f;
        bool is_nan[NP], some = false;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            kp[i] = in ? kp[i] : 0;
            const uint32_t w = in ? vp[i] : 0;
            s[i] = s_of(w);
            mid[i] = mid_of(w);
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
        // f = 2^(8 - e) for a largest of 2^e (at most 2^17), and at most 2^15
        const int e = max((int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127, -7);
        const float f = __builtin_bit_cast(float, (uint32_t)(127 + 8 - e) << 23);
        const bool one = __any(some);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int g = h + 4 * i;
            if (g < NG) lds_s[wave][g][col] = (uint16_t)kvc_f2h(s[i] * f * 512.0f);
        }
        if (d0 == 0) {  // the first of a tile's waves writes what is its keys'
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int g = h + 4 * i;
                if (g < NG) {
                    to.ks[kgt][half][g][col] = s_of(kp[i]);
                    const float m = mid[i] * f;
                    const uint32_t hi = kvc_f2h(m);
                    uint16_t *const row = &to.z[kgt][g / 8][2 * g % 16 + 16 * (col / 4)][4 * half + col % 4];
                    row[0] = (uint16_t)hi;
                    row[8] = (uint16_t)kvc_f2h(m - kvc_h2f(hi));
                    if (one) to.nan[kgt][g + 16 * (col / 4)][4 * half + col % 4] = is_nan[i] ? 0x3C00 : 0;
                }
                to.kp[kgt][half][i][lane] = kp[i];
            }
            if (h == 0) {
                to.z[kgt][NZ - 1][2 * NG % 16 + 16 * (col / 4)][4 * half + col % 4] = (uint16_t)kvc_f2h(f);
                to.e[kgt][half][col] = (float)(e - 8);
                to.f[kgt][half][col] = f;
            }
            if (lane == 0) to.any_nan[kgt][half] = one;
        }
    };
    // Part `part` of `parts` of the operands themselves, after lay_params.
    constexpr int VN = ND > 1 ? 2 : 1, V_ITEMS = ND / VN * 4;  // dwords of V at once
    const auto lay_operands = [&](T &to, int part, int parts) {
        const int kgt = tile >> 1, half = tile & 1;
#pragma unroll
        for (int i = 0; i < ND; ++i)
            if (i * parts / ND == part) to.k[kgt][half][d0 + i][lane] = code_octet(kw[i]);
        // V with s of this lane's four keys
#pragma unroll
        for (int item = 0; item < V_ITEMS; ++item) {
            if (item * parts / V_ITEMS != part) continue;
            const int i = item / 4 * VN, n = item % 4, c = (d0 + i) / 2 * 4 + n;
            u32x2 hi, lo;
#pragma unroll
            for (int k = 0; k < VN; ++k) {
                const u16x2 sp = *(const u16x2 *)&lds_s[wave][16 * c / G][4 * h + 2 * ((d0 + i + k) & 1)];
                const f16x2 t2 = __builtin_bit_cast(f16x2, centred_pair(vw[i + k], n)), s2 = __builtin_bit_cast(f16x2, sp);
                const f16x2 first = t2 * s2;
                hi[k] = __builtin_bit_cast(uint32_t, first);
                lo[k] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(t2, s2, -first));
            }
            if (VN > 1) {
                to.v[kgt][c][0][half][lane] = hi;
                to.v[kgt][c][1][half][lane] = lo;
            } else {
                ((uint32_t *)&to.v[kgt][c][0][half][lane])[d0 & 1] = hi[0];
                ((uint32_t *)&to.v[kgt][c][1][half][lane])[d0 & 1] = lo[0];
            }
        }
    };
    const auto lay_out = [&](int t, T &to) {
        lay_params(t, to);
        lay_operands(to, 0, 1);
    };
    // which rows of a column tile see how many of which groups' NaN: a product of its own
    const auto meet_nan = [&](const T &now, int ct, uint32_t see) {
        u32x4 is = *(const u32x4 *)&now.nan[kg][lane][0], sees;
        if (!now.any_nan[kg][0]) is[0] = is[1] = 0;
        if (!now.any_nan[kg][1]) is[2] = is[3] = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const int at = 16 * (i / 4) + i % 4;
            sees[i / 2] = (see >> at & 1 ? 0x3C00u : 0) | (see >> (at + 1) & 1 ? 0x3C000000u : 0);
        }
        const f32x4 n = mfma(is, sees, f32x4{0, 0, 0, 0});
        uint32_t met = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) met |= n[i] > 0.0f ? 1u << i : 0;
        if (met) atomicOr(&lds_nan[32 * rg + 16 * ct + col], met << (4 * h));
    };
    // rows of which some p passes the largest so far by 2^8
    const auto pass_on = [&](int ct, float top) {
        float pass = ref[ct] + 15.0f, mu;  // as rescale leaves it
        const float by = rescale(top, pass, ref[ct], mu);
        l[ct] *= by;
#pragma unroll
        for (int i = 0; i < NZ; ++i) z[ct][i] *= by;
#pragma unroll
        for (int c = 0; c < NT; ++c) o[ct][c] *= by;
    };
    const auto load_v = [&](const T &now, int c, u32x4 *v) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const u32x2 a0 = now.v[kg][c][k][0][lane], a1 = now.v[kg][c][k][1][lane];
            v[k] = u32x4{a0[0], a0[1], a1[0], a1[1]};
        }
    };
    // A turn that every row of the wave sees whole, without a cap, and what the next one needs laid out
    // meanwhile: the matrix unit takes 16 cycles an instruction, of which a wave's vector instructions can have 12.
    const auto both = [&](int t, const T &now, T &to) {
        u32x4 k[2][NW];
        uint32_t prm[2][NP];
        const u32x4 sums[2] = {lds_sums[2 * rg][lane], lds_sums[2 * rg + 1][lane]};
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
            for (int s = 0; s < NW; ++s) k[tt][s] = now.k[kg][tt][s][lane];
#pragma unroll
            for (int i = 0; i < NP; ++i) prm[tt][i] = now.kp[kg][tt][i][lane];
        }
        const uint32_t some_nan = now.any_nan[kg][0] | now.any_nan[kg][1];
        __builtin_amdgcn_sched_barrier(0);
        float y[2][8], top[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            f32x4 x[2], c[2][NG], ks[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) ks[g] = *(const f32x4 *)&now.ks[kg][tt][g][4 * h];
            const f32x4 e = *(const f32x4 *)&now.e[kg][tt][4 * h];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) c[ct][g] = mfma(k[tt][s], q[ct][s], s == g * (G / 32) ? f32x4{0, 0, 0, 0} : c[ct][g]);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                x[ct] = mfma(lo_operand<NG>(prm[tt], h), sums[ct], f32x4{0, 0, 0, 0});
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) x[ct][i] = __builtin_fmaf(ks[g][i], c[ct][g][i], x[ct][i]);
                    y[ct][4 * tt + i] = __builtin_fmaf(x[ct][i], up[ct], e[i]);
                    top[ct] = tt + i == 0 ? y[ct][0] : fmaxf(top[ct], y[ct][4 * tt + i]);
                }
            }
        }
        // the first tile's vector work among the second's products
        __builtin_amdgcn_sched_group_barrier(0x8, 2 * (NW + 1), 0);
#pragma unroll
        for (int i = 0; i < 2 * (NW + 1); ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
        }
        lay_params(t + 1, to);
        if (__any(top[0] > ref[0] + 15.0f || top[1] > ref[1] + 15.0f || some_nan)) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                pass_on(ct, top[ct]);
                if (some_nan) meet_nan(now, ct, ~0u);
            }
        }
        f32x4 f[2];
        if (!TWO) f[0] = *(const f32x4 *)&now.f[kg][0][4 * h], f[1] = *(const f32x4 *)&now.f[kg][1][4 * h];
        u32x4 va[2][2][2], zo[NZ], hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < NZ; ++i) zo[i] = *(const u32x4 *)&now.z[kg][i][lane][0];
        load_v(now, 0, va[0][0]);
        load_v(now, 1, va[0][1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const float mu = ref[ct] == -__builtin_inff() ? 0.0f : ref[ct];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const f32x2 p = {exp2_fast(y[ct][i] - mu), exp2_fast(y[ct][i + 1] - mu)};
                const f16x2 t2 = __builtin_convertvector(p, f16x2);
                hi[ct][i / 2] = __builtin_bit_cast(uint32_t, t2);
                if (TWO) {
                    const f32x2 r = {p[0] - (float)t2[0], p[1] - (float)t2[1]};
                    lo[ct][i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(r, f16x2));
                } else {
                    l[ct] = __builtin_fmaf(p[0], f[i / 4][i % 4], l[ct]);
                    l[ct] = __builtin_fmaf(p[1], f[i / 4][i % 4 + 1], l[ct]);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        constexpr int PAIRS = NT / 2, EACH = TWO ? 6 : 4;  // of channel tiles, and a pair's products
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            // a pair's operands are on their way since the one before
            if (p + 1 < PAIRS) load_v(now, 2 * p + 2, va[(p + 1) & 1][0]), load_v(now, 2 * p + 3, va[(p + 1) & 1][1]);
            lay_operands(to, p, PAIRS);
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
    const auto work = [&](int t, const T &now) {
        const int blk = t * KG + kg, key0 = blk * 32;
        if (key0 >= any_hi || key0 + 32 <= any_lo) return;
        const bool partial = key0 + 32 > j.pos0 || key0 < all_lo;
        // K's operands: a tile's are on their way while the other's are worked on
        f32x4 x[2][2];
        u32x4 k[2][NW];
        const u32x4 sums[2] = {lds_sums[2 * rg][lane], lds_sums[2 * rg + 1][lane]};
#pragma unroll
        for (int s = 0; s < NW; ++s) k[0][s] = now.k[kg][0][s][lane];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            uint32_t prm[NP];
            f32x4 ks[NG];
#pragma unroll
            for (int i = 0; i < NP; ++i) prm[i] = now.kp[kg][tt][i][lane];
#pragma unroll
            for (int g = 0; g < NG; ++g) ks[g] = *(const f32x4 *)&now.ks[kg][tt][g][4 * h];
            if (tt == 0)
#pragma unroll
                for (int s = 0; s < NW; ++s) k[1][s] = now.k[kg][1][s][lane];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x4 c[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int s = g * (G / 32); s < (g + 1) * (G / 32); ++s) {
                    c[0] = mfma(k[tt][s], q[0][s], c[0]);
                    c[1] = mfma(k[tt][s], q[1][s], c[1]);
                }
                if (g == 0) {
                    const u32x4 klo = lo_operand<NG>(prm, h);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) x[ct][tt] = mfma(klo, sums[ct], f32x4{0, 0, 0, 0});
                }
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[ct][tt][i] = __builtin_fmaf(ks[g][i], c[ct][i], x[ct][tt][i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const f32x4 e[2] = {*(const f32x4 *)&now.e[kg][0][4 * h], *(const f32x4 *)&now.e[kg][1][4 * h]};
        f32x4 f[2];
        if (!TWO) f[0] = *(const f32x4 *)&now.f[kg][0][4 * h], f[1] = *(const f32x4 *)&now.f[kg][1][4 * h];
        // V's operands are on their way while the ones before are worked on
        u32x4 va[2][2][2];
        load_v(now, 0, va[0][0]);
        load_v(now, 1, va[0][1]);
        u32x4 hi[2], lo[2];
        uint32_t see[2];  // the keys that the lane's row sees, of its own
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            float mul = up[ct], y[8], top = -__builtin_inff();
            if (a.softcap > 0.0f) {
                float cap = a.softcap;
                __asm__ volatile("" : "+s"(cap), "+v"(mul));  // or what the cap makes of them is kept in registers
                cap_logits(cap, x[ct], mul);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(x[ct][i / 4][i % 4], mul, e[i / 4][i % 4]);
            see[ct] = ~0u;
            if (partial) {
                // keys before the tree from k_lo on, and the path's
                const int tok = toks >> (16 * ct) & 0xFFFF;
                const int k_lo = a.window ? max(0, j.pos0 + lds_steps[tok] - a.window) : 0;
                const int n = min(max(j.pos0 - key0, 0), 32), m = min(max(k_lo - key0, 0), 32);
                uint32_t ok = (uint32_t)((1ull << n) - 1) & ~(uint32_t)((1ull << m) - 1);
                if (blk >= paths.first) ok |= lds_bits[tok * paths.words + blk - paths.first];
                see[ct] = ok >>= 4 * h;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = ok >> (16 * (i / 4) + i % 4) & 1 ? y[i] : -__builtin_inff();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, y[i]);
            if (__any(top > ref[ct] + 15.0f)) pass_on(ct, top);
            const float mu = ref[ct] == -__builtin_inff() ? 0.0f : ref[ct];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float p0 = exp2_fast(y[i] - mu), p1 = exp2_fast(y[i + 1] - mu);
                const f32x2 p = {p0, p1};
                const f16x2 t = __builtin_convertvector(p, f16x2);
                hi[ct][i / 2] = __builtin_bit_cast(uint32_t, t);
                if (TWO) {
                    const f32x2 r = {p0 - (float)t[0], p1 - (float)t[1]};
                    lo[ct][i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(r, f16x2));
                } else {
                    l[ct] = __builtin_fmaf(p0, f[i / 4][i % 4], l[ct]);
                    l[ct] = __builtin_fmaf(p1, f[i / 4][i % 4 + 1], l[ct]);
                }
            }
        }
        if (now.any_nan[kg][0] | now.any_nan[kg][1]) {
            meet_nan(now, 0, see[0]);
            meet_nan(now, 1, see[1]);
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            const u32x4 zo = *(const u32x4 *)&now.z[kg][i][lane][0];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                z[ct][i] = mfma(zo, hi[ct], z[ct][i]);
                if (TWO) z[ct][i] = mfma(zo, lo[ct], z[ct][i]);
            }
        }
#pragma unroll
        for (int c = 0; c < NT; c += 2) {
            const int now_v = c / 2 & 1;
            if (c + 2 < NT) {
                load_v(now, c + 2, va[now_v ^ 1][0]);
                load_v(now, c + 3, va[now_v ^ 1][1]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int term = 0; term < (TWO ? 3 : 2); ++term)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
                        o[ct][c + k] = mfma(va[now_v][k][term == 1], term == 2 ? lo[ct] : hi[ct], o[ct][c + k]);
        }
    };
    if (turn < t_end) {
        look_up(turn);
        fetch(turn);
        look_up(turn + 1);
        if (BUFS == 2) lay_out(turn, turns[0]);
    }
    // what follows from the lane is worked out in each turn: kept, it takes the queries' registers
    const auto begin = [&]() {
        __asm__ volatile("" : "+v"(lane));
        col = lane & 15, h = lane >> 4;
        lds_barrier();
    };
    // turns that every row sees whole, without a cap: a loop of their own, in which the sums stay where they are
    const int from = max(turn, (max(all_lo, 0) + 32 * KG - 1) / (32 * KG));
    const int to = BUFS == 2 && a.softcap == 0.0f ? min(t_end, max(j.pos0, 0) / (32 * KG)) : 0;
    int side = 0;
    while (turn < t_end) {
        if (turn >= from && turn < to) {
            if (row_w < j.rows) {
                for (; turn < to; ++turn, side ^= 1) {
                    begin();
                    fetch(turn + 1);
                    look_up(turn + 2);
                    both(turn, turns[side], turns[side ^ 1]);
                }
            } else {
                for (; turn < to; ++turn, side ^= 1) {
                    begin();
                    fetch(turn + 1);
                    look_up(turn + 2);
                    lay_out(turn + 1, turns[side ^ 1]);
                }
            }
            continue;
        }
        begin();
        if (BUFS == 1) {
            lay_out(turn, turns[0]);
            lds_barrier();
        }
        fetch(turn + 1);  // past the end: the last tile again
        look_up(turn + 2);
        work(turn, turns[side]);
        // the other side: nobody reads it before the next barrier, nor since the last
        if (BUFS == 2) lay_out(turn + 1, turns[side ^ 1]);
        ++turn, side ^= BUFS - 1;
    }
    if (bad_page && lane == 0) kvc_flag(a.pool.status, KVC_DEV_BAD_INDEX);

    // a row's sums, in the lanes that hold its channels
    lds_barrier();
    float L[2];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int at_l = 2 * NG % 16;
        const float lhat = __shfl(z[ct][NZ - 1][at_l % 4], col + 16 * (at_l / 4), 64);
        L[ct] = TWO ? lhat : row_sum(l[ct]);
        // p's one term: an average with the weights as they were rounded, times the sum of those that were not
        const float fix = TWO || lhat == 0.0f ? 1.0f : L[ct] / lhat;
        const uint32_t met = lds_nan[32 * rg + 16 * ct + col];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const f32x4 zg = z[ct][g / 8];
            float mid = __shfl(g & 1 ? zg[2] + zg[3] : zg[0] + zg[1], col + 16 * (g % 8 / 2), 64);
            if (met >> g & 1) mid = __builtin_nanf("");
#pragma unroll
            for (int c = g * (G / 16); c < (g + 1) * (G / 16); ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[ct][c][i] = (o[ct][c][i] + mid) * fix;
        }
    }
    // the groups of keys joined: the others hand theirs to the first
    if constexpr (KG > 1) {
        static_assert(KG == 2, "one hands over");
        f32x4 *const part = (f32x4 *)lds_raw + rg * (2 * NT + 1) * 64;
        static_assert(RG * (2 * NT + 1) * 64 * 16 <= sizeof(T), "the parts fit where the operands were");
        lds_barrier();
        if (kg == 1) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                for (int c = 0; c < NT; ++c) part[(ct * NT + c) * 64 + lane] = o[ct][c];
            part[2 * NT * 64 + lane] = f32x4{ref[0], L[0], ref[1], L[1]};
        }
        lds_barrier();
        if (kg == 1) return;
        const f32x4 ml = part[2 * NT * 64 + lane];
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const float M = fmaxf(ref[ct], ml[2 * ct]);
            const float w0 = ref[ct] == -__builtin_inff() ? 0.0f : exp2_fast(ref[ct] - M);
            const float w1 = ml[2 * ct] == -__builtin_inff() ? 0.0f : exp2_fast(ml[2 * ct] - M);
#pragma unroll
            for (int c = 0; c < NT; ++c) o[ct][c] = w0 * o[ct][c] + w1 * part[(ct * NT + c) * 64 + lane];
            L[ct] = w0 * L[ct] + w1 * ml[2 * ct + 1];
            ref[ct] = M;
        }
    }
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int row = row_w + 16 * ct + col;
        if (row >= j.rows) continue;
        const int head = j.h * a.R + row % a.R;
        const int64_t tok = j.q0 + row / a.R, grow = tok * a.Hq + head;
        const int64_t prow = (int64_t)j.split * a.n_q * a.Hq + grow;
        const float inv = a.ns > 1 ? 1.0f : (L[ct] == 0.0f ? 0.0f : 1.0f / L[ct]);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const f32x4 y = o[ct][c] * inv;
            if (a.ns > 1)
                *(f32x4 *)(a.part_o + prow * D + 16 * c + 4 * h) = y;
            else
                store_out<BF>(a, tok, head, 16 * c + 4 * h, y);
        }
        if (h == 0) {
            if (a.ns > 1) {
                a.part_ml[prow * 2] = ref[ct];
                a.part_ml[prow * 2 + 1] = L[ct];
            } else if (a.lse) {
                a.lse[grow] = lse_of(ref[ct], L[ct]);
            }
        }
    }
}

template <int D, int G, bool BF, int RG>
hipError_t attend_wide(const Kv4Attn &a, dim3 grid, hipStream_t s)
{
    constexpr int rows = 32 * RG, turns = sizeof(Turn<D, G, 4 / RG>) * (RG == 4 ? 2 : 1);
    const int lds = turns + 2 * rows + (a.max_q + 1) / 2 * 4 + 4 * rows * ((a.max_q + 62) / 32);
    // above 64 KB LDS has to be asked for; the attribute is per device, and cheap
    const hipError_t e = hipFuncSetAttribute((const void *)k_kv4_tree_wide<D, G, BF, RG>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    k_kv4_tree_wide<D, G, BF, RG><<<grid, dim3(256), lds, s>>>(a);
    return hipGetLastError();
}

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const dim3 grid((uint32_t)((int64_t)a.ns * a.pool.H * a.B * a.tiles)), block(64 * kWaves);
    hipError_t e;
    if (a.rows == 128)
        e = attend_wide<D, G, BF, 4>(a, grid, s);
    else if (a.rows == 64)
        e = attend_wide<D, G, BF, 2>(a, grid, s);
    else {
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

int64_t splits(const Kv4Pool &p, int64_t blocks, int64_t keys)
{
    int64_t ns = 1;
    if (keys > 512)
        for (const auto &l : {std::pair<int64_t, int64_t>{256, 256}, {512, 512}})
            ns = std::max(ns, std::min(l.first / blocks, (keys + l.second - 1) / l.second));
    return std::min<int64_t>(ns, 128);
}

}  // namespace

Kv4Plan kv4_tree_plan(const Kv4Pool &p, int64_t n_seqs, int R, int64_t max_q, int64_t max_keys, int64_t window)
{
    Kv4Plan plan = {};
    const int64_t most = max_q * R;
    const int rows = most > 64 ? 128 : most > 32 ? 64 : most > 16 ? 32 : 16;
    plan.rows = rows;
    plan.tiles = (int32_t)((max_q * R + rows - 1) / rows);
    const int64_t blocks = std::max<int64_t>(n_seqs * p.H * plan.tiles, 1);
    // a window reaches back from the tree's first token, and its keys go on to the last
    const int64_t keys = window ? std::min(max_keys, window + max_q) : max_keys;
    plan.ns = (int32_t)splits(p, blocks, keys);
    plan.most_ns = (int32_t)splits(p, blocks, max_keys);
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
