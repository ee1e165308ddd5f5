// kvc_kv4_tree.hip - attention of a tree of drafted tokens over the resident
// 4-bit cache.
//
// The arithmetic is that of kvc_kv4_attn.hip (codes as matrix operands, s and lo
// outside of them, p s as two fp16 terms relative to the row's largest p s); what
// differs is which keys a row sees and how many rows there are: a tree's tokens
// times the heads of a group, typically 32 to 512, all over the same keys.  Two
// kernels: k_kv4_tree, whose waves have CT tiles of 16 rows each and unpack a
// block of 32 keys once for all of them, and blocks of 128 rows (kv4_rows.h),
// whose waves unpack for each other.
//
// Of the drafted keys a row sees its own path.  A block that holds such keys
// walks the parents of its tokens once, in LDS, and keeps the path as bits, one word
// per token and block of 32 keys.
#include <algorithm>
#include <type_traits>

#include "kv4_rows.h"

namespace {

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
    // the same for the whole block; a tile without a key walks for its bad parents
    const bool walks = b_end > paths.first || a.window || j.kend == 0;
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

// Which shapes blocks of 128 rows are faster for (16 sequences of up to 8192 keys, 8 KV heads, trees of 128 rows, bf16; 8
// sequences with D = 256): D = 128 G = 32, 64, 128: 176, 127, 114 us, tiles of 32 rows 219, 147, 122 (fp16, G = 64: 127, 142;
// soft cap: 148, 160); D = 256 G = 32 359, 400.  The others: D = 64 G = 32, 64: 102, 106 and 87, 89; D = 256 G = 64, 128: 224,
// 198 and 183, 175.
constexpr bool has_rows(int D, int G) { return D == 128 || (D == 256 && G == 32); }

template <int D, int G, bool BF>
hipError_t attend(const Kv4Attn &a, hipStream_t s)
{
    const dim3 grid((uint32_t)((int64_t)a.ns * a.pool.H * a.B * a.tiles)), block(64 * kWaves);
    hipError_t e = hipErrorInvalidValue;
    if (a.rows == kRows) {
        if constexpr (has_rows(D, G)) e = launch_rows<D, G, BF, true>(a, grid.x, s);
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
//   Blocks of 128 rows.  {512, 512}: 128 of 8192 129 in 4, 181 in 3, 137 in 8; 32 of 80000 374 in 16, 528 in 8, 382 in 32.
// {1024, 2048} for sequences of several lengths: 128 of 16000 252 in 8, 304 in 4, 293 in 16; of a single one 64 of 30000
// 309 in 8, 312 in 16.
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
    const int64_t tiles = (most + narrow - 1) / narrow, wide_tiles = (most + kRows - 1) / kRows;
    // a window reaches back from the tree's first token, and its keys go on to the last
    const int64_t keys = window ? std::min(max_keys, window + max_q) : max_keys;
    // blocks of 128 rows where the longest tree gives at least 7/8 of their waves rows (trees of up to 112 rows: 126 us for
    // 124, G = 32 176 for 193; of up to 96: 122 for 118, since most are smaller, G = 32 168 for 174, D = 256 343 for 332), the
    // keys fill the chip (8 heads of 2 sequences of 2000 keys: 27 us for 25) and the paths leave a compute unit the blocks
    // that its registers hold (16 trees of 128 tokens with a head each: 221 us for 145)
    const int64_t full = p.D == 128 && p.G == 32 ? 24 : 28;  // of 32
    const bool fits = rows_lds(p.D, p.G) + tree_lds(R, (int)max_q) <= (p.D == 256 ? kLds : kLds / 2);
    const bool wide = has_rows(p.D, p.G) && fits && tiles * 8 >= wide_tiles * full && heads * wide_tiles * ((keys + 511) / 512) >= 512;
    plan.rows = wide ? kRows : (int32_t)narrow;
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
