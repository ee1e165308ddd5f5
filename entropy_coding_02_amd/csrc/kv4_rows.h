// kv4_rows.h - blocks of 128 query rows over the resident 4-bit cache: prompt
// pieces (kvc_kv4_attn.hip) and trees of many rows (kvc_kv4_tree.hip).
#pragma once

#include <algorithm>

#include "kv4_tile.h"

namespace {

constexpr int kRows = 128;   // query rows of a block, 32 a wave
constexpr int kKeys = 64;    // keys a turn
constexpr int kLds = 163840;  // of a compute unit

// ------------------------------------------------------- a tree's own keys

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

// Tokens that 128 rows may belong to.
__host__ __device__ constexpr int tile_tokens(int R, int max_q)
{
    const int most = (kRows - 2) / R + 2 < kRows ? (kRows - 2) / R + 2 : kRows;
    return max_q < most ? max_q : most;
}

// Which of the keys key0 .. key0 + 31 a token of the tile sees: those before the tree, from its window's first on, and its path's.
__device__ __forceinline__ uint32_t sees(const Kv4Attn &a, const Job &j, const Paths &p, const int16_t *steps, int tok, int key0)
{
    const int k_lo = a.window ? max(0, j.pos0 + steps[tok] - a.window) : 0;
    const int n = min(max(j.pos0 - key0, 0), 32), m = min(max(k_lo - key0, 0), 32), w = (key0 >> 5) - p.first;
    uint32_t see = (uint32_t)((1ull << n) - 1) & ~(uint32_t)((1ull << m) - 1);
    if (w >= 0 && w < p.words) see |= p.bits[tok * p.words + w];
    return see;
}

// ------------------------------------------------------- blocks of 128 rows

// LDS of such a block, and what a tree's paths take more.
constexpr int rows_lds(int D, int G)
{
    return 2 * (4 * (D / 32) * 1024 + 2 * (D / 16) * 1024 + 4 * 1024 + 3 * 4 * 64 * ((D / G + 3) / 4) * 4 + kKeys * 4);
}
constexpr int tree_lds(int R, int max_q)
{
    return (tile_tokens(R, max_q) + 1) / 2 * 4 + 4 * tile_tokens(R, max_q) * ((max_q + 62) / 32);
}

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
// TREE: the rows are a tree's tokens and see their own paths.  What they do not see takes no part, whatever its size: neither
// the scale of p s nor any operand of a row goes by it.  60 tokens of 8 heads a KV head, 80000 keys, 8 KV heads, bf16: 374 us,
// 0.42 PFLOP/s of products (tiles of 32 rows 403).  Tried: V's s in its operand, scaled by the largest value of 16 keys, and p
// as one term for bf16 (358 us) or two: keys whose tile also held one of far larger values, seen or not, were lost among fp16's
// subnormals (sizes 2^16 apart: outputs off by 5%, or by anything).
template <int D, int G, bool BF, bool TREE>
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
    static_assert(2 * sizeof(Turn) == rows_lds(D, G));
    extern __shared__ __align__(16) uint8_t lds_raw[];
    Turn *const turns = (Turn *)lds_raw;
    Job j;
    if (!make_job<kRows, TREE>(a, j)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, h = lane >> 4;
    const int t_end = min(j.u1 * 2, (j.kend + kKeys - 1) / kKeys);
    int turn = j.u0 * 2;
    const WaveAt<D, G> wat(a, j);
    const LaneAt<D, G> at(lane, a.pool);

    // a tree's paths lie behind the turns (tree_lds); its parents, done with before, where the first turn goes
    int16_t *const lds_steps = (int16_t *)(turns + 2), *const lds_parent = (int16_t *)lds_raw;
    static_assert(2 * kTreeMost <= sizeof(Turn), "the parents fit there");
    Paths paths;
    const int last_row = min(j.row0 + kRows, j.rows) - 1, tok0 = j.row0 / a.R;
    if constexpr (TREE) {
        paths.bits = (uint32_t *)(lds_steps + (tile_tokens(a.R, a.max_q) + 1) / 2 * 2);
        paths.base = j.pos0;
        paths.first = max(j.pos0, 0) >> 5;
        paths.words = max(((j.kend + 31) >> 5) - paths.first, 0);
        // the same for the whole block; a tile without a key walks for its bad parents
        if (t_end * 2 > paths.first || a.window || j.kend == 0) {
            stage_parents(a, j, last_row / a.R, lds_parent);
            lds_barrier();
            walk(a, paths, lds_parent, tok0, last_row / a.R, lds_steps);
        }
        lds_barrier();
    }

    // the wave's rows: two column tiles of 16.  Where trees have fewer, the same waves would idle in every block.
    const int row_w = j.row0 + 32 * (TREE ? (wave + (int)blockIdx.x) & 3 : wave);
    u32x4 q[2][NW];
    u32x4 sums[2];
    float up[2];
    int k_lo[2], k_hi[2];
    uint32_t toks = 0;  // which of the tile's tokens the lane's rows are
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int row = row_w + 16 * ct + col, qi = row / a.R;
        const bool real = row < j.rows;
        if constexpr (TREE) {
            toks |= (uint32_t)(min(row, last_row) / a.R - tok0) << (16 * ct);
        } else {
            const int pos = j.pos0 + qi;
            k_hi[ct] = a.causal ? min(j.len, pos + 1) : j.len;
            k_lo[ct] = a.window ? max(0, pos - a.window + 1) : 0;
        }
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
    const int any_lo = a.window ? j.pos0 + (TREE ? 0 : row_w / a.R) - a.window + 1 : 0;
    const int all_hi = TREE ? j.pos0 : a.causal ? min(j.len, j.pos0 + row_w / a.R + 1) : j.len;
    const int all_lo = a.window ? j.pos0 + (TREE ? j.nq - 1 : last / a.R) - a.window + 1 : 0;

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
                    if (TREE && partial) {
                        const uint32_t see = sees(a, j, paths, lds_steps, toks >> (16 * ct) & 0xFFFF, key0) >> (4 * h);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (!(see >> (16 * (i / 4) + i % 4) & 1)) x[ct][i / 4][i % 4] = -__builtin_inff();
                    } else if (partial) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int key = key0 + 16 * (i / 4) + 4 * h + i % 4;
                            if (key < k_lo[ct] || key >= k_hi[ct]) x[ct][i / 4][i % 4] = -__builtin_inff();
                        }
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
                                if (x[ct][i / 4][i % 4] == -__builtin_inff()) {
                                    vmid[i / 4][i % 4] = 0.0f;
                                    if (TREE) vs[i / 4][i % 4] = 0.0f;
                                }
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

template <int D, int G, bool BF, bool TREE>
hipError_t launch_rows(const Kv4Attn &a, uint32_t blocks, hipStream_t s)
{
    // above 64 KB LDS has to be asked for; the attribute is per device, and cheap.  As much as any call takes, always: calls of
    // several threads must not lower it for each other.
    constexpr int turns = rows_lds(D, G), most = TREE ? std::min(kLds, turns + tree_lds(1, kTreeMost)) : turns;
    const int lds = TREE ? turns + tree_lds(a.R, a.max_q) : turns;
    if (most > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)k_kv4_prompt<D, G, BF, TREE>, hipFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != hipSuccess) return e;
    }
    k_kv4_prompt<D, G, BF, TREE><<<dim3(blocks), dim3(256), lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace
