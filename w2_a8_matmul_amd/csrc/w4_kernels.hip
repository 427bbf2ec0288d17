// The linear layer with 4-bit weights and group scales ("W4") for gfx950:
// tiled weight layout, the product kernel for few token rows, entry points.
//
// Mathematics: y[m][n] = xs[m] * sum_g s[n][g] * sum_{k in g} xq[m][k] * (q[n][k] - z[n][g]).
// The inner sums are exact INT32 products on the INT8 matrix instructions;
// only the outer sum over the groups is fp32.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

// --------------------------------------------------------------- tiled layout

// Fragment (tile t of 16 channels, block b of 128 columns) is 1 KiB at
// (t * KB + b) * 1024, KB = ceil(K/128).  Lane L = n + 16 g of a wave owns 16
// bytes of it, those of channel 16 t + n; byte i holds the code of column
// 128 b + c(g, i) in its low nibble and of column 128 b + 64 + c(g, i) in its
// high one.  The low nibbles of a fragment are thus one B operand of the INT8
// products over columns 0..63 of the block, and the high ones one over
// 64..127, each after one mask.  c(g, i) is 16 g + i (v_mfma_i32_16x16x64_i8
// on activations read 16 bytes at a time), or, with 4 scales a block,
// 32 (i / 8) + 8 g + i % 8: each half of 8 bytes is then an operand of
// v_mfma_i32_16x16x32_i8, whose sum stays inside one 32-column group.
// Without zero points the nibbles are q - 8 in two's complement: masked into
// the high half of a byte they are 16 (q - 8), an INT8 operand in one or two
// instructions for four weights, and the factor 16 is taken out of the scale
// (exactly: a bf16 scale is a multiple of 2^-133, a sixteenth of it an fp32 number;
// taken out of the sum instead, it made sums over 2^124 infinite).  With zero points the
// nibbles are q.
//
// The scales follow the fragments: P = 1, 2 or 4 per channel and block (the
// group size a multiple of 128, of 64 or of 32; larger groups repeat theirs),
// [t][b][n][P] bf16, then the zero points in the same order, a byte each.
constexpr int kBlk = 128;

int per_block(int64_t K, int64_t group) {
    if (group % 128 == 0 || group >= K) return 1;
    return group % 64 == 0 ? 2 : 4;
}

int64_t w4_bytes(int64_t N, int64_t K, int64_t group, bool zeros) {
    const int64_t frags = ((N + 15) / 16) * ((K + kBlk - 1) / kBlk);
    return frags * (1024 + per_block(K, group) * (zeros ? 48 : 32));
}

__host__ __device__ constexpr int frag_column(int P, int g, int i) {
    return P == 4 ? 32 * (i >> 3) + 8 * g + (i & 7) : 16 * g + i;
}

constexpr int kTileThreads = 256;

// One thread per 16-byte piece, then one per (channel, block) of the scales.
__global__ __launch_bounds__(kTileThreads) void w4_tile_kernel(const uint8_t *__restrict__ packed,
                                                               const uint16_t *__restrict__ scales,
                                                               const uint8_t *__restrict__ zeros, int N, int K,
                                                               int64_t group, int G, int P, int64_t frags,
                                                               uint8_t *__restrict__ tiled) {
    const int KB = (K + kBlk - 1) / kBlk;
    uint16_t *sc = reinterpret_cast<uint16_t *>(tiled + frags * 1024);
    uint8_t *zp = tiled + frags * (1024 + 32 * P);
    const int64_t pieces = frags * 64, total = pieces + frags * 16;
    for (int64_t c = (int64_t)blockIdx.x * kTileThreads + threadIdx.x; c < total;
         c += (int64_t)gridDim.x * kTileThreads) {
        const bool piece = c < pieces;
        const int64_t f = piece ? c >> 6 : (c - pieces) >> 4;
        const int l = piece ? (int)(c & 63) : (int)((c - pieces) & 15);
        const int64_t tile = f / KB;
        const int64_t n = tile * 16 + (l & 15);
        const int k0 = (int)(f - tile * KB) * kBlk;
        if (piece) {
            auto code = [&](int k) -> uint32_t {
                if (n >= N || k >= K) return 0u;
                const uint32_t q = (packed[n * (K / 2) + k / 2] >> (4 * (k & 1))) & 15u;
                return zeros ? q : q ^ 8u;
            };
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int k = k0 + frag_column(P, l >> 4, i);
                w[i >> 2] |= (code(k) | (code(k + 64) << 4)) << (8 * (i & 3));
            }
            *reinterpret_cast<uint4 *>(tiled + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int p = 0; p < P; ++p) {
                const int k = k0 + p * (kBlk / P);
                const bool ok = n < N && k < K;
                const int64_t at = ok ? n * G + k / group : 0;
                sc[(f * 16 + l) * P + p] = ok ? scales[at] : (uint16_t)0;
                if (zeros) zp[(f * 16 + l) * P + p] = ok ? zeros[at] : (uint8_t)0;
            }
        }
    }
}

// --------------------------------------------------------------- decode

// INT8 B operand dwords of the low (h = 0) or high (h = 1) nibbles of packed
// dword w.  Without zero points: 16 (q - 8) per byte.  With: q - z, where zrep
// holds z in every byte (the set top bit keeps each byte's difference from
// borrowing out of it; clearing it by exclusive or leaves q - z).
template <bool kZeros>
__device__ __forceinline__ int32_t nibbles(uint32_t w, int h, uint32_t zrep) {
    if constexpr (kZeros) {
        const uint32_t q = (h ? w >> 4 : w) & 0x0F0F0F0Fu;
        return (int32_t)(((q | 0x80808080u) - zrep) ^ 0x80808080u);
    } else {
        return (int32_t)((h ? w : w << 4) & 0xF0F0F0F0u);
    }
}

// What an INT32 sum of such operands is multiplied by, from a scale's bits in the upper
// half of a dword.
template <bool kZeros>
__device__ __forceinline__ float scale_of(uint32_t bits) {
    return kZeros ? __uint_as_float(bits) : __uint_as_float(bits) * 0.0625f;
}

// --------------------------------------------------------------- product, few rows

// Up to 16 token rows: one read of the weights.  A workgroup's 16 waves form
// 16 / KS teams; a team takes a group of NT tiles of 16 channels at a time, its KS
// waves every KS-th block of 128 columns.  Both operands go straight from memory to
// registers in operand order (lane L = n + 16 g: B column n; A row n, 16-byte
// piece g), kDepth blocks ahead; nothing passes through LDS but the waves'
// partial sums, which a team adds in wave order.
//
// A row r is token 4 (r % 4) + r / 4, so that result register i of lane group g
// belongs to token 4 i + g: with up to 4 tokens only register 0 of every result is
// converted and scaled, with up to 8 two (Q registers).
//
// Bound by the weight stream where there is one: 8 x 4096 -> 128256 with groups
// of 128 moves 275 MB in 50.8 us (5.4 TB/s, what a copy of 1 GiB reaches is
// 5.2), 1 x 4096 -> 14336 31 MB in 9.2 us (3.4 TB/s: 448 groups on 256 CUs take two
// rounds, and each join waits for its token scales, which the next group's
// loads are ahead of, so that the ring drains); 1 x 4096 -> 1024 takes 4.5 us, nearly
// all of it the launch and two memory round trips, the operands' and at the
// end the token scale's, on 64 of the CUs.
constexpr int kRowWaves = 16;

template <int NT, int Q, int P, bool kZeros>
__global__ __launch_bounds__(kRowWaves * 64) void w4_rows_kernel(
    const int8_t *__restrict__ xq, const uint8_t *__restrict__ tiled, int M, int K, int N, int KS, int rounds, int wgs,
    const float *__restrict__ xs, void *__restrict__ y, int obf) {
    constexpr int kDepth = 2;  // (three and four measured 1 to 8% slower)
    __shared__ float red[kRowWaves * NT * Q * 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int KB = (K + kBlk - 1) / kBlk, tiles = (N + 15) >> 4;
    const int teams = kRowWaves / KS, team = wave / KS, part = wave - team * KS;
    const uint32_t frags = (uint32_t)tiles * (uint32_t)KB;
    const auto rx = make_rsrc(xq, (uint32_t)M * (uint32_t)K);
    const auto rw = make_rsrc(tiled, frags * 1024u);
    const auto rs = make_rsrc(tiled + (int64_t)frags * 1024, frags * (32u * P));
    const auto rz = make_rsrc(tiled + (int64_t)frags * (1024 + 32 * P), kZeros ? frags * (16u * P) : 0u);

    struct Stage {
        uint4 w[NT];
        uint32_t s[NT][P == 4 ? 2 : 1], z[NT];
        uint4 a[2];
    };
    const int mine = (KB - part + KS - 1) / KS;     // this wave's blocks of a tile group
    int group = (int)blockIdx.x * teams + team;
    const int stride = wgs * teams;
    const int token = 4 * (n & 3) + (n >> 2);
    const uint32_t arow = token < M ? (uint32_t)token * (uint32_t)K : kOOB;
    auto load = [&](Stage &st, int grp, int step) {
        const int kb = part + KS * step;
        const bool live = step < mine;
        const uint32_t alive = live ? arow : kOOB;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (P == 4) {
                // the columns of byte halves 0..7 and 8..15 of the fragment's lane
                const int k = kb * kBlk + 64 * h + 8 * g;
                const auto lo = __builtin_amdgcn_raw_buffer_load_b64(
                    rx, alive != kOOB && k < K ? alive + (uint32_t)k : kOOB, 0, 0);
                const auto hi = __builtin_amdgcn_raw_buffer_load_b64(
                    rx, alive != kOOB && k + 32 < K ? alive + (uint32_t)k + 32u : kOOB, 0, 0);
                st.a[h] = make_uint4(lo[0], lo[1], hi[0], hi[1]);
            } else {
                const int k = kb * kBlk + 64 * h + 16 * g;
                st.a[h] = bload16(rx, alive != kOOB && k < K ? alive + (uint32_t)k : kOOB);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tile = grp * NT + t;
            const uint32_t f = (uint32_t)tile * (uint32_t)KB + (uint32_t)kb;
            const bool ok = live && tile < tiles;
            st.w[t] = bload16(rw, ok ? f * 1024u + 16u * (uint32_t)lane : kOOB);
            const uint32_t so = ok ? (f * 16u + (uint32_t)n) * (2u * P) : kOOB;
            if constexpr (P == 1) st.s[t][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, so, 0, 0);
            if constexpr (P == 2) st.s[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, so, 0, 0);
            if constexpr (P == 4) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, so, 0, 0);
                st.s[t][0] = v[0];
                st.s[t][1] = v[1];
            }
            if constexpr (kZeros) {
                const uint32_t zo = ok ? (f * 16u + (uint32_t)n) * (uint32_t)P : kOOB;
                if constexpr (P == 1) st.z[t] = __builtin_amdgcn_raw_buffer_load_b8(rz, zo, 0, 0);
                if constexpr (P == 2) st.z[t] = __builtin_amdgcn_raw_buffer_load_b16(rz, zo, 0, 0);
                if constexpr (P == 4) st.z[t] = __builtin_amdgcn_raw_buffer_load_b32(rz, zo, 0, 0);
            }
        }
    };
    float sum[NT][Q];
    auto consume = [&](const Stage &st) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t wv[4] = {st.w[t].x, st.w[t].y, st.w[t].z, st.w[t].w};
            auto add = [&](const v4i &c, uint32_t sbits) {
                const float s = scale_of<kZeros>(sbits << 16);
#pragma unroll
                for (int i = 0; i < Q; ++i) sum[t][i] = __builtin_fmaf(s, (float)c[i], sum[t][i]);
            };
            const v4i zero = {0, 0, 0, 0};
            v4i acc;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i b;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int p = P == 1 ? 0 : P == 2 ? h : 2 * h + (d >> 1);
                    b[d] = nibbles<kZeros>(wv[d], h, kZeros ? ((st.z[t] >> (8 * p)) & 0xFFu) * 0x01010101u : 0u);
                }
                const uint4 av = st.a[h];
                const v4i a = {(int)av.x, (int)av.y, (int)av.z, (int)av.w};
                if constexpr (P == 4) {
                    auto two = [](const v4i &v, int e) {
                        return (long)((uint64_t)(uint32_t)v[e] | (uint64_t)(uint32_t)v[e + 1] << 32);
                    };
                    add(__builtin_amdgcn_mfma_i32_16x16x32_i8(two(a, 0), two(b, 0), zero, 0, 0, 0), st.s[t][h]);
                    add(__builtin_amdgcn_mfma_i32_16x16x32_i8(two(a, 2), two(b, 2), zero, 0, 0, 0), st.s[t][h] >> 16);
                } else if constexpr (P == 2) {
                    add(__builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, zero, 0, 0, 0), h ? st.s[t][0] >> 16 : st.s[t][0]);
                } else {
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, h ? acc : zero, 0, 0, 0);
                    if (h) add(acc, st.s[t][0]);
                }
            }
        }
    };

    Stage ring[kDepth];
    // (group, step) of the next load; every wave takes steps_max steps per group, so
    // that barriers line up (blocks past its share are predicated off)
    const int steps_max = (KB + KS - 1) / KS;
    int ld_group = group, ld_step = 0;
    auto load_next = [&](Stage &st) {
        load(st, ld_group, ld_step);
        if (++ld_step == steps_max) {
            ld_step = 0;
            ld_group += stride;
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load_next(ring[d]);

    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < Q; ++i) sum[t][i] = 0.0f;
    };
    clear();
    int step = 0;
    const int total = rounds * steps_max;
#pragma unroll 1
    for (int st0 = 0; st0 < total; st0 += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (st0 + u >= total) break;  // uniform
            consume(ring[u]);
            load_next(ring[u]);
            if (++step < steps_max) continue;
            // the team's partial sums of this tile group, added in wave order
            step = 0;
            float *own = red + wave * (NT * Q * 64);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < Q; ++i) own[(t * Q + i) * 64 + lane] = sum[t][i];
            clear();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const float *from = red + team * KS * (NT * Q * 64);
            for (int o = part * 64 + lane; o < NT * Q * 64; o += KS * 64) {
                // o = token (16 NT) + channel, token 4 i + g'
                const int ch = o % (16 * NT), m = o / (16 * NT), c = group * (16 * NT) + ch;
                const float *at = from + ((ch >> 4) * Q + (m >> 2)) * 64 + (ch & 15) + 16 * (m & 3);
                float v = 0.0f;
                for (int w = 0; w < KS; ++w) v += at[w * (NT * Q * 64)];
                if (m < M && c < N) {
                    v = xs[m] * v;
                    if (obf)
                        static_cast<uint16_t *>(y)[(int64_t)m * N + c] = f32_to_bf16_rne(v);
                    else
                        static_cast<float *>(y)[(int64_t)m * N + c] = v;
                }
            }
            group += stride;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
    }
}

// --------------------------------------------------------------- product, many rows

// Workgroup tile of 32 TR token rows on eight waves, each with TR results of 32 x 32
// on v_mfma_i32_32x32x32_i8.  The waves form KP column ranges (range q takes blocks
// q, q + KP, ...) of 8 / KP waves, which side by side cover 32 (8 / KP) channels;
// the ranges' sums meet in LDS at the end, in their order.
//
// Everything a block of 128 columns needs is copied to LDS by LDS-DMA, S - 1
// blocks ahead: the activations, shared by the waves of a range and stored in
// 16-byte chunks by row, and each wave's own fragments, scales and zero points.
// (With the fragments loaded into registers instead, the compiler's waits for
// them count only the loads it knows and so also wait for younger activation
// copies.)
//
// What bounds it is issue: every group of every result costs a conversion and a
// multiply-add (2 P per result and block of 128) beside the product itself.
// The 32 x 32 products take half the issue slots of 16 x 16 ones per
// multiplication, and their K = 32 serves 32-column groups at full rate.
// 2048 x 4096 -> 14336 takes 159 us with groups of 64 (1.51 POP/s; 157 to 187 by
// card and by how long it has been running), 190 to 212 with zero points (four registers spill, and
// the scratch loads that bring two back in every step wait for the copies of the
// next block), 132 with 128, 230 with 32 and zero points: at 64, vector instructions issue 96% of
// the time and the matrix cores run 37% of it, LDS has no bank conflict.  At the end
// the token scales of each quad of rows are loaded between the stores, a wait for
// each: a fixed cost that counts where a CU has about one tile.
//
// K order.  Product operands hold 16 consecutive columns in lane half h of a row
// or channel.  With P = 1 or 2 those are chunk 2 h + s of a 64-column half
// (s = 0, 1: two products a half), the low or high nibbles of piece 2 h + s of
// the fragment; with P = 4, chunk h of a 32-column group, the halves of pieces
// 2 h and 2 h + 1.
typedef int32_t v16i __attribute__((ext_vector_type(16)));

template <int KP, int S, bool kZeros, int kARows>
struct GemmLds {
    static constexpr int kActs = KP * S * kARows * kBlk, kSums = KP > 1 ? 8 * kARows * 128 : 0;
    // activations; the ranges' partial sums after the last block
    __attribute__((aligned(16))) int8_t a[kActs > kSums ? kActs : kSums];
    __attribute__((aligned(16))) uint8_t w[S][8][2048];
    __attribute__((aligned(16))) uint8_t s[S][8][256], z[kZeros ? S : 1][8][256];
};

// One tile of 32 TR rows from row0, channels from 32 (8 / KP) bn; kARows >= 32 TR: what
// the LDS has room for.
template <int TR, int KP, int S, int P, bool kZeros, int kARows>
__device__ __forceinline__ void w4_gemm_tile(GemmLds<KP, S, kZeros, kARows> &lds, const int8_t *__restrict__ xq,
                                             const uint8_t *__restrict__ tiled, int M, int K, int N, int row0, int bn,
                                             const float *__restrict__ xs, void *__restrict__ y, int obf) {
    constexpr int WP = 8 / KP;                   // waves of a column range
    constexpr int BM = 32 * TR;
    constexpr int NA = BM / 8 / WP;              // activation loads (1 KiB) per wave and block
    constexpr int NL = NA + (kZeros ? 4 : 3);    // all loads per wave and block
    static_assert(BM / 8 % WP == 0, "the waves of a range share its activation loads evenly");
    constexpr int kRangeBytes = BM * kBlk;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int KB = (K + kBlk - 1) / kBlk, tiles = (N + 15) >> 4;
    const int part = wave / WP, pw = wave - part * WP;  // column range, wave of it
    const int tile0 = 2 * (bn * WP + pw);
    const int steps = (KB + KP - 1) / KP;

    const uint32_t frags = (uint32_t)tiles * (uint32_t)KB;
    const v4i rx = rsrc_words(xq, (uint32_t)M * (uint32_t)K);
    const v4i rw = rsrc_words(tiled, frags * 1024u);
    const v4i rs = rsrc_words(tiled + (int64_t)frags * 1024, frags * (32u * P));
    const v4i rz = rsrc_words(tiled + (int64_t)frags * (1024 + 32 * P), kZeros ? frags * (16u * P) : 0u);

    // activation load L = pw + WP j: rows 16 (L / 2) .., columns 64 (L % 2) .. of a
    // block; lane l moves 16-byte chunk l / 16 of row l % 16 to 16 l of KiB L
    uint32_t aoff[NA], atail[NA];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
        const int L = pw + WP * j, row = row0 + 16 * (L >> 1) + (lane & 15), col = 64 * (L & 1) + 16 * (lane >> 4);
        aoff[j] = row < M ? (uint32_t)row * (uint32_t)K + (uint32_t)col : kOOB;
        atail[j] = (KB - 1) * kBlk + col < K ? aoff[j] : kOOB;
    }
    // scale load: dword `lane` of the wave's two tiles of 8 P dwords; zero points:
    // of 4 P dwords.  (A tile past the last one re-reads that one: its channels
    // are not stored.)
    auto first = [&](int t) { return (uint32_t)min(tile0 + t, tiles - 1) * (uint32_t)KB; };
    const int st = lane / (8 * P), zt = lane / (4 * P);
    const uint32_t soff = st < 2 ? first(st) * (32u * P) + 4u * (lane % (8 * P)) : kOOB;
    const uint32_t zoff = zt < 2 ? first(zt) * (16u * P) + 4u * (lane % (4 * P)) : kOOB;
    const uint32_t wfirst[2] = {(uint32_t)__builtin_amdgcn_readfirstlane(first(0) * 1024u),
                                (uint32_t)__builtin_amdgcn_readfirstlane(first(1) * 1024u)};
    const uint32_t alds = S3D8_LDS_OFFSET(&lds.a[0]) + (uint32_t)(kRangeBytes * part) + 1024u * (uint32_t)pw;
    const uint32_t wlds = S3D8_LDS_OFFSET(&lds.w[0][wave][0]);
    const uint32_t slds = S3D8_LDS_OFFSET(&lds.s[0][wave][0]), zlds = S3D8_LDS_OFFSET(&lds.z[0][wave][0]);
    // step i of column range `part` is block part + KP i.  Past the last block
    // the activations are zeros and the weights those of the last one, so
    // that every wait counts the same and every range takes as many steps.
    auto issue = [&](int i, int slot) {
        const int kb = part + KP * i;
        const uint32_t kbc = (uint32_t)min(kb, KB - 1);
#pragma unroll
        for (int j = 0; j < NA; ++j)
            load_to_lds16_so(alds + (uint32_t)(KP * kRangeBytes) * slot + (uint32_t)(WP * 1024) * j,
                             kb < KB - 1 ? aoff[j] : kb == KB - 1 ? atail[j] : kOOB, kbc * kBlk, rx);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            load_to_lds16_so(wlds + 16384u * slot + 1024u * t, 16u * lane, wfirst[t] + kbc * 1024u, rw);
        load_to_lds4_so(slds + 2048u * slot, soff, kbc * (32u * P), rs);
        if constexpr (kZeros) load_to_lds4_so(zlds + 2048u * slot, zoff, kbc * (16u * P), rz);
    };

    float sum[TR][16];
#pragma unroll
    for (int r = 0; r < TR; ++r)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[r][e] = 0.0f;

#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i, i);
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
        // this wave's copies of step i have landed, everyone's after the
        // barrier, which also ends every read of step i - 1's slot
        wait_vmcnt_barrier<(S - 2) * NL>();
        issue(i + S - 1, slot == 0 ? S - 1 : slot - 1);

        // this lane's channel: pieces 2 h and 2 h + 1 of its fragment, scales, zero points
        const uint8_t *wp = &lds.w[slot][wave][1024 * (n >> 4) + 16 * (n & 15) + 512 * h];
        const uint4 w0 = *reinterpret_cast<const uint4 *>(wp), w1 = *reinterpret_cast<const uint4 *>(wp + 256);
        const uint32_t w[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
        const uint8_t *sp = &lds.s[slot][wave][2 * P * n], *zp = &lds.z[kZeros ? slot : 0][wave][P * n];
        uint32_t sv[2] = {0, 0}, zv = 0;
        if constexpr (P == 1) sv[0] = *reinterpret_cast<const uint16_t *>(sp);
        if constexpr (P == 2) sv[0] = *reinterpret_cast<const uint32_t *>(sp);
        if constexpr (P == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(sp);
            sv[0] = v.x;
            sv[1] = v.y;
        }
        if constexpr (kZeros) {
            if constexpr (P == 1) zv = *zp;
            if constexpr (P == 2) zv = *reinterpret_cast<const uint16_t *>(zp);
            if constexpr (P == 4) zv = *reinterpret_cast<const uint32_t *>(zp);
        }
        float s[P];
        uint32_t z[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            s[p] = scale_of<kZeros>(p & 1 ? sv[p >> 1] & 0xFFFF0000u : sv[p >> 1] << 16);
            z[p] = kZeros ? ((zv >> (8 * p)) & 0xFFu) * 0x01010101u : 0u;
        }
        // operand j of the block's four (j = 2 half + s, or the 32-column group)
        v4i b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint32_t wd = P == 4 ? w[d >> 1][2 * (j & 1) + (d & 1)] : w[j & 1][d];
                b[j][d] = nibbles<kZeros>(wd, j >> 1, z[P == 1 ? 0 : P == 2 ? j >> 1 : j]);
            }
        // row 32 r + n of the tile, chunk of 16 columns as above
        const int8_t *at = &lds.a[kRangeBytes * (KP * slot + part) + 2048 * (n >> 4) + 16 * (n & 15) +
                                 (P == 4 ? 256 : 512) * h];
        auto read_a = [&](int r, int j) {
            return *reinterpret_cast<const v4i *>(at + 4096 * r + 1024 * (j >> 1) + (P == 4 ? 512 : 256) * (j & 1));
        };
        constexpr int kChain = 4 / P;  // products of one group
        // A group's products back to back, the next group's activations behind
        // them, then the scaling: a wave's vector operations do not run in the
        // shadow of its own products but do beside another wave's (interleaved
        // with the products they cost 187 us for 170 at 2048 x 4096 x 14336).
        v4i a[2][kChain];
#pragma unroll
        for (int q = 0; q < kChain; ++q) a[0][q] = read_a(0, q);
#pragma unroll
        for (int k = 0; k < TR * P; ++k) {
            const int r = k / P, p = k % P;
            v16i c = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < kChain; ++q)
                c = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[k & 1][q], b[kChain * p + q], c, 0, 0, 0);
            if (k + 1 < TR * P)
#pragma unroll
                for (int q = 0; q < kChain; ++q)
                    a[(k + 1) & 1][q] = read_a((k + 1) / P, kChain * ((k + 1) % P) + q);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[r][e] = __builtin_fmaf(s[p], (float)c[e], sum[r][e]);
            __builtin_amdgcn_sched_barrier(0);
        }
        slot = slot == S - 1 ? 0 : slot + 1;
    }
    wait_vmcnt<0>();  // loads of blocks past the end

    // Result lane (n, h), element 4 q + e of row tile r: row 32 r + 8 q + 4 h + e, channel
    // n.  In quads of rows (quad 4 r + q): the ranges' sums are added in their
    // order, and the waves of a range store their share of the quads.
    constexpr int TO = 4 * TR / KP;
    static_assert(4 * TR % KP == 0, "the ranges share the quads evenly");
    float4 out[TO];
    if constexpr (KP == 1) {
#pragma unroll
        for (int o = 0; o < TO; ++o) {
            const float *v = &sum[o >> 2][4 * (o & 3)];
            out[o] = make_float4(v[0], v[1], v[2], v[3]);
        }
    } else {
        wait_vmcnt_barrier<0>();  // every wave has read its last block
        float4 *red = reinterpret_cast<float4 *>(&lds.a[0]);
#pragma unroll
        for (int o = 0; o < 4 * TR; ++o) {
            const float *v = &sum[o >> 2][4 * (o & 3)];
            red[((part * WP + pw) * 4 * TR + o) * 64 + lane] = make_float4(v[0], v[1], v[2], v[3]);
        }
        wait_vmcnt_barrier<0>();
#pragma unroll
        for (int o = 0; o < TO; ++o) {
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < KP; ++q) {
                const float4 u = red[((q * WP + pw) * 4 * TR + part * TO + o) * 64 + lane];
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            out[o] = v;
        }
    }
    // Rows past M lie past the end of the buffer and channels past N get an
    // offset that does: those stores are dropped.
    const int wrow = row0 + 8 * TO * part, nrows = min(M - wrow, 8 * TO);
    if (nrows <= 0) return;
    const uint32_t size = obf ? 2u : 4u, rowb = size * (uint32_t)N;
    const auto ry = make_rsrc(static_cast<char *>(y) + (int64_t)wrow * N * size, rowb * (uint32_t)nrows);
    const auto rxs = make_rsrc(xs + wrow, 4u * (uint32_t)nrows);
    const int ch = 16 * tile0 + n;
    const uint32_t base = ch < N ? 4u * h * rowb + size * (uint32_t)ch : kOOB;
#pragma unroll
    for (int o = 0; o < TO; ++o) {
        const uint4 sx = bload16(rxs, 32u * o + 16u * h);
        const float f[4] = {__uint_as_float(sx.x) * out[o].x, __uint_as_float(sx.y) * out[o].y,
                            __uint_as_float(sx.z) * out[o].z, __uint_as_float(sx.w) * out[o].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t off = base + (uint32_t)(8 * o + e) * rowb;
            if (obf)
                __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_rne(f[e]), ry, off, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[e]), ry, off, 0, 0);
        }
    }
}

// Workgroups as gemm_tile, but the tiles past the first `big` of an XCD go to two
// workgroups of half the rows each: what would be less than half a round of
// tiles on the XCD's CUs is then less than a round of halves.
template <int TR, int KP, int S, int P, bool kZeros>
__global__ __launch_bounds__(512, 4) void w4_gemm_kernel(const int8_t *__restrict__ xq,
                                                         const uint8_t *__restrict__ tiled, int M, int K, int N,
                                                         int nbm, int nbn, int big, const float *__restrict__ xs,
                                                         void *__restrict__ y, int obf) {
    __shared__ GemmLds<KP, S, kZeros, 32 * TR> lds;
    const int nt = nbm * nbn, per_xcd = (nt + kXcds - 1) / kXcds;
    const int i = (int)(blockIdx.x / kXcds);
    const int L = (int)(blockIdx.x % kXcds) * per_xcd + (i < big ? i : big + ((i - big) >> 1));
    if (L >= nt) return;  // padding workgroup
    int bm, bn;
    gemm_tile_at(L, nbm, nbn, bm, bn);
    const int row0 = bm * 32 * TR;
    if constexpr (TR == 4 && KP == 1) {
        if (i >= big) {
            const int half = row0 + 16 * TR * ((i - big) & 1);
            if (half < M) w4_gemm_tile<TR / 2, KP, S, P, kZeros>(lds, xq, tiled, M, K, N, half, bn, xs, y, obf);
            return;
        }
    }
    w4_gemm_tile<TR, KP, S, P, kZeros>(lds, xq, tiled, M, K, N, row0, bn, xs, y, obf);
}

// --------------------------------------------------------------- launches

struct W4Args {
    const int8_t *xq;
    const float *xs;
    const uint8_t *tiled;
    int M, K, N;
    void *y;
    int obf;
};

template <int NT, int Q>
void launch_rows(const W4Args &a, int P, bool zeros, int cus, hipStream_t stream) {
    const int KB = (a.K + kBlk - 1) / kBlk, groups = ((a.N + 15) / 16 + NT - 1) / NT;
    // as many waves on a group's columns as it has blocks, fewer (at least 4) once
    // the groups give every wave of every CU two: 128256 channels at one token
    // take 48.9 us with 4, 55.6 with 2; 28672 take 14.7 with 8, 16.0 with 16
    int KS = kRowWaves;
    while (KS > 1 && (KS / 2 >= KB || (KS > 4 && (int64_t)groups * KS > (int64_t)cus * kRowWaves * 2))) KS /= 2;
    const int teams = kRowWaves / KS;
    const int wgs = std::min((groups + teams - 1) / teams, cus);
    const int rounds = (groups + wgs * teams - 1) / (wgs * teams);
    typedef void (*Fn)(const int8_t *, const uint8_t *, int, int, int, int, int, int, const float *, void *, int);
    static const Fn fns[3][2] = {
        {w4_rows_kernel<NT, Q, 1, false>, w4_rows_kernel<NT, Q, 1, true>},
        {w4_rows_kernel<NT, Q, 2, false>, w4_rows_kernel<NT, Q, 2, true>},
        {w4_rows_kernel<NT, Q, 4, false>, w4_rows_kernel<NT, Q, 4, true>},
    };
    hipLaunchKernelGGL(fns[P == 4 ? 2 : P - 1][zeros], dim3(wgs), dim3(kRowWaves * 64), 0, stream, a.xq, a.tiled, a.M,
                       a.K, a.N, KS, rounds, wgs, a.xs, a.y, a.obf);
}

// Workgroup tiles of the GEMM: rows and channels, column ranges (waves split
// between them), and the time of a step of `ranges` blocks and of everything
// else, in ns, from K = 4096 with one workgroup on a CU (a second one beside
// it gains little: a workgroup keeps its SIMDs' issue busy).  They are those of groups of
// 64 without zero points and rank the tiles; as times they are low for zero points:
// 1600 x 5120 -> 1280 with groups of 128 is put at 20.8 us and takes 28.
struct GemmTile {
    int rows, channels, ranges, step_ns, fixed_ns;
};
constexpr GemmTile kGemmTiles[] = {
    {128, 256, 1, 1400, 3000}, {64, 256, 1, 825, 3000}, {64, 128, 2, 890, 3000},
    {64, 64, 4, 970, 3000},    {32, 128, 2, 510, 3000}, {32, 64, 4, 575, 3000},
};

struct GemmPlan {
    int tile, big;  // tile of kGemmTiles; whole tiles of an XCD (the rest are halved)
    int64_t ns;     // estimated time
};

// The tile with the least estimated time: rounds of workgroups on an XCD's CUs
// times a workgroup's time.  On the largest tile a last round that is at most
// half full is taken in halves, beside the workgroups before them on a CU (0.3 of a
// round: 2048 x 4096 -> 14336 has 3.5 rounds and takes 159 us, a round 47; 0.6 alone).
GemmPlan gemm_plan(int64_t M, int64_t K, int64_t N, int cus) {
    const int64_t KB = (K + kBlk - 1) / kBlk, cus_xcd = std::max(1, cus / kXcds);
    GemmPlan best{};
    for (int i = 0; i < (int)(sizeof(kGemmTiles) / sizeof(kGemmTiles[0])); ++i) {
        const GemmTile &t = kGemmTiles[i];
        const int64_t wgs = ((M + t.rows - 1) / t.rows) * ((N + t.channels - 1) / t.channels);
        const int64_t per_xcd = (wgs + kXcds - 1) / kXcds, rest = per_xcd % cus_xcd;
        const bool halves = i == 0 && rest > 0 && 2 * rest <= cus_xcd;
        const int64_t rounds = per_xcd / cus_xcd, tenths = 10 * rounds + (halves ? (rounds ? 3 : 6) : rest ? 10 : 0);
        const int64_t ns = tenths * ((KB + t.ranges - 1) / t.ranges * t.step_ns + t.fixed_ns) / 10;
        if (i == 0 || ns < best.ns) best = {i, (int)(halves ? per_xcd - rest : per_xcd), ns};
    }
    return best;
}

// a wave's rows of output stay under 2^31 bytes (32-bit store offsets)
constexpr int64_t kGemmMaxN = (int64_t(1) << 31) / (4 * 128) - 1;

template <int TR, int KP, int S>
void launch_gemm(const W4Args &a, int P, bool zeros, int big, hipStream_t stream) {
    constexpr int BM = 32 * TR, BN = 32 * (8 / KP);
    const int nbm = (a.M + BM - 1) / BM, nbn = (a.N + BN - 1) / BN;
    const int per_xcd = (nbm * nbn + kXcds - 1) / kXcds;
    typedef void (*Fn)(const int8_t *, const uint8_t *, int, int, int, int, int, int, const float *, void *, int);
    static const Fn fns[3][2] = {
        {w4_gemm_kernel<TR, KP, S, 1, false>, w4_gemm_kernel<TR, KP, S, 1, true>},
        {w4_gemm_kernel<TR, KP, S, 2, false>, w4_gemm_kernel<TR, KP, S, 2, true>},
        {w4_gemm_kernel<TR, KP, S, 4, false>, w4_gemm_kernel<TR, KP, S, 4, true>},
    };
    hipLaunchKernelGGL(fns[P == 4 ? 2 : P - 1][zeros], dim3((2 * per_xcd - big) * kXcds), dim3(512), 0, stream, a.xq,
                       a.tiled, a.M, a.K, a.N, nbm, nbn, big, a.xs, a.y, a.obf);
}

// Token rows of one call: keeps every launch under 2^32 threads.
constexpr int64_t kMaxRows = 1 << 19;

int check_w4(int64_t M, int64_t K, int64_t N, int64_t group, bool zeros) {
    if (M <= 0 || K <= 0 || N <= 0 || group <= 0)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes and group must be positive");
    if (K % 16 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "K must be a multiple of 16");
    if (group % 32 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "group must be a multiple of 32");
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (M > kMaxRows || K > lim - kBlk || N > lim - 64 || M > lim / K || M > lim / N || (N + 15) / 16 > lim / (K + kBlk) ||
        w4_bytes(N, K, group, zeros) > lim)
        return s3d8::fail(S3D8_ERR_SHAPE, "tensor too large (more than 2^31 elements or tiled bytes, or 524288 rows)");
    return S3D8_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                 int64_t tiled_bytes, int64_t group, int32_t has_zeros, const void *y, int32_t out_type) {
    if (!xq || !xs || !tiled || !y) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    if (out_type != S3D8_OUT_F32 && out_type != S3D8_OUT_BF16)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown output type");
    if (has_zeros != 0 && has_zeros != 1) return s3d8::fail(S3D8_ERR_INVALID_ARG, "has_zeros must be 0 or 1");
    int rc = check_w4(M, K, N, group, has_zeros != 0);
    if (rc) return rc;
    if (M > 16 && N > kGemmMaxN)
        return s3d8::fail(S3D8_ERR_SHAPE, "N over 4194303 is not supported for M > 16");
    if (tiled_bytes != w4_bytes(N, K, group, has_zeros != 0))
        return s3d8::fail(S3D8_ERR_INVALID_ARG,
                          "tiled_bytes is not s3d8_w4_tiled_bytes(N, K, group, has_zeros): pass the matrix as "
                          "s3d8_w4_tile laid it out for these arguments");
    if (!aligned16(xq) || !aligned16(tiled))
        return s3d8::fail(S3D8_ERR_ALIGN, "xq and the tiled weights must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(xs) & 3u || reinterpret_cast<uintptr_t>(y) & (out_type == S3D8_OUT_F32 ? 3u : 1u))
        return s3d8::fail(S3D8_ERR_ALIGN, "xs and y must be aligned to their elements");
    return S3D8_OK;
}

// Up to 16 rows.  Tiles per group: one while a CU has no more than one (4096 -> 1024 at
// one token 4.3 us, 4.6 with two), else two (4096 -> 14336: 9.4 us, 9.8 with one, 9.3
// with four; 8192: 6.7, 7.4, 7.8), or four where the activations that each group reads
// again are many (16 tokens, 14336: 10.5, 11.8 with two; the build for groups of 32 or 96
// with zero points does not fit the registers: 87 spill, and it takes 31 to 37 us).
void launch_few(const W4Args &a, int P, bool zeros, int cus, hipStream_t stream) {
    const int64_t tiles = ((int64_t)a.N + 15) / 16;
    const int nt = tiles <= cus ? 1 : a.M > 8 && tiles > 3 * cus ? 4 : 2;
    if (a.M <= 4)
        nt == 1 ? launch_rows<1, 1>(a, P, zeros, cus, stream) : launch_rows<2, 1>(a, P, zeros, cus, stream);
    else if (a.M <= 8)
        nt == 1 ? launch_rows<1, 2>(a, P, zeros, cus, stream) : launch_rows<2, 2>(a, P, zeros, cus, stream);
    else if (nt == 4)
        launch_rows<4, 4>(a, P, zeros, cus, stream);
    else
        nt == 1 ? launch_rows<1, 4>(a, P, zeros, cus, stream) : launch_rows<2, 4>(a, P, zeros, cus, stream);
}

void launch_many(const W4Args &a, const GemmPlan &plan, int P, bool zeros, hipStream_t stream) {
    switch (plan.tile) {
        case 0: launch_gemm<4, 1, 2>(a, P, zeros, plan.big, stream); break;
        case 1: launch_gemm<2, 1, 3>(a, P, zeros, plan.big, stream); break;
        case 2: launch_gemm<2, 2, 3>(a, P, zeros, plan.big, stream); break;
        case 3: launch_gemm<2, 4, 3>(a, P, zeros, plan.big, stream); break;
        case 4: launch_gemm<1, 2, 3>(a, P, zeros, plan.big, stream); break;
        default: launch_gemm<1, 4, 3>(a, P, zeros, plan.big, stream); break;
    }
}

int launch_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                  int64_t group, bool zeros, void *y, int32_t out_type, int cus, hipStream_t stream) {
    const bool bf = out_type == S3D8_OUT_BF16;
    const W4Args a{xq, xs, tiled, (int)M, (int)K, (int)N, y, bf};
    const int P = per_block(K, group);
    if (M <= 16) {
        launch_few(a, P, zeros, cus, stream);
        return s3d8::launch_status();
    }
    GemmPlan plan = gemm_plan(M, K, N, cus);
    // Up to 16 rows past a multiple of 64 (the 1601 tokens of an image) cost the
    // GEMM a row of tiles; where that is more than a launch of the kernel for
    // few rows (its weights at 4 TB/s and 3.5 us), they go there: 1601 x 5120 ->
    // 1280 takes 32.7 us in one launch, 30.1 in two.
    const int64_t rest = M % 64, whole = M - rest;
    if (rest > 0 && rest <= 16 && whole > 16) {
        const GemmPlan most = gemm_plan(whole, K, N, cus);
        if (most.ns + 3500 + w4_bytes(N, K, group, zeros) / 4000 < plan.ns) {
            const W4Args last{xq + whole * K, xs + whole, tiled, (int)rest, (int)K, (int)N,
                              static_cast<char *>(y) + whole * N * (bf ? 2 : 4), bf};
            launch_few(last, P, zeros, cus, stream);
            launch_many({xq, xs, tiled, (int)whole, (int)K, (int)N, y, bf}, most, P, zeros, stream);
            return s3d8::launch_status();
        }
    }
    launch_many(a, plan, P, zeros, stream);
    return s3d8::launch_status();
}

}  // namespace

extern "C" {

int64_t s3d8_w4_tiled_bytes(int64_t N, int64_t K, int64_t group, int32_t has_zeros) {
    if (N <= 0 || K <= 0 || group <= 0 || group % 32 != 0) return -1;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (N > lim || K > lim || (N + 15) / 16 > (int64_t(1) << 50) / (K + kBlk)) return -1;
    return w4_bytes(N, K, group, has_zeros != 0);
}

int32_t s3d8_w4_tile(const uint8_t *packed, const uint16_t *scales_bf16, const uint8_t *zeros, int64_t N, int64_t K,
                     int64_t group, uint8_t *tiled, void *stream) {
    if (!packed || !scales_bf16 || !tiled) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    int rc = check_w4(1, K, N, group, zeros != nullptr);
    if (rc) return rc;
    if (!aligned16(tiled)) return s3d8::fail(S3D8_ERR_ALIGN, "tiled must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(scales_bf16) & 1u)
        return s3d8::fail(S3D8_ERR_ALIGN, "scales_bf16 must be 2-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    const int64_t frags = ((N + 15) / 16) * ((K + kBlk - 1) / kBlk);
    const int64_t blocks = std::min<int64_t>((frags * 80 + kTileThreads - 1) / kTileThreads, (int64_t)cus * 8);
    hipLaunchKernelGGL(w4_tile_kernel, dim3((unsigned)blocks), dim3(kTileThreads), 0, (hipStream_t)stream, packed,
                       scales_bf16, zeros, (int)N, (int)K, group, (int)((K - 1) / group + 1), per_block(K, group),
                       frags, tiled);
    return s3d8::launch_status();
}

int32_t s3d8_w4_linear(const int8_t *xq, const float *xs, int64_t M, int64_t K, int64_t N, const uint8_t *tiled,
                       int64_t tiled_bytes, int64_t group, int32_t has_zeros, void *y, int32_t out_type,
                       void *stream) {
    int rc = check_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type);
    if (rc) return rc;
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    return launch_linear(xq, xs, M, K, N, tiled, group, has_zeros != 0, y, out_type, cus, (hipStream_t)stream);
}

int32_t s3d8_w4_forward(const float *x, int64_t M, int64_t K, int64_t N, const uint8_t *tiled, int64_t tiled_bytes,
                        int64_t group, int32_t has_zeros, void *y, int32_t out_type, int8_t *xq, float *xs,
                        void *stream) {
    int rc = check_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type);
    if (rc) return rc;
    rc = s3d8_quant_act(x, M, K, xq, xs, stream);
    if (rc) return rc;
    return s3d8_w4_linear(xq, xs, M, K, N, tiled, tiled_bytes, group, has_zeros, y, out_type, stream);
}

}  // extern "C"
