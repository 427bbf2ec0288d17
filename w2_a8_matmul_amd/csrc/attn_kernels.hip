// Attention of query tokens to an encoder's states, for gfx950.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kKeys = 64;       // keys in a block
constexpr int kRows = 32;       // query rows of a wave
constexpr int kMaxSplits = 64;
// The maximum that is taken off the scores is only raised when a score is past it by this power
// of 2: p up to 2^8 is as exact in bf16 and fp32 as p up to 1, and most blocks scale nothing.
constexpr float kSlack = 8.0f;

// What the kernels read: a pair is a sequence and a key head, whose R = T * G rows are
// its T query tokens (of all sequences, where they share their states) times the G query
// heads that read this key head, head fastest.
struct Attn {
    const uint16_t *q, *k, *v;
    const int32_t *lens;
    const uint64_t *words;  // [mask sequences][blocks][mask rows] bits of 64 keys, or NULL
    uint16_t *o;
    float *part;            // [splits][pairs][R][D] sums, then [splits][pairs][R] maximum and sum of p
    int64_t q_seq, q_row, q_head, k_seq, k_row, k_head, v_seq, v_row, v_head;
    int64_t word_seq, word_block, word_row;
    int Lq, Lk, G, Hk, D, R, pairs, tiles, splits, shared;
    float scale;            // times log2(e)
};

// Chunk (16 bytes, 8 entries) c of row r of a tile lies at chunk place(c, r) of the row's
// CPR chunks in LDS, so that the sixteen rows that a wide read takes a column from lie in
// different banks (keys), and the four rows that a transposed read takes four
// chunks from (values).
template <int CPR>
__device__ __forceinline__ int key_place(int c, int r) {
    return CPR == 16 ? c ^ (r & 15) : CPR == 8 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
}
template <int CPR>
__device__ __forceinline__ int value_place(int c, int r) {
    return CPR == 16 ? c ^ ((r & 3) << 2) : CPR == 8 ? c ^ (((r >> 1) & 1) << 2) : c;
}

// The larger of a lane's value and that of the lane 32 further.
__device__ __forceinline__ float halves_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// sum_j p_j v_j of one row over the keys from `begin` to `end` that it sees: entries
// `lane` and `lane` + 64.
__device__ __forceinline__ void visible_sum(const Attn &a, int64_t q_at, const uint16_t *kp, const uint16_t *vp, int64_t word_at,
                                         float most, int begin, int end, float (&e)[2]) {
    const int lane = threadIdx.x & 63;
    const uint64_t *words = a.words + word_at;
    float q[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) q[n] = lane + 64 * n < a.D ? bf16_to_f32(a.q[q_at + lane + 64 * n]) : 0.0f;
    for (int key = begin; key < end; ++key) {
        if (!(words[(key / kKeys) * a.word_block] >> (key % kKeys) & 1)) continue;
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
            if (lane + 64 * n < a.D) s = __builtin_fmaf(q[n], bf16_to_f32(kp[key * a.k_row + lane + 64 * n]), s);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
        const float p = (float)(__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s, a.scale, -most));
#pragma unroll
        for (int n = 0; n < 2; ++n)
            if (lane + 64 * n < a.D) e[n] = __builtin_fmaf(p, bf16_to_f32(vp[key * a.v_row + lane + 64 * n]), e[n]);
    }
}

template <int NK, int ND, int kW>
__global__ __launch_bounds__(64 * kW, 2) void attn_kernel(const Attn a) {
    constexpr int Dp = 32 * ND;         // entries of a row in LDS
    constexpr int CPR = Dp / 8;
    constexpr int kTile = kKeys * CPR;  // chunks
    static_assert(16 * NK <= Dp && CPR % kW == 0, "");
    __shared__ __attribute__((aligned(1024))) uint4 tiles[2][2][kTile];

    const int lane = threadIdx.x & 63, col = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int pair = (int)blockIdx.x % a.pairs, rest = (int)blockIdx.x / a.pairs;
    const int tile = rest % a.tiles, split = rest / a.tiles;
    const int seq = pair / a.Hk, head = pair % a.Hk;

    // this lane's row (past the last: the last again, not stored)
    const int row = (tile * kW + wave) * kRows + col;
    const bool live = row < a.R;
    const int rr = min(row, a.R - 1), t = rr / a.G, g = rr % a.G;
    const int b = a.shared ? t / a.Lq : seq, i = a.shared ? t % a.Lq : t;

    int len = a.lens ? a.lens[a.shared ? 0 : seq] : a.Lk;
    len = max(0, min(len, a.Lk));
    const int blocks = (len + kKeys - 1) / kKeys;
    const int first = (int)((int64_t)blocks * split / a.splits), last = (int)((int64_t)blocks * (split + 1) / a.splits);

    bf8 qf[NK];
    const uint16_t *qp = a.q + b * a.q_seq + i * a.q_row + (int64_t)(head * a.G + g) * a.q_head;
#pragma unroll
    for (int s = 0; s < NK; ++s) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (16 * s + 8 * h < a.D) u = *reinterpret_cast<const uint4 *>(qp + 16 * s + 8 * h);
        qf[s] = __builtin_bit_cast(bf8, u);
    }
    const int64_t word_at = b * a.word_seq + i * a.word_row;

    // the lane's part of each copy of a tile into LDS
    constexpr int kCopies = CPR / kW;
    uint32_t koff[kCopies], voff[kCopies];
#pragma unroll
    for (int n = 0; n < kCopies; ++n) {
        const int c = (wave + n * kW) * 64 + lane, r = c / CPR, p = c % CPR;
        const int kc = key_place<CPR>(p, r), vc = value_place<CPR>(p, r);  // (its own inverse)
        koff[n] = 8 * kc < a.D ? (uint32_t)r * (uint32_t)a.k_row * 2 + kc * 16 : kOOB;
        voff[n] = 8 * vc < a.D ? (uint32_t)r * (uint32_t)a.v_row * 2 + vc * 16 : kOOB;
    }
    const uint16_t *kp = a.k + seq * a.k_seq + head * a.k_head, *vp = a.v + seq * a.v_seq + head * a.v_head;
    auto copy_keys = [&](int block) {
        const int rows = min(kKeys, len - block * kKeys) - 1;
        const v4i r = rsrc_words(kp + (int64_t)block * kKeys * a.k_row, (uint32_t)(rows * a.k_row + a.D) * 2);
#pragma unroll
        for (int n = 0; n < kCopies; ++n)
            load_to_lds16_so(S3D8_LDS_OFFSET(&tiles[0][block & 1][(wave + n * kW) * 64]), koff[n], 0, r);
    };
    auto copy_values = [&](int block) {
        const int rows = min(kKeys, len - block * kKeys) - 1;
        const v4i r = rsrc_words(vp + (int64_t)block * kKeys * a.v_row, (uint32_t)(rows * a.v_row + a.D) * 2);
#pragma unroll
        for (int n = 0; n < kCopies; ++n)
            load_to_lds16_so(S3D8_LDS_OFFSET(&tiles[1][block & 1][(wave + n * kW) * 64]), voff[n], 0, r);
    };

    f16v acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
    float most = -FLT_MAX, sum = 0.0f;  // of scaled scores, in powers of 2; this lane's part of the sum

    // a score operand (32 keys, 16 entries) and a value operand (32 entries, 16 keys; transposed by the
    // read: entry by lane, four keys in a row) of a block
    auto key_operand = [&](int block, int i) {
        const int n = i / 2, r = i % 2 * 32 + col;
        return *reinterpret_cast<const bf8 *>(reinterpret_cast<const char *>(tiles[0][block & 1]) +
                                              (r * CPR + key_place<CPR>(2 * n + h, r)) * 16);
    };
    auto value_operand = [&](int block, int i) {
        const int n = i / ND, d = i % ND;
        struct Two {
            s4 x[2];
        } two;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 16 * n + 8 * j + 4 * h + ((lane & 15) >> 2);
            const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            two.x[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s4 *)(reinterpret_cast<const char *>(tiles[1][block & 1]) +
                                                         (r * CPR + value_place<CPR>(c, r)) * 16 + 8 * (lane & 1)));
        }
        return __builtin_bit_cast(bf8, two);
    };
    auto word_of = [&](int block, uint64_t word) {
        const int inside = len - block * kKeys;
        return inside < kKeys ? word & ((1ull << max(inside, 0)) - 1) : word;
    };
    auto load_word = [&](int block) { return a.words[word_at + block * a.word_block]; };
    auto most_of = [&](const f16v(&s)[2]) {
        float m = s[0][0];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) m = fmaxf(m, s[kt][r]);
        return m;
    };

    // Scores are transposed: key by register, row by lane.  Block n is weighed and added while the
    // scores of block n + 1 are computed: their products run beside the exponentials, and the
    // largest of them is found beside the products with the values.
    if (first < last) {
        uint64_t word = ~0ull, next_word = ~0ull;
        if (a.words) word = load_word(first);
        copy_keys(first);
        copy_values(first);
        wait_vmcnt_barrier<0>();
        word = word_of(first, word);
        if (first + 1 < last) {
            if (a.words) next_word = load_word(first + 1);
            copy_keys(first + 1);
        }
        f16v s[2], t[2];
#pragma unroll
        for (int r = 0; r < 16; ++r) s[0][r] = s[1][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * NK; ++i)
            s[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_operand(first, i), qf[i / 2], s[i % 2], 0, 0, 0);
        float m = most_of(s);

        auto step = [&](int block, f16v(&s)[2], f16v(&t)[2]) {
            wait_vmcnt_barrier<0>();
            const uint64_t after = word_of(block + 1, next_word);
            if (block + 2 < last) {
                if (a.words) next_word = load_word(block + 2);
                copy_keys(block + 2);
            }
            if (block + 1 < last) copy_values(block + 1);
            if (__ballot(word != ~0ull)) {
                const uint64_t mine = word >> (4 * h);
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const uint32_t bits = (uint32_t)(mine >> (32 * kt));
                        s[kt][r] = bits >> (8 * (r / 4) + r % 4) & 1 ? s[kt][r] : -INFINITY;
                    }
                m = most_of(s);
            }
            word = after;
            m = halves_max(m) * a.scale;
            if (__ballot(m > most + kSlack)) {
                m = fmaxf(most, m);
                const float f = __builtin_amdgcn_exp2f(most - m);
                most = m;
                sum *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= f;
            }
            constexpr int kAhead = 4;  // operands in flight
            bf8 operand[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) operand[i] = key_operand(block + 1, i);
            uint32_t pf[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) t[0][r] = t[1][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * NK; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                t[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[i % kAhead], qf[i / 2], t[i % 2], 0, 0, 0);
                operand[i % kAhead] = i + kAhead < 2 * NK ? key_operand(block + 1, i + kAhead)
                                                          : value_operand(block, i + kAhead - 2 * NK);
#pragma unroll
                for (int e = i * 16 / (2 * NK); e < (i + 1) * 16 / (2 * NK); ++e) {
                    bf2 pair;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        pair[x] = (__bf16)__builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 8][2 * (e % 8) + x], a.scale, -most));
                    sum = __builtin_amdgcn_fdot2_f32_bf16(pair, bf2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
                    pf[e] = __builtin_bit_cast(uint32_t, pair);
                }
            }
            m = t[0][0];
#pragma unroll
            for (int i = 0; i < 4 * ND; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                const uint4 p = make_uint4(pf[i / ND * 4], pf[i / ND * 4 + 1], pf[i / ND * 4 + 2], pf[i / ND * 4 + 3]);
                acc[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand[(i + 2 * NK) % kAhead], __builtin_bit_cast(bf8, p),
                                                                      acc[i % ND], 0, 0, 0);
                if (i + kAhead < 4 * ND) operand[(i + 2 * NK) % kAhead] = value_operand(block, i + kAhead);
#pragma unroll
                for (int e = i * 32 / (4 * ND); e < (i + 1) * 32 / (4 * ND); ++e) m = fmaxf(m, t[e / 16][e % 16]);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int block = first;;) {
            step(block, s, t);
            if (++block >= last) break;
            step(block, t, s);
            if (++block >= last) break;
        }
    }
    if (a.words) {
        // A hidden key has p = 0, but the product with an infinite or NaN value of it is NaN. Rows that
        // are not finite are summed again, one by one, over what they see.
        float z = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) z = __builtin_fmaf(acc[d][r], 0.0f, z);
        uint64_t bad = __ballot(z != z);
        bad = (bad | bad >> 32) & 0xFFFFFFFFull;
        while (bad) {
            const int lost = __builtin_ctzll(bad);
            bad &= bad - 1;
            float e[2] = {0.0f, 0.0f};
            visible_sum(a, __shfl((long long)(qp - a.q), lost), kp, vp, __shfl((long long)word_at, lost),
                        __shfl(most, lost), first * kKeys, min(last * kKeys, len), e);
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float x = __shfl(e[d / 2], (32 * d + 8 * (r / 4) + 4 * h + r % 4) & 63);
                    if (col == lost) acc[d][r] = x;
                }
        }
    }
    sum += __shfl_xor(sum, 32);

    if (!live) return;
    if (a.splits > 1) {
        const int64_t at = ((int64_t)split * a.pairs + pair) * a.R + row;
        float *p = a.part + at * a.D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int e = 32 * d + 2 * r + 4 * h;
                if (e < a.D) *reinterpret_cast<float4 *>(p + e) = make_float4(acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]);
            }
        if (h == 0) {
            float *ms = a.part + (int64_t)a.splits * a.pairs * a.R * a.D;
            *reinterpret_cast<float2 *>(ms + 2 * at) = make_float2(most, sum);
        }
        return;
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *o = a.o + (((int64_t)b * a.Lq + i) * a.Hk * a.G + head * a.G + g) * a.D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
            const int e = 32 * d + 2 * r + 4 * h;
            if (e < a.D)
                *reinterpret_cast<bf4 *>(o + e) = bf4{(__bf16)(acc[d][r] * f), (__bf16)(acc[d][r + 1] * f),
                                                      (__bf16)(acc[d][r + 2] * f), (__bf16)(acc[d][r + 3] * f)};
        }
}

// Partial sums of the splits joined: 4 entries of a row a thread, kLanes threads of a
// row's entries sharing its splits, so that a row's loads are all on their way at once (one
// thread for all of them: 10 us instead of 3 for 32 rows of 26 splits).
struct Partial {
    float most, sum;
    float4 x;
    __device__ __forceinline__ void join(float m, float n, float4 y) {
        const float top = fmaxf(most, m), f = __builtin_amdgcn_exp2f(most - top), g = __builtin_amdgcn_exp2f(m - top);
        most = top;
        sum = __builtin_fmaf(f, sum, g * n);
        x.x = __builtin_fmaf(f, x.x, g * y.x);
        x.y = __builtin_fmaf(f, x.y, g * y.y);
        x.z = __builtin_fmaf(f, x.z, g * y.z);
        x.w = __builtin_fmaf(f, x.w, g * y.w);
    }
};
template <int kLanes>
__global__ __launch_bounds__(256) void attn_join_kernel(const Attn a) {
    constexpr int kRowsHere = 8 / kLanes, kAtOnce = 4;
    __shared__ Partial parts[256];
    const int e = (threadIdx.x & 31) * 4, lane = (threadIdx.x >> 5) % kLanes, here = (threadIdx.x >> 5) / kLanes;
    const int64_t rows = (int64_t)a.pairs * a.R, at = (int64_t)blockIdx.x * kRowsHere + here;
    const bool in = at < rows && e < a.D;
    const float *ms = a.part + a.splits * rows * a.D;
    Partial p{-FLT_MAX, 0.0f, make_float4(0, 0, 0, 0)};
    if (in)
        for (int s0 = lane; s0 < a.splits; s0 += kAtOnce * kLanes) {
            float2 u[kAtOnce];
            float4 y[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int s = min(s0 + n * kLanes, a.splits - 1);
                u[n] = *reinterpret_cast<const float2 *>(ms + 2 * (s * rows + at));
                y[n] = *reinterpret_cast<const float4 *>(a.part + (s * rows + at) * a.D + e);
            }
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n)
                if (s0 + n * kLanes < a.splits) p.join(u[n].x, u[n].y, y[n]);
        }
    if constexpr (kLanes > 1) {
        parts[threadIdx.x] = p;
        __syncthreads();
        if (lane) return;
#pragma unroll
        for (int n = 1; n < kLanes; ++n) {
            const Partial &o = parts[threadIdx.x + 32 * n];
            p.join(o.most, o.sum, o.x);
        }
    }
    if (!in) return;
    const int pair = (int)(at / a.R), row = (int)(at % a.R), seq = pair / a.Hk, head = pair % a.Hk, t = row / a.G, g = row % a.G;
    const int64_t token = a.shared ? t : (int64_t)seq * a.Lq + t;
    const float f = p.sum == 0.0f ? 0.0f : 1.0f / p.sum;
    typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf4 *>(a.o + ((token * a.Hk + head) * a.G + g) * a.D + e) =
        bf4{(__bf16)(p.x.x * f), (__bf16)(p.x.y * f), (__bf16)(p.x.z * f), (__bf16)(p.x.w * f)};
}

// The mask as bits: a wave takes a row's eight blocks of 64 keys.
constexpr int kMaskBlocks = 8;
__global__ __launch_bounds__(256) void attn_mask_kernel(const uint8_t *mask, int64_t mask_seq, int64_t mask_row, int64_t rows,
                                                        int Lk, int blocks, uint64_t *words) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), seq = blockIdx.z;
    if (row >= rows) return;
    const uint8_t *p = mask + seq * mask_seq + row * mask_row;
    const int first = blockIdx.y * kMaskBlocks;
    uint64_t w[kMaskBlocks];
#pragma unroll
    for (int n = 0; n < kMaskBlocks; ++n) {
        const int key = (first + n) * kKeys + lane;
        w[n] = __ballot(key < Lk && p[key] != 0);
    }
    uint64_t mine = 0;
#pragma unroll
    for (int n = 0; n < kMaskBlocks; ++n) mine = lane == n ? w[n] : mine;
    if (lane < kMaskBlocks && first + lane < blocks) words[(seq * blocks + first + lane) * rows + row] = mine;
}

// --------------------------------------------------------------- host

struct Plan {
    int64_t pairs, R, tiles, splits, waves;
    int64_t word_seqs, word_rows, blocks;
    int64_t words, part;  // bytes
};

int check_sizes(const s3d8_cross_attention_args &a) {
    if (a.B <= 0 || a.Lq <= 0 || a.Lk <= 0 || a.heads <= 0 || a.kv_heads <= 0 || a.D <= 0)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (a.B > 65535 || a.Lq > 1 << 24 || a.Lk > 1 << 24 || a.heads > 4096)
        return s3d8::fail(S3D8_ERR_SHAPE, "more than 65535 sequences, 2^24 tokens or keys or 4096 heads are not supported");
    if (a.D % 16 || a.D > 128) return s3d8::fail(S3D8_ERR_SHAPE, "heads must be a multiple of 16 up to 128");
    if (a.heads % a.kv_heads) return s3d8::fail(S3D8_ERR_SHAPE, "heads must be a multiple of kv_heads");
    if (a.B * a.Lq * a.heads > 1 << 30) return s3d8::fail(S3D8_ERR_SHAPE, "B Lq heads over 2^30 is not supported");
    return S3D8_OK;
}

Plan plan(const s3d8_cross_attention_args &a, int cus) {
    Plan p{};
    const int64_t G = a.heads / a.kv_heads;
    p.pairs = (a.shared ? 1 : a.B) * a.kv_heads;
    p.R = (a.shared ? a.B * a.Lq : a.Lq) * G;
    p.blocks = (a.Lk + kKeys - 1) / kKeys;
    p.waves = p.R <= 96 ? 1 : 4;
    p.tiles = (p.R + kRows * p.waves - 1) / (kRows * p.waves);
    const int64_t groups = p.pairs * p.tiles, most = p.waves == 1 ? p.blocks : p.blocks / 4;
    p.splits = std::max<int64_t>(1, std::min<int64_t>({2 * cus / groups, most, kMaxSplits}));
    if (a.mask) {
        p.word_seqs = a.mask_seq ? a.B : 1;
        p.word_rows = a.mask_row ? a.Lq : 1;
        p.words = (p.word_seqs * p.word_rows * p.blocks * 8 + 15) / 16 * 16;
    }
    if (p.splits > 1) p.part = p.splits * p.pairs * p.R * (a.D + 2) * 4;
    return p;
}

template <int kW>
auto attn_build(int64_t D) {
    return D <= 64 ? attn_kernel<4, 2, kW> : D <= 80 ? attn_kernel<5, 3, kW> : D <= 96 ? attn_kernel<6, 3, kW> : attn_kernel<8, 4, kW>;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

int64_t s3d8_cross_attention_workspace_bytes(const s3d8_cross_attention_args *args, int32_t num_cus) {
    if (!args || num_cus <= 0 || check_sizes(*args)) return -1;
    const Plan p = plan(*args, num_cus);
    s3d8::clear_error();
    return p.words + p.part;
}

int32_t s3d8_cross_attention(const s3d8_cross_attention_args *args, void *stream) {
    if (!args || !args->q || !args->k || !args->v || !args->o) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_cross_attention_args &a = *args;
    int rc = check_sizes(a);
    if (rc) return rc;
    if ((a.xq != nullptr) != (a.xs != nullptr)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "xq and xs go together");
    if (!(a.scale > 0.0f && a.scale <= 0x1p100f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "scale must be positive (at most 2^100)");
    if (a.xq && a.heads * a.D > 65536) return s3d8::fail(S3D8_ERR_SHAPE, "codes of rows over 65536 are not supported");
    if (a.xq && a.B * a.Lq > 1 << 19) return s3d8::fail(S3D8_ERR_SHAPE, "codes of more than 524288 rows are not supported");
    const int64_t lim = int64_t(1) << 40;
    for (int64_t s : {a.q_seq, a.q_row, a.q_head, a.k_seq, a.k_row, a.k_head, a.v_seq, a.v_row, a.v_head}) {
        if (s < 0 || s > lim) return s3d8::fail(S3D8_ERR_INVALID_ARG, "strides must not be negative (and at most 2^40)");
        if (s % 8) return s3d8::fail(S3D8_ERR_ALIGN, "strides must be multiples of 8");
    }
    if (a.Lk > 1 && (a.k_row < a.D || a.v_row < a.D || a.k_row >= 1 << 23 || a.v_row >= 1 << 23))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "k_row and v_row must be at least D and below 2^23");
    if (a.mask && (a.mask_seq < 0 || a.mask_row < 0 || a.mask_seq > lim || a.mask_row > lim))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "mask strides must not be negative (and at most 2^40)");
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.o, 16) || !aligned(a.xq, 16) ||
        !aligned(a.workspace, 16))
        return s3d8::fail(S3D8_ERR_ALIGN, "q, k, v, o, xq and workspace must be 16-byte aligned");
    if (!aligned(a.kv_lens, 4) || !aligned(a.xs, 4)) return s3d8::fail(S3D8_ERR_ALIGN, "kv_lens and xs must be 4-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    const Plan p = plan(a, cus);
    if (p.words + p.part > 0 && (!a.workspace || a.workspace_bytes < p.words + p.part))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "workspace smaller than s3d8_cross_attention_workspace_bytes");
    if (p.pairs * p.tiles * p.splits * 64 * p.waves >= int64_t(1) << 32)
        return s3d8::fail(S3D8_ERR_SHAPE, "more than 2^32 threads are not supported");
    Attn d{};
    d.q = a.q;
    d.k = a.k;
    d.v = a.v;
    d.lens = a.kv_lens;
    d.o = a.o;
    d.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + p.words);
    d.q_seq = a.q_seq;
    d.q_row = a.q_row;
    d.q_head = a.q_head;
    d.k_seq = a.k_seq;
    d.k_row = a.Lk > 1 ? a.k_row : a.D;
    d.k_head = a.k_head;
    d.v_seq = a.v_seq;
    d.v_row = a.Lk > 1 ? a.v_row : a.D;
    d.v_head = a.v_head;
    d.Lq = (int)a.Lq;
    d.Lk = (int)a.Lk;
    d.G = (int)(a.heads / a.kv_heads);
    d.Hk = (int)a.kv_heads;
    d.D = (int)a.D;
    d.R = (int)p.R;
    d.pairs = (int)p.pairs;
    d.tiles = (int)p.tiles;
    d.splits = (int)p.splits;
    d.shared = a.shared != 0;
    d.scale = a.scale * 0x1.715476p+0f;
    if (a.mask) {
        uint64_t *words = static_cast<uint64_t *>(a.workspace);
        d.words = words;
        d.word_seq = a.mask_seq ? p.blocks * p.word_rows : 0;
        d.word_block = p.word_rows;
        d.word_row = a.mask_row ? 1 : 0;
        hipLaunchKernelGGL(attn_mask_kernel,
                           dim3((unsigned)((p.word_rows + 3) / 4), (unsigned)((p.blocks + kMaskBlocks - 1) / kMaskBlocks),
                                (unsigned)p.word_seqs),
                           dim3(256), 0, (hipStream_t)stream, a.mask, a.mask_seq, a.mask_row, p.word_rows, (int)a.Lk,
                           (int)p.blocks, words);
    }
    const auto fn = p.waves == 1 ? attn_build<1>(a.D) : attn_build<4>(a.D);
    hipLaunchKernelGGL(fn, dim3((unsigned)(p.pairs * p.tiles * p.splits)), dim3((unsigned)(64 * p.waves)), 0,
                       (hipStream_t)stream, d);
    if (p.splits > 1) {
        const int64_t rows = p.pairs * p.R;
        if (p.splits > 4)
            hipLaunchKernelGGL(attn_join_kernel<8>, dim3((unsigned)rows), dim3(256), 0, (hipStream_t)stream, d);
        else
            hipLaunchKernelGGL(attn_join_kernel<1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, (hipStream_t)stream, d);
    }
    if (a.xq) s3d8::codes_of_rows(a.o, a.B * a.Lq, a.heads * a.D, a.xq, a.xs, cus, stream);
    return s3d8::launch_status();
}

}  // extern "C"
