// Query and key heads between their projections and attention, for gfx950: the RMS
// norm of each head and its rotary position, queries and keys in one launch.
//
// A head x becomes n = (x r) w, r = 1 / sqrt(mean(x^2) + eps), and pairs (a, b) of n become
// (a c - b s, b c + a s).  It is read once into the registers of 8 to 64 lanes, its squares are
// summed there, and it is written once: memory bounds it (8192 tokens of 40 heads of 128, bf16, 168
// MB: 34 us, 4.9 TB/s; a copy reaches 5.1), and with few tokens the launch (one token 3.4 us).
// Lanes take up to eight pairs, 16 bytes of either side at once for bf16 and for fp32 values.  Angles are
// position * frequency in 64 bits, reduced to a part of a turn before anything is rounded
// to fp32, so that far positions keep their phase; a workgroup computes cosine and sine
// once per token and pair and takes them, like the weights, from LDS for all of the token's
// heads (2048 tokens of 40 heads: 11.8 us; with the weights in registers 18.6).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

constexpr int kMaxHead = 256;
constexpr int64_t kMaxTokens = 1 << 19;
constexpr int64_t kMaxHeads = 1 << 26;     // of all tokens
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kThreads = 256;
constexpr int64_t kCosines = 32 << 10;  // bytes of LDS

// Cosine and sine of `angle` radians, each times `factor`, as fp32.  The angle goes to
// turns and their fraction in 64 bits, from there to the nearest quarter turn and a
// rest of at most an eighth, on which the Taylor series to the ninth and tenth
// degree are off by less than 2^-29 (sine) and 2^-32 (cosine).
__device__ __forceinline__ float2 turned(double angle, float factor) {
    const double t = angle * 0x1.45f306dc9c883p-3;  // 1 / (2 pi)
    const double r = 4.0 * (t - __builtin_rint(t));
    const double quarter = __builtin_rint(r);
    const float x = (float)((r - quarter) * 0x1.921fb54442d18p+0);  // pi / 2
    const float z = x * x;
    float s = __builtin_fmaf(z, 1.0f / 362880, -1.0f / 5040);
    s = __builtin_fmaf(z, s, 1.0f / 120);
    s = __builtin_fmaf(z, s, -1.0f / 6);
    s = __builtin_fmaf(z * x, s, x);
    float c = __builtin_fmaf(z, -1.0f / 3628800, 1.0f / 40320);
    c = __builtin_fmaf(z, c, -1.0f / 720);
    c = __builtin_fmaf(z, c, 1.0f / 24);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    const int q = (int)quarter & 3;
    const float cq = q & 1 ? s : c, sq = q & 1 ? c : s;
    return make_float2(factor * (q == 1 || q == 2 ? -cq : cq), factor * (q >= 2 ? -sq : sq));
}

// V values from element `at` of fp32 or bf16 rows, and to them: aligned to V elements or 16 bytes.
template <class T, int N>
using Vec = T __attribute__((ext_vector_type(N)));

template <int V, bool kBF>
__device__ __forceinline__ void load(float (&x)[V], const void *p, int64_t at) {
    if constexpr (kBF && V > 1) {
        const auto u = *global(reinterpret_cast<const Vec<uint32_t, V / 2> *>(static_cast<const uint16_t *>(p) + at));
#pragma unroll
        for (int v = 0; v < V / 2; ++v) {
            const uint32_t w = u[v];
            x[2 * v] = __uint_as_float(w << 16);
            x[2 * v + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    } else if constexpr (kBF) {
        x[0] = bf16_to_f32(global(static_cast<const uint16_t *>(p))[at]);
    } else if constexpr (V > 1) {
        const auto u = *global(reinterpret_cast<const Vec<float, V> *>(static_cast<const float *>(p) + at));
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = u[v];
    } else {
        x[0] = global(static_cast<const float *>(p))[at];
    }
}
template <int V>
__device__ __forceinline__ void store(void *p, int64_t at, const float (&x)[V], bool bf) {
    if (bf) {
        if constexpr (V > 1) {
            Vec<__bf16, V> u;
#pragma unroll
            for (int v = 0; v < V; ++v) u[v] = (__bf16)x[v];
            *global(reinterpret_cast<Vec<__bf16, V> *>(static_cast<__bf16 *>(p) + at)) = u;
        } else {
            global(static_cast<__bf16 *>(p))[at] = (__bf16)x[0];
        }
    } else if constexpr (V > 1) {
        constexpr int kN = V < 4 ? V : 4;
#pragma unroll
        for (int n = 0; n < V; n += kN) {
            Vec<float, kN> u;
#pragma unroll
            for (int v = 0; v < kN; ++v) u[v] = x[n + v];
            *global(reinterpret_cast<Vec<float, kN> *>(static_cast<float *>(p) + at + n)) = u;
        }
    } else {
        global(static_cast<float *>(p))[at] = x[0];
    }
}

// Sum over groups of G lanes (a power of two), in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xF,
                                                                     0xF, false));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>());
    v += dpp(v, std::integral_constant<int, 0x4E>());
    v += dpp(v, std::integral_constant<int, 0x141>());
    if constexpr (G >= 16) v += dpp(v, std::integral_constant<int, 0x140>());
    if constexpr (G >= 32) v += __shfl_xor(v, 16);
    if constexpr (G >= 64) v += __shfl_xor(v, 32);
    return v;
}

// One group of G lanes per head: lane i holds the V pairs of chunks i, i + G, ...,
// NC of them, a chunk being V elements at `first` and V at `second`.  In the turned
// part these are the two sides of V pairs (half layout: rot / 2 apart;
// interleaved: 2 V elements in a row, whose pairs are side by side); past it 2 V
// elements in a row that stay as they are.
// A workgroup takes `heads` heads in a row, queries and keys of a token one after the other, of as
// many tokens as that may be.
template <int V, int G, int NC, bool kBF>
__global__ __launch_bounds__(kThreads) void head_rope_kernel(const s3d8_head_rope_args a, int heads) {
    extern __shared__ float2 turn[];
    __shared__ __attribute__((aligned(16))) float weights[2 * kMaxHead];
    constexpr int kGroups = kThreads / G;
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const int D = (int)a.D, half = (int)a.rotary_dim / 2, all = (int)(a.q_heads + a.k_heads);
    const int64_t head0 = (int64_t)blockIdx.x * heads, token0 = head0 / all;
    const int skip = (int)(head0 - token0 * all);  // heads of its first token that are another's
    const int items = (int)min((int64_t)heads, a.M * all - head0);
    const bool side_by_side = a.interleaved != 0;

    int first[NC], second[NC];
    bool in[NC], turns[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int p = (lane + c * G) * V;  // the chunk's first pair
        in[c] = 2 * p < D;
        turns[c] = p < half;
        first[c] = turns[c] && !side_by_side ? p : 2 * p;
        second[c] = first[c] + (turns[c] && !side_by_side ? half : V);
    }
    struct Head {
        float x[NC][2][V];
    };
    // a head's place: token0 + t, and its number among the token's
    struct Place {
        int t, head;
    };
    const int more = kGroups / all, rest = kGroups - more * all;
    auto after = [&](Place p) {
        p.t += more;
        p.head += rest;
        if (p.head >= all) {
            p.head -= all;
            ++p.t;
        }
        return p;
    };
    auto load_head = [&](Place p, Head &h) {
        const int64_t token = token0 + p.t;
        const bool q = p.head < a.q_heads;
        const int64_t at = q ? token * a.q_row + p.head * a.q_head : token * a.k_row + (p.head - a.q_heads) * a.k_head;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (in[c]) {
                load<V, kBF>(h.x[c][0], q ? a.q : a.k, at + first[c]);
                load<V, kBF>(h.x[c][1], q ? a.q : a.k, at + second[c]);
            }
    };
    Head next;
    Place place{(skip + group) / all, (skip + group) % all};
    if (group < items) load_head(place, next);
    // weights and cosines in LDS, once for the workgroup's heads
    if (a.q_weight)
        for (int i = threadIdx.x; i < D; i += kThreads) weights[i] = global(a.q_weight)[i];
    if (a.k_weight)
        for (int i = threadIdx.x; i < D; i += kThreads) weights[kMaxHead + i] = global(a.k_weight)[i];
    const int tokens = (skip + items - 1) / all + 1;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int64_t token = token0 + i / half;
        const double pos = a.positions_64 ? (double)global(static_cast<const int64_t *>(a.positions))[token]
                                          : (double)global(static_cast<const int32_t *>(a.positions))[token];
        turn[i] = turned(pos * global(a.frequencies)[i % half], a.factor);
    }
    lds_barrier();
    const float inv_d = 1.0f / (float)D;
    for (int item = group; item < items; item += kGroups) {
        Head h = next;
        const int t = place.t, head = place.head;
        place = after(place);
        if (item + kGroups < items) load_head(place, next);
        const bool q = head < a.q_heads;
        if (q ? a.q_weight : a.k_weight) {
            const float *w = weights + (q ? 0 : kMaxHead);
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c])
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int v = 0; v < V; ++v) sum = __builtin_fmaf(h.x[c][s][v], h.x[c][s][v], sum);
            const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<G>(sum), inv_d, a.eps));
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (in[c])
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        using W = Vec<float, V < 4 ? V : 4>;
                        const W *ws = reinterpret_cast<const W *>(w + (s ? second[c] : first[c]));
#pragma unroll
                        for (int v = 0; v < V; ++v) h.x[c][s][v] = h.x[c][s][v] * r * ws[v / 4][v % 4];
                    }
        }
        void *p = q ? a.q_out : a.k_out;
        const int64_t token = token0 + t;
        const int64_t at = q ? token * a.q_out_row + head * a.q_out_head
                             : token * a.k_out_row + (head - a.q_heads) * a.k_out_head;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (!in[c]) continue;
            if (turns[c]) {
                const float2 *cs = turn + t * half + (lane + c * G) * V;
                auto rotate = [](float &x, float &y, float2 f) {
                    const float u = __builtin_fmaf(x, f.x, -(y * f.y));
                    y = __builtin_fmaf(y, f.x, x * f.y);
                    x = u;
                };
                if (V > 1 && side_by_side) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {  // pair v: elements 2 v and 2 v + 1 of the 2 V in a row
                        float *e = &h.x[c][0][0] + 2 * v;
                        rotate(e[0], e[1], cs[v]);
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) rotate(h.x[c][0][v], h.x[c][1][v], cs[v]);
                }
            }
            store<V>(p, at + first[c], h.x[c][0], a.out_type == S3D8_ROWS_BF16);
            store<V>(p, at + second[c], h.x[c][1], a.out_type == S3D8_ROWS_BF16);
        }
    }
}

using HeadRopeFn = void (*)(s3d8_head_rope_args, int);

// The build for V pairs a lane, and the lanes of a head.
template <bool kBF>
HeadRopeFn head_rope_build(int pairs, int64_t D, int &lanes) {
    if (pairs == 1) {
        lanes = 64;
        return D <= 128 ? head_rope_kernel<1, 64, 1, kBF> : head_rope_kernel<1, 64, 2, kBF>;
    }
    if (pairs == 2) {
        lanes = D <= 128 ? 32 : 64;
        return D <= 128 ? head_rope_kernel<2, 32, 1, kBF> : head_rope_kernel<2, 64, 1, kBF>;
    }
    if (kBF && pairs == 8) {
        lanes = D <= 128 ? 8 : 16;
        return D <= 128 ? head_rope_kernel<8, 8, 1, true> : head_rope_kernel<8, 16, 1, true>;
    }
    lanes = D <= 64 ? 8 : D <= 128 ? 16 : 32;
    return D <= 64    ? head_rope_kernel<4, 8, 1, kBF>
           : D <= 128 ? head_rope_kernel<4, 16, 1, kBF>
                      : head_rope_kernel<4, 32, 1, kBF>;
}

bool row_type(int32_t t) { return t == S3D8_ROWS_F32 || t == S3D8_ROWS_BF16; }

// Row and head strides of M x heads heads of D, and the pointer's alignment to an element.
int check_heads(const void *p, int64_t M, int64_t heads, int64_t D, int64_t row, int64_t head, int32_t type) {
    if (reinterpret_cast<uintptr_t>(p) & (type == S3D8_ROWS_F32 ? 3 : 1))
        return s3d8::fail(S3D8_ERR_ALIGN, "heads must be aligned to an element");
    if ((heads > 1 && head < D) || (M > 1 && row < D) || head < 0 || row < 0 || head > kMaxStride || row > kMaxStride)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "row and head strides must be at least the head's size (and at most 2^40)");
    return S3D8_OK;
}

// Whether heads can be read (or written) V elements at a time.
bool by(int V, const void *p, int64_t row, int64_t head, int32_t type) {
    const uintptr_t bytes = std::min(V * (type == S3D8_ROWS_F32 ? 4 : 2), 16);
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 && row % V == 0 && head % V == 0;
}

}  // namespace

extern "C" {

int32_t s3d8_rope_frequencies(int64_t rotary_dim, double base, int32_t scaling, double factor, double original_length,
                              double low, double high, double *frequencies, double *attention_factor) {
    if (!frequencies || !attention_factor) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    if (rotary_dim <= 0 || rotary_dim % 2 || rotary_dim > kMaxHead)
        return s3d8::fail(S3D8_ERR_SHAPE, "rotary_dim must be even, from 2 to 256");
    if (!(base > 1.0 && base <= 1e30)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "base must be over 1 (and at most 1e30)");
    if (scaling < S3D8_ROPE_PLAIN || scaling > S3D8_ROPE_YARN)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown kind of scaling");
    if (scaling != S3D8_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e9))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "factor must be at least 1 (and at most 1e9)");
    const bool by_length = scaling == S3D8_ROPE_LLAMA3 || scaling == S3D8_ROPE_YARN;
    if (by_length && !(original_length >= 1.0 && original_length <= 1e12 && low > 0.0 && low < high && high <= 1e9))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "original_length must be positive, and low and high turns 0 < low < high");
    const double pi = 3.14159265358979323846;
    double first = 0.0, last = 0.0;
    if (scaling == S3D8_ROPE_YARN) {  // the pairs that make `high` and `low` turns over the original length
        auto pair = [&](double turns) {
            return (double)rotary_dim * std::log(original_length / (turns * 2.0 * pi)) / (2.0 * std::log(base));
        };
        first = std::fmax(std::floor(pair(high)), 0.0);
        last = std::fmin(std::ceil(pair(low)), (double)(rotary_dim - 1));
    }
    for (int64_t j = 0; j < rotary_dim / 2; ++j) {
        const double f = std::pow(base, -2.0 * (double)j / (double)rotary_dim);
        double stretch = 0.0;  // share of the frequency divided by factor
        if (scaling == S3D8_ROPE_LINEAR) stretch = 1.0;
        if (scaling == S3D8_ROPE_LLAMA3)
            stretch = 1.0 - std::fmin(std::fmax((original_length * f / (2.0 * pi) - low) / (high - low), 0.0), 1.0);
        if (scaling == S3D8_ROPE_YARN)
            stretch = std::fmin(std::fmax(((double)j - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
        frequencies[j] = f * (1.0 - stretch) + (stretch > 0.0 ? f / factor * stretch : 0.0);
    }
    *attention_factor = scaling == S3D8_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    s3d8::clear_error();
    return S3D8_OK;
}

int32_t s3d8_head_rope(const s3d8_head_rope_args *args, void *stream) {
    if (!args || !args->q || !args->q_out) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    s3d8_head_rope_args a = *args;
    if ((a.k != nullptr) != (a.k_out != nullptr) || (a.k != nullptr) != (a.k_heads != 0))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "k, k_out and k_heads go together");
    if (!a.k && a.k_weight) return s3d8::fail(S3D8_ERR_INVALID_ARG, "k_weight needs k");
    if (a.M <= 0 || a.q_heads <= 0 || a.k_heads < 0 || a.D <= 0 || a.rotary_dim < 0)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (a.D % 2 || a.D > kMaxHead) return s3d8::fail(S3D8_ERR_SHAPE, "heads must be of an even size up to 256");
    if (a.rotary_dim % 2 || a.rotary_dim > a.D)
        return s3d8::fail(S3D8_ERR_SHAPE, "rotary_dim must be even and at most the head's size");
    if (a.M > kMaxTokens || a.q_heads > 4096 || a.k_heads > 4096)
        return s3d8::fail(S3D8_ERR_SHAPE, "more than 524288 tokens or 4096 heads are not supported");
    // (a workgroup takes 8 heads or more where there are many: 2^31 threads at most)
    if (a.M * (a.q_heads + a.k_heads) > kMaxHeads) return s3d8::fail(S3D8_ERR_SHAPE, "more than 2^26 heads are not supported");
    if (a.rotary_dim && (!a.positions || !a.frequencies))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "rotary_dim needs positions and frequencies");
    if (!a.rotary_dim && !a.q_weight && !a.k_weight)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "neither a norm nor a rotary position");
    if (!row_type(a.in_type) || !row_type(a.out_type)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    if (!(a.eps >= 0x1p-126f && a.eps <= 0x1p126f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "eps must be positive (2^-126 to 2^126)");
    if (!(std::fabs(a.factor) <= 0x1p100f)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "factor must be finite (at most 2^100)");
    int rc = check_heads(a.q, a.M, a.q_heads, a.D, a.q_row, a.q_head, a.in_type);
    if (!rc) rc = check_heads(a.q_out, a.M, a.q_heads, a.D, a.q_out_row, a.q_out_head, a.out_type);
    if (!rc && a.k) rc = check_heads(a.k, a.M, a.k_heads, a.D, a.k_row, a.k_head, a.in_type);
    if (!rc && a.k) rc = check_heads(a.k_out, a.M, a.k_heads, a.D, a.k_out_row, a.k_out_head, a.out_type);
    if (rc) return rc;
    if ((reinterpret_cast<uintptr_t>(a.q_weight) | reinterpret_cast<uintptr_t>(a.k_weight)) & 3 ||
        reinterpret_cast<uintptr_t>(a.frequencies) & 7 || reinterpret_cast<uintptr_t>(a.positions) & (a.positions_64 ? 7 : 3))
        return s3d8::fail(S3D8_ERR_ALIGN, "weights, frequencies and positions must be aligned to an element");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    // The most pairs a lane that fall together: loads of 16 bytes where they can be.
    int pairs = a.in_type == S3D8_ROWS_BF16 ? 8 : 4;
    while (pairs > 1 && !(a.D % (2 * pairs) == 0 && a.rotary_dim % (2 * pairs) == 0 && by(pairs, a.q, a.q_row, a.q_head, a.in_type) &&
                          by(pairs, a.q_out, a.q_out_row, a.q_out_head, a.out_type) &&
                          (!a.k || (by(pairs, a.k, a.k_row, a.k_head, a.in_type) &&
                                    by(pairs, a.k_out, a.k_out_row, a.k_out_head, a.out_type)))))
        pairs /= 2;
    int lanes = 0;
    const HeadRopeFn fn =
        a.in_type == S3D8_ROWS_BF16 ? head_rope_build<true>(pairs, a.D, lanes) : head_rope_build<false>(pairs, a.D, lanes);
    // Heads that a group of lanes takes in turn, by how often one for each would fill the device: with
    // more, the next head is on its way while one is turned, and a token's cosines serve more
    // heads, but fewer workgroups share the work.  With 1, 2 and 4, in us: 512 tokens of 40 heads of 128
    // (2.5 times) 5.2, 6.2, 8.0; 1601 of 32 heads of 80 (6.3) 8.1, 7.2, 8.7; 2048 of 40 (10) 12.8, 11.8, 12.4;
    // 8192 of 40 (40) 43.2, 37.6, 34.2.
    const int64_t groups = kThreads / lanes, all = a.q_heads + a.k_heads, total = a.M * all, full = total / (groups * cus);
    int64_t heads, cosines;
    for (int64_t each = full >= 20 ? 4 : full >= 6 ? 2 : 1;; each /= 2) {
        heads = groups * each;
        cosines = ((heads + all - 2) / all + 1) * (a.rotary_dim / 2) * (int64_t)sizeof(float2);  // of the tokens they are of
        if (each == 1 || cosines <= kCosines) break;
    }
    hipLaunchKernelGGL(fn, dim3((unsigned)((total + heads - 1) / heads)), dim3(kThreads),
                       (size_t)cosines, (hipStream_t)stream, a, (int)heads);
    return s3d8::launch_status();
}

}  // extern "C"
