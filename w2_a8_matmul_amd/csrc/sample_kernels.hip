// The choice of the next token from a row of logits, for gfx950.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

constexpr int64_t kMaxVocabulary = 1 << 18;  // 2^18 weights of 2^44 stay below 2^63
constexpr int64_t kMaxRows = 1 << 19;
constexpr int kT = 1024;
constexpr int kDigit = 11, kBins = 1 << kDigit;
constexpr int kIndexBits = 18;
constexpr int kOrderBits = 32 + kIndexBits;
constexpr int kListed = 4096;
constexpr uint32_t kNothing = 0x007FFFFFu;  // order_key(-infinity)

// fp32 values as whole numbers that order like them (-0 as 0, NaN as -infinity).
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return l != l ? kNothing : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// Place of a token in the order of falling logits, then rising index.
__device__ __forceinline__ uint64_t place(uint32_t key, uint32_t index) {
    return (uint64_t)(~key) << kIndexBits | index;
}
__device__ __forceinline__ uint32_t place_key(uint64_t p) { return ~(uint32_t)(p >> kIndexBits); }
__device__ __forceinline__ uint32_t place_index(uint64_t p) { return (uint32_t)p & ((1u << kIndexBits) - 1); }

// W = rne(2^44 exp((l - m) / t)).  The quotient is l - m times 1 / t with its
// remainder's share, so that it is rounded once; below -60 the weight is 0.
struct Weights {
    uint32_t top;
    double m, t, rt;
    __device__ __forceinline__ uint64_t operator()(uint32_t key) const {
        if (key == top) return 1ull << 44;
        if (key <= kNothing) return 0;
        const double d = (double)key_value(key) - m;
        double x = d * rt;
        x = __builtin_fma(__builtin_fma(-x, t, d), rt, x);
        if (!(x > -60.0)) return 0;
        const Exp e = exp_parts(x);
        const double s = e.two_n * 0x1p44;
        // 2^52 added rounds to a whole number, which the sum's low bits then are
        return (uint64_t)__double_as_longlong(__builtin_fma(s, e.less_one, s) + 0x1p52) & ((1ull << 52) - 1);
    }
};

// Element i of a row, all of them, each by one thread of the workgroup.
template <bool kBF, class F>
__device__ __forceinline__ void each(const void *row, int V, F f) {
    constexpr int kV = kBF ? 8 : 4;  // elements in 16 bytes
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    const int head = min(V, (int)((16 - (at & 15)) & 15) / (kBF ? 2 : 4));
    const int vectors = (V - head) / kV, tail = head + vectors * kV;
    auto one = [&](int i) {
        if constexpr (kBF)
            f(i, bf16_to_f32(static_cast<const uint16_t *>(row)[i]));
        else
            f(i, static_cast<const float *>(row)[i]);
    };
    if ((int)threadIdx.x < head) one(threadIdx.x);
    if ((int)threadIdx.x < V - tail) one(tail + threadIdx.x);
    const uint4 *p = reinterpret_cast<const uint4 *>(at + head * (kBF ? 2 : 4));
    auto four = [&](uint4 u, int v) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        const int i = head + v * kV;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kBF) {
                f(i + 2 * j, __uint_as_float(w[j] << 16));
                f(i + 2 * j + 1, __uint_as_float(w[j] & 0xFFFF0000u));
            } else {
                f(i + j, __uint_as_float(w[j]));
            }
        }
    };
    constexpr int kAhead = 4;  // loads in flight
    int v = threadIdx.x;
    for (; v + (kAhead - 1) * kT < vectors; v += kAhead * kT) {
        uint4 u[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) u[a] = p[v + a * kT];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) four(u[a], v + a * kT);
    }
    for (; v < vectors; v += kT) four(p[v], v);
}

struct Shared {
    uint64_t bins[kBins];
    uint64_t list[kListed];  // places
    uint64_t sums[kT / 64];
    uint64_t found[3];  // bin, sum before it, sum in it
    int listed;
};

// Sum of the workgroup's values before this thread's and in all.
__device__ __forceinline__ uint64_t scan(uint64_t v, uint64_t *sums, uint64_t &total) {
    uint64_t s = v;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t u = __shfl_up((unsigned long long)s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 63) sums[threadIdx.x >> 6] = s;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) {
        const uint64_t u = sums[w];
        if (w < (int)(threadIdx.x >> 6)) before += u;
        total += u;
    }
    return before + s - v;
}

// Where the running sum of `value` over the tokens, in the order of `order` (whole
// numbers of `bits` bits, no two the same), reaches limit(total): all ones where it
// does not.  Digit by digit: sums of the values by the next bits of the order, then the bin in
// which the running sum reaches the limit.  go(f) calls f(place) once for every token.
// kLast: any number between that token's and the next one's will do.
template <bool kLast, class Go, class Order, class Value, class Limit>
__device__ uint64_t reach(Shared &sh, int bits, Go go, Order order, Value value, Limit limit, uint64_t &total) {
    uint64_t prefix = 0, left = 0;
    bool first = true;
    while (bits > 0) {
        const int digit = min(kDigit, bits), shift = bits - digit;
        for (int i = threadIdx.x; i < kBins; i += kT) sh.bins[i] = 0;
        __syncthreads();
        go([&](uint64_t p) {
            const uint64_t o = order(p);
            if (!first && o >> bits != prefix) return;
            const uint64_t w = value(p);
            if (w) atomicAdd((unsigned long long *)&sh.bins[(o >> shift) & ((1u << digit) - 1)], (unsigned long long)w);
        });
        __syncthreads();
        const uint64_t a = sh.bins[2 * threadIdx.x], b = sh.bins[2 * threadIdx.x + 1];
        uint64_t sum;
        const uint64_t before = scan(a + b, sh.sums, sum);
        if (first) {
            total = sum;
            left = limit(total);
            if (left > total) return ~0ull;
        }
        if (before < left && left <= before + a + b) {
            const bool second = left > before + a;
            sh.found[0] = 2 * threadIdx.x + second;
            sh.found[1] = before + (second ? a : 0);
            sh.found[2] = second ? b : a;
        }
        __syncthreads();
        prefix = prefix << digit | sh.found[0];
        left -= sh.found[1];
        bits = shift;
        const bool whole = left == sh.found[2];  // the bin's last token
        __syncthreads();
        if (kLast && whole) return ((prefix + 1) << shift) - 1;
        first = false;
    }
    return prefix;
}

template <bool kBF>
__global__ __launch_bounds__(kT) void sample_kernel(const s3d8_sample_args a) {
    __shared__ Shared sh;
    const int64_t r = blockIdx.x;
    const int V = (int)a.V;
    const void *row = static_cast<const char *>(a.logits) + r * a.row * (kBF ? 2 : 4);
    auto go_row = [&](auto f) { each<kBF>(row, V, [&](int i, float l) { f(place(order_key(l), i)); }); };

    uint64_t first = ~0ull;
    go_row([&](uint64_t p) { first = min(first, p); });
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) first = min(first, (uint64_t)__shfl_xor((unsigned long long)first, o));
    if ((threadIdx.x & 63) == 0) sh.sums[threadIdx.x >> 6] = first;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kT / 64; ++w) first = min(first, sh.sums[w]);
    __syncthreads();

    const uint32_t top = place_key(first);
    const float t = a.temperature ? a.temperature[r] : a.temperature_all;
    if (top <= kNothing || !(t > 0.0f)) {  // (NaN too)
        if (threadIdx.x == 0) {
            a.token[r] = top <= kNothing ? -1 : (int32_t)place_index(first);
            if (a.prob) a.prob[r] = top <= kNothing ? 0.0f : 1.0f;
        }
        return;
    }
    const double T = fminf(t, 0x1p100f);
    const int k = a.top_k ? a.top_k[r] : a.top_k_all;
    const float top_p = fmaxf(a.top_p ? a.top_p[r] : a.top_p_all, 0.0f);
    const float min_p = fminf(fmaxf(a.min_p ? a.min_p[r] : a.min_p_all, 0.0f), 1.0f);
    const Weights weight{top, (double)key_value(top), T, 1.0 / T};

    // The last place that is kept: by number, then by sum.
    uint64_t last = ~0ull, total;
    bool listed = false;
    auto go_list = [&](auto f) {
        for (int i = threadIdx.x; i < sh.listed; i += kT) f(sh.list[i]);
    };
    auto by_place = [](uint64_t p) { return p; };
    if (k > 0 && k < V) {
        last = reach<true>(
            sh, kOrderBits, go_row, by_place, [](uint64_t) { return 1ull; }, [&](uint64_t) { return (uint64_t)k; }, total);
        if (k <= kListed) {
            if (threadIdx.x == 0) sh.listed = 0;
            __syncthreads();
            go_row([&](uint64_t p) {
                if (p <= last) sh.list[atomicAdd(&sh.listed, 1)] = p;
            });
            __syncthreads();
            listed = true;
        }
    }
    auto draw = [&](auto go) {
        auto ranked = [&](uint64_t p) { return p <= last ? weight(place_key(p)) : 0ull; };
        if (top_p < 1.0f) {
            const uint64_t end = reach<true>(
                sh, kOrderBits, go, by_place, ranked,
                [&](uint64_t s) { return max(1ull, (unsigned long long)ceil((double)top_p * (double)s)); }, total);
            last = min(last, end);
        }
        const uint64_t least = (uint64_t)ceil((double)min_p * 0x1p44);
        const float u = fmaxf(a.u[r], 0.0f);
        return reach<false>(
            sh, kIndexBits, go, [](uint64_t p) { return (uint64_t)place_index(p); },
            [&](uint64_t p) {
                const uint64_t w = ranked(p);
                return w >= least ? w : 0ull;
            },
            [&](uint64_t s) { return 1 + min((uint64_t)((double)u * (double)s), s - 1); }, total);
    };
    const uint64_t at = listed ? draw(go_list) : draw(go_row);
    if (threadIdx.x == 0) a.token[r] = (int32_t)at;
    if (a.prob && threadIdx.x == 0) {
        const float l = kBF ? bf16_to_f32(static_cast<const uint16_t *>(row)[at]) : static_cast<const float *>(row)[at];
        a.prob[r] = (float)((double)weight(order_key(l)) / (double)total);
    }
}

}  // namespace

extern "C" int32_t s3d8_sample(const s3d8_sample_args *args, void *stream) {
    if (!args || !args->logits || !args->u || !args->token) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_sample_args &a = *args;
    if (a.M <= 0 || a.V <= 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (a.V > kMaxVocabulary) return s3d8::fail(S3D8_ERR_SHAPE, "more than 262144 tokens are not supported");
    if (a.M > kMaxRows) return s3d8::fail(S3D8_ERR_SHAPE, "more than 524288 rows are not supported");
    if (a.type != S3D8_ROWS_F32 && a.type != S3D8_ROWS_BF16) return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    if ((a.M > 1 && a.row < a.V) || a.row < 0 || a.row > int64_t(1) << 40)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "rows must be at least V elements apart (and at most 2^40)");
    if (!a.temperature && !(a.temperature_all >= 0.0f && a.temperature_all <= 0x1p100f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "temperature must be from 0 to 2^100");
    if (!a.top_k && a.top_k_all < 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "top_k must not be negative");
    if (!a.top_p && !(a.top_p_all >= 0.0f && a.top_p_all <= 1.0f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "top_p must be from 0 to 1");
    if (!a.min_p && !(a.min_p_all >= 0.0f && a.min_p_all <= 1.0f))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "min_p must be from 0 to 1");
    auto odd = [](const void *p, uintptr_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; };
    if (odd(a.logits, a.type == S3D8_ROWS_F32 ? 4 : 2) || odd(a.u, 4) || odd(a.temperature, 4) || odd(a.top_k, 4) ||
        odd(a.top_p, 4) || odd(a.min_p, 4) || odd(a.token, 4) || odd(a.prob, 4))
        return s3d8::fail(S3D8_ERR_ALIGN, "arrays must be aligned to an element");
    const int rc = s3d8::check_device(nullptr);
    if (rc) return rc;
    const auto fn = a.type == S3D8_ROWS_BF16 ? sample_kernel<true> : sample_kernel<false>;
    hipLaunchKernelGGL(fn, dim3((unsigned)a.M), dim3(kT), 0, (hipStream_t)stream, a);
    return s3d8::launch_status();
}
