// What stands between the linear layers of a block, for gfx950: the norms
// before and after it with its gate and the residual sum, and the gated
// activation, each ending in the INT8 codes that the linear kernels read.
//
// A row is read once, stays in the registers of one workgroup through its
// reductions, and is written once.  So the bytes moved are the floor, but the
// arithmetic is close to it: statistics and values are held in 64 bits so that
// the codes are the correctly rounded ones, and vector instructions issue most
// of the time a launch takes (70% and 84% at the large sizes below).  Rows of more
// than 28672 values, 16 float4 to each of 1024 threads, do not fit: 324 to 840 bytes
// a lane spill to scratch memory, and 64 rows of 53248 in bf16 take 25 us in the
// norm and 100 us in the gated activation.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "s3d8.h"
#include "s3d8_device.h"
#include "s3d8_internal.h"

namespace {

constexpr int64_t kMaxWidth = 65536;    // 16 float4 per thread of 1024
constexpr int64_t kMaxRows = 1 << 19;   // keeps a launch under 2^32 threads

__device__ __forceinline__ float4 bf16x4_values(uint2 u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// A workgroup's share of a row of K fp32 or bf16 values from element `base`, as it
// lies in memory: thread t of T takes four values at 4 (t + T j), j < NV (zeros
// past the row).
template <bool kBF>
using Raw = std::conditional_t<kBF, uint2, float4>;
__device__ __forceinline__ float4 values(float4 r) { return r; }
__device__ __forceinline__ float4 values(uint2 r) { return bf16x4_values(r); }

template <int T, int NV, bool kBF>
__device__ __forceinline__ void load_row(Raw<kBF> (&r)[NV], const void *p, int64_t base, int n4) {
    using E = std::conditional_t<kBF, uint16_t, float>;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        r[j] = i < n4 ? reinterpret_cast<const Raw<kBF> *>(static_cast<const E *>(p) + base)[i] : Raw<kBF>{};
    }
}

// Workgroup barrier for LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Four values rounded to bf16, to nearest even.
__device__ __forceinline__ uint2 bf16x4(float4 v) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 lo = {(__bf16)v.x, (__bf16)v.y}, hi = {(__bf16)v.z, (__bf16)v.w};  // v_cvt_pk_bf16_f32
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

__device__ __forceinline__ void store4(void *p, int64_t at, float4 v, bool bf) {
    if (bf)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) = bf16x4(v);
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = v;
}

template <class F>
__device__ __forceinline__ float4 map4(float4 a, F f) {
    return make_float4(f(a.x), f(a.y), f(a.z), f(a.w));
}
template <class F>
__device__ __forceinline__ float4 zip4(float4 a, float4 b, F f) {
    return make_float4(f(a.x, b.x), f(a.y, b.y), f(a.z, b.z), f(a.w, b.w));
}

// v plus lane-permuted v, both halves of the double through DPP.
template <int kCtrl>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, 0xF, 0xF, false);
    return v + __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Sum over the wave, wave-uniform (the moves of row16_max: within pairs, within
// quads, halves of 8 mirrored, the row of 16 mirrored, then the four rows).
__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Sum and maximum over the workgroup's T threads, the same in every thread.
// `slot` is LDS not used by the previous reduction (one barrier per reduction,
// none for a workgroup of one wave).
template <int T>
__device__ __forceinline__ double block_sum(double v, double *slot) {
    v = wave_sum(v);
    if constexpr (T == 64) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    lds_barrier();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += slot[w];
    return v;
}

template <int T>
__device__ __forceinline__ float block_max(float v, float *slot) {
    v = wave_max(v);
    if constexpr (T == 64) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    lds_barrier();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = fmaxf(v, slot[w]);
    return v;
}

// Codes rne(x rs) of four values, |x rs| < 2^22, and in `far` the largest distance of
// an x rs from its code.  Adding 1.5 2^23 rounds to an integer, whose low byte
// is then the low byte of the sum.
__device__ __forceinline__ uint32_t codes4(float4 x, float rs, float &far) {
    constexpr float kRound = 12582912.0f;
    const float m[4] = {__builtin_fmaf(x.x, rs, kRound), __builtin_fmaf(x.y, rs, kRound), __builtin_fmaf(x.z, rs, kRound),
                        __builtin_fmaf(x.w, rs, kRound)};
    const float d[4] = {__builtin_fmaf(x.x, rs, kRound - m[0]), __builtin_fmaf(x.y, rs, kRound - m[1]),
                        __builtin_fmaf(x.z, rs, kRound - m[2]), __builtin_fmaf(x.w, rs, kRound - m[3])};
    far = fmaxf(fmaxf(far, fmaxf(fabsf(d[0]), fabsf(d[1]))), fmaxf(fabsf(d[2]), fabsf(d[3])));
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m[1]), __float_as_uint(m[0]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(m[3]), __float_as_uint(m[2]), 0x04000C0Cu);
    return lo | hi;
}

// The row (NV float4 per thread, zeros past n4) out: fp32, bf16, or its codes
// and scale as s3d8_quant_act makes them.
template <int T, int NV>
__device__ __forceinline__ void row_out(const float4 (&v)[NV], int64_t row, int K, int out_type, void *rows, int8_t *xq,
                                        float *xs, float *slot) {
    const int n4 = K >> 2;
    if (out_type != S3D8_ROWS_CODES) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = threadIdx.x + j * T;
            if (i < n4) store4(rows, row * K + 4 * i, v[j], out_type == S3D8_ROWS_BF16);
        }
        return;
    }
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        a = fmaxf(a, fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w))));
    a = block_max<T>(a, slot);
    const float s = a / 127.0f;
    if (threadIdx.x == 0) xs[row] = s;
    // The code is rne(fl(x / s)).  t = x rcp(s), the reciprocal good to an ulp, differs
    // from x / s by less than 127 2^-23, fl(x / s) by less than 127 2^-24: where t is further than 2^-15
    // from a border k + 1/2, rne(t) is the code.  Four values of which one is nearer
    // than that (or 1 / s infinite or 0) divide: few, but where u is a bf16 row but for a
    // factor, half the row's maximum is an exact tie, which most rows hold.
    // (A finite s is at most 2^121, so that its reciprocal is no subnormal number; that of
    // a subnormal s may be infinite, and finite operands can have infinite products.)
    const float rs = __builtin_amdgcn_rcpf(s);
    const bool usable = rs > 0.0f && rs < INFINITY;
    auto code = [&](float x) {
        return a == 0.0f ? 0u : (uint32_t)(uint8_t)(int8_t)fminf(127.0f, fmaxf(-127.0f, rintf(x / s)));
    };
    uint32_t q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float far = 0.0f;
        q[j] = codes4(v[j], rs, far);
        if (!(far <= 0.5f - 0x1p-15f && usable))
            q[j] = code(v[j].x) | code(v[j].y) << 8 | code(v[j].z) << 16 | code(v[j].w) << 24;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        if (i < n4) reinterpret_cast<uint32_t *>(xq + row * K)[i] = q[j];
    }
}

// N(v; w, b) of a row.  The statistics are sums of exact products in 64 bits,
// rounded to fp32 once: an fp32 sum would depend on its order, and its last
// bit moves codes across their rounding borders.
template <int T, int NV, bool kLayer>
__device__ __forceinline__ void normalise(float4 (&v)[NV], int K, double inv_k, double eps,
                                          const float *__restrict__ w, const float *__restrict__ b, double *slot) {
    const int n4 = K >> 2;
    // x / K with inv_k = fl(1 / K): the product and its remainder's share
    auto mean = [&](double x) {
        const double m = x * inv_k;
        return __builtin_fma(__builtin_fma(-m, (double)K, x), inv_k, m);
    };
    double mu = 0.0;
    if constexpr (kLayer) {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) s += ((double)v[j].x + (double)v[j].y) + ((double)v[j].z + (double)v[j].w);
        mu = mean(block_sum<T>(s, slot));
        slot += T / 64;
    }
    double qs[2] = {0.0, 0.0};  // two chains
    auto square = [&](float x, double &q) {
        const double y = kLayer ? (double)x - mu : (double)x;
        q = __builtin_fma(y, y, q);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (kLayer && (int)threadIdx.x + j * T >= n4) continue;  // (past the row v is 0, not mu)
        square(v[j].x, qs[0]);
        square(v[j].y, qs[1]);
        square(v[j].z, qs[0]);
        square(v[j].w, qs[1]);
    }
    // 1 / sqrt(d): two Newton steps on the hardware's estimate, to a relative 2^-51
    const double d = mean(block_sum<T>(qs[0] + qs[1], slot)) + eps;
    double y = __builtin_amdgcn_rsq(d);
    y = __builtin_fma(0.5 * y, __builtin_fma(-d * y, y, 1.0), y);
    y = __builtin_fma(0.5 * y, __builtin_fma(-d * y, y, 1.0), y);
    const float r = (float)y;
    const float m = (float)mu;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        if (i >= n4) continue;
        // both vectors asked for before either is used
        const float4 wv = reinterpret_cast<const float4 *>(w)[i];
        float4 bv;
        if (kLayer && b) bv = reinterpret_cast<const float4 *>(b)[i];
        float4 u = v[j];
        if constexpr (kLayer) u = map4(u, [&](float x) { return x - m; });
        u = zip4(map4(u, [&](float x) { return x * r; }), wv, [](float x, float y) { return x * y; });
        if constexpr (kLayer)
            if (b) u = zip4(u, bv, [](float x, float y) { return x + y; });
        v[j] = u;
    }
}

// exp(x) - 1 = 2^n (p(r) - 1) + (2^n - 1) and its parts: x = n ln 2 + r with ln 2 in two
// parts (Cody and Waite's reduction), p a polynomial of degree 11 on |r| <= ln 2 / 2
// (Chebyshev interpolation, relative error 2^-55.7).
struct Exp {
    double less_one, two_n;  // p(r) - 1, 2^n
};
__device__ __forceinline__ Exp exp_parts(double x) {
    const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
    const double r = __builtin_fma(n, -0x1.a39ef35793c76p-33, __builtin_fma(n, -0x1.62e42fee00000p-1, x));
    double e = 0x1.af631d203b4edp-26;
    e = __builtin_fma(e, r, 0x1.28b405992d897p-22);
    e = __builtin_fma(e, r, 0x1.71ddf5748bd71p-19);
    e = __builtin_fma(e, r, 0x1.a01991ac6b2ddp-16);
    e = __builtin_fma(e, r, 0x1.a01a01b1437f6p-13);
    e = __builtin_fma(e, r, 0x1.6c16c187fbea9p-10);
    e = __builtin_fma(e, r, 0x1.111111110f225p-7);
    e = __builtin_fma(e, r, 0x1.555555554f0cep-5);
    e = __builtin_fma(e, r, 0x1.555555555555ap-3);
    e = __builtin_fma(e, r, 0x1.0000000000011p-1);
    e = __builtin_fma(e, r, 1.0);
    return {e * r, __builtin_amdgcn_ldexp(1.0, (int)n)};
}
// 1 / d to a relative 2^-52: two Newton steps on the hardware reciprocal.
__device__ __forceinline__ double reciprocal(double d) {
    double q = __builtin_amdgcn_rcp(d);
    q = __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
    return __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
}

// tanh(g) = (e^2g - 1) / (e^2g + 1) in 64 bits, rounded to fp32.  (The clamp takes a NaN to
// a bound.)
__device__ __forceinline__ float tanh_rounded(float g) {
    const Exp e = exp_parts(2.0 * (double)__builtin_amdgcn_fmed3f(g, -20.0f, 20.0f));
    const double m = __builtin_fma(e.two_n, e.less_one, e.two_n - 1.0);
    return g != g ? g : __builtin_copysignf((float)(m * reciprocal(m + 2.0)), g);
}

// One workgroup per row: h += gate * norm(branch), then the norm of h and its
// codes, with the row in registers from the loads to the last store.
//
// Measured, RMS with a branch and its post norm, codes out: 2048 x 4096 in bf16
// 15.1 us (58.7 MB at 3.9 TB/s), 17.2 with operands in no cache; RMS of one row
// 2.9 us; layer norm, 1601 x 1280 in fp32 with a gate to bf16, 8.3 us.  34 vector
// instructions per element of the first issue 70% of its time, most of them
// 64-bit (34 us with sums by shuffles through LDS and the same workgroup for every
// width).  The last one is a wave per row, fewer than two a SIMD, whose loads, mean,
// squares, weights and stores follow one another.  The weights loaded before the sums rather than after them gain at some
// sizes what they lose at others (8192 x 4096: 52.8 us for 56.3, 1601 x 5120: 25.7
// for 24.9).  More than one row a workgroup (the weights kept in registers, the
// next row's loads ahead) takes 172 registers and 31 us.
template <int T, int NV, bool kLayer>
__global__ __launch_bounds__(T) void block_norm_kernel(const s3d8_block_norm_args p, double inv_k) {
    __shared__ double sums[4][T / 64];
    __shared__ float maxima[T / 64];
    const int64_t row = blockIdx.x;
    const int K = (int)p.K, n4 = K >> 2;
    const int64_t base = row * K;
    auto load = [&](float4 (&v)[NV], const void *x, bool bf) {
        if (bf) {
            Raw<true> r[NV];
            load_row<T, NV, true>(r, x, base, n4);
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = values(r[j]);
        } else {
            load_row<T, NV, false>(v, x, base, n4);
        }
    };
    // one gate for all: by a scalar load, and its tanh while the row is on its way
    const bool one = !p.gate_channels, squash = p.gate_tanh;
    float g1 = 1.0f;
    if (p.gate && one) g1 = *p.gate;
    float4 h[NV];
    load(h, p.h, p.h_type == S3D8_ROWS_BF16);
    if (p.branch) {
        float4 t[NV];
        load(t, p.branch, p.branch_type == S3D8_ROWS_BF16);
        if (squash) g1 = tanh_rounded(g1);
        if (p.post_weight) normalise<T, NV, kLayer>(t, K, inv_k, p.eps, p.post_weight, p.post_bias, sums[0]);
        if (p.gate) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = threadIdx.x + j * T;
                float4 g = make_float4(g1, g1, g1, g1);
                if (!one && i < n4) {
                    g = reinterpret_cast<const float4 *>(p.gate)[i];
                    if (squash) g = map4(g, tanh_rounded);
                }
                t[j] = zip4(g, t[j], [](float x, float y) { return x * y; });
            }
        }
        const float rs = p.residual_scale;
        if (rs != 1.0f)
#pragma unroll
            for (int j = 0; j < NV; ++j) h[j] = map4(h[j], [&](float x) { return rs * x; });
#pragma unroll
        for (int j = 0; j < NV; ++j) h[j] = zip4(h[j], t[j], [](float x, float y) { return x + y; });
        if (p.h_type == S3D8_ROWS_BF16) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = threadIdx.x + j * T;
                const uint2 u = bf16x4(h[j]);
                h[j] = bf16x4_values(u);  // the norm reads the residual as it is stored
                if (i < n4) reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.h_out) + base)[i] = u;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = threadIdx.x + j * T;
                if (i < n4) reinterpret_cast<float4 *>(static_cast<float *>(p.h_out) + base)[i] = h[j];
            }
        }
    }
    normalise<T, NV, kLayer>(h, K, inv_k, p.eps, p.weight, p.bias, sums[2]);
    row_out<T, NV>(h, row, K, p.out_type, p.rows, p.xq, p.xs, maxima);
}

// SiLU(g) * u = g u / (1 + exp(-g)) in 64 bits, rounded to fp32 once, to a
// relative 2^-50 before that (so that it is the correctly rounded product but
// for one value in some 2^25).  |g| is cut at 700, where the result is already
// g u or, below 2^-149, a zero of its sign; the denominator stays finite.
__device__ __forceinline__ float gated(float g, float u) {
    const Exp e = exp_parts((double)-__builtin_amdgcn_fmed3f(g, -700.0f, 700.0f));
    const double d = 1.0 + __builtin_fma(e.two_n, e.less_one, e.two_n);
    return (float)((double)g * (double)u * reciprocal(d));
}

// The same in fp32, off by less than a relative 2^-20 while g >= -64 and g u is
// neither infinite nor subnormal: exp2 and the reciprocal by at most an ulp
// (2^-23) each, the exponent -g log2(e) in two parts by nothing that counts, and
// five more roundings of 2^-24.
__device__ __forceinline__ float gated_near(float g, float u) {
    const float c = fminf(g, 200.0f);
    const float h = c * -0x1.715476p+0f;
    const float l = __builtin_fmaf(c, -0x1.4ae0c0p-26f, __builtin_fmaf(c, -0x1.715476p+0f, -h));
    float e = __builtin_amdgcn_exp2f(h);
    e = __builtin_fmaf(e, l * 0x1.62e430p-1f, e);
    return g * u * __builtin_amdgcn_rcpf(1.0f + e);
}

// Codes and scale of a row, equal to what row_out makes of gated() of every element,
// but with gated() (some 45 instructions) only where fp32 cannot tell:
//   - the row's maximum is gated() of the elements whose gated_near() is
//     within 2^-18 of the largest one (the true maximum's is within 2^-19);
//   - t = near rcp(s) is off from x / s by less than 127 (2^-20 + 2^-22) < 2^-12.6,
//     fl(x / s) by 127 2^-24: where t is further than 2^-12 from a border k + 1/2
//     its nearest integer is the code (all but one value in 2^11).
// Both kinds go through a list in LDS, so that the few of them take one pass of
// the workgroup.  False where the row is outside gated_near()'s range or a list
// overflows: nothing is then said about the row, whose codes may be partly
// written.
constexpr int kListed = 256;
template <int T, int NV, bool kBF>
__device__ __forceinline__ bool glu_codes(const Raw<kBF> (&g4)[NV], const Raw<kBF> (&u4)[NV], int64_t row, int K,
                                          int8_t *xq, float *xs, float (*slots)[T / 64]) {
    __shared__ int counts[2];
    __shared__ int place[kListed];
    __shared__ float4 gs[kListed], us[kListed];
    const int n4 = K >> 2;
    if (threadIdx.x < 2) counts[threadIdx.x] = 0;
    float4 near[NV];
    float lowest = 0.0f, most = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const float4 g = values(g4[j]);
        near[j] = zip4(g, values(u4[j]), gated_near);
        lowest = fminf(fminf(lowest, fminf(g.x, g.y)), fminf(g.z, g.w));
        most = fmaxf(fmaxf(most, fmaxf(fabsf(near[j].x), fabsf(near[j].y))), fmaxf(fabsf(near[j].z), fabsf(near[j].w)));
    }
    const float top = block_max<T>(lowest < -64.0f ? INFINITY : most, slots[0]);
    if (!(top >= 0x1p-100f && top < INFINITY)) return false;  // uniform
    lds_barrier();  // (a workgroup of one wave has had none)
    const float bar = top * (1.0f - 0x1p-18f);
    auto list = [&](int j, int which) {
        const int k = atomicAdd(&counts[which], 1);
        if (k < kListed) {
            place[k] = threadIdx.x + j * T;
            gs[k] = values(g4[j]);
            us[k] = values(u4[j]);
        }
    };
    if (most >= bar) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (fmaxf(fmaxf(fabsf(near[j].x), fabsf(near[j].y)), fmaxf(fabsf(near[j].z), fabsf(near[j].w))) >= bar)
                list(j, 0);
    }
    lds_barrier();
    int listed = counts[0];
    if (listed > kListed) return false;
    float a = 0.0f;
    const float *gl = reinterpret_cast<const float *>(gs), *ul = reinterpret_cast<const float *>(us);
    for (int k = threadIdx.x; k < 4 * listed; k += T) a = fmaxf(a, fabsf(gated(gl[k], ul[k])));
    a = block_max<T>(a, slots[1]);
    lds_barrier();
    const float s = a / 127.0f, rs = __builtin_amdgcn_rcpf(s);
    if (threadIdx.x == 0) xs[row] = s;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = threadIdx.x + j * T;
        float far = 0.0f;
        const uint32_t q = codes4(near[j], rs, far);
        if (far > 0.5f - 0x1p-12f)
            list(j, 1);
        else if (i < n4)
            reinterpret_cast<uint32_t *>(xq + row * K)[i] = q;
    }
    lds_barrier();
    listed = counts[1];
    if (listed > kListed) return false;
    for (int k = threadIdx.x; k < 4 * listed; k += T) {
        const float x = fminf(127.0f, fmaxf(-127.0f, rintf(gated(gl[k], ul[k]) / s)));
        const int at = 4 * place[k >> 2] + (k & 3);
        if (at < K) xq[row * K + at] = (int8_t)x;
    }
    return true;
}

// One workgroup per row.  Measured in bf16, codes out: 2048 x 14336 31-33 us (147 MB
// at 4.5 TB/s; 27 vector instructions per element, issuing 84% of the time), 58.7 us
// with gated() for every element, which is what a row with one gate below -64 takes
// (62 us with one in each row), and rows out in bf16 or fp32 too (47 us in bf16, 176 MB);
// one row of 14336 in fp32 5.2 us,
// 5 x 1744 to fp32 2.5 us (both little more than a launch and their latency).
template <int T, int NV, bool kBF>
__global__ __launch_bounds__(T) void glu_act_kernel(const void *__restrict__ gate, int64_t ldg,
                                                    const void *__restrict__ up, int64_t ldu, int K, int out_type,
                                                    void *__restrict__ rows, int8_t *__restrict__ xq,
                                                    float *__restrict__ xs) {
    __shared__ float maxima[3][T / 64];
    const int64_t row = blockIdx.x;
    const int n4 = K >> 2;
    Raw<kBF> g4[NV], u4[NV];
    load_row<T, NV, kBF>(g4, gate, row * ldg, n4);
    load_row<T, NV, kBF>(u4, up, row * ldu, n4);
    if (out_type == S3D8_ROWS_CODES && glu_codes<T, NV, kBF>(g4, u4, row, K, xq, xs, maxima)) return;
    float4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = zip4(values(g4[j]), values(u4[j]), gated);
    row_out<T, NV>(v, row, K, out_type, rows, xq, xs, maxima[2]);
}

// --------------------------------------------------------------- host

// Kernels by workgroup and row width.
template <bool kLayer>
struct BlockNorm {
    template <int T, int NV>
    static constexpr auto kernel() { return &block_norm_kernel<T, NV, kLayer>; }
};
template <bool kBF>
struct GluAct {
    template <int T, int NV>
    static constexpr auto kernel() { return &glu_act_kernel<T, NV, kBF>; }
};

// The workgroup of a row: where there are rows for every CU, the fewest threads
// that hold it in `most` float4 each (few waves to join, several rows on a CU at
// once); else as many as it has float4 (short chains).
template <class Op>
auto row_kernel(int64_t M, int64_t K, int cus, int most, int &threads) {
    const int64_t n4 = K / 4;
    threads = 1024;
    for (int t : {512, 256, 64})
        if (n4 <= t * (M >= 2 * cus ? most : 1)) threads = t;
    const int64_t nv = (n4 + threads - 1) / threads;
    auto pick = [&](auto t) {
        constexpr int T = decltype(t)::value;
        constexpr int kTwo = T == 512 ? 4 : 2;  // (up to 1024 float4 with 2 to 7 a thread go to 256 threads)
        return nv <= 1   ? Op::template kernel<T, 1>()
               : nv <= 2 ? Op::template kernel<T, kTwo>()
               : nv <= 4 ? Op::template kernel<T, 4>()
               : nv <= 5 ? Op::template kernel<T, 5>()
                         : Op::template kernel<T, 7>();
    };
    if (threads == 64) return pick(std::integral_constant<int, 64>());
    if (threads == 256) return pick(std::integral_constant<int, 256>());
    if (threads == 512) return pick(std::integral_constant<int, 512>());
    return nv > 7 ? Op::template kernel<1024, 16>() : pick(std::integral_constant<int, 1024>());
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_rows(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0) return s3d8::fail(S3D8_ERR_INVALID_ARG, "sizes must be positive");
    if (K % 16 != 0) return s3d8::fail(S3D8_ERR_SHAPE, "K must be a multiple of 16");
    if (K > kMaxWidth) return s3d8::fail(S3D8_ERR_SHAPE, "K over 65536 is not supported");
    if (M > kMaxRows) return s3d8::fail(S3D8_ERR_SHAPE, "more than 524288 rows are not supported");
    return S3D8_OK;
}

bool row_type(int32_t t) { return t == S3D8_ROWS_F32 || t == S3D8_ROWS_BF16; }

int check_out(int32_t out_type, const void *rows, const int8_t *xq, const float *xs) {
    if (!row_type(out_type) && out_type != S3D8_ROWS_CODES)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown output type");
    const bool codes = out_type == S3D8_ROWS_CODES;
    if (codes ? rows || !xq || !xs : !rows || xq || xs)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "codes need xq and xs and no rows, other outputs rows alone");
    if (!aligned(rows, 16) || !aligned(xq, 16))
        return s3d8::fail(S3D8_ERR_ALIGN, "output rows and xq must be 16-byte aligned");
    if (!aligned(xs, 4)) return s3d8::fail(S3D8_ERR_ALIGN, "xs must be 4-byte aligned");
    return S3D8_OK;
}

}  // namespace

extern "C" {

int32_t s3d8_block_norm(const s3d8_block_norm_args *args, void *stream) {
    if (!args || !args->h || !args->weight) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    const s3d8_block_norm_args &a = *args;
    if ((a.branch != nullptr) != (a.h_out != nullptr))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "h_out goes with branch");
    if (!a.branch && (a.post_weight || a.gate))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "a post norm or gate needs a branch");
    if (a.kind != S3D8_NORM_RMS && a.kind != S3D8_NORM_LAYER)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown norm kind");
    if (a.kind == S3D8_NORM_RMS && (a.bias || a.post_bias))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "an RMS norm has no bias");
    if (a.post_bias && !a.post_weight) return s3d8::fail(S3D8_ERR_INVALID_ARG, "post_bias needs post_weight");
    if (!row_type(a.h_type) || (a.branch && !row_type(a.branch_type)))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    // 1 / sqrt(eps), a zero row's factor, is then between 2^-126 and 2^126 (infinite, it made zeros NaN)
    if (!(a.eps >= 0x1p-252 && a.eps <= 0x1p252))
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "eps must be positive (2^-252 to 2^252)");
    int rc = check_rows(a.M, a.K);
    if (rc) return rc;
    rc = check_out(a.out_type, a.rows, a.xq, a.xs);
    if (rc) return rc;
    if (!aligned(a.h, 16) || !aligned(a.branch, 16) || !aligned(a.h_out, 16) || !aligned(a.weight, 16) ||
        !aligned(a.bias, 16) || !aligned(a.post_weight, 16) || !aligned(a.post_bias, 16) ||
        !aligned(a.gate, a.gate_channels ? 16 : 4))
        return s3d8::fail(S3D8_ERR_ALIGN, "rows and [K] vectors must be 16-byte aligned");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    int threads = 0;
    const auto fn = a.kind == S3D8_NORM_LAYER ? row_kernel<BlockNorm<true>>(a.M, a.K, cus, 7, threads)
                                              : row_kernel<BlockNorm<false>>(a.M, a.K, cus, 7, threads);
    hipLaunchKernelGGL(fn, dim3((unsigned)a.M), dim3(threads), 0, (hipStream_t)stream, a, 1.0 / (double)a.K);
    return s3d8::launch_status();
}

int32_t s3d8_glu_act(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int64_t M, int64_t K,
                     int32_t in_type, int32_t out_type, void *rows, int8_t *xq, float *xs, void *stream) {
    if (!gate || !up) return s3d8::fail(S3D8_ERR_INVALID_ARG, "null pointer argument");
    if (!row_type(in_type)) return s3d8::fail(S3D8_ERR_INVALID_ARG, "unknown row type");
    int rc = check_rows(M, K);
    if (rc) return rc;
    rc = check_out(out_type, rows, xq, xs);
    if (rc) return rc;
    const int64_t lim = int64_t(1) << 40;
    if (ld_gate < K || ld_up < K || ld_gate > lim || ld_up > lim)
        return s3d8::fail(S3D8_ERR_INVALID_ARG, "row strides must be at least K (and below 2^40)");
    const uintptr_t four = in_type == S3D8_ROWS_F32 ? 16 : 8;
    if (ld_gate % 4 || ld_up % 4 || !aligned(gate, four) || !aligned(up, four))
        return s3d8::fail(S3D8_ERR_ALIGN, "gate and up rows must be aligned to 4 elements");
    int cus = 0;
    rc = s3d8::check_device(&cus);
    if (rc) return rc;
    int threads = 0;
    const auto fn = in_type == S3D8_ROWS_BF16 ? row_kernel<GluAct<true>>(M, K, cus, 7, threads)
                                              : row_kernel<GluAct<false>>(M, K, cus, 7, threads);
    hipLaunchKernelGGL(fn, dim3((unsigned)M), dim3(threads), 0, (hipStream_t)stream, gate, ld_gate, up, ld_up,
                       (int)K, out_type, rows, xq, xs);
    return s3d8::launch_status();
}

}  // extern "C"
