// Device helpers shared by the kernel sources of libs3d8: operand types,
// bfloat16 conversion, raw buffer access, LDS-destination loads and wave
// reductions.  Not part of the public ABI.
#ifndef S3D8_DEVICE_H
#define S3D8_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

namespace {

typedef int32_t v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
// Round to nearest even of a finite fp32 to bfloat16 bits.
__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
    const uint32_t u = __float_as_uint(f);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// Raw buffer loads (buffer_load_dwordx4): an offset at or past the buffer
// size returns zeros without touching memory, so predicated-off lanes need no
// branch around the load.  kOOB is past every buffer (sizes are < 2^31).
constexpr uint32_t kOOB = 0x80000000u;
constexpr int32_t kRsrcWord3 = 0x00020000;  // gfx9 family: raw, 32-bit data format

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, kRsrcWord3);
}
__device__ __forceinline__ uint4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// LDS byte offset of a __shared__ object (the value M0 takes for an
// LDS-destination buffer load).
#define S3D8_LDS_OFFSET(p) ((uint32_t)(size_t)((__attribute__((address_space(3))) const char *)(p)))

// Buffer resource as four SGPRs for inline assembly (raw, no swizzle).
__device__ __forceinline__ v4i rsrc_words(const void *p, uint32_t bytes) {
    const uint64_t a = (uint64_t)p;
    return v4i{(int32_t)(uint32_t)a, (int32_t)((uint32_t)(a >> 32) & 0xFFFFu), (int32_t)bytes, kRsrcWord3};
}

// 16 bytes per lane from buffer offset voff + soff into LDS at lds + 16 *
// lane (buffer_load_dwordx4 with the LDS bit; M0 holds the LDS base and is
// restored afterwards).  soff, the instruction's scalar offset, lets per-lane
// offsets stay loop-invariant.  A lane whose voff is at or past the buffer
// size (kOOB) writes zeros; callers keep soff below 2^31 so that voff + soff
// never wraps, and keep voff + soff inside the buffer for every other lane.
// The load counts in vmcnt like any vector load; the compiler does not see
// it, so the caller waits for it explicitly.
__device__ __forceinline__ void load_to_lds16_so(uint32_t lds, uint32_t voff, uint32_t soff, v4i rsrc) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
        : "memory");
}

// The same with 4 bytes per lane, into LDS at lds + 4 * lane.
__device__ __forceinline__ void load_to_lds4_so(uint32_t lds, uint32_t voff, uint32_t soff, v4i rsrc) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %2, %3, %4 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
        : "memory");
}

// Maxima of non-negative floats (absolute values and their maxima, never
// NaN): for x >= +0 the IEEE bit patterns order like the values, so the
// reductions compare them as unsigned integers (0 is the identity, and the
// DPP moves fold into the max instructions).
// max over each row of 16 lanes, result in every lane of the row (DPP:
// swap neighbours, swap pairs, mirror halves of 8, mirror the row)
__device__ __forceinline__ float row16_max(float v) {
    uint32_t u = __float_as_uint(v);
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xB1, 0xF, 0xF, false));
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4E, 0xF, 0xF, false));
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xF, 0xF, false));
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x140, 0xF, 0xF, false));
    return __uint_as_float(u);
}
// max over the wave, wave-uniform
__device__ __forceinline__ float wave_max(float v) {
    const uint32_t u = __float_as_uint(row16_max(v));
    const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)u, 0), (uint32_t)__builtin_amdgcn_readlane((int)u, 16));
    const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)u, 32), (uint32_t)__builtin_amdgcn_readlane((int)u, 48));
    return __uint_as_float(max(a, b));
}

// --------------------------------------------------------------- GEMM tiles

constexpr int kXcds = 8;

// Tile of workgroup blockIdx.x.  Workgroup w runs on XCD w % 8; each XCD
// takes a contiguous range of tile indices, and tile indices run over
// groups of kGroupM row blocks, row block fastest within a group and
// column block next: the ~32 workgroups resident on one XCD then cover
// about 8 row blocks x 4 column blocks, so their activation and weight
// tiles are shared through that XCD's L2 instead of each workgroup
// streaming its own weight stripe.
//
// With the input columns split into `splits` ranges, the range index ks is
// the slowest: an XCD's workgroups then share a k range as well.
constexpr int kGroupM = 8;
__device__ __forceinline__ void gemm_tile_at(int L, int nbm, int nbn, int &bm, int &bn) {
    const int group = L / (kGroupM * nbn), r = L - group * (kGroupM * nbn);
    const int gm = min(kGroupM, nbm - group * kGroupM);
    bm = group * kGroupM + r % gm;
    bn = r / gm;
}
__device__ __forceinline__ bool gemm_tile(int nbm, int nbn, int splits, int &bm, int &bn, int &ks) {
    const int nt = nbm * nbn;
    const int nwg = nt * splits;
    const int per_xcd = (nwg + kXcds - 1) / kXcds;
    const int L0 = (int)(blockIdx.x % kXcds) * per_xcd + (int)(blockIdx.x / kXcds);
    if (L0 >= nwg) return false;
    ks = L0 / nt;
    gemm_tile_at(L0 - ks * nt, nbm, nbn, bm, bn);
    return true;
}
__device__ __forceinline__ bool gemm_tile(int nbm, int nbn, int &bm, int &bn) {
    int ks;
    return gemm_tile(nbm, nbn, 1, bm, bn, ks);
}

// s_waitcnt vmcnt(N) for the loads the compiler does not see (LDS-DMA), and
// the same followed by lgkmcnt(0) and a workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N <= 63, "vmcnt is a 6-bit count");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vmcnt_barrier() {
    static_assert(N >= 0 && N <= 63, "vmcnt is a 6-bit count");
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

}  // namespace

#endif
