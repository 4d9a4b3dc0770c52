// What the launches of the chunked gated delta rule share: the operands' layout in memory and the arithmetic of f16 pairs.
#pragma once
#include "common.cuh"
#include "delta.h"
#include "tc.cuh"

namespace moestep {
namespace delta {

constexpr int C = 64;  // tokens of a chunk
// X and P are lower triangular: of their 16 x 16 blocks (f16, 512 bytes) the ten on and below the diagonal are kept
constexpr int kTri = 10 * 512;
// What a chunk of one value head has: X high, X low and factors for the states, P and factors for the outputs
enum { kA, kBeta, kD, kGamma };  // [4][64] floats
enum { kSince, kPi };            // [2][64] floats
constexpr int kXBytes = 2 * kTri + 4 * C * 4, kPBytes = kTri + 2 * C * 4, kHeadBytes = kXBytes + kPBytes;

template <int DK>
struct Tile {
    static constexpr int kBytes = C * DK * 2;  // K or Q of a chunk
};

struct Scratch {
    char* qk;     // [R][chunks][Hk][K tile, Q tile]
    char* heads;  // [R][chunks][Hv][kHeadBytes]
    int chunks;
};

// Tiles are made of 8 x 8 matrices of 128 contiguous bytes, eight rows of 16: what ldmatrix reads without a bank conflict, and
// the unit of tcgen05's layout without swizzle.  K and Q: the matrices of eight columns below each other, so that
// steps along tokens and along columns are both constant (K is an operand either way).  X and P: 16 x 16 blocks of four
// matrices, row by row; the blocks on and below the diagonal, column by column.  An ldmatrix address is the lane's place in
// 16 x 16 elements, found once, plus a constant.
constexpr int kRows16 = 256, kCols16 = 2048;  // bytes of K or Q from 16 tokens, 16 columns to the next
__device__ __forceinline__ int in_tile(int r, int c) { return c * 1024 + r * 16; }  // 8 columns c of row r of K or Q
__device__ __forceinline__ int in_block(int r, int c) { return (r >> 3) * 256 + c * 128 + (r & 7) * 16; }  // half c of row r
__device__ __forceinline__ constexpr int tri(int bi, int bj) { return (bj * (7 - bj) / 2 + bi) * 512; }  // of a lower triangle

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(tc::smem_addr(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// two values as the sum of two f16 pairs
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack(x, y);
    float lx, ly;  // x - hi
    asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tfma.rn.f32.f16 %0, p, %5, %3;\n\tfma.rn.f32.f16 %1, q, %5, %4;\n\t}"
        : "=f"(lx), "=f"(ly)
        : "r"(hi), "f"(x), "f"(y), "h"(static_cast<unsigned short>(0xbc00)));  // -1
    lo = pack(lx, ly);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // |e| <= 126
// a power of two that brings `most` to [2^to, 2^(to+1)); 1 for zeros and what is not finite
__device__ __forceinline__ float scale_to(float most, int to) {
    const int e = static_cast<int>(__float_as_uint(most) >> 23);
    if (most == 0.f || e == 255) return 1.f;
    return pow2(min(max(to + 127 - e, -126), 126));
}
// 1 / x of a power of two, |exponent| <= 126
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// Requests in the order of their lengths, long ones first, so that none begins when the others end
__device__ __forceinline__ int longest_first(const DeltaArgs& a, int r, int* found) {
    if (!a.length || a.R > 64) return r;
    const int tid = threadIdx.x;
    if (tid < a.R) {
        const int len = __ldg(&a.length[tid]);
        int rank = 0;
        for (int j = 0; j < a.R; ++j) {
            const int other = __ldg(&a.length[j]);
            rank += other > len || (other == len && j < tid);
        }
        if (rank == r) *found = tid;
    }
    __syncthreads();
    return *found;
}

}  // namespace delta

// The second launch for heads with Dv = 128, a block a head
cudaError_t launch_delta_heads(const DeltaArgs& a, const delta::Scratch& w, cudaStream_t s);

}  // namespace moestep
