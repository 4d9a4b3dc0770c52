// The paged key-value cache: new tokens' keys and values stored into pages (quantised
// on the way with MOESTEP_FP8) and read back.
//
// FP8: a (token, head) vector x is stored as code = e4m3(x * 2^-e) with one exponent e, the
// smallest with max|x| <= 448 * 2^e.  A power of two costs no accuracy against a free scale
// (E4M3 is a floating-point format: a factor below 2 only moves values within their
// binades) and buys exactness: the quantisation rounds once, and code * 2^e is a bf16 value,
// so every reader sees the same numbers.  amax = m * 2^x (m in [0.5, 1)) gives e = x - 9 if
// m <= 0.875 (448 = 0.875 * 2^9) else x - 8: integer work on the float's bits, no division.
#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

#include <type_traits>

namespace moestep {
namespace {

struct CopyArgs {
    const void* k;  // new keys / values, or where they are read back to
    const void* v;
    long long ld;
    const int32_t* pos;
    void* kc;
    void* vc;
    uint8_t* ke;
    uint8_t* ve;
    const int32_t* table;
    int n, Hkv, page_log2, n_pages, max_pages;
    uint32_t per_magic, n_magic;  // ceil(2^32 / divisor) of 2 * Hkv and, where n is in [2, 65000], of n
    long long vectors;            // tokens * 2 * Hkv
    int* err;
};

// A thread handles 16 elements of kPer vectors; D / 16 lanes share a vector, and
// consecutive vectors are a token's key heads, then its value heads, so a warp reads and
// writes whole lines.  A block takes 2 * 256 / (D / 16) vectors: their tokens and requests are
// found with 32-bit divisions (a wide one only in a launch of more than 2^32 vectors) and from
// there on with multiplications by reciprocals, which give x / d exactly while x (d - 1) < 2^32: j < 2 Hkv + 128
// (2176 at most), tl < n + 64 (a block has 128 vectors where D = 64, two at least to a token).
// Both kernels are copies, bound by memory: 32768 tokens of 8 heads of 128 (134 MB of bf16 on
// one side, 69 MB of codes on the other) are written in 34.7 us and read back in 33.8 us, 5.8
// and 6.0 TB/s.  Four vectors a thread take 3 and 1 us longer (fewer blocks, a longer tail), one
// 0.5 and 2 us and a read of 777 tokens 6.6 us against 6.0 us (too few loads in flight).  Six
// resident blocks for the write (40 registers) against five 35.0 : 36.0 us, eight for the read
// (32 registers) against six 36.3 : 40.2 us (then with 16 consecutive elements a thread, whose
// stores of half sectors cost 2.5 us).  fp32 (537 MB in all), with four: 79 us each way, 6.8 TB/s.
constexpr int kPer = 2;

struct Vector {
    long long t;  // token
    int r;        // its request
    int h;
    bool v, on;
};

// x / d of a quotient that fits 31 bits; 64-bit arithmetic only where x needs it
__device__ __forceinline__ unsigned divide(long long x, unsigned d) {
    return x >> 32 ? static_cast<unsigned>(x / d) : static_cast<unsigned>(x) / d;
}

template <int L>
__device__ __forceinline__ Vector vector_of(const CopyArgs& a, unsigned t0, unsigned rem, unsigned r0, unsigned tl0, int q,
                                            long long first) {
    const unsigned local = q * (256 / L) + threadIdx.x / L, per = 2 * a.Hkv;
    const unsigned j = rem + local, dt = __umulhi(j, a.per_magic), w = j - dt * per, tl = tl0 + dt;
    const unsigned dr = a.n_magic ? __umulhi(tl, a.n_magic) : a.n == 1 ? tl : tl >= static_cast<unsigned>(a.n);
    Vector x;
    x.t = static_cast<long long>(t0) + dt;
    x.r = static_cast<int>(r0 + dr);
    x.v = w >= static_cast<unsigned>(a.Hkv);
    x.h = static_cast<int>(x.v ? w - a.Hkv : w);
    x.on = first + local < a.vectors;
    return x;
}

// Place of a token's vector: its row index (vectors of D elements from the pool's start), -1
// for a token that is not stored, -2 for a bad position or page.
__device__ __forceinline__ long long place(const CopyArgs& a, int p, const Vector& x) {
    if (p < 0) return -1;
    const int pg = p >> a.page_log2;
    if (pg >= a.max_pages) return -2;
    const int id = __ldg(&a.table[static_cast<long long>(x.r) * a.max_pages + pg]);
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.n_pages)) return -2;
    return ((static_cast<long long>(id) * a.Hkv + x.h) << a.page_log2) + (p & ((1 << a.page_log2) - 1));
}

// e of a vector whose largest finite magnitude (or infinity) is amax >= 0
__device__ __forceinline__ int kv_exponent(float amax) {
    if (amax == 0.f) return -100;
    amax = fminf(amax, 3.402823466e38f);
    const uint32_t b = __float_as_uint(amax);
    if (b < 0x00800000u) return -100;                   // subnormal: far below 448 * 2^-100
    const int x = static_cast<int>(b >> 23) - 126;      // amax = m * 2^x
    const int e = (b & 0x7fffffu) > 0x600000u ? x - 8 : x - 9;  // m > 0.875
    return min(max(e, -100), 119);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ float2 from_e4m3x2(uint16_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// 16 elements as they are loaded: 2 (bf16) or 4 (fp32) 16-byte pieces, D / N elements apart, so that
// the lanes of a vector read and write whole sectors together
template <int DT>
struct Sixteen {
    static constexpr int N = DT == MOESTEP_F32 ? 4 : 2;
    uint4 p[N];
};

template <int DT, int D>
__global__ void __launch_bounds__(256, DT == MOESTEP_F32 ? 4 : 6) kv_write_kernel(const CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    using T = typename std::conditional<DT == MOESTEP_F32, float, bf16>::type;
    using S = Sixteen<DT>;
    constexpr int L = D / 16;
    const long long first = static_cast<long long>(blockIdx.x) * (256 / L * kPer);
    const unsigned t0 = divide(first, 2 * a.Hkv), rem = static_cast<unsigned>(first - static_cast<long long>(t0) * (2 * a.Hkv));
    const unsigned r0 = t0 / a.n, tl0 = t0 - r0 * a.n;
    const int lane = threadIdx.x % L;
    Vector vec[kPer];
    int pos[kPer];
    S in[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {  // the tokens' rows do not wait for their places
        vec[q] = vector_of<L>(a, t0, rem, r0, tl0, q, first);
        pos[q] = -1;
        if (vec[q].on) {
            pos[q] = __ldg(&a.pos[vec[q].t]);
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(vec[q].v ? a.v : a.k) + vec[q].t * a.ld + vec[q].h * D) + lane;
#pragma unroll
            for (int i = 0; i < S::N; ++i) in[q].p[i] = __ldg(src + i * L);
        }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const long long row = vec[q].on ? place(a, pos[q], vec[q]) : -1;
        if (row == -2 && lane == 0) record_error(a.err, kErrBadInput);
        void* cache = vec[q].v ? a.vc : a.kc;
        if (DT != MOESTEP_FP8) {
            if (row < 0) continue;
            uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(cache) + row * D) + lane;
#pragma unroll
            for (int i = 0; i < S::N; ++i) d[i * L] = in[q].p[i];
            continue;
        }
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 u = in[q].p[i / 4];
            const uint32_t w = vec[q].on ? (i % 4 == 0 ? u.x : i % 4 == 1 ? u.y : i % 4 == 2 ? u.z : u.w) : 0u;
            x[2 * i] = __uint_as_float(w << 16);
            x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));  // fmaxf passes over NaN
#pragma unroll
        for (int o = L / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (row < 0) continue;
        const int e = kv_exponent(amax);
        const float s = pow2f(-e);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = to_e4m3x2(x[4 * i] * s, x[4 * i + 1] * s) | to_e4m3x2(x[4 * i + 2] * s, x[4 * i + 3] * s) << 16;
        uint2* d = reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D) + lane;
        d[0] = make_uint2(w[0], w[1]);
        d[L] = make_uint2(w[2], w[3]);
        if (lane == 0) (vec[q].v ? a.ve : a.ke)[row] = static_cast<uint8_t>(e + 127);
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(256, DT == MOESTEP_F32 ? 4 : 8) kv_read_kernel(const CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    using T = typename std::conditional<DT == MOESTEP_F32, float, bf16>::type;
    using S = Sixteen<DT>;
    constexpr int L = D / 16;
    const long long first = static_cast<long long>(blockIdx.x) * (256 / L * kPer);
    const unsigned t0 = divide(first, 2 * a.Hkv), rem = static_cast<unsigned>(first - static_cast<long long>(t0) * (2 * a.Hkv));
    const unsigned r0 = t0 / a.n, tl0 = t0 - r0 * a.n;
    const int lane = threadIdx.x % L;
    Vector vec[kPer];
    long long row[kPer];
    int pos[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        vec[q] = vector_of<L>(a, t0, rem, r0, tl0, q, first);
        pos[q] = vec[q].on ? __ldg(&a.pos[vec[q].t]) : -1;
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        row[q] = place(a, pos[q], vec[q]);
        if (row[q] == -2 && lane == 0) record_error(a.err, kErrBadInput);
    }
    S o[kPer];
    uint4 codes[kPer];
    int ex[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {  // all loads before the first use
        const void* cache = vec[q].v ? a.vc : a.kc;
#pragma unroll
        for (int i = 0; i < S::N; ++i) o[q].p[i] = make_uint4(0, 0, 0, 0);
        codes[q] = make_uint4(0, 0, 0, 0);
        ex[q] = 127;
        if (row[q] < 0) continue;
        if (DT == MOESTEP_FP8) {
            const uint2* s = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + row[q] * D) + lane;
            const uint2 lo = __ldg(s), hi = __ldg(s + L);
            codes[q] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            ex[q] = __ldg(&(vec[q].v ? a.ve : a.ke)[row[q]]);
        } else {
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(cache) + row[q] * D) + lane;
#pragma unroll
            for (int i = 0; i < S::N; ++i) o[q].p[i] = __ldg(s + i * L);
        }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        if (!vec[q].on) continue;
        if (DT == MOESTEP_FP8) {
            // 2^(exp - 127) in two factors: the byte of a corrupted cache may name any power
            const int e = ex[q] - 127, e1 = e >> 1;
            const float s1 = pow2f(e1), s2 = pow2f(e - e1);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c4 = i / 2 == 0 ? codes[q].x : i / 2 == 1 ? codes[q].y : i / 2 == 2 ? codes[q].z : codes[q].w;
                const float2 f = from_e4m3x2(static_cast<uint16_t>(c4 >> (16 * (i & 1))));
                const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s1 * s2, f.y * s1 * s2);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            o[q].p[0] = make_uint4(w[0], w[1], w[2], w[3]);
            o[q].p[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        uint4* d = reinterpret_cast<uint4*>(const_cast<T*>(static_cast<const T*>(vec[q].v ? a.v : a.k)) +
                                            vec[q].t * a.ld + vec[q].h * D) + lane;
#pragma unroll
        for (int i = 0; i < S::N; ++i) d[i * L] = o[q].p[i];
    }
}

template <int DT, int D>
cudaError_t launch_copy(bool write, const CopyArgs& a, cudaStream_t s) {
    constexpr int per_block = 256 / (D / 16) * kPer;
    const dim3 grid(static_cast<unsigned>((a.vectors + per_block - 1) / per_block));
    return write ? launch_pdl(kv_write_kernel<DT, D>, grid, dim3(256), 0, s, a)
                 : launch_pdl(kv_read_kernel<DT, D>, grid, dim3(256), 0, s, a);
}

int copy_call(bool write, const moestep_kv_dims* kd, int R, int n, const void* k, const void* v, long long ld,
              const int32_t* pos, const moestep_kv_cache* c, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_kv_dims(kd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n <= 0 || !pos) return MOESTEP_EINVAL;
    const long long width = 1ll * kd->Hkv * kd->D;
    if ((rc = check_kv_cache(kd, c)) != MOESTEP_OK) return rc;
    if ((rc = check_kv_rows(k, ld, width, kd->dtype)) != MOESTEP_OK) return rc;
    if ((rc = check_kv_rows(v, ld, width, kd->dtype)) != MOESTEP_OK) return rc;
    const long long tokens = 1ll * R * n;
    // (one block handles at least 64 vectors)
    if (tokens > (1ll << 31) - 1 || tokens * kd->Hkv > (1ll << 35)) return MOESTEP_EUNSUPPORTED;
    if ((rc = check_kv_ws(ws, ws_bytes, kKvHeader)) != MOESTEP_OK) return rc;
    if ((rc = device_ok(nullptr)) != MOESTEP_OK) return rc;
    CopyArgs a{};
    a.k = k;
    a.v = v;
    a.ld = ld;
    a.pos = pos;
    a.kc = c->k;
    a.vc = c->v;
    a.ke = c->k_exp;
    a.ve = c->v_exp;
    a.table = c->table;
    a.n = n;
    a.Hkv = kd->Hkv;
    a.page_log2 = kd->page == 16 ? 4 : kd->page == 32 ? 5 : kd->page == 64 ? 6 : 7;
    a.n_pages = kd->n_pages;
    a.max_pages = kd->max_pages;
    a.per_magic = static_cast<uint32_t>(((1ull << 32) + 2 * kd->Hkv - 1) / (2 * kd->Hkv));
    a.n_magic = n >= 2 && n <= 65000 ? static_cast<uint32_t>(((1ull << 32) + n - 1) / n) : 0;
    a.vectors = tokens * 2 * kd->Hkv;
    a.err = static_cast<int*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    cudaError_t e;
    const bool wide = kd->D == 128;
    if (kd->dtype == MOESTEP_F32)
        e = wide ? launch_copy<MOESTEP_F32, 128>(write, a, s) : launch_copy<MOESTEP_F32, 64>(write, a, s);
    else if (kd->dtype == MOESTEP_BF16)
        e = wide ? launch_copy<MOESTEP_BF16, 128>(write, a, s) : launch_copy<MOESTEP_BF16, 64>(write, a, s);
    else
        e = wide ? launch_copy<MOESTEP_FP8, 128>(write, a, s) : launch_copy<MOESTEP_FP8, 64>(write, a, s);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}

}  // namespace
}  // namespace moestep

extern "C" int kv_cache_write(const moestep_kv_dims* kd, int R, int n, const void* k, const void* v, long long ld,
                              const int32_t* pos, const moestep_kv_cache* cache, void* ws, size_t ws_bytes,
                              void* stream) {
    return moestep::copy_call(true, kd, R, n, k, v, ld, pos, cache, ws, ws_bytes, stream);
}

extern "C" int kv_cache_read(const moestep_kv_dims* kd, int R, int n, const int32_t* pos,
                             const moestep_kv_cache* cache, void* k, void* v, void* ws, size_t ws_bytes,
                             void* stream) {
    const long long ld = kd ? 1ll * kd->Hkv * kd->D : 0;
    return moestep::copy_call(false, kd, R, n, k, v, ld, pos, cache, ws, ws_bytes, stream);
}
