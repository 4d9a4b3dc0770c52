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
    long long tokens;
    int* err;
};

// Place of a token's vector of one head: its row index (vectors of D elements from the
// pool's start), -1 for a token that is not stored, -2 for a bad position or page.
__device__ __forceinline__ long long place(const CopyArgs& a, long long t, int h) {
    const int p = __ldg(&a.pos[t]);
    if (p < 0) return -1;
    const int pg = p >> a.page_log2;
    if (pg >= a.max_pages) return -2;
    const int id = __ldg(&a.table[t / a.n * a.max_pages + pg]);
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.n_pages)) return -2;
    return ((static_cast<long long>(id) * a.Hkv + h) << a.page_log2) + (p & ((1 << a.page_log2) - 1));
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

__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// Eight consecutive elements of a vector a thread: D / 8 lanes share a vector, and
// consecutive lane groups are the heads of one token's row, so a warp reads whole lines.
// `a` works on item = (token, k or v, head, lane); kPer items a thread keep enough loads in flight.
constexpr int kPer = 4;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<bf16>(const bf16* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(256) kv_write_kernel(const CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    using T = typename std::conditional<DT == MOESTEP_F32, float, bf16>::type;
    constexpr int L = D / 8;
    const long long items = a.tokens * 2 * a.Hkv * L;
    const long long base = static_cast<long long>(blockIdx.x) * (256 * kPer) + threadIdx.x;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const long long it = base + q * 256;
        const bool on = it < items;  // whole warps' lane groups agree: items is a multiple of L
        const int lane = static_cast<int>(it % L);
        const long long vec = it / L;
        const int h = static_cast<int>(vec % a.Hkv);
        const long long tv = vec / a.Hkv;
        const int isv = static_cast<int>(tv & 1);
        const long long t = tv >> 1;
        long long row = -1;
        if (on) row = place(a, t, h);
        if (row == -2 && lane == 0) record_error(a.err, kErrBadInput);
        const T* src = static_cast<const T*>(isv ? a.v : a.k) + t * a.ld + h * D + lane * 8;
        if (DT != MOESTEP_FP8) {
            if (row < 0) continue;
            const uint4* s = reinterpret_cast<const uint4*>(src);
            uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(isv ? a.vc : a.kc) + row * D + lane * 8);
            d[0] = __ldg(s);
            if (DT == MOESTEP_F32) d[1] = __ldg(s + 1);
            continue;
        }
        float x[8] = {};
        if (row >= 0) load8<T>(src, x);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));  // fmaxf passes over NaN
#pragma unroll
        for (int o = L / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (row < 0) continue;
        const int e = kv_exponent(amax);
        const float s = pow2f(-e);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = to_e4m3x2(x[4 * i] * s, x[4 * i + 1] * s) |
                   static_cast<uint32_t>(to_e4m3x2(x[4 * i + 2] * s, x[4 * i + 3] * s)) << 16;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(isv ? a.vc : a.kc) + row * D + lane * 8) =
            make_uint2(w[0], w[1]);
        if (lane == 0) (isv ? a.ve : a.ke)[row] = static_cast<uint8_t>(e + 127);
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    using T = typename std::conditional<DT == MOESTEP_F32, float, bf16>::type;
    constexpr int L = D / 8;
    const long long items = a.tokens * 2 * a.Hkv * L;
    const long long base = static_cast<long long>(blockIdx.x) * (256 * kPer) + threadIdx.x;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const long long it = base + q * 256;
        if (it >= items) continue;
        const int lane = static_cast<int>(it % L);
        const long long vec = it / L;
        const int h = static_cast<int>(vec % a.Hkv);
        const long long tv = vec / a.Hkv;
        const int isv = static_cast<int>(tv & 1);
        const long long t = tv >> 1;
        const long long row = place(a, t, h);
        if (row == -2 && lane == 0) record_error(a.err, kErrBadInput);
        uint4 o[2] = {};
        if (row >= 0) {
            if (DT != MOESTEP_FP8) {
                const uint4* s =
                    reinterpret_cast<const uint4*>(static_cast<const T*>(isv ? a.vc : a.kc) + row * D + lane * 8);
                o[0] = __ldg(s);
                if (DT == MOESTEP_F32) o[1] = __ldg(s + 1);
            } else {
                const uint2 w = __ldg(
                    reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(isv ? a.vc : a.kc) + row * D + lane * 8));
                // 2^(exp - 127) in two factors: the byte of a corrupted cache may name any power
                const int e = __ldg(&(isv ? a.ve : a.ke)[row]) - 127, e1 = e >> 1;
                const float s1 = pow2f(e1), s2 = pow2f(e - e1);
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint16_t c = static_cast<uint16_t>((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
                    const float2 f = from_e4m3x2(c);
                    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s1 * s2, f.y * s1 * s2);
                    r[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                o[0] = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        uint4* d = reinterpret_cast<uint4*>(const_cast<T*>(static_cast<const T*>(isv ? a.v : a.k)) + t * a.ld + h * D +
                                            lane * 8);
        d[0] = o[0];
        if (DT == MOESTEP_F32) d[1] = o[1];
    }
}

template <int DT, int D>
cudaError_t launch_copy(bool write, const CopyArgs& a, cudaStream_t s) {
    const long long items = a.tokens * 2 * a.Hkv * (D / 8);
    const long long ctas = (items + 256 * kPer - 1) / (256 * kPer);
    return write ? launch_pdl(kv_write_kernel<DT, D>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, a)
                 : launch_pdl(kv_read_kernel<DT, D>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, a);
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
    if (tokens > (1ll << 31) - 1 || tokens * 2 * width / 8 > (1ll << 40)) return MOESTEP_EUNSUPPORTED;
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
    a.tokens = tokens;
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
