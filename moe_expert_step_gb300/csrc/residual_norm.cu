// The gated residual update after a block and the norm before the next one, one pass:
//   h' = h + s * g * (w_post * y * rsqrt(mean(y^2) + eps)),   x = w_pre * h' * rsqrt(mean(h'^2) + eps)
// One CTA a token.  A token's y and h are read once, held in registers through both
// reductions, and h' and x are written once: 12 to 16 bytes an element, memory-bound.
#include "combine.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

#include <cmath>

namespace moestep {
namespace {

struct NormArgs {
    const void* y;
    const void* w_post;
    const float* gate;
    long long gate_ld;
    float res_scale;
    const float* h_in;
    float* h_out;
    const void* w_pre;
    void* x;
    float eps;
    int H, P;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<bf16>(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// Columns c = 4 (tid + 256 i), i < N: N = ceil(H / 1024)
template <typename TY, typename TX, int N>
__global__ void __launch_bounds__(256) residual_norm_kernel(const NormArgs a) {
    __shared__ float red[9];
    pdl_trigger();
    pdl_wait();
    const size_t row = static_cast<size_t>(blockIdx.x) * a.H;
    const TY* y = static_cast<const TY*>(a.y) + row;
    float4 yv[N], hv[N];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 4 * (threadIdx.x + 256 * i);
        yv[i] = hv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < a.H) {
            yv[i] = load4<TY>(y + c);
            hv[i] = load4<float>(a.h_in + row + c);
        }
    }
    float ry = 1.f;
    if (a.w_post) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            ss += yv[i].x * yv[i].x + yv[i].y * yv[i].y + yv[i].z * yv[i].z + yv[i].w * yv[i].w;
        ry = 1.0f / sqrtf(group_sum_256(ss, red) / a.H + a.eps);
    }
    const float* g = a.gate ? a.gate + (blockIdx.x / a.P) * a.gate_ld : nullptr;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 4 * (threadIdx.x + 256 * i);
        if (c >= a.H) continue;
        float4 v = yv[i];
        if (a.w_post) {
            const float4 w = load4<TX>(static_cast<const TX*>(a.w_post) + c);
            v = make_float4(v.x * ry * w.x, v.y * ry * w.y, v.z * ry * w.z, v.w * ry * w.w);
        }
        if (g) {
            const float4 w = load4<float>(g + c);
            v = make_float4(v.x * w.x, v.y * w.y, v.z * w.z, v.w * w.w);
        }
        float4 h = hv[i];
        h = make_float4(h.x + a.res_scale * v.x, h.y + a.res_scale * v.y, h.z + a.res_scale * v.z,
                        h.w + a.res_scale * v.w);
        hv[i] = h;
        ss += h.x * h.x + h.y * h.y + h.z * h.z + h.w * h.w;
        *reinterpret_cast<float4*>(a.h_out + row + c) = h;
    }
    if (a.x == nullptr) return;
    const float rh = 1.0f / sqrtf(group_sum_256(ss, red) / a.H + a.eps);
    TX* x = static_cast<TX*>(a.x) + row;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 4 * (threadIdx.x + 256 * i);
        if (c >= a.H) continue;
        const float4 w = a.w_pre ? load4<TX>(static_cast<const TX*>(a.w_pre) + c) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 h = hv[i];
        store4<TX>(x + c, make_float4(h.x * rh * w.x, h.y * rh * w.y, h.z * rh * w.z, h.w * rh * w.w));
    }
}

template <typename TY, typename TX>
cudaError_t launch_norm(int T, const NormArgs& a, cudaStream_t s) {
    const dim3 grid(T), block(256);
    switch ((a.H + 1023) / 1024) {
        case 1: return launch_pdl(residual_norm_kernel<TY, TX, 1>, grid, block, 0, s, a);
        case 2: return launch_pdl(residual_norm_kernel<TY, TX, 2>, grid, block, 0, s, a);
        case 3:
        case 4: return launch_pdl(residual_norm_kernel<TY, TX, 4>, grid, block, 0, s, a);
        default: return launch_pdl(residual_norm_kernel<TY, TX, 7>, grid, block, 0, s, a);
    }
}

}  // namespace
}  // namespace moestep

extern "C" int block_residual_norm(const moestep_dims* dims, int T, const void* y, int y_dtype, const void* w_post,
                                   const float* gate, long long gate_ld, float res_scale, const float* h_in,
                                   float* h_out, const void* w_pre, void* x, float eps, void* stream) {
    using namespace moestep;
    int rc = validate_dims(dims);
    if (rc != MOESTEP_OK) return rc;
    if (T <= 0 || !y || !h_in || !h_out) return MOESTEP_EINVAL;
    if (y_dtype != MOESTEP_BF16 && y_dtype != MOESTEP_F32) return MOESTEP_EINVAL;
    if (!std::isfinite(res_scale) || !std::isfinite(eps) || !(eps > 0.f)) return MOESTEP_EINVAL;
    if (gate && (gate_ld < 0 || (gate_ld > 0 && gate_ld < dims->H))) return MOESTEP_EINVAL;
    for (const void* p : {y, w_post, static_cast<const void*>(gate), static_cast<const void*>(h_in),
                          static_cast<const void*>(h_out), w_pre, static_cast<const void*>(x)})
        if (!kv_aligned16(p)) return MOESTEP_EALIGN;
    if (gate && gate_ld % 4) return MOESTEP_EALIGN;
    if (dims->H > 7168) return MOESTEP_EUNSUPPORTED;
    if ((rc = device_ok(nullptr)) != MOESTEP_OK) return rc;
    NormArgs a{y, w_post, gate, gate_ld, res_scale, h_in, h_out, w_pre, x, eps, dims->H, dims->P};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    cudaError_t e;
    if (dims->dtype == MOESTEP_F32)
        e = y_dtype == MOESTEP_F32 ? launch_norm<float, float>(T, a, s) : launch_norm<bf16, float>(T, a, s);
    else
        e = y_dtype == MOESTEP_F32 ? launch_norm<float, bf16>(T, a, s) : launch_norm<bf16, bf16>(T, a, s);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}
