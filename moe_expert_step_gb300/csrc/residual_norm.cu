// The gated residual update after a block and the norm before the next one, one pass:
//   h' = h + s * g * (w_post * y * rsqrt(mean(y^2) + eps)),   x = w_pre * h' * rsqrt(mean(h'^2) + eps)
// A token's y and h are read once, held in registers through both reductions, and h' and x are
// written once: 12 to 16 bytes an element, memory-bound.  Four warps a row up to H = 2048 (8192
// tokens x 2048, bf16 y: 38.1 us, 5.3 TB/s; eight warps 39.7, two 41.2, one warp a row without
// barriers 52: too few rows in flight), eight above, 8 columns a lane at a time.
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
    int H, P, T;
};

// Eight consecutive columns, as loaded
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Eight<bf16> {
    uint4 u;
    __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the W warps of a row
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();  // the last sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += red[w];
    return t;
}

// A row on the W warps of a block: lane i of warp w holds columns 8 (i + 32 (w + W j)) .. + 7, j < N.
template <typename TY, typename TX, int W, int N>
__global__ void __launch_bounds__(32 * W) residual_norm_kernel(const NormArgs a) {
    __shared__ float red[W];
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, c0 = 8 * threadIdx.x;
    const size_t row = static_cast<size_t>(t) * a.H;
    Eight<TY> yv[N];
    float h[N][8];
    // y and h of the whole row in flight at once
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 256 * W * j;
        if (c < a.H) yv[j].load(static_cast<const TY*>(a.y) + row + c);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 256 * W * j;
        Eight<float> e;
        if (c < a.H) {
            e.load(a.h_in + row + c);
            e.get(h[j]);
        }
    }
    float ry = 1.f, ss = 0.f;
    if (a.w_post) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (c0 + 256 * W * j >= a.H) continue;
            float y[8];
            yv[j].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
        }
        ry = 1.0f / sqrtf(row_sum<W>(ss, red) / a.H + a.eps);
    }
    const float* g = a.gate ? a.gate + (t / a.P) * a.gate_ld : nullptr;
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 256 * W * j;
        if (c >= a.H) continue;
        float y[8], w[8];
        yv[j].get(y);
        if (a.w_post) {
            Eight<TX> e;
            e.load(static_cast<const TX*>(a.w_post) + c);
            e.get(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * ry * w[i];
        }
        if (g) {
            Eight<float> e;
            e.load(g + c);
            e.get(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[j][i] += a.res_scale * y[i];
            ss += h[j][i] * h[j][i];
        }
        store8(a.h_out + row + c, h[j]);
    }
    if (a.x == nullptr) return;
    const float rh = 1.0f / sqrtf(row_sum<W>(ss, red) / a.H + a.eps);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 256 * W * j;
        if (c >= a.H) continue;
        float w[8];
        if (a.w_pre) {
            Eight<TX> e;
            e.load(static_cast<const TX*>(a.w_pre) + c);
            e.get(w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= h[j][i] * rh;
        store8(static_cast<TX*>(a.x) + row + c, w);
    }
}

template <typename TY, typename TX>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    const dim3 grid(a.T);
    if (a.H <= 1024) return launch_pdl(residual_norm_kernel<TY, TX, 4, 1>, grid, dim3(128), 0, s, a);
    if (a.H <= 2048) return launch_pdl(residual_norm_kernel<TY, TX, 4, 2>, grid, dim3(128), 0, s, a);
    if (a.H <= 4096) return launch_pdl(residual_norm_kernel<TY, TX, 8, 2>, grid, dim3(256), 0, s, a);
    return launch_pdl(residual_norm_kernel<TY, TX, 8, 4>, grid, dim3(256), 0, s, a);
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
    if (dims->H > 8192) return MOESTEP_EUNSUPPORTED;
    if ((rc = device_ok(nullptr)) != MOESTEP_OK) return rc;
    NormArgs a{y, w_post, gate, gate_ld, res_scale, h_in, h_out, w_pre, x, eps, dims->H, dims->P, T};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    cudaError_t e;
    if (dims->dtype == MOESTEP_F32)
        e = y_dtype == MOESTEP_F32 ? launch_norm<float, float>(a, s) : launch_norm<bf16, float>(a, s);
    else
        e = y_dtype == MOESTEP_F32 ? launch_norm<float, bf16>(a, s) : launch_norm<bf16, bf16>(a, s);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}
