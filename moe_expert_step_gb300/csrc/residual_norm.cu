// The gated residual update after a block and the norm before the next one, one pass:
//   h' = h + s * g * (w_post * y * rsqrt(mean(y^2) + eps)),   x = w_pre * h' * rsqrt(mean(h'^2) + eps)
// A token's y and h are read once, held in registers through both reductions, and h' and x are
// written once: 12 to 16 bytes an element, memory-bound.  Four warps a row up to H = 2048, eight up
// to 4096, sixteen above, 4 columns a lane at a time.  Everything that a row needs is loaded before
// the first sum, the weights and the gate too: 8192 tokens x 2048, bf16 y, 32.4 us, 6.3 TB/s (fp32 y 37.5, all in fp32 43.6 us, 6.2 TB/s), against
// 33.3 with w_pre and 41 with all three loaded where they are used (two more latencies a row
// with nothing else in flight).  8 columns a lane 34.1 us (half sectors a store of h').  Rows
// brought through shared memory by persistent blocks, two to four ahead, took 43 to 50 us.
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

// Four consecutive columns, as loaded
template <typename T>
struct Four;
template <>
struct Four<float> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w; }
};
template <>
struct Four<bf16> {
    uint2 u;
    __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
    }
};
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&x)[4]) {
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(x[0], x[1]), b1 = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
}

// Sum over the W warps of a row (each sum of a block in words of its own)
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += red[w];
    return t;
}

// A row on the W warps of a block: lane i of warp w holds columns 4 (i + 32 (w + W j)) .. + 3, j < N,
// so that a warp's loads and stores are of whole lines.
template <typename TY, typename TX, int W, int N>
__global__ void __launch_bounds__(32 * W) residual_norm_kernel(const NormArgs a) {
    __shared__ float red[2 * W];
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, c0 = 4 * threadIdx.x;
    const size_t row = static_cast<size_t>(t) * a.H;
    Four<TY> yv[N];
    float h[N][4];
    // the whole row in flight at once
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 128 * W * j;
        if (c < a.H) yv[j].load(static_cast<const TY*>(a.y) + row + c);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 128 * W * j;
        Four<float> e;
        if (c < a.H) {
            e.load(a.h_in + row + c);
            e.get(h[j]);
        }
    }
    const float* g = a.gate ? a.gate + (t / a.P) * a.gate_ld : nullptr;
    Four<TX> post[N], pre[N];
    Four<float> gt[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 128 * W * j;
        if (c >= a.H) continue;
        if (a.w_post) post[j].load(static_cast<const TX*>(a.w_post) + c);
        if (g) gt[j].load(g + c);
        if (a.x && a.w_pre) pre[j].load(static_cast<const TX*>(a.w_pre) + c);
    }
    float ry = 1.f, ss = 0.f;
    if (a.w_post) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (c0 + 128 * W * j >= a.H) continue;
            float y[4];
            yv[j].get(y);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss += y[i] * y[i];
        }
        ry = 1.0f / sqrtf(row_sum<W>(ss, red) / a.H + a.eps);
    }
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 128 * W * j;
        if (c >= a.H) continue;
        float y[4], w[4];
        yv[j].get(y);
        if (a.w_post) {
            post[j].get(w);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = y[i] * ry * w[i];
        }
        if (g) {
            gt[j].get(w);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[j][i] += a.res_scale * y[i];
            ss += h[j][i] * h[j][i];
        }
        store4(a.h_out + row + c, h[j]);
    }
    if (a.x == nullptr) return;
    const float rh = 1.0f / sqrtf(row_sum<W>(ss, red + W) / a.H + a.eps);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = c0 + 128 * W * j;
        if (c >= a.H) continue;
        float w[4];
        if (a.w_pre) {
            pre[j].get(w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] *= h[j][i] * rh;
        store4(static_cast<TX*>(a.x) + row + c, w);
    }
}

template <typename TY, typename TX>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    const dim3 grid(a.T);
    if (a.H <= 1024) return launch_pdl(residual_norm_kernel<TY, TX, 4, 2>, grid, dim3(128), 0, s, a);
    if (a.H <= 2048) return launch_pdl(residual_norm_kernel<TY, TX, 4, 4>, grid, dim3(128), 0, s, a);
    if (a.H <= 4096) return launch_pdl(residual_norm_kernel<TY, TX, 8, 4>, grid, dim3(256), 0, s, a);
    return launch_pdl(residual_norm_kernel<TY, TX, 16, 4>, grid, dim3(512), 0, s, a);
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
