// The gated delta rule token by token, for a few tokens a request and for fp32, and the C entries
// of both forms.
//
//   S <- a S + b k (v - a S^T k)^T,  o = scale S^T q,  a = e^g
//
// The state is kept transposed, [Dv][Dk]: every row is a recurrence of its own (row j needs
// only v_j), so rows are spread over warps that never speak to each other.  Eight lanes share a row,
// Dk / 8 elements each, four rows a step of a warp.  Both products of a token are taken on the state
// before it: with p = S k, s = S q and c = k . q,
//
//   u = b (v - a p),  o = scale (a s + u c),  S <- a S + u k,
//
// so a token costs one round of lane exchanges (three steps for p and s together).  Queries, keys and
// the tokens' scalars are staged in shared memory, kTokens at a time.
//
// Bound: with one token the state's bytes, read and written once (128 requests of 32 heads of 128 x 128,
// 537 MB); with tens of tokens the chain of tokens.
#include <cmath>

#include "common.cuh"
#include "delta.h"
#include "kernels.h"
#include "launch.cuh"

namespace moestep {
namespace {

constexpr int kTokens = 16;  // staged at a time
constexpr int kWarps = 4;

// NR: rows of a lane group (a warp has 4 NR rows, a block kWarps * 4 NR)
template <typename T, int DK, int NR>
__global__ void __launch_bounds__(32 * kWarps) delta_recurrent_kernel(const DeltaArgs a) {
    constexpr int N = DK / 32;             // 16-byte pieces of a lane's share of a row
    constexpr int ROWS = kWarps * 4 * NR;  // rows of a block
    __shared__ float ks[kTokens][DK], qs[kTokens][DK];
    __shared__ float vs[kTokens][ROWS];
    __shared__ float gate[kTokens], rate[kTokens], kq[kTokens];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % 8;
    const int slices = a.Dv / ROWS;
    const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.Hv, r = blockIdx.x / slices / a.Hv;
    int tokens, slot;
    if (!delta_request(a, r, threadIdx.x == 0 && slice == 0 && hv == 0, tokens, slot)) return;
    const int row0 = slice * ROWS + warp * 4 * NR + lane / 8;  // + 4 i
    const long long state0 = (1ll * slot * a.Hv + hv) * a.Dv * DK + 4 * sub;
    float S[NR][N][4];
    const bool fresh = a.fresh && a.fresh[r];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!fresh) x = *reinterpret_cast<const float4*>(a.state + state0 + 1ll * (row0 + 4 * i) * DK + 32 * j);
            S[i][j][0] = x.x, S[i][j][1] = x.y, S[i][j][2] = x.z, S[i][j][3] = x.w;
        }
    const int hk = hv / (a.Hv / a.Hk);
    for (int t0 = 0; t0 < tokens; t0 += kTokens) {
        const int m = min(kTokens, tokens - t0);
        if (t0) __syncthreads();
        for (int t = warp; t < m; t += kWarps) {  // a warp stages a token
            const long long tok = 1ll * r * a.n + t0 + t;
            const T* kp = static_cast<const T*>(a.k) + tok * a.k_ld + hk * DK;
            const T* qp = static_cast<const T*>(a.q) + tok * a.q_ld + hk * DK;
            float kk[DK / 32], qq[DK / 32], sk = 0.f, sq = 0.f, c = 0.f;
#pragma unroll
            for (int j = 0; j < DK / 32; ++j) {
                kk[j] = to_f32(kp[lane + 32 * j]);
                qq[j] = to_f32(qp[lane + 32 * j]);
                sk += kk[j] * kk[j];
                sq += qq[j] * qq[j];
                c += kk[j] * qq[j];
            }
            sk = warp_sum(sk);
            sq = warp_sum(sq);
            c = warp_sum(c);
            const float rk = a.eps > 0.f ? 1.0f / sqrtf(sk + a.eps) : 1.f, rq = a.eps > 0.f ? 1.0f / sqrtf(sq + a.eps) : 1.f;
#pragma unroll
            for (int j = 0; j < DK / 32; ++j) {
                ks[t][lane + 32 * j] = kk[j] * rk;
                qs[t][lane + 32 * j] = qq[j] * rq;
            }
            if (lane == 0) {
                gate[t] = expf(a.g[tok * a.Hv + hv]);
                rate[t] = a.beta[tok * a.Hv + hv];
                kq[t] = c * rk * rq;
            }
            for (int j = lane; j < ROWS; j += 32)
                vs[t][j] = to_f32(static_cast<const T*>(a.v)[tok * a.v_ld + hv * a.Dv + slice * ROWS + j]);
        }
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            float p[NR], s[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) p[i] = s[i] = 0.f;
            float kk[N][4];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&ks[t][32 * j + 4 * sub]);
                const float4 y = *reinterpret_cast<const float4*>(&qs[t][32 * j + 4 * sub]);
                kk[j][0] = x.x, kk[j][1] = x.y, kk[j][2] = x.z, kk[j][3] = x.w;
                const float qq[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[i] += S[i][j][e] * kk[j][e];
                        s[i] += S[i][j][e] * qq[e];
                    }
            }
#pragma unroll
            for (int o = 4; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    p[i] += __shfl_xor_sync(0xffffffffu, p[i], o);
                    s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
                }
            const float al = gate[t], be = rate[t], c = kq[t];
            T* out = static_cast<T*>(a.out) + ((1ll * r * a.n + t0 + t) * a.Hv + hv) * a.Dv + row0;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float u = be * (vs[t][warp * 4 * NR + lane / 8 + 4 * i] - al * p[i]);
                if (sub == 0) out[4 * i] = from_f32<T>(a.scale * (al * s[i] + u * c));
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][j][e] = al * S[i][j][e] + u * kk[j][e];
            }
        }
    }
    if (!a.state_out) return;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
            *reinterpret_cast<float4*>(a.state_out + state0 + 1ll * (row0 + 4 * i) * DK + 32 * j) =
                make_float4(S[i][j][0], S[i][j][1], S[i][j][2], S[i][j][3]);
}

template <typename T, int DK>
cudaError_t launch_rows(const DeltaArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(1ll * a.R * a.Hv * (a.Dv / (kWarps * 8))));
    return launch_pdl(delta_recurrent_kernel<T, DK, 2>, grid, dim3(32 * kWarps), 0, s, a);
}

int check_delta(const moestep_delta_dims* dd, int R, int n) {
    const int rc = check_delta_dims(dd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n <= 0) return MOESTEP_EINVAL;
    if (1ll * R * dd->Hv > (1 << 24)) return MOESTEP_EUNSUPPORTED;
    if (1ll * R * n > (1ll << 31) - 1 || (1ll * R * n + 64ll * R) * dd->Hk > 64 * ((1ll << 31) - 1)) return MOESTEP_EUNSUPPORTED;
    return MOESTEP_OK;
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs& a, int dtype, cudaStream_t s) {
    if (dtype == MOESTEP_F32) return a.Dk == 128 ? launch_rows<float, 128>(a, s) : launch_rows<float, 64>(a, s);
    return a.Dk == 128 ? launch_rows<bf16, 128>(a, s) : launch_rows<bf16, 64>(a, s);
}

}  // namespace moestep

extern "C" int moestep_delta_workspace_size(const moestep_delta_dims* dd, int R, int n, size_t* bytes) {
    using namespace moestep;
    const int rc = check_delta(dd, R, n);
    if (rc != MOESTEP_OK) return rc;
    if (bytes == nullptr) return MOESTEP_EINVAL;
    *bytes = kKvHeader + delta_chunk_bytes(*dd, R, n);
    return MOESTEP_OK;
}

extern "C" int block_delta_rule(const moestep_delta_dims* dd, int R, int n, const void* q, long long q_ld, const void* k,
                                long long k_ld, const void* v, long long v_ld, const float* g, const float* beta,
                                const int32_t* length, const int32_t* slot, const uint8_t* fresh, const float* state,
                                float* state_out, float scale, float qk_eps, void* out, void* ws, size_t ws_bytes,
                                void* stream) {
    using namespace moestep;
    int rc = check_delta(dd, R, n);
    if (rc != MOESTEP_OK) return rc;
    if (!g || !beta || !state || !out || !std::isfinite(scale) || !std::isfinite(qk_eps) || qk_eps < 0.f)
        return MOESTEP_EINVAL;
    if (!slot && R > dd->n_slots) return MOESTEP_EINVAL;
    if ((rc = check_kv_rows(q, q_ld, 1ll * dd->Hk * dd->Dk, dd->dtype)) != MOESTEP_OK) return rc;
    if ((rc = check_kv_rows(k, k_ld, 1ll * dd->Hk * dd->Dk, dd->dtype)) != MOESTEP_OK) return rc;
    if ((rc = check_kv_rows(v, v_ld, 1ll * dd->Hv * dd->Dv, dd->dtype)) != MOESTEP_OK) return rc;
    for (const void* p : {static_cast<const void*>(state), static_cast<const void*>(state_out), static_cast<const void*>(out)})
        if (!kv_aligned16(p)) return MOESTEP_EALIGN;
    for (const void* p : {static_cast<const void*>(g), static_cast<const void*>(beta), static_cast<const void*>(length),
                          static_cast<const void*>(slot)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return MOESTEP_EALIGN;
    if ((rc = check_kv_ws(ws, ws_bytes, kKvHeader + delta_chunk_bytes(*dd, R, n))) != MOESTEP_OK) return rc;
    int sms = 0;
    if ((rc = device_ok(&sms)) != MOESTEP_OK) return rc;
    const DeltaArgs a{q,         k,         v,     q_ld,   k_ld,   v_ld,          g,     beta,   length, slot,
                      fresh,     state,     state_out, out, static_cast<int*>(ws), R,   n,      dd->Hk, dd->Hv,
                      dd->Dk,    dd->Dv,    dd->n_slots, scale, qk_eps,    wait_timeout_ns()};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    const cudaError_t e = delta_chunked(*dd, R, n) ? launch_delta_chunks(a, static_cast<char*>(ws) + kKvHeader, sms, s)
                                                   : launch_delta_recurrent(a, dd->dtype, s);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}
