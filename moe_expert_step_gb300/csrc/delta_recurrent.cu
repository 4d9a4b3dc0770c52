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
// the tokens' scalars are staged in shared memory, Stage::kTokens at a time in two buffers.
//
// Bound: with one token the state's bytes, read and written once (128 requests of 32 heads of 128 x 128, 540 MB:
// 80 us, 6.7 TB/s, 99 % of the copy rate); with tens of tokens the chain of a token: its queries and keys come
// from shared memory to every lane group (4 KB a warp), then the sums over lanes.  77 fp32 tokens of 3 requests of 4 heads
// of 64 x 64: 15.9 us in a graph, 200 ns a token.
#include <cmath>

#include "common.cuh"
#include "delta.h"
#include "kernels.h"
#include "launch.cuh"

namespace moestep {
namespace {

constexpr int kWarps = 4;
// Rows of a lane group (a warp has 4 NR rows, a block kWarps * 4 NR), which share the reads of a token.  us with one / two /
// four of them: 12 heads of 64 x 64, 77 fp32 tokens 16.3 / 15.9 / 23.3; 32 heads of 128 x 128, 31 tokens 13.9 / 13.5 / 16.6,
// 16 requests of that 103 / 73 / 79.
constexpr int NR = 2;

// N pieces of four elements, 32 apart
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float (&x)[N][4]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if constexpr (sizeof(T) == 4) {
            const float4 y = __ldg(reinterpret_cast<const float4*>(p + 32 * j));
            x[j][0] = y.x, x[j][1] = y.y, x[j][2] = y.z, x[j][3] = y.w;
        } else {
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(p + 32 * j));
            x[j][0] = __uint_as_float(y.x << 16), x[j][1] = __uint_as_float(y.x & 0xffff0000u);
            x[j][2] = __uint_as_float(y.y << 16), x[j][3] = __uint_as_float(y.y & 0xffff0000u);
        }
    }
}

// One token of a head for the lane group of a row: everything that does not depend on the state
template <typename T, int DK>
struct Staged {
    static constexpr int kTokens = 16;  // at a time
    float k[kTokens][DK], q[kTokens][DK];
    float gate[kTokens], rate[kTokens], kq[kTokens];
};

__device__ __forceinline__ float inverse_norm(float ss, float eps) { return eps > 0.f ? 1.0f / sqrtf(ss + eps) : 1.f; }

__device__ __forceinline__ float decay(float g) { return fabsf(g) < 0.25f ? 1.f + grown(g) : expf(g); }

// ONE: a token a request, nothing is staged and each warp forms the token's sums itself
template <typename T, int DK, bool ONE>
__global__ void __launch_bounds__(32 * kWarps) delta_recurrent_kernel(const DeltaArgs a) {
    constexpr int N = DK / 32;             // 16-byte pieces of a lane's share of a row
    constexpr int ROWS = kWarps * 4 * NR;  // rows of a block
    using Stage = Staged<T, DK>;
    __shared__ Stage sm[ONE ? 1 : 2];
    __shared__ float vs[ONE ? 1 : 2][Stage::kTokens][ROWS];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % 8;
    const int slices = a.Dv / ROWS;
    const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.Hv, r = blockIdx.x / slices / a.Hv;
    int tokens, slot;
    if (!delta_request(a, r, threadIdx.x == 0 && slice == 0 && hv == 0, tokens, slot)) return;
    const int hk = hv / (a.Hv / a.Hk);
    const long long tok0 = 1ll * r * a.n;
    const T* const kp = static_cast<const T*>(a.k) + tok0 * a.k_ld + hk * DK;
    const T* const qp = static_cast<const T*>(a.q) + tok0 * a.q_ld + hk * DK;
    const T* const vp = static_cast<const T*>(a.v) + tok0 * a.v_ld + hv * a.Dv + slice * ROWS;
    const int row = warp * 4 * NR + lane / 8;  // + 4 i, of the block's
    const long long state0 = ((1ll * slot * a.Hv + hv) * a.Dv + slice * ROWS + row) * DK + 4 * sub;
    float S[NR][N][4];
    const bool fresh = a.fresh && a.fresh[r];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!fresh) x = *reinterpret_cast<const float4*>(a.state + state0 + 4 * i * DK + 32 * j);
            S[i][j][0] = x.x, S[i][j][1] = x.y, S[i][j][2] = x.z, S[i][j][3] = x.w;
        }
    T* const out = static_cast<T*>(a.out) + (tok0 * a.Hv + hv) * a.Dv + slice * ROWS + row;
    // a token of the lane group's rows, from its key and query and their scalars
    auto step = [&](const float(&kk)[N][4], const float(&qq)[N][4], float al, float be, float c, const float(&v)[NR], T* o) {
        float p[NR], s[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            p[i] = s[i] = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[i] += S[i][j][e] * kk[j][e];
                    s[i] += S[i][j][e] * qq[j][e];
                }
        }
#pragma unroll
        for (int m = 4; m; m >>= 1)
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                p[i] += __shfl_xor_sync(0xffffffffu, p[i], m);
                s[i] += __shfl_xor_sync(0xffffffffu, s[i], m);
            }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float u = be * (v[i] - al * p[i]);
            if (sub == 0) o[4 * i] = from_f32<T>(a.scale * (al * s[i] + u * c));
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][j][e] = al * S[i][j][e] + u * kk[j][e];
        }
    };
    if constexpr (ONE) {
        if (tokens > 0) {
            float kk[N][4], qq[N][4], sk = 0.f, sq = 0.f, c = 0.f, v[NR];
            load_row<T, N>(kp + 4 * sub, kk);
            load_row<T, N>(qp + 4 * sub, qq);
#pragma unroll
            for (int i = 0; i < NR; ++i) v[i] = to_f32(vp[row + 4 * i]);
            const float al = decay(a.g[tok0 * a.Hv + hv]), be = a.beta[tok0 * a.Hv + hv];
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sk += kk[j][e] * kk[j][e];
                    sq += qq[j][e] * qq[j][e];
                    c += kk[j][e] * qq[j][e];
                }
#pragma unroll
            for (int m = 4; m; m >>= 1) {
                sk += __shfl_xor_sync(0xffffffffu, sk, m);
                sq += __shfl_xor_sync(0xffffffffu, sq, m);
                c += __shfl_xor_sync(0xffffffffu, c, m);
            }
            const float rk = inverse_norm(sk, a.eps), rq = inverse_norm(sq, a.eps);
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) kk[j][e] *= rk, qq[j][e] *= rq;
            step(kk, qq, al, be, c * rk * rq, v, out);
        }
    } else {
        // a warp stages four tokens of kTokens, eight lanes each; the next ones while these are computed
        auto stage = [&](int t0, int which) {
            Stage& s = sm[which];
            const int t = warp * 4 + lane / 8;
            if (t0 + t < tokens) {
                float kk[N][4], qq[N][4], sk = 0.f, sq = 0.f, c = 0.f;
                load_row<T, N>(kp + (t0 + t) * a.k_ld + 4 * sub, kk);
                load_row<T, N>(qp + (t0 + t) * a.q_ld + 4 * sub, qq);
                float v[ROWS / 8];
#pragma unroll
                for (int i = 0; i < ROWS / 8; ++i) v[i] = to_f32(vp[(t0 + t) * a.v_ld + sub + 8 * i]);
                const float g = a.g[(tok0 + t0 + t) * a.Hv + hv], be = a.beta[(tok0 + t0 + t) * a.Hv + hv];
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sk += kk[j][e] * kk[j][e];
                        sq += qq[j][e] * qq[j][e];
                        c += kk[j][e] * qq[j][e];
                    }
                const unsigned group = 0xffu << (lane & 24);
#pragma unroll
                for (int m = 4; m; m >>= 1) {
                    sk += __shfl_xor_sync(group, sk, m);
                    sq += __shfl_xor_sync(group, sq, m);
                    c += __shfl_xor_sync(group, c, m);
                }
                const float rk = inverse_norm(sk, a.eps), rq = inverse_norm(sq, a.eps);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    *reinterpret_cast<float4*>(&s.k[t][32 * j + 4 * sub]) =
                        make_float4(kk[j][0] * rk, kk[j][1] * rk, kk[j][2] * rk, kk[j][3] * rk);
                    *reinterpret_cast<float4*>(&s.q[t][32 * j + 4 * sub]) =
                        make_float4(qq[j][0] * rq, qq[j][1] * rq, qq[j][2] * rq, qq[j][3] * rq);
                }
#pragma unroll
                for (int i = 0; i < ROWS / 8; ++i) vs[which][t][sub + 8 * i] = v[i];
                if (sub == 0) {
                    s.gate[t] = decay(g);
                    s.rate[t] = be;
                    s.kq[t] = c * rk * rq;
                }
            }
        };
        stage(0, 0);
        __syncthreads();
#pragma unroll 1
        for (int t0 = 0; t0 < tokens; t0 += Stage::kTokens) {
            const int which = t0 / Stage::kTokens & 1, m = min(Stage::kTokens, tokens - t0);
            const Stage& s = sm[which];
            if (t0 + Stage::kTokens < tokens) stage(t0 + Stage::kTokens, which ^ 1);
#pragma unroll 1
            for (int t = 0; t < m; ++t) {
                float kk[N][4], qq[N][4], v[NR];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(&s.k[t][32 * j + 4 * sub]);
                    const float4 y = *reinterpret_cast<const float4*>(&s.q[t][32 * j + 4 * sub]);
                    kk[j][0] = x.x, kk[j][1] = x.y, kk[j][2] = x.z, kk[j][3] = x.w;
                    qq[j][0] = y.x, qq[j][1] = y.y, qq[j][2] = y.z, qq[j][3] = y.w;
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) v[i] = vs[which][t][row + 4 * i];
                step(kk, qq, s.gate[t], s.rate[t], s.kq[t], v, out + static_cast<long long>(t0 + t) * a.Hv * a.Dv);
            }
            __syncthreads();
        }
    }
    if (!a.state_out) return;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
            *reinterpret_cast<float4*>(a.state_out + state0 + 4 * i * DK + 32 * j) = make_float4(S[i][j][0], S[i][j][1], S[i][j][2], S[i][j][3]);
}

template <typename T, int DK, bool ONE>
cudaError_t launch_rows(const DeltaArgs& a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(1ll * a.R * a.Hv * (a.Dv / (kWarps * 4 * NR))));
    return launch_pdl(delta_recurrent_kernel<T, DK, ONE>, grid, dim3(32 * kWarps), 0, s, a);
}

template <typename T, int DK>
cudaError_t launch_dk(const DeltaArgs& a, cudaStream_t s) {
    if (a.n == 1) return launch_rows<T, DK, true>(a, s);
    return launch_rows<T, DK, false>(a, s);
}

int check_delta(const moestep_delta_dims* dd, int R, int n) {
    const int rc = check_delta_dims(dd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n <= 0) return MOESTEP_EINVAL;
    if (1ll * R * dd->Hv > (1 << 24)) return MOESTEP_EUNSUPPORTED;
    if (n > (1 << 30) || 1ll * R * n > (1ll << 31) - 1 || (1ll * R * n + 64ll * R) * dd->Hk > 64 * ((1ll << 31) - 1)) return MOESTEP_EUNSUPPORTED;
    return MOESTEP_OK;
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs& a, int dtype, cudaStream_t s) {
    if (dtype == MOESTEP_F32) return a.Dk == 128 ? launch_dk<float, 128>(a, s) : launch_dk<float, 64>(a, s);
    return a.Dk == 128 ? launch_dk<bf16, 128>(a, s) : launch_dk<bf16, 64>(a, s);
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
    // blocks read all of a head's queries, keys and states while others write theirs
    if (out == q || out == k || out == state || out == state_out) return MOESTEP_EINVAL;
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
