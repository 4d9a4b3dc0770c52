// The gated delta rule in chunks of 64 tokens on tensor cores (bf16 queries, keys and values).
//
// With G_i the sum of g over a chunk's tokens up to i, S0 the state before it (both transposed here:
// S0 is [Dv][Dk]) and
//
//   A_ij = beta_i e^(G_i - G_j) k_i.k_j  (j < i),   X = (I + A)^-1,   P_ij = scale e^(G_i - G_j) q_i.k_j  (j <= i)
//
// the recurrence over the chunk is
//
//   R_i = beta_i (v_i - e^G_i S0 k_i),  U = X R,  o_i = scale e^G_i S0 q_i + sum_j P_ij U_j,
//   S = e^G_C S0 + sum_j e^(G_C - G_j) U_j k_j^T
//
// Two launches.  The first, parallel over (chunk, key head), has no states in it: it makes X and P.  The second walks
// the chunks of each (request, head) in order.  Its unit is a warp with 16 rows of the transposed state (16 of the
// Dv columns): rows need nothing from one another, so warps never meet.  All its products have those 16 rows
// as the MMA's M, so that each accumulator is the next product's A operand as it stands in the registers:
// S0 -> S0 K^T -> R -> R X^T = U -> U P^T and U K, without shared memory or lane exchanges in between; the B
// operands (K, Q, X, P) are shared-memory tiles that the first launch has laid out swizzled, brought by bulk copies.
//
// Accuracy.  States and sums are fp32.  An fp32 operand enters as the sum of two f16 numbers after a power of two that
// brings its row's largest element to 2^12: 22 bits, and 2^-37 of the row's largest for small elements.  Queries and
// keys are f16 numbers exactly after a power of two a row (elements below 2^-14 of the row's largest are off by 2^-25 of
// it at most), their norms are fp32 factors beside the products.  Only the output's products take one f16 number each
// for S0, U and P (2^-12, against the 2^-9 to which outputs are rounded).  Exponents of decays are differences of sums
// held in two floats, so strong decays before a token do not blur the weak ones after it.
#include "common.cuh"
#include "delta.h"
#include "kernels.h"
#include "launch.cuh"
#include "tc.cuh"

namespace moestep {
namespace {

constexpr int C = 64;             // tokens of a chunk
constexpr int kSquare = C * C * 2;  // bytes of a 64 x 64 f16 tile
constexpr int kVec = 2048;        // bytes of a chunk's factors
constexpr int kHeadBytes = 3 * kSquare + kVec;  // X high, X low, P, factors of one value head
// factors of a token (float [8][64])
enum { kA, kBeta, kB, kD, kTau, kPi, kGamma };

template <int DK>
struct Tile {
    static constexpr int kBytes = C * DK * 2;  // K or Q of a chunk: DK / 64 tiles of [64 tokens][64]
};

struct Scratch {
    char* qk;     // [R][chunks][Hk][K tile, Q tile]
    char* heads;  // [R][chunks][Hv][kHeadBytes]
    int chunks;
};

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
// two values as the sum of two f16 pairs
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack(x, y);
    const float2 h = unpack(hi);
    lo = pack(x - h.x, y - h.y);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // |e| <= 126
// a power of two that brings `most` to [2^to, 2^(to+1)); 1 for zeros and what is not finite
__device__ __forceinline__ float scale_to(float most, int to) {
    const int e = static_cast<int>(__float_as_uint(most) >> 23);
    if (most == 0.f || e == 255) return 1.f;
    return pow2(min(max(to + 127 - e, -126), 126));
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// byte offset of 16-byte piece c of row r in a tile of 128-byte rows
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// ---------------------------------------------------------------- first launch: X and P of every chunk
// A block has one chunk of one key head, four warps with 16 tokens each for the products k.k and q.k.  The inverse of
// I + A of a value head is 64 columns that 64 threads find by elimination, each holding its column in registers.
template <int DK>
struct PrepSmem {
    alignas(128) char k[Tile<DK>::kBytes];
    char q[Tile<DK>::kBytes];
    float at[2][C][C + 4];  // A transposed, then X, of two value heads
    float ck[C], cq[C];     // factors of the keys and queries
    float ghi[2][C], glo[2][C], beta[2][C];
};

template <int DK>
__global__ void __launch_bounds__(128) delta_prep_kernel(const DeltaArgs a, const Scratch w) {
    extern __shared__ __align__(128) char raw[];
    PrepSmem<DK>& sm = *reinterpret_cast<PrepSmem<DK>*>(raw);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int hk = blockIdx.x % a.Hk, chunk = blockIdx.x / a.Hk % w.chunks, r = blockIdx.x / a.Hk / w.chunks;
    int tokens, slot;
    if (!delta_request(a, r, false, tokens, slot)) return;
    const int m = min(C, tokens - chunk * C);
    if (m <= 0) return;
    const long long tok0 = 1ll * r * a.n + chunk * C;
    const long long unit = 1ll * r * w.chunks + chunk;

    // keys and queries: f16 after a power of two a row, DK / 8 lanes a row
    constexpr int L = DK / 8, RPW = 32 / L;
    char* to = w.qk + (unit * a.Hk + hk) * 2 * Tile<DK>::kBytes;
    const int sub = lane % L;
#pragma unroll 4
    for (int i = 0; i < 16 / RPW * 2; ++i) {
        const bool query = i >= 16 / RPW;
        const int t = warp * 16 + (i % (16 / RPW)) * RPW + lane / L;
        const bf16* p = static_cast<const bf16*>(query ? a.q : a.k) + (tok0 + t) * (query ? a.q_ld : a.k_ld) + hk * DK + 8 * sub;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t < m) x = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        float f[8], most = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(xs[j] << 16);
            f[2 * j + 1] = __uint_as_float(xs[j] & 0xffff0000u);
            most = fmaxf(most, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float up = scale_to(most, 0), down = 1.f / up;
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] *= up;
            ss += f[j] * f[j];
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (sub == 0) (query ? sm.cq : sm.ck)[t] = a.eps > 0.f ? 1.f / sqrtf(ss + a.eps * up * up) : down;
        const uint4 y = make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
        const int at = sub / 8 * (C * 128) + swz(t, sub % 8);
        *reinterpret_cast<uint4*>((query ? sm.q : sm.k) + at) = y;
        *reinterpret_cast<uint4*>(to + (query ? Tile<DK>::kBytes : 0) + at) = y;
    }
    __syncthreads();

    // k.k and q.k of this warp's 16 tokens with the tokens up to them
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[t][e] = qk[t][e] = 0.f;
    const uint32_t ks = tc::smem_addr(sm.k), qs = tc::smem_addr(sm.q);
    const int lr = lane & 7, lm = lane >> 3;  // row within a matrix, matrix of ldmatrix.x4
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        const int base = kt / 4 * (C * 128), c = kt % 4 * 2;
        uint32_t ak[4], aq[4];
        const int arow = warp * 16 + (lm & 1) * 8 + lr, acol = c + (lm >> 1);
        ldsm4(ak, ks + base + swz(arow, acol));
        ldsm4(aq, qs + base + swz(arow, acol));
#pragma unroll
        for (int t2 = 0; t2 < 4; ++t2) {
            if (t2 > warp) continue;
            uint32_t b[4];
            ldsm4(b, ks + base + swz(t2 * 16 + (lm >> 1) * 8 + lr, c + (lm & 1)));
            mma(kk[2 * t2], ak, b[0], b[1]);
            mma(kk[2 * t2 + 1], ak, b[2], b[3]);
            mma(qk[2 * t2], aq, b[0], b[1]);
            mma(qk[2 * t2 + 1], aq, b[2], b[3]);
        }
    }

    const int group = a.Hv / a.Hk, g4 = lane / 4, q4 = lane % 4;
    for (int v0 = 0; v0 < group; v0 += 2) {  // two value heads at a time, a pair of warps each
        const int pair = warp / 2, hv = hk * group + v0 + pair;
        const bool on = v0 + pair < group;
        char* head = w.heads + (unit * a.Hv + hv) * kHeadBytes;
        float* vec = reinterpret_cast<float*>(head + 3 * kSquare);
        if (v0) __syncthreads();  // at[] is free
        if (on && warp % 2 == 0) {
            // sums of g, in 64 bits: lane holds tokens 2 lane and 2 lane + 1
            double s[2];
            float be[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                float g = t < m ? a.g[(tok0 + t) * a.Hv + hv] : 0.f;
                if (g < -200.f) g = -200.f;  // e^-200 is 0 in fp32 as well
                s[i] = g;
                be[i] = t < m ? a.beta[(tok0 + t) * a.Hv + hv] : 0.f;
            }
            const double mine = s[0] + s[1];
            double run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += x;
            }
            const double all = __shfl_sync(0xffffffffu, run, 31);
            s[0] = run - mine + s[0];
            s[1] = run;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const float hi = static_cast<float>(s[i]);
                sm.ghi[pair][t] = hi;
                sm.glo[pair][t] = static_cast<float>(s[i] - hi);
                sm.beta[pair][t] = be[i];
                const float since = expf(hi), left = expf(static_cast<float>(all - s[i]));
                vec[kA * C + t] = since * sm.ck[t];
                vec[kBeta * C + t] = be[i];
                vec[kB * C + t] = since * sm.cq[t] * a.scale;
                vec[kD * C + t] = left * sm.ck[t];
            }
            if (lane == 0) vec[kGamma * C] = expf(static_cast<float>(all));
        }
        __syncthreads();
        // A (transposed) and P of both heads, from every warp's products
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (v0 + p >= group) continue;
            char* ph = w.heads + (unit * a.Hv + hk * group + v0 + p) * kHeadBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // rows g4 and g4 + 8 of the warp's 16
                const int i = warp * 16 + h * 8 + g4;
                const float gh = sm.ghi[p][i], gl = sm.glo[p][i], bc = sm.beta[p][i] * sm.ck[i], qc = sm.cq[i] * a.scale;
                float pv[16], most = 0.f;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 8 * t + 2 * q4 + e;
                        float x = 0.f;
                        if (t / 2 <= warp && j <= i) {
                            const float decay = expf((gh - sm.ghi[p][j]) + (gl - sm.glo[p][j])) * sm.ck[j];
                            x = decay * qc * qk[t][2 * h + e];
                            if (j < i) sm.at[p][j][i] = decay * bc * kk[t][2 * h + e];
                        }
                        pv[2 * t + e] = x;
                        most = fmaxf(most, fabsf(x));
                    }
                const float up = scale_to(quad_max(most), 0);
                if (q4 == 0) reinterpret_cast<float*>(ph + 3 * kSquare)[kPi * C + i] = 1.f / up;
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    *reinterpret_cast<uint32_t*>(ph + 2 * kSquare + swz(i, t) + 4 * q4) = pack(pv[2 * t] * up, pv[2 * t + 1] * up);
            }
        }
        __syncthreads();
        if (on) {
            // column c of X: x_i = (i == c) - sum_{j < i} A_ij x_j, every x_j taken off the later rows as it is final
            const int c = warp % 2 * 32 + lane;
            float x[C];
#pragma unroll
            for (int i = 0; i < C; ++i) x[i] = i == c ? 1.f : 0.f;
            const float(*at)[C + 4] = sm.at[pair];
            if (warp % 2 == 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
#pragma unroll
                    for (int i = j + 1; i < C; ++i) x[i] -= at[j][i] * x[j];
            }
#pragma unroll
            for (int j = 32; j < C - 1; ++j)
#pragma unroll
                for (int i = j + 1; i < C; ++i) x[i] -= at[j][i] * x[j];
            tc::named_bar_sync(1 + pair, 64);
#pragma unroll
            for (int i = 0; i < C; ++i) sm.at[pair][i][c] = x[i];
            tc::named_bar_sync(1 + pair, 64);
            const int i = c;  // now a row each
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < C; j += 4) {
                const float4 y = *reinterpret_cast<const float4*>(&sm.at[pair][i][j]);
                most = fmaxf(fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y))), fmaxf(fabsf(y.z), fabsf(y.w)));
            }
            const float up = scale_to(most, 10);
            vec[kTau * C + i] = 1.f / up;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(&sm.at[pair][i][8 * j]);
                const float4 z = *reinterpret_cast<const float4*>(&sm.at[pair][i][8 * j + 4]);
                uint4 hi, lo;
                split(y.x * up, y.y * up, hi.x, lo.x);
                split(y.z * up, y.w * up, hi.y, lo.y);
                split(z.x * up, z.y * up, hi.z, lo.z);
                split(z.z * up, z.w * up, hi.w, lo.w);
                *reinterpret_cast<uint4*>(head + swz(i, j)) = hi;
                *reinterpret_cast<uint4*>(head + kSquare + swz(i, j)) = lo;
            }
        }
    }
}

// ---------------------------------------------------------------- second launch: the states' walk
template <int DK, int W>
struct WalkSmem {
    static constexpr int kStages = 2;
    struct Stage {
        char k[Tile<DK>::kBytes];
        char q[Tile<DK>::kBytes];
        char head[kHeadBytes];
    };
    alignas(128) Stage st[kStages];
    char v[W][2][C * 32];  // a warp's 16 columns of the values, then of the outputs
    uint64_t full[kStages], empty[kStages];
    int abort;
};

template <int DK, int W>
__global__ void __launch_bounds__(32 * W, 1) delta_walk_kernel(const DeltaArgs a, const Scratch w) {
    extern __shared__ __align__(128) char raw[];
    using Smem = WalkSmem<DK, W>;
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    constexpr int NS = Smem::kStages;
    constexpr uint32_t kQk = 2 * Tile<DK>::kBytes;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g4 = lane / 4, q4 = lane % 4;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&sm.full[i], 1);
            tc::mbar_init(&sm.empty[i], W);
        }
        sm.abort = 0;
        tc::fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();
    const int slices = a.Dv / (16 * W);
    const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.Hv, r = blockIdx.x / slices / a.Hv;
    int tokens, slot;
    if (!delta_request(a, r, tid == 0 && slice == 0 && hv == 0, tokens, slot)) return;
    __syncthreads();
    const int hk = hv / (a.Hv / a.Hk), n_chunks = (tokens + C - 1) / C;
    const int row0 = (slice * W + warp) * 16;  // first of the warp's rows
    const long long tok0 = 1ll * r * a.n, unit0 = 1ll * r * w.chunks;

    auto fetch = [&](int c) {  // by one thread: chunk c into its stage
        typename Smem::Stage& s = sm.st[c % NS];
        uint64_t* bar = &sm.full[c % NS];
        tc::mbar_arrive_expect_tx(bar, kQk + kHeadBytes);
        bulk_load(tc::smem_addr(s.k), w.qk + ((unit0 + c) * a.Hk + hk) * kQk, kQk, bar);
        bulk_load(tc::smem_addr(s.head), w.heads + ((unit0 + c) * a.Hv + hv) * kHeadBytes, kHeadBytes, bar);
    };
    const uint32_t vs = tc::smem_addr(sm.v[warp]);
    auto at_v = [&](int t, int c) { return t * 32 + ((c ^ (t >> 2 & 1)) << 4); };
    auto fetch_v = [&](int c) {  // a warp's 16 columns of the values, zeros behind the request's tokens
        const bf16* p = static_cast<const bf16*>(a.v) + hv * a.Dv + row0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = i * 16 + lane / 2, tok = c * C + t;
            const bool on = tok < tokens;
            cp16(vs + (c & 1) * (C * 32) + at_v(t, lane & 1), p + (tok0 + (on ? tok : 0)) * a.v_ld + 8 * (lane & 1), on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (tid == 0)
        for (int c = 0; c < NS && c < n_chunks; ++c) fetch(c);
    if (n_chunks > 0) fetch_v(0);

    // rows g4 and g4 + 8 of the transposed state, columns 8 t + 2 q4 + {0, 1}; times sigma of the row
    float S[DK / 8][4], sigma[2] = {1.f, 1.f};
    const long long state0 = ((1ll * slot * a.Hv + hv) * a.Dv + row0 + g4) * DK + 2 * q4;
    const bool fresh = a.fresh && a.fresh[r];
#pragma unroll
    for (int t = 0; t < DK / 8; ++t) {
        float2 x = make_float2(0.f, 0.f), y = x;
        if (!fresh) {
            x = *reinterpret_cast<const float2*>(a.state + state0 + 8 * t);
            y = *reinterpret_cast<const float2*>(a.state + state0 + 8 * DK + 8 * t);
        }
        S[t][0] = x.x, S[t][1] = x.y, S[t][2] = y.x, S[t][3] = y.y;
    }

    const int lr = lane & 7, lm = lane >> 3;
    bool ok = true;
    int c = 0;
    for (; c < n_chunks; ++c) {
        const int st = c % NS;
        ok = tc::mbar_wait(&sm.full[st], (c / NS) & 1, &sm.abort, a.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (c + 1 < n_chunks) {
            fetch_v(c + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        typename Smem::Stage& s = sm.st[st];
        const uint32_t ks = tc::smem_addr(s.k), qs = tc::smem_addr(s.q), xs = tc::smem_addr(s.head);
        const float* vec = reinterpret_cast<const float*>(s.head + 3 * kSquare);
        const uint32_t vc = vs + (c & 1) * (C * 32);

        // S0 K^T (pairs of f16) and S0 Q^T (one f16)
        float most[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < DK / 8; ++t) {
            most[0] = fmaxf(most[0], fmaxf(fabsf(S[t][0]), fabsf(S[t][1])));
            most[1] = fmaxf(most[1], fmaxf(fabsf(S[t][2]), fabsf(S[t][3])));
        }
        float up[2], down[2];  // S is brought to 2^12 by `up`; products are brought back by `down`
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            most[h] = quad_max(most[h]);
            up[h] = scale_to(most[h], 12);
            down[h] = 1.f / up[h] * sigma[h];
            most[h] *= sigma[h];
        }
        float sk[8][4], sq[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sk[t][e] = sq[t][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                split(S[2 * kt + j][0] * up[0], S[2 * kt + j][1] * up[0], hi[2 * j], lo[2 * j]);
                split(S[2 * kt + j][2] * up[1], S[2 * kt + j][3] * up[1], hi[2 * j + 1], lo[2 * j + 1]);
            }
            const int base = kt / 4 * (C * 128), cc = kt % 4 * 2;
#pragma unroll
            for (int t2 = 0; t2 < 4; ++t2) {
                uint32_t b[4];
                const int off = base + swz(t2 * 16 + (lm >> 1) * 8 + lr, cc + (lm & 1));
                ldsm4(b, ks + off);
                mma(sk[2 * t2], hi, b[0], b[1]);
                mma(sk[2 * t2 + 1], hi, b[2], b[3]);
                mma(sk[2 * t2], lo, b[0], b[1]);
                mma(sk[2 * t2 + 1], lo, b[2], b[3]);
                ldsm4(b, qs + off);
                mma(sq[2 * t2], hi, b[0], b[1]);
                mma(sq[2 * t2 + 1], hi, b[2], b[3]);
            }
        }
        // R = beta (v - e^G S0 k), in place of S0 K^T
        float rmost[2] = {0.f, 0.f};
#pragma unroll
        for (int t2 = 0; t2 < 4; ++t2) {
            uint32_t vv[4];  // tokens 16 t2 ..: columns 0-7, 8-15; tokens 16 t2 + 8 ..: the same
            ldsm4_t(vv, vc + at_v(t2 * 16 + (lm >> 1) * 8 + lr, lm & 1));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * t2 + j;
                const float2 av = *reinterpret_cast<const float2*>(vec + kA * C + 8 * t + 2 * q4);
                const float2 be = *reinterpret_cast<const float2*>(vec + kBeta * C + 8 * t + 2 * q4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = vv[2 * j + h];
                    float& r0 = sk[t][2 * h];
                    float& r1 = sk[t][2 * h + 1];
                    r0 = be.x * (__uint_as_float(x << 16) - av.x * (r0 * down[h]));
                    r1 = be.y * (__uint_as_float(x & 0xffff0000u) - av.y * (r1 * down[h]));
                    rmost[h] = fmaxf(rmost[h], fmaxf(fabsf(r0), fabsf(r1)));
                }
            }
        }
        // U = X R
        float rup[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) rup[h] = scale_to(quad_max(rmost[h]), 12);
        float u[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[t][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                split(sk[2 * kt + j][0] * rup[0], sk[2 * kt + j][1] * rup[0], hi[2 * j], lo[2 * j]);
                split(sk[2 * kt + j][2] * rup[1], sk[2 * kt + j][3] * rup[1], hi[2 * j + 1], lo[2 * j + 1]);
            }
#pragma unroll
            for (int t2 = kt; t2 < 4; ++t2) {  // X is lower triangular
                uint32_t b[4], bl[4];
                const int off = swz(t2 * 16 + (lm >> 1) * 8 + lr, kt * 2 + (lm & 1));
                ldsm4(b, xs + off);
                ldsm4(bl, xs + kSquare + off);
                mma(u[2 * t2], hi, b[0], b[1]);
                mma(u[2 * t2 + 1], hi, b[2], b[3]);
                mma(u[2 * t2], lo, b[0], b[1]);
                mma(u[2 * t2 + 1], lo, b[2], b[3]);
                mma(u[2 * t2], hi, bl[0], bl[1]);
                mma(u[2 * t2 + 1], hi, bl[2], bl[3]);
            }
        }
        float umost[2] = {0.f, 0.f}, dmost[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float2 tau = *reinterpret_cast<const float2*>(vec + kTau * C + 8 * t + 2 * q4);
            const float2 dd = *reinterpret_cast<const float2*>(vec + kD * C + 8 * t + 2 * q4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float back = 1.f / rup[h];
                float& u0 = u[t][2 * h];
                float& u1 = u[t][2 * h + 1];
                u0 *= tau.x * back;
                u1 *= tau.y * back;
                umost[h] = fmaxf(umost[h], fmaxf(fabsf(u0), fabsf(u1)));
                dmost[h] = fmaxf(dmost[h], fmaxf(fabsf(u0 * dd.x), fabsf(u1 * dd.y)));
            }
        }
        // O = e^G scale S0 Q^T + U P^T
        float uup[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) uup[h] = scale_to(quad_max(umost[h]), 12);
        float o[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t hi[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                hi[2 * j] = pack(u[2 * kt + j][0] * uup[0], u[2 * kt + j][1] * uup[0]);
                hi[2 * j + 1] = pack(u[2 * kt + j][2] * uup[1], u[2 * kt + j][3] * uup[1]);
            }
#pragma unroll
            for (int t2 = kt; t2 < 4; ++t2) {
                uint32_t b[4];
                ldsm4(b, xs + 2 * kSquare + swz(t2 * 16 + (lm >> 1) * 8 + lr, kt * 2 + (lm & 1)));
                mma(o[2 * t2], hi, b[0], b[1]);
                mma(o[2 * t2 + 1], hi, b[2], b[3]);
            }
        }
        __syncwarp();  // the values have been read: their place takes the outputs
#pragma unroll
        for (int t2 = 0; t2 < 4; ++t2) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * t2 + j;
                const float2 b = *reinterpret_cast<const float2*>(vec + kB * C + 8 * t + 2 * q4);
                const float2 pi = *reinterpret_cast<const float2*>(vec + kPi * C + 8 * t + 2 * q4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float back = 1.f / uup[h];
                    const __nv_bfloat162 x =
                        __floats2bfloat162_rn(b.x * (sq[t][2 * h] * down[h]) + pi.x * (o[t][2 * h] * back),
                                              b.y * (sq[t][2 * h + 1] * down[h]) + pi.y * (o[t][2 * h + 1] * back));
                    y[2 * j + h] = *reinterpret_cast<const uint32_t*>(&x);
                }
            }
            stsm4_t(vc + at_v(t2 * 16 + (lm >> 1) * 8 + lr, lm & 1), y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
        {
            bf16* p = static_cast<bf16*>(a.out) + hv * a.Dv + row0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = i * 16 + lane / 2, tok = c * C + t;
                if (tok < tokens)
                    *reinterpret_cast<uint4*>(p + (tok0 + tok) * a.Hv * a.Dv + 8 * (lane & 1)) =
                        *reinterpret_cast<const uint4*>(sm.v[warp][c & 1] + at_v(t, lane & 1));
            }
        }
        __syncwarp();  // read before the next values are fetched into it
        // S = e^G_C S0 + U' K, U' = e^(G_C - G) U; S and U' share the row's new power of two
        const float gamma = vec[kGamma * C];
        float dup[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            dup[h] = scale_to(fmaxf(quad_max(dmost[h]), most[h] * gamma * 0x1p-8f), 12);
            const float f = gamma * sigma[h] * dup[h];
            sigma[h] = 1.f / dup[h];
#pragma unroll
            for (int t = 0; t < DK / 8; ++t) S[t][2 * h] *= f, S[t][2 * h + 1] *= f;
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 dd = *reinterpret_cast<const float2*>(vec + kD * C + 8 * (2 * kt + j) + 2 * q4);
                split(u[2 * kt + j][0] * dd.x * dup[0], u[2 * kt + j][1] * dd.y * dup[0], hi[2 * j], lo[2 * j]);
                split(u[2 * kt + j][2] * dd.x * dup[1], u[2 * kt + j][3] * dd.y * dup[1], hi[2 * j + 1], lo[2 * j + 1]);
            }
#pragma unroll
            for (int t2 = 0; t2 < DK / 16; ++t2) {
                uint32_t b[4];
                ldsm4_t(b, ks + t2 / 4 * (C * 128) + swz(kt * 16 + (lm & 1) * 8 + lr, t2 % 4 * 2 + (lm >> 1)));
                mma(S[2 * t2], hi, b[0], b[1]);
                mma(S[2 * t2 + 1], hi, b[2], b[3]);
                mma(S[2 * t2], lo, b[0], b[1]);
                mma(S[2 * t2 + 1], lo, b[2], b[3]);
            }
        }
        // the stage is free for chunk c + NS
        if (c + NS < n_chunks) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.empty[st]);
            if (tid == 0) {
                if (tc::mbar_wait(&sm.empty[st], (c / NS) & 1, &sm.abort, a.timeout_ns))
                    fetch(c + NS);
                else
                    *const_cast<volatile int*>(&sm.abort) = 1;  // every warp leaves at its next wait
            }
        }
    }
    if (!ok) {  // a wait ran out: record it, let the copies that were issued land, leave the state as it was
        if (lane == 0) {
            *const_cast<volatile int*>(&sm.abort) = 1;
            record_error(a.err, kErrTimeoutMma);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (tid == 0) {
            int zero = 0;
            for (int i = c; i < c + NS && i < n_chunks; ++i)
                tc::mbar_wait(&sm.full[i % NS], (i / NS) & 1, &zero, 1000000000ull);
        }
        return;
    }
    if (!a.state_out) return;
#pragma unroll
    for (int t = 0; t < DK / 8; ++t) {
        *reinterpret_cast<float2*>(a.state_out + state0 + 8 * t) = make_float2(S[t][0] * sigma[0], S[t][1] * sigma[0]);
        *reinterpret_cast<float2*>(a.state_out + state0 + 8 * DK + 8 * t) = make_float2(S[t][2] * sigma[1], S[t][3] * sigma[1]);
    }
}

template <int DK>
cudaError_t launch_prep(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    static int done[64];
    cudaError_t e = ensure_smem(delta_prep_kernel<DK>, sizeof(PrepSmem<DK>), done);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(1ll * a.R * w.chunks * a.Hk));
    return launch_pdl(delta_prep_kernel<DK>, grid, dim3(128), sizeof(PrepSmem<DK>), s, a, w);
}

template <int DK, int W>
cudaError_t launch_walk(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    static int done[64];
    cudaError_t e = ensure_smem(delta_walk_kernel<DK, W>, sizeof(WalkSmem<DK, W>), done);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.R * a.Hv * (a.Dv / (16 * W))));
    return launch_pdl(delta_walk_kernel<DK, W>, grid, dim3(32 * W), sizeof(WalkSmem<DK, W>), s, a, w);
}

template <int DK>
cudaError_t launch_chunks(const DeltaArgs& a, const Scratch& w, int sms, cudaStream_t s) {
    cudaError_t e = launch_prep<DK>(a, w, s);
    if (e != cudaSuccess) return e;
    count_launch();
    // as few warps a block as keep the multiprocessors busy: a block's tiles are shared by its warps
    const long long slices = 1ll * a.R * a.Hv * (a.Dv / 16);
    if (slices <= 2ll * sms) return launch_walk<DK, 2>(a, w, s);
    return launch_walk<DK, 4>(a, w, s);
}

size_t qk_bytes(const moestep_delta_dims& d, long long units) { return static_cast<size_t>(units) * d.Hk * 2 * C * d.Dk * 2; }

}  // namespace

bool delta_chunked(const moestep_delta_dims& d, int R, int n) { return d.dtype == MOESTEP_BF16 && n >= 64; }

size_t delta_chunk_bytes(const moestep_delta_dims& d, int R, int n) {
    if (!delta_chunked(d, R, n)) return 0;
    const long long units = 1ll * R * ((n + C - 1) / C);
    return qk_bytes(d, units) + static_cast<size_t>(units) * d.Hv * kHeadBytes;
}

cudaError_t launch_delta_chunks(const DeltaArgs& a, void* scratch, int sms, cudaStream_t s) {
    Scratch w;
    w.chunks = (a.n + C - 1) / C;
    w.qk = static_cast<char*>(scratch);
    const moestep_delta_dims d{a.Hk, a.Hv, a.Dk, a.Dv, a.n_slots, MOESTEP_BF16};
    w.heads = w.qk + qk_bytes(d, 1ll * a.R * w.chunks);
    return a.Dk == 128 ? launch_chunks<128>(a, w, sms, s) : launch_chunks<64>(a, w, sms, s);
}

}  // namespace moestep
