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
// the chunks of each (request, head) in order.  Its unit is a slice of 16 rows of the transposed state (16 of the Dv
// columns): rows need nothing from one another.  All its products have those 16 rows as the MMA's M, so that an
// accumulator is the next product's A operand as it stands in the registers, S0 -> S0 K^T -> R -> R X^T = U -> U P^T and
// U K; the B operands (K, Q, X, P) are tiles that the first launch has laid out for ldmatrix, brought by bulk copies.
// (On mma.sync: with few heads the chain counts, and every link of it would pass through tensor memory on tcgen05.  Many heads
// of 128 values are walked there, in delta_heads.cu.)
//
// 8192 tokens of 16 and 32 heads of 128: 60 and 296 us (354 together; 206 MB that have to be moved, 30 us); 8 requests of up
// to 4096 tokens: 140 and 300 us (517 MB, 76 us).
//
// Accuracy.  States and sums are fp32.  An fp32 operand enters as the sum of two f16 numbers after a power of two that
// brings its row's largest element to 2^12: 22 bits, and 2^-37 of the row's largest for small elements.  Queries and
// keys are f16 numbers exactly after a power of two a row (elements below 2^-14 of the row's largest are off by 2^-25 of
// it at most), their norms are fp32 factors beside the products.  Only the output's products take one f16 number each
// for S0, U and P (2^-12, against the 2^-9 to which outputs are rounded).  Exponents of decays are differences of sums
// held in two floats, so strong decays before a token do not blur the weak ones after it.
#include "common.cuh"
#include "delta_chunk.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc.cuh"

#include <type_traits>

namespace moestep {
using namespace delta;
namespace {

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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the first product of a sum
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
        "%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool FIRST>
__device__ __forceinline__ void mma_(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FIRST)
        mma0(d, a, b0, b1);
    else
        mma(d, a, b0, b1);
}
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// x^-1/2, rsqrtf and a step of Newton's iteration (1 / sqrtf in its place: 16 blocks of 32 tokens 43.9 -> 44.2 us)
__device__ __forceinline__ float inverse_root(float x) {
    const float y = rsqrtf(x);
    return x < 3e38f ? y * (1.5f - 0.5f * x * y * y) : 0.f;
}
// Factor that divides a row by sqrt(|x|^2 + eps), of elements that are `up` times the row's, their squares' sum ss: (ss +
// eps up^2)^-1/2.  ss is 2^9 at most, so for rows so small that eps up^2 leaves fp32's range eps is all that counts.
__device__ __forceinline__ float inverse_norm(float ss, float eps, float up) {
    const float more = eps * up * up;
    return more < 1e38f ? inverse_root(ss + more) : inverse_root(eps) * inverse(up);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

__device__ __forceinline__ constexpr int below(int bi, int bj) { return (bi * (bi - 1) / 2 + bj) * 512; }  // of one without its diagonal
// Values and outputs of a slice: 16 rows of 32 bytes, whose halves change places in every second group of four rows
__device__ __forceinline__ int in_slice(int r, int c) { return r * 32 + ((c ^ (r >> 2 & 1)) << 4); }
// lanes' places for ldmatrix.x4: with the 8 x 8 matrices in the order of the rows (B operands; A operands transposed), and
// in the order of the columns (A operands; B operands transposed)
__device__ __forceinline__ int by_rows(int lane) { return in_block((lane >> 4) * 8 + (lane & 7), lane >> 3 & 1); }
__device__ __forceinline__ int slice_by_rows(int lane) { return in_slice((lane >> 4) * 8 + (lane & 7), lane >> 3 & 1); }
__device__ __forceinline__ int tile_by_rows(int lane) { return in_tile((lane >> 4) * 8 + (lane & 7), lane >> 3 & 1); }
__device__ __forceinline__ int tile_by_cols(int lane) { return in_tile((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4); }

// ---------------------------------------------------------------- first launch: X and P of every chunk
// A block has one chunk of one key head, four warps with 16 tokens each for the products k.k and q.k.  Bound by latency: 38 %
// of the issue slots and 2.5 to 3.2 TB/s with four blocks a multiprocessor.
//
// Rows of keys are brought to [1, 2) by a power of two and their norms left out: with c_i the factor between key and row,
// the system is solved for U' = c U, whose matrix A'_ij = beta_i c_i^2 e^(G_i - G_j) k_i.k_j has entries of the size of 1
// whatever the keys' scale (up to 23 for normalised ones, as long as beta |k|^2 <= 2 without).
//
// X = (I + A')^-1 of a value head by a pair of warps: the 16 x 16 blocks on the diagonal by elimination in fp32, a column
// a thread; then blocks of 32 and of 64 from X_BA = -X_B A_BA X_A, on tensor cores with operands of two f16
// numbers.  Computed transposed, (X_A^T A_BA^T) X_B^T, the first product is the second one's A operand in place.
// (64 steps of elimination in registers, unrolled, ran at the speed of their instruction fetches: 208 us for 8192 tokens
// of 32 heads; in loops of 16 rows 150 us; by blocks 91 us, now 60 us.)
template <int DK>
struct PrepSmem {
    union {
        struct {
            alignas(128) char k[Tile<DK>::kBytes];  // K and Q as they go to global memory
            char q[Tile<DK>::kBytes];
        };
        // then of two value heads: X high, X low, factors, P, factors, as they go to global memory.  Before X is there,
        // its place has the tokens' sums of g and beta c^2.
        char x[2][kHeadBytes];
    };
    struct Blocks {
        char ahi[6 * 512], alo[6 * 512];  // A' below its diagonal blocks
        float at[4][16][16];              // the diagonal blocks, transposed
    } blocks[2];
    float ck[C], cq[C];  // factors of the keys and queries
};
struct Gates {  // in x
    float ghi[C], glo[C], beta[C];
};

// A number as the sum of two floats, of which the high one is the nearest float: about 2^-46 of the larger term is lost a sum
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ Sum sum_of(float a, float b) {  // a b
    const float p = a * b;
    return Sum{p, fmaf(a, b, -p)};
}
__device__ __forceinline__ Sum operator+(const Sum& a, const Sum& b) {
    const float s = a.hi + b.hi, v = s - a.hi;
    const float e = (a.hi - (s - v)) + (b.hi - v) + (a.lo + b.lo);
    const float h = s + e;
    return Sum{h, e - (h - s)};
}

__device__ __forceinline__ float exp2_fast(float x) {  // (2^-22 of the value; to 0 below 2^-126)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d += a b for operands of two f16 numbers (the product of the low ones is below the others' error), two tiles at a time
template <bool FIRST>
__device__ __forceinline__ void mma3(float (&d0)[4], float (&d1)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                     const uint32_t (&b)[4], const uint32_t (&bl)[4]) {
    mma_<FIRST>(d0, hi, b[0], b[1]);
    mma_<FIRST>(d1, hi, b[2], b[3]);
    mma(d0, lo, b[0], b[1]);
    mma(d1, lo, b[2], b[3]);
    mma(d0, hi, bl[0], bl[1]);
    mma(d1, hi, bl[2], bl[3]);
}

// Blocks [bn, bn + NB) x m of X, below the diagonal, from the finished ones: X_A is block rows and columns from ma on,
// X_B from bn on, NB each; m is one of X_A's block columns.
template <int NB>
__device__ __forceinline__ void merge_blocks(uint32_t xh, uint32_t xl, uint32_t ah, uint32_t al, int ma, int m, int bn) {
    const int lane = threadIdx.x % 32, rows = by_rows(lane);
    float d[2 * NB][4];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[t][e] = 0.f;
    // T^T [m][n] = sum_k X_A[k][m] A_BA[n][k]: block rows k before m are zero
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
        const int k = ma + kb;
        if (k < m) continue;
        uint32_t a[4], l[4];
        ldsm4_t(a, xh + tri(k, m) + rows);
        ldsm4_t(l, xl + tri(k, m) + rows);
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            uint32_t b[4], bl[4];
            ldsm4(b, ah + below(bn + t, k) + rows);
            ldsm4(bl, al + below(bn + t, k) + rows);
            mma3<false>(d[2 * t], d[2 * t + 1], a, l, b, bl);
        }
    }
    // X_BA^T [m][n] = - sum_k T^T[m][k] X_B[n][k]
    float y[2 * NB][4];
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[t][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < NB; ++kb) {
        uint32_t a[4], l[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            split(-d[2 * kb + j][0], -d[2 * kb + j][1], a[2 * j], l[2 * j]);
            split(-d[2 * kb + j][2], -d[2 * kb + j][3], a[2 * j + 1], l[2 * j + 1]);
        }
#pragma unroll
        for (int t = kb; t < NB; ++t) {
            uint32_t b[4], bl[4];
            ldsm4(b, xh + tri(bn + t, bn + kb) + rows);
            ldsm4(bl, xl + tri(bn + t, bn + kb) + rows);
            mma3<false>(y[2 * t], y[2 * t + 1], a, l, b, bl);
        }
    }
#pragma unroll
    for (int t = 0; t < NB; ++t) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) split(y[2 * t + j][2 * h], y[2 * t + j][2 * h + 1], hi[2 * j + h], lo[2 * j + h]);
        stsm4_t(xh + tri(bn + t, m) + rows, hi[0], hi[1], hi[2], hi[3]);
        stsm4_t(xl + tri(bn + t, m) + rows, lo[0], lo[1], lo[2], lo[3]);
    }
}

// 2^x of a chunk's decay
__device__ __forceinline__ float chunk_decay(float x) { return fabsf(x) < 0.25f ? 1.f + grown(x * 0.6931471805599453f) : exp2f(x); }

// BRIEF: at most 32 tokens a request, whose products are half as many rows and columns
template <int DK, bool BRIEF>
__global__ void __launch_bounds__(128, 4) delta_prep_kernel(const DeltaArgs a, const Scratch w) {
    extern __shared__ __align__(128) char raw[];
    PrepSmem<DK>& sm = *reinterpret_cast<PrepSmem<DK>*>(raw);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, pair = warp / 2;
    const int hk = blockIdx.x % a.Hk, chunk = blockIdx.x / a.Hk % w.chunks, r = blockIdx.x / a.Hk / w.chunks;
    const long long tok0 = 1ll * r * a.n + chunk * C;
    // A first chunk's rows are on their way before it is known how many are tokens (they are the request's memory in any
    // case); later ones, of which ragged batches have many without a token, wait for it.
    int tokens = a.n, slot = 0;
    if (chunk && !delta_request(a, r, false, tokens, slot)) return;
    const int there = tokens - chunk * C;
    if (there <= 0) return;
    const long long unit = 1ll * r * w.chunks + chunk;
    const int group = a.Hv / a.Hk;

    // keys and queries: f16 after a power of two a row, four lanes a row
    constexpr int PIECES = DK / 32;  // 16-byte pieces of a lane: 64 bytes of a row together
    constexpr int EIGHTS = BRIEF ? 1 : 2;  // of a warp's tokens
    const int sub = (lane & 1) + (lane >> 4) * 2, row = lane >> 1 & 7;  // (a load's and a store's eight lanes: whole sectors, few conflicts)
    uint4 in[2][EIGHTS][PIECES];
#pragma unroll
    for (int i = 0; i < EIGHTS; ++i) {
        const int t = (warp * EIGHTS + i) * 8 + row;
        const bf16* kp = static_cast<const bf16*>(a.k) + (tok0 + t) * a.k_ld + hk * DK + 8 * sub;
        const bf16* qp = static_cast<const bf16*>(a.q) + (tok0 + t) * a.q_ld + hk * DK + 8 * sub;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            in[0][i][j] = in[1][i][j] = make_uint4(0, 0, 0, 0);
            if (t < there) {
                in[0][i][j] = __ldg(reinterpret_cast<const uint4*>(kp + 32 * j));
                in[1][i][j] = __ldg(reinterpret_cast<const uint4*>(qp + 32 * j));
            }
        }
    }
    if (!chunk && !delta_request(a, r, false, tokens, slot)) return;
    const int m = min(C, tokens - chunk * C);
    if (m <= 0) return;
    float gs[2], be[2];  // of the first two value heads, by an even warp each: tokens 2 lane and 2 lane + 1
    auto load_gates = [&](int v) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const bool on = v < group && t < m;
            gs[i] = on ? a.g[(tok0 + t) * a.Hv + hk * group + v] : 0.f;
            be[i] = on ? a.beta[(tok0 + t) * a.Hv + hk * group + v] : 0.f;
        }
    };
    if (warp % 2 == 0) load_gates(pair);
#pragma unroll
    for (int i = 0; i < EIGHTS; ++i)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int t = (warp * EIGHTS + i) * 8 + row;
            float f[8 * PIECES], most = 0.f;
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                if (t >= m) in[which][i][j] = make_uint4(0, 0, 0, 0);
                const uint32_t xs[4] = {in[which][i][j].x, in[which][i][j].y, in[which][i][j].z, in[which][i][j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[8 * j + 2 * e] = __uint_as_float(xs[e] << 16);
                    f[8 * j + 2 * e + 1] = __uint_as_float(xs[e] & 0xffff0000u);
                    most = fmaxf(most, fmaxf(fabsf(f[8 * j + 2 * e]), fabsf(f[8 * j + 2 * e + 1])));
                }
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            const float up = scale_to(fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16)), 0);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8 * PIECES; ++j) {
                f[j] *= up;
                ss += f[j] * f[j];
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 16);
            if (sub == 0)
                (which ? sm.cq : sm.ck)[t] = ss == 0.f ? 0.f : a.eps > 0.f ? inverse_norm(ss, a.eps, up) : inverse(up);
#pragma unroll
            for (int j = 0; j < PIECES; ++j)
                *reinterpret_cast<uint4*>((which ? sm.q : sm.k) + in_tile(t, 4 * j + sub)) =
                    make_uint4(pack(f[8 * j], f[8 * j + 1]), pack(f[8 * j + 2], f[8 * j + 3]), pack(f[8 * j + 4], f[8 * j + 5]),
                               pack(f[8 * j + 6], f[8 * j + 7]));
        }
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
        bulk_store(w.qk + (unit * a.Hk + hk) * 2 * Tile<DK>::kBytes, sm.k, 2 * Tile<DK>::kBytes);
        bulk_commit();
    }

    // k.k and q.k of this warp's tokens with the tokens up to them: eight tokens from the front and eight from the back, so
    // that every warp has as many pairs (BRIEF: k.k by the first two warps, q.k by the others)
    const int front = BRIEF ? warp % 2 : warp, back = (BRIEF ? 3 : 7) - front;  // in eights
    constexpr int COLS = BRIEF ? 4 : 8;                                        // eights of tokens
    const bool of_keys = !BRIEF || warp < 2, of_queries = !BRIEF || warp >= 2;
    float kk[COLS][4], qk[COLS][4];
#pragma unroll
    for (int t = 0; t < COLS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[t][e] = qk[t][e] = 0.f;
    const uint32_t ks = tc::smem_addr(sm.k), qs = tc::smem_addr(sm.q);
    {
        const int eight = lane >> 3 & 1 ? back : front;
        const int own = in_tile(8 * eight + (lane & 7), lane >> 4), rows = tile_by_rows(lane);
#pragma unroll 2
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t ak[4], aq[4];
            if (of_keys) ldsm4(ak, ks + kt * kCols16 + own);
            if (of_queries) ldsm4(aq, qs + kt * kCols16 + own);
#pragma unroll
            for (int t2 = 0; t2 < COLS / 2; ++t2) {
                if (2 * t2 > back) continue;
                uint32_t b[4];
                ldsm4(b, ks + t2 * kRows16 + kt * kCols16 + rows);
                if (of_keys) {
                    mma(kk[2 * t2], ak, b[0], b[1]);
                    mma(kk[2 * t2 + 1], ak, b[2], b[3]);
                }
                if (of_queries) {
                    mma(qk[2 * t2], aq, b[0], b[1]);
                    mma(qk[2 * t2 + 1], aq, b[2], b[3]);
                }
            }
        }
    }

    const int g4 = lane / 4, q4 = lane % 4;
#pragma unroll 1
    for (int v0 = 0; v0 < group; v0 += 2) {  // two value heads at a time, a pair of warps each
        const bool on = v0 + pair < group;
        if (tid == 0) bulk_wait_read();
        __syncthreads();  // K and Q, or x[], have been read: their place is free
        if (v0 && warp % 2 == 0) load_gates(v0 + pair);
        if (on && warp % 2 == 0) {
            Gates& gates = *reinterpret_cast<Gates*>(sm.x[pair]);
            float* vec = reinterpret_cast<float*>(sm.x[pair] + 2 * kTri);
            float* out = reinterpret_cast<float*>(sm.x[pair] + kXBytes + kTri);
            Sum s[2];  // sums of g, to base 2
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float g = gs[i] < -200.f ? -200.f : gs[i];  // (e^-200 is 0 as well)
                s[i] = sum_of(g, 1.4426950408889634f);
                s[i].lo = fmaf(g, 1.925963033500811e-8f, s[i].lo);  // log2(e) = 1.4426950216293335 + 1.92596299e-8
            }
            const Sum mine = s[0] + s[1];
            Sum run = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const Sum x{__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
                if (lane >= o) run = x + run;
            }
            const Sum all{__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
            Sum before{__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
            if (lane == 0) before = Sum{0.f, 0.f};
            s[0] = before + s[0];
            s[1] = run;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                const float hi = s[i].hi;
                gates.ghi[t] = hi;
                gates.glo[t] = s[i].lo;
                const float ck = sm.ck[t], cq = sm.cq[t] * a.scale, since = exp2f(hi + s[i].lo);
                gates.beta[t] = be[i] * ck * ck;
                vec[kA * C + t] = since * ck;
                vec[kBeta * C + t] = be[i] * ck;
                out[kSince * C + t] = since;
                out[kPi * C + t] = cq;
                vec[kD * C + t] = exp2f((all.hi - hi) + (all.lo - s[i].lo));
            }
            if (lane == 0) vec[kGamma * C] = chunk_decay(all.hi + all.lo);
        }
        __syncthreads();
        // A' and P of both heads, from every warp's products
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            if (v0 + p >= group) break;
            char* const ps = sm.x[p] + kXBytes;
            typename PrepSmem<DK>::Blocks& bl = sm.blocks[p];
            const Gates& gates = *reinterpret_cast<const Gates*>(sm.x[p]);
            const int i0[2] = {8 * front + g4, 8 * back + g4};
            const float gh[2] = {gates.ghi[i0[0]], gates.ghi[i0[1]]}, gl[2] = {gates.glo[i0[0]], gates.glo[i0[1]]};
            const float bc[2] = {gates.beta[i0[0]], gates.beta[i0[1]]};
#pragma unroll
            for (int t = 0; t < COLS; ++t) {
                if (t > (back | 1)) continue;
                const float2 jh = *reinterpret_cast<const float2*>(&gates.ghi[8 * t + 2 * q4]);
                const float2 jl = *reinterpret_cast<const float2*>(&gates.glo[8 * t + 2 * q4]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int eight = h ? back : front;
                    if (t > (eight | 1)) continue;
                    const int i = i0[h], j = 8 * t + 2 * q4, at = in_block(eight % 2 * 8 + g4, t % 2) + 4 * q4;
                    const float e0 = exp2_fast((gh[h] - jh.x) + (gl[h] - jl.x)), e1 = exp2_fast((gh[h] - jh.y) + (gl[h] - jl.y));
                    const float a0 = e0 * bc[h] * kk[t][2 * h], a1 = e1 * bc[h] * kk[t][2 * h + 1];
                    float p0 = e0 * qk[t][2 * h], p1 = e1 * qk[t][2 * h + 1];
                    if (t / 2 == eight / 2) {  // (the elements of A' on and above the diagonal are not looked at)
                        if (of_keys) {
                            bl.at[t / 2][j % 16][i % 16] = a0;
                            bl.at[t / 2][j % 16 + 1][i % 16] = a1;
                        }
                        if (j > i) p0 = 0.f;
                        if (j + 1 > i) p1 = 0.f;
                    } else if (of_keys) {
                        uint32_t hi, lo;
                        split(a0, a1, hi, lo);
                        *reinterpret_cast<uint32_t*>(bl.ahi + below(eight / 2, t / 2) + at) = hi;
                        *reinterpret_cast<uint32_t*>(bl.alo + below(eight / 2, t / 2) + at) = lo;
                    }
                    if (of_queries) *reinterpret_cast<uint32_t*>(ps + tri(eight / 2, t / 2) + at) = pack(p0, p1);
                }
            }
        }
        tc::fence_proxy_async_smem();
        __syncthreads();
        if (on && (!BRIEF || warp % 2 == 0)) {
            char* const xp = sm.x[pair];
            {  // diagonal blocks: column c of block b, an elimination in registers
                const int c = warp % 2 * 32 + lane, b = c / 16;
                const float(*at)[16] = sm.blocks[pair].at[b];
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = i == c % 16 ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < 15; ++j)
#pragma unroll
                    for (int i = j + 1; i < 16; ++i) x[i] -= at[j][i] * x[j];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int o = tri(b, b) + in_block(i, c % 16 / 8) + 2 * (c % 8);
                    const __half hi = __float2half_rn(x[i]);
                    *reinterpret_cast<__half*>(xp + o) = hi;
                    *reinterpret_cast<__half*>(xp + kTri + o) = __float2half_rn(x[i] - __half2float(hi));
                }
            }
            const uint32_t xh = tc::smem_addr(xp), xl = xh + kTri;
            const uint32_t ah = tc::smem_addr(sm.blocks[pair].ahi), al = tc::smem_addr(sm.blocks[pair].alo);
            const int w2 = warp % 2;
            __syncwarp();
            merge_blocks<1>(xh, xl, ah, al, 2 * w2, 2 * w2, 2 * w2 + 1);
            if constexpr (!BRIEF) {
                tc::named_bar_sync(1 + pair, 64);
                merge_blocks<2>(xh, xl, ah, al, 0, w2, 2);
            }
            tc::fence_proxy_async_smem();
            if constexpr (BRIEF)
                __syncwarp();
            else
                tc::named_bar_sync(1 + pair, 64);
        }
        if (group - v0 > 1) __syncthreads();  // (thread 0 stores both heads)
        if (tid == 0) {
            for (int p = 0; p < 2 && v0 + p < group; ++p)
                bulk_store(w.heads + (unit * a.Hv + hk * group + v0 + p) * kHeadBytes, sm.x[p], kHeadBytes);
            bulk_commit();
        }
    }
    if (tid == 0) bulk_wait();
}

// ---------------------------------------------------------------- second launch: the states' walk
// A slice of 16 rows of the transposed state is walked by two warps.  Warp p keeps columns [DK / 2 p, DK / 2 (p + 1)) of
// the rows and takes tokens [32 p, 32 p + 32) of R and U; the operands that the other one needs (its half of the
// state, R of the first tokens, U') pass through shared memory as f16 pairs in the A operand's layout, each
// half with row scales of its own, so that nothing has to be agreed on before.  The outputs are no part of the chain of
// states: a third warp makes them from the same operands, up to a chunk later.
//
// Bound: with one slice a multiprocessor the chain, 3500 cycles a chunk (170 MMAs at 8 cycles a warp, the rest is the latency
// of scales, splits and exchanges between them); with two 4400 (the third warps share the schedulers); with four 6400,
// shared memory at 72 % (ldmatrix half of it) and the tensor pipe at 50 %.
// Slower: one warp a slice (448 us for the 8192 tokens); four warps a slice, a quarter of columns and tokens each (333); the
// products of neighbouring chunks' keys from the first launch, which take the states off the chain but cost a quarter
// more MMAs (273, and 13 us more in the first launch; 648 for the batch).
template <int DK, int W, int NS, int TT>
struct WalkSmem {
    static constexpr int QS = NS == 1 ? 1 : 2;
    struct ForStates {
        char k[Tile<DK>::kBytes];
        char x[kXBytes];
    };
    struct ForOutputs {
        char q[Tile<DK>::kBytes];
        char p[kPBytes];
    };
    alignas(128) ForStates x[NS];
    ForOutputs q[QS];
    struct Pass {                     // of a slice, from warp p to the others
        uint4 s[QS][2][DK / 32][32];  // [chunk % 2][p][k step][lane]: S0, high
        uint4 sl[2][DK / 32][32];     // low
        uint4 u[QS][2][TT][32];       // [chunk % 2][p][k step][lane]: U', high
        uint4 d[2][TT][2][32];        // [p][k step][high, low][lane]: U' e^(G_C - G)
        uint4 r[TT][2][32];           // R of the first tokens
        float ds[QS][2][16], du[QS][2][16], dd[2][16], dr[16];  // factors of their rows
    } pass[W];
    char v[2 * W][QS][TT * 16 * 32];  // a warp's tokens of 16 values
    char o[W][2 * TT * 16 * 32];      // the chunk's tokens of 16 outputs
    uint64_t x_full[NS], x_empty[NS], q_full[QS], q_empty[QS];
    uint64_t given[W][2], taken[W][2];  // S0 and U' of chunk % 2 for the third warp
    int abort, request;
};

// Warps of a block: two a slice, then those of the outputs; with two slices an idle one between these, so that each shares
// its scheduler (warp modulo 4) with the lighter warp of another slice
template <int W>
constexpr int kWalkWarps = 3 * W + (W == 2);

// TT: sixteens of tokens of each of the two warps.  2; or 1, for at most 32 tokens a request, with tiles for one chunk (NS = 1)
template <int DK, int W, int NS, int TT>
__global__ void __launch_bounds__(32 * kWalkWarps<W>, TT == 1 ? 2 : 1) delta_walk_kernel(const DeltaArgs a, const Scratch w) {
    extern __shared__ __align__(128) char raw[];
    using Smem = WalkSmem<DK, W, NS, TT>;
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    constexpr int QS = Smem::QS;
    constexpr int NK = DK / 32;        // k steps of 16 of a half of the state's columns
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g4 = lane / 4, q4 = lane % 4;
    const bool outputs = warp >= 2 * W;
    const int mine = !outputs ? warp / 2 : W == 2 ? (warp - 4) / 2 : warp - 2 * W, p = warp % 2;  // slice of the block, part of it
    typename Smem::Pass& ps = sm.pass[mine];
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&sm.x_full[i], 1);
            tc::mbar_init(&sm.x_empty[i], 2 * W);
        }
        for (int i = 0; i < QS; ++i) {
            tc::mbar_init(&sm.q_full[i], 1);
            tc::mbar_init(&sm.q_empty[i], W);
        }
        for (int i = 0; i < 2 * W; ++i) {
            tc::mbar_init(&sm.given[0][i], 2);
            tc::mbar_init(&sm.taken[0][i], 1);
        }
        sm.abort = 0;
        tc::fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();
    const int slices = a.Dv / (16 * W);
    const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.Hv;
    int r = blockIdx.x / slices / a.Hv;
    r = longest_first(a, r, &sm.request);
    int tokens, slot;
    if (!delta_request(a, r, tid == 0 && slice == 0 && hv == 0, tokens, slot)) return;
    __syncthreads();
    const int hk = hv / (a.Hv / a.Hk), n_chunks = (tokens + C - 1) / C;
    const int row0 = (slice * W + mine) * 16;  // first of the slice's rows
    const long long tok0 = 1ll * r * a.n, unit0 = 1ll * r * w.chunks;
    const int rows = by_rows(lane), slice_rows = slice_by_rows(lane), tile_rows = tile_by_rows(lane), tile_cols = tile_by_cols(lane);
    // (after a wait that ran out the other waits end at once and no more is fetched: the walk goes on, bounded, over
    // whatever stands in the tiles, so that nobody is left at a barrier, the error is recorded and no state is stored: the
    // warps of the states learn at a barrier, which those of the outputs only pass, whether all of the block's waits ended well)
    bool ok = true;
    constexpr int kBarEnd = 13, kEnd = 3 * W * 32;
    auto wait = [&](uint64_t* bar, int phase) {
        if (tc::mbar_wait(bar, phase & 1, &sm.abort, a.timeout_ns)) return;
        ok = false;
        *const_cast<volatile int*>(&sm.abort) = 1;
    };

    // tiles: those of the states are fetched by the first warp, those of the outputs by the first of these.  A stage is
    // filled again in the middle of the next chunk, when nobody uses it any more, so that no wait costs anything.
    int issued = 0;
    auto keys = [&](int c) { return w.qk + ((unit0 + c) * a.Hk + hk) * 2 * Tile<DK>::kBytes; };
    auto head = [&](int c) { return w.heads + ((unit0 + c) * a.Hv + hv) * kHeadBytes; };

    if (outputs) {
        if (W == 2 && p) return;
        const bool fetches = mine == 0 && lane == 0;
        auto fetch = [&]() {
            const int st = issued % QS;
            if (issued >= QS) wait(&sm.q_empty[st], issued / QS - 1);
            if (!ok) return;
            tc::mbar_arrive_expect_tx(&sm.q_full[st], Tile<DK>::kBytes + kPBytes);
            bulk_load(tc::smem_addr(sm.q[st].q), keys(issued) + Tile<DK>::kBytes, Tile<DK>::kBytes, &sm.q_full[st]);
            bulk_load(tc::smem_addr(sm.q[st].p), head(issued) + kXBytes, kPBytes, &sm.q_full[st]);
            ++issued;
        };
        if (fetches && n_chunks) fetch();
        const uint32_t os = tc::smem_addr(sm.o[mine]);
#pragma unroll 1
        for (int c = 0; c < n_chunks; ++c) {
            const int cb = c & 1;
            if (fetches && ok && issued < n_chunks) fetch();
            __syncwarp();
            wait(&sm.q_full[c % QS], c / QS);
            wait(&sm.given[mine][cb], c >> 1);
            __syncwarp();
            if (a.state_out && c + 1 == n_chunks) bar_arrive(kBarEnd, kEnd);  // (the last wait is over)
            typename Smem::ForOutputs& s = sm.q[c % QS];
            const uint32_t qr = tc::smem_addr(s.q) + tile_rows, pr = tc::smem_addr(s.p) + rows;
            const float* vec = reinterpret_cast<const float*>(s.p + kTri) + 2 * q4;
            // S0 Q^T, with the columns of each half of S0 and their scale
            float o[4 * TT][4];
            {
                float x[4 * TT][4];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int kt = 0; kt < NK; ++kt) {
                        const uint4 y = ps.s[cb][half][kt][lane];
                        const uint32_t hi[4] = {y.x, y.y, y.z, y.w};
                        uint32_t b[2 * TT][4];
#pragma unroll
                        for (int t2 = 0; t2 < 2 * TT; ++t2) ldsm4(b[t2], qr + t2 * kRows16 + (half * NK + kt) * kCols16);
#pragma unroll
                        for (int t2 = 0; t2 < 2 * TT; ++t2) {
                            if (kt == 0) {
                                mma0(x[2 * t2], hi, b[t2][0], b[t2][1]);
                                mma0(x[2 * t2 + 1], hi, b[t2][2], b[t2][3]);
                            } else {
                                mma(x[2 * t2], hi, b[t2][0], b[t2][1]);
                                mma(x[2 * t2 + 1], hi, b[t2][2], b[t2][3]);
                            }
                        }
                    }
                    const float f[2] = {ps.ds[cb][half][g4], ps.ds[cb][half][g4 + 8]};
#pragma unroll
                    for (int t = 0; t < 4 * TT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[t][e] = half ? o[t][e] + x[t][e] * f[e / 2] : x[t][e] * f[e / 2];
                }
            }
            // e^G of that, + P U', scaled by the token's factor
#pragma unroll
            for (int t = 0; t < 4 * TT; ++t) {
                const float2 b = *reinterpret_cast<const float2*>(vec + kSince * C + 8 * t);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][e] *= e % 2 ? b.y : b.x;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[4 * TT][4];
#pragma unroll
                for (int kt = 0; kt < TT; ++kt) {
                    const uint4 y = ps.u[cb][half][kt][lane];
                    const uint32_t uh[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int t2 = TT * half + kt; t2 < 2 * TT; ++t2) {
                        uint32_t b[4];
                        ldsm4(b, pr + tri(t2, TT * half + kt));
                        if (kt == 0) {
                            mma0(x[2 * t2], uh, b[0], b[1]);
                            mma0(x[2 * t2 + 1], uh, b[2], b[3]);
                        } else {
                            mma(x[2 * t2], uh, b[0], b[1]);
                            mma(x[2 * t2 + 1], uh, b[2], b[3]);
                        }
                    }
                }
                const float f[2] = {ps.du[cb][half][g4], ps.du[cb][half][g4 + 8]};
#pragma unroll
                for (int t = 2 * TT * half; t < 4 * TT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][e] += x[t][e] * f[e / 2];
            }
#pragma unroll
            for (int t = 0; t < 4 * TT; ++t) {
                const float2 pi = *reinterpret_cast<const float2*>(vec + kPi * C + 8 * t);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][e] *= e % 2 ? pi.y : pi.x;
            }
            __syncwarp();  // S0, U' and the tiles have been read
            if (lane == 0) {
                tc::mbar_arrive(&sm.taken[mine][cb]);
                tc::mbar_arrive(&sm.q_empty[c % QS]);
            }
#pragma unroll
            for (int t2 = 0; t2 < 2 * TT; ++t2) {
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const __nv_bfloat162 both = __floats2bfloat162_rn(o[2 * t2 + j][2 * h], o[2 * t2 + j][2 * h + 1]);
                        x[2 * j + h] = *reinterpret_cast<const uint32_t*>(&both);
                    }
                stsm4_t(os + t2 * 512 + slice_rows, x[0], x[1], x[2], x[3]);
            }
            __syncwarp();
            bf16* op = static_cast<bf16*>(a.out) + hv * a.Dv + row0;
#pragma unroll
            for (int i = 0; i < 2 * TT; ++i) {
                const int tok = c * C + i * 16 + lane / 2;
                if (tok < tokens)
                    *reinterpret_cast<uint4*>(op + (tok0 + tok) * a.Hv * a.Dv + 8 * (lane & 1)) =
                        *reinterpret_cast<const uint4*>(sm.o[mine] + i * 512 + in_slice(lane / 2, lane & 1));
            }
            __syncwarp();
        }
        if (!__all_sync(0xffffffffu, ok)) {  // a wait ran out: record it and let the copies that were issued land
            if (lane == 0) record_error(a.err, kErrTimeoutEpilogue);
            if (fetches) {
                int zero = 0;
                for (int i = max(0, issued - QS); i < issued; ++i)
                    tc::mbar_wait(&sm.q_full[i % QS], (i / QS) & 1, &zero, 1000000000ull);
            }
        }
        return;
    }

    auto fetch = [&]() {
        const int st = issued % NS;
        if (issued >= NS) wait(&sm.x_empty[st], issued / NS - 1);
        if (!ok) return;
        tc::mbar_arrive_expect_tx(&sm.x_full[st], Tile<DK>::kBytes + kXBytes);
        bulk_load(tc::smem_addr(sm.x[st].k), keys(issued), Tile<DK>::kBytes, &sm.x_full[st]);
        bulk_load(tc::smem_addr(sm.x[st].x), head(issued), kXBytes, &sm.x_full[st]);
        ++issued;
    };
    if (tid == 0)
        while (issued < (NS == 1 ? 1 : NS - 1) && issued < n_chunks) fetch();

    const uint32_t vs = tc::smem_addr(sm.v[warp]);
    auto fetch_v = [&](int c) {  // the warp's values, zeros behind the request's tokens
        const bf16* vp = static_cast<const bf16*>(a.v) + hv * a.Dv + row0;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = i * 16 + lane / 2, tok = c * C + 16 * TT * p + t;
            const bool on = tok < tokens;
            cp16(vs + (c & 1) * (TT * 512) + i * 512 + in_slice(lane / 2, lane & 1), vp + (tok0 + (on ? tok : 0)) * a.v_ld + 8 * (lane & 1), on);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (n_chunks > 0) fetch_v(0);

    // rows g4 and g4 + 8 of the slice, columns DK / 2 p + 8 t + 2 q4 + {0, 1}
    float S[DK / 16][4];
    const long long state0 = ((1ll * slot * a.Hv + hv) * a.Dv + row0 + g4) * DK + p * (DK / 2) + 2 * q4;
    const bool fresh = a.fresh && a.fresh[r];
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
        float2 x = make_float2(0.f, 0.f), y = x;
        if (!fresh) {
            x = *reinterpret_cast<const float2*>(a.state + state0 + 8 * t);
            y = *reinterpret_cast<const float2*>(a.state + state0 + 8 * DK + 8 * t);
        }
        S[t][0] = x.x, S[t][1] = x.y, S[t][2] = y.x, S[t][3] = y.y;
    }

    // Barriers of the slice's warps.  A: both halves of S0 are there, and later U' of the first tokens (the second warp
    // waits for it before it reports at C, so that the first cannot be at A again before it has passed); B: R of the
    // first tokens; C: U' of the later ones.
    const int bar_a = 1 + 3 * mine, bar_b = bar_a + 1, bar_c = bar_a + 2;
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
        const int st = c % NS, cb = c & 1;
        wait(&sm.x_full[st], c / NS);
        if (c >= 2) wait(&sm.taken[mine][cb], (c >> 1) - 1);
        if (c + 1 < n_chunks) {
            fetch_v(c + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        typename Smem::ForStates& s = sm.x[st];
        const uint32_t kr = tc::smem_addr(s.k) + TT * p * kRows16 + tile_rows, xr = tc::smem_addr(s.x) + rows;
        const float* vec = reinterpret_cast<const float*>(s.x + 2 * kTri) + 16 * TT * p + 2 * q4;  // of this warp's tokens
        const uint32_t vc = vs + (c & 1) * (TT * 512);

        // S0 K^T of the warp's tokens: first with its own columns of S0, then with the other's
        float most[2] = {0.f, 0.f}, up[2], own[2], other[2];
#pragma unroll
        for (int t = 0; t < DK / 16; ++t) {
            most[0] = fmaxf(most[0], fmaxf(fabsf(S[t][0]), fabsf(S[t][1])));
            most[1] = fmaxf(most[1], fmaxf(fabsf(S[t][2]), fabsf(S[t][3])));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            up[h] = scale_to(quad_max(most[h]), 12);
            own[h] = inverse(up[h]);
            if (q4 == 0) ps.ds[cb][p][g4 + 8 * h] = own[h];
        }
        float sk[2 * TT][4], zk[2 * TT][4];
        auto half_product = [&](auto first, const uint32_t(&hi)[4], const uint32_t(&lo)[4], uint32_t kb, float(&x)[2 * TT][4]) {
            constexpr bool F = decltype(first)::value;
            uint32_t b[TT][4];
#pragma unroll
            for (int t2 = 0; t2 < TT; ++t2) ldsm4(b[t2], kb + t2 * kRows16);
#pragma unroll
            for (int t2 = 0; t2 < TT; ++t2) {
                mma_<F>(x[2 * t2], hi, b[t2][0], b[t2][1]);
                mma_<F>(x[2 * t2 + 1], hi, b[t2][2], b[t2][3]);
            }
#pragma unroll
            for (int t2 = 0; t2 < TT; ++t2) {
                mma(x[2 * t2], lo, b[t2][0], b[t2][1]);
                mma(x[2 * t2 + 1], lo, b[t2][2], b[t2][3]);
            }
        };
        const std::true_type first{};
        const std::false_type then{};
        const uint32_t k_own = kr + p * (NK * kCols16), k_other = kr + (1 - p) * (NK * kCols16);
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                split(S[2 * kt + j][0] * up[0], S[2 * kt + j][1] * up[0], hi[2 * j], lo[2 * j]);
                split(S[2 * kt + j][2] * up[1], S[2 * kt + j][3] * up[1], hi[2 * j + 1], lo[2 * j + 1]);
            }
            ps.s[cb][p][kt][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            ps.sl[p][kt][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (kt == 0)
                half_product(first, hi, lo, k_own + kt * kCols16, sk);
            else
                half_product(then, hi, lo, k_own + kt * kCols16, sk);
        }
        tc::named_bar_sync(bar_a, 64);
        if (tid == 0 && ok && issued < n_chunks) fetch();
        __syncwarp();
        other[0] = ps.ds[cb][1 - p][g4], other[1] = ps.ds[cb][1 - p][g4 + 8];
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
            const uint4 x = ps.s[cb][1 - p][kt][lane], y = ps.sl[1 - p][kt][lane];
            const uint32_t hi[4] = {x.x, x.y, x.z, x.w}, lo[4] = {y.x, y.y, y.z, y.w};
            if (kt == 0)
                half_product(first, hi, lo, k_other + kt * kCols16, zk);
            else
                half_product(then, hi, lo, k_other + kt * kCols16, zk);
        }
        // R = beta c (v - e^G c S0 k), in place of S0 K^T
        float rmost[2] = {0.f, 0.f};
#pragma unroll
        for (int t2 = 0; t2 < TT; ++t2) {
            uint32_t vv[4];  // tokens 16 t2 ..: columns 0-7, 8-15; tokens 16 t2 + 8 ..: the same
            ldsm4_t(vv, vc + t2 * 512 + slice_rows);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * t2 + j;
                const float2 av = *reinterpret_cast<const float2*>(vec + kA * C + 8 * t);
                const float2 be = *reinterpret_cast<const float2*>(vec + kBeta * C + 8 * t);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = vv[2 * j + h];
                    float& r0 = sk[t][2 * h];
                    float& r1 = sk[t][2 * h + 1];
                    r0 = be.x * (__uint_as_float(x << 16) - av.x * (r0 * own[h] + zk[t][2 * h] * other[h]));
                    r1 = be.y * (__uint_as_float(x & 0xffff0000u) - av.y * (r1 * own[h] + zk[t][2 * h + 1] * other[h]));
                    rmost[h] = fmaxf(rmost[h], fmaxf(fabsf(r0), fabsf(r1)));
                }
            }
        }
        // U' = X R: of the warp's own tokens, and for the later tokens of the first ones
        float rup[2], rdown[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            rup[h] = scale_to(quad_max(rmost[h]), 12);
            rdown[h] = inverse(rup[h]);
            if (p == 0 && q4 == 0) ps.dr[g4 + 8 * h] = rdown[h];
        }
        float u[2 * TT][4];
        {
            uint32_t hi[TT][4], lo[TT][4];
#pragma unroll
            for (int kt = 0; kt < TT; ++kt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    split(sk[2 * kt + j][0] * rup[0], sk[2 * kt + j][1] * rup[0], hi[kt][2 * j], lo[kt][2 * j]);
                    split(sk[2 * kt + j][2] * rup[1], sk[2 * kt + j][3] * rup[1], hi[kt][2 * j + 1], lo[kt][2 * j + 1]);
                }
                if (p == 0) {
                    ps.r[kt][0][lane] = make_uint4(hi[kt][0], hi[kt][1], hi[kt][2], hi[kt][3]);
                    ps.r[kt][1][lane] = make_uint4(lo[kt][0], lo[kt][1], lo[kt][2], lo[kt][3]);
                }
            }
            if (p == 0) bar_arrive(bar_b, 64);
            uint32_t b[TT][TT][4], l[TT][TT][4];
#pragma unroll
            for (int t2 = 0; t2 < TT; ++t2)
#pragma unroll
                for (int kt = 0; kt <= t2; ++kt) {
                    const uint32_t x = xr + (p ? tri(TT + t2, TT + kt) : tri(t2, kt));
                    ldsm4(b[t2][kt], x);
                    ldsm4(l[t2][kt], x + kTri);
                }
#pragma unroll
            for (int kt = 0; kt < TT; ++kt)
#pragma unroll
                for (int t2 = kt; t2 < TT; ++t2) {
                    if (kt == 0)
                        mma3<true>(u[2 * t2], u[2 * t2 + 1], hi[kt], lo[kt], b[t2][kt], l[t2][kt]);
                    else
                        mma3<false>(u[2 * t2], u[2 * t2 + 1], hi[kt], lo[kt], b[t2][kt], l[t2][kt]);
                }
        }
#pragma unroll
        for (int t = 0; t < 2 * TT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[t][e] *= rdown[e / 2];
        if (p == 1) {
            float z[2 * TT][4];
            uint32_t b[TT][TT][4], l[TT][TT][4];
#pragma unroll
            for (int t2 = 0; t2 < TT; ++t2)
#pragma unroll
                for (int kt = 0; kt < TT; ++kt) {
                    ldsm4(b[t2][kt], xr + tri(TT + t2, kt));
                    ldsm4(l[t2][kt], xr + tri(TT + t2, kt) + kTri);
                }
            tc::named_bar_sync(bar_b, 64);
            const float f[2] = {ps.dr[g4], ps.dr[g4 + 8]};
#pragma unroll
            for (int kt = 0; kt < TT; ++kt) {
                const uint4 x = ps.r[kt][0][lane], y = ps.r[kt][1][lane];
                const uint32_t hi[4] = {x.x, x.y, x.z, x.w}, lo[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int t2 = 0; t2 < TT; ++t2) {
                    if (kt == 0)
                        mma3<true>(z[2 * t2], z[2 * t2 + 1], hi, lo, b[t2][kt], l[t2][kt]);
                    else
                        mma3<false>(z[2 * t2], z[2 * t2 + 1], hi, lo, b[t2][kt], l[t2][kt]);
                }
            }
#pragma unroll
            for (int t = 0; t < 2 * TT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) u[t][e] += z[t][e] * f[e / 2];
        }
        // U' and U' e^(G_C - G), each brought to 2^12
        float umost[2] = {0.f, 0.f}, dmost[2] = {0.f, 0.f}, dx[2 * TT][4];
#pragma unroll
        for (int t = 0; t < 2 * TT; ++t) {
            const float2 left = *reinterpret_cast<const float2*>(vec + kD * C + 8 * t);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                dx[t][2 * h] = u[t][2 * h] * left.x;
                dx[t][2 * h + 1] = u[t][2 * h + 1] * left.y;
                umost[h] = fmaxf(umost[h], fmaxf(fabsf(u[t][2 * h]), fabsf(u[t][2 * h + 1])));
                dmost[h] = fmaxf(dmost[h], fmaxf(fabsf(dx[t][2 * h]), fabsf(dx[t][2 * h + 1])));
            }
        }
        float uup[2], dup[2], ddown[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uup[h] = scale_to(quad_max(umost[h]), 12);
            dup[h] = scale_to(quad_max(dmost[h]), 12);
            ddown[h] = inverse(dup[h]);
            if (q4 == 0) {
                ps.dd[p][g4 + 8 * h] = ddown[h];
                ps.du[cb][p][g4 + 8 * h] = inverse(uup[h]);
            }
        }
        uint32_t dhi[TT][4], dlo[TT][4];
#pragma unroll
        for (int kt = 0; kt < TT; ++kt) {
            uint32_t uh[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = 2 * kt + j;
                    split(dx[t][2 * h] * dup[h], dx[t][2 * h + 1] * dup[h], dhi[kt][2 * j + h], dlo[kt][2 * j + h]);
                    uh[2 * j + h] = pack(u[t][2 * h] * uup[h], u[t][2 * h + 1] * uup[h]);
                }
            ps.d[p][kt][0][lane] = make_uint4(dhi[kt][0], dhi[kt][1], dhi[kt][2], dhi[kt][3]);
            ps.d[p][kt][1][lane] = make_uint4(dlo[kt][0], dlo[kt][1], dlo[kt][2], dlo[kt][3]);
            ps.u[cb][p][kt][lane] = make_uint4(uh[0], uh[1], uh[2], uh[3]);
        }
        if (!a.state_out && c + 1 == n_chunks) {  // the states behind the last chunk are not wanted
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.given[mine][cb]);
            break;
        }
        if (p == 0) {
            bar_arrive(bar_a, 64);
        } else {
            tc::named_bar_sync(bar_a, 64);
            bar_arrive(bar_c, 64);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.given[mine][cb]);
        // S = e^G_C S0 + U' e^(G_C - G) K on the warp's columns, with its own tokens and then with the other's (sums of
        // their own, added in fp32: an MMA cuts off what it adds to a large accumulator)
        float d[DK / 16][4];
        auto state_product = [&](const uint32_t(&hi)[TT][4], const uint32_t(&lo)[TT][4], int half) {
            const uint32_t kc = tc::smem_addr(s.k) + half * (TT * kRows16) + p * (NK * kCols16) + tile_cols;
#pragma unroll
            for (int kt = 0; kt < TT; ++kt)
#pragma unroll
                for (int t2 = 0; t2 < NK; t2 += 2) {
                    uint32_t b0[4], b1[4];
                    ldsm4_t(b0, kc + kt * kRows16 + t2 * kCols16);
                    ldsm4_t(b1, kc + kt * kRows16 + (t2 + 1) * kCols16);
                    if (kt == 0) {
                        mma0(d[2 * t2], hi[kt], b0[0], b0[1]);
                        mma0(d[2 * t2 + 1], hi[kt], b0[2], b0[3]);
                        mma0(d[2 * t2 + 2], hi[kt], b1[0], b1[1]);
                        mma0(d[2 * t2 + 3], hi[kt], b1[2], b1[3]);
                    } else {
                        mma(d[2 * t2], hi[kt], b0[0], b0[1]);
                        mma(d[2 * t2 + 1], hi[kt], b0[2], b0[3]);
                        mma(d[2 * t2 + 2], hi[kt], b1[0], b1[1]);
                        mma(d[2 * t2 + 3], hi[kt], b1[2], b1[3]);
                    }
                    mma(d[2 * t2], lo[kt], b0[0], b0[1]);
                    mma(d[2 * t2 + 1], lo[kt], b0[2], b0[3]);
                    mma(d[2 * t2 + 2], lo[kt], b1[0], b1[1]);
                    mma(d[2 * t2 + 3], lo[kt], b1[2], b1[3]);
                }
        };
        state_product(dhi, dlo, p);
        {
            const float gamma = *(reinterpret_cast<const float*>(s.x + 2 * kTri) + kGamma * C);
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][e] = S[t][e] * gamma + d[t][e] * ddown[e / 2];
        }
        // the other warp's tokens
        if (p == 0) tc::named_bar_sync(bar_c, 64);
        {
            const float f[2] = {ps.dd[1 - p][g4], ps.dd[1 - p][g4 + 8]};
            uint32_t ehi[TT][4], elo[TT][4];
#pragma unroll
            for (int kt = 0; kt < TT; ++kt) {
                const uint4 x = ps.d[1 - p][kt][0][lane], y = ps.d[1 - p][kt][1][lane];
                ehi[kt][0] = x.x, ehi[kt][1] = x.y, ehi[kt][2] = x.z, ehi[kt][3] = x.w;
                elo[kt][0] = y.x, elo[kt][1] = y.y, elo[kt][2] = y.z, elo[kt][3] = y.w;
            }
            state_product(ehi, elo, 1 - p);
#pragma unroll
            for (int t = 0; t < DK / 16; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][e] += d[t][e] * f[e / 2];
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.x_empty[st]);
    }
    if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) record_error(a.err, kErrTimeoutMma);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (tid == 0) {
            int zero = 0;
            for (int i = max(0, issued - NS); i < issued; ++i)
                tc::mbar_wait(&sm.x_full[i % NS], (i / NS) & 1, &zero, 1000000000ull);
        }
        __syncwarp();
    }
    if (!a.state_out) return;
    if (n_chunks) {
        tc::named_bar_sync(kBarEnd, kEnd);
        if (*const_cast<volatile int*>(&sm.abort)) return;
    }
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
        *reinterpret_cast<float2*>(a.state_out + state0 + 8 * t) = make_float2(S[t][0], S[t][1]);
        *reinterpret_cast<float2*>(a.state_out + state0 + 8 * DK + 8 * t) = make_float2(S[t][2], S[t][3]);
    }
}

template <int DK, bool BRIEF>
cudaError_t launch_prep(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    static int done[64];
    cudaError_t e = ensure_smem(delta_prep_kernel<DK, BRIEF>, sizeof(PrepSmem<DK>), done);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(1ll * a.R * w.chunks * a.Hk));
    return launch_pdl(delta_prep_kernel<DK, BRIEF>, grid, dim3(128), sizeof(PrepSmem<DK>), s, a, w);
}

template <int DK, int W, int NS, int TT>
cudaError_t launch_walk(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    constexpr size_t bytes = sizeof(WalkSmem<DK, W, NS, TT>);
    static_assert(bytes <= (TT == 1 ? 113 : 227) * 1024);
    static int done[64];
    cudaError_t e = ensure_smem(delta_walk_kernel<DK, W, NS, TT>, bytes, done);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.R * a.Hv * (a.Dv / (16 * W))));
    return launch_pdl(delta_walk_kernel<DK, W, NS, TT>, grid, dim3(32 * kWalkWarps<W>), bytes, s, a, w);
}

template <int DK>
cudaError_t launch_chunks(const DeltaArgs& a, const Scratch& w, int sms, cudaStream_t s) {
    const bool brief = a.n <= 32;
    cudaError_t e = brief ? launch_prep<DK, true>(a, w, s) : launch_prep<DK, false>(a, w, s);
    if (e != cudaSuccess) return e;
    count_launch();
    // As few slices a block as leave no multiprocessor a second block (blocks of more share their tiles, but also the chain
    // of a chunk gets longer).  us for 1000 tokens with 1 / 2 / 4 slices a block: 128 slices 41 / 48 / 65, 256 slices
    // 73 / 52 / 68, 384 slices of 500 tokens 59 / 51 / 40.  Where four fill the multiprocessors more than once and there is more
    // than one chunk, whole heads on tcgen05 are faster (1000 tokens, 512 slices 91 against 76, 768 slices 100 : 140, 1024
    // slices 105 : 145).
    const long long slices = 1ll * a.R * a.Hv * (a.Dv / 16);
    // One chunk in halves of 16 tokens leaves room for two blocks a multiprocessor (us for 32 tokens with 1 / 2 / 4 slices a
    // block: 256 slices 11.4 / 11.5 / 12.4, 512 slices 14.0 / 13.1 / 15.0, 1024 slices 21.6 / 18.9 / 16.6).
    if (brief) {
        if (slices <= 2ll * sms) return launch_walk<DK, 1, 1, 1>(a, w, s);
        if (slices <= 4ll * sms) return launch_walk<DK, 2, 1, 1>(a, w, s);
        return launch_walk<DK, 4, 1, 1>(a, w, s);
    }
    if (slices <= sms) return launch_walk<DK, 1, 3, 2>(a, w, s);
    if (slices <= 2ll * sms) return launch_walk<DK, 2, 3, 2>(a, w, s);
    if (a.Dv == 128 && a.n > C && slices > 4ll * sms) return launch_delta_heads(a, w, s);
    return launch_walk<DK, 4, 2, 2>(a, w, s);
}

size_t qk_bytes(const moestep_delta_dims& d, long long units) { return static_cast<size_t>(units) * d.Hk * 2 * C * d.Dk * 2; }

}  // namespace

// From 24 tokens on the two launches are faster than the recurrence but for one request or few small heads, which they hardly
// slow down (us against the recurrence's with 20 / 24 / 28 tokens; 16 and 32 heads of 128: one request 11.2 : 9.6 / 11.2 : 10.6 /
// 11.3 : 11.9, 4 requests 15.2 : 18.1 / 15.2 : 20.8 / 15.4 : 23.8, 16 requests 40.7 : 50.3 / 41.1 : 57.9 / 41.6 : 66.1; 2 and 4
// heads of 64, one request 7.4 : 5.8 / 7.4 : 6.3 / 7.4 : 7.0).
bool delta_chunked(const moestep_delta_dims& d, int R, int n) { return d.dtype == MOESTEP_BF16 && n >= 24; }

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
