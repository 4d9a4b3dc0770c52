// The second launch of the chunked gated delta rule for many heads of 128 values, on tcgen05.
//
// A block walks the chunks of one (request, head).  The 128 rows of its transposed state are the M of every MMA and the lanes
// of tensor memory; four threads share a row and keep a quarter of it each, in fp32 registers.  A chunk is a chain of
//
//   S0 K^T  ->  R = beta c (v - e^G c S0 k)  ->  U' = R X^T  ->  e^G S0 Q^T + U' P^T  and  S = e^G_C S0 + U' e^(G_C - G) K
//
// whose left operands the threads write to tensor memory, as f16 pairs where the states depend on them, and whose right ones
// are the first launch's tiles: 8 x 8 matrices at constant distances, so that K is an operand both ways and the
// columns of a lower triangle are operands of 64, 48, 32 and 16 rows without their zeros.
//
// MMAs that are in flight together are ordered only among those of one accumulator and one shape.  So products of 64, 48, 32 and
// 16 tokens have accumulators of their own, which the threads add up, and none is written to columns that another one in flight
// reads or writes.
//
// Bound: the chain, 7350 cycles a chunk.  An MMA with its left operand in tensor memory takes 64 cycles whatever its N, and 40 of
// the 48 are on the chain (S0 K^T 1050 cycles, U' 1050, the outputs' and the state's 770); the threads' part is 3500 issue
// slots of a scheduler.  Against the walk of slices of 16 rows with mma.sync (four slices a block; us with both launches, 16 / 32 heads of
// 128): 4 requests of 1000 tokens 105 : 145, 8 requests 200 : 282, 16 requests 390 : 501, 8 ragged ones of up to 4096 tokens
// 440 : 580; but 2 requests of 1000 tokens 91 : 76, and with one chunk the same or more (4 requests of 64 tokens 26 : 23).
// Slower (where these took 435): two threads a row and two blocks a multiprocessor (514), a warp of its own for the MMAs (518,
// 96 registers a thread spill), accumulators of their own for the low parts, issued by other warps (457).
#include "attn_tc.cuh"
#include "common.cuh"
#include "delta_chunk.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace moestep {
using namespace delta;
namespace {

constexpr int kDv = 128, kParts = 4, kThreads = kParts * kDv;  // kParts threads share a row of the state
// Places in tensor memory, 64 columns each (lane = row of the state), and what they hold in the course of a chunk
constexpr uint32_t kS = 0;     // S0, high parts; e^G S0 Q^T, to which the products with U' of the first 16 tokens are added
constexpr uint32_t kL = 64;    // S0, low parts; U' from R of the first 16; U' e^(G_C - G), high and low parts (32 columns each)
constexpr uint32_t kR = 128;   // S0 K^T; R, high and low parts (32 each); U' (32)
constexpr uint32_t kO = 192;   // S0 Q^T
constexpr uint32_t kM = 256;   // (96 columns) U' from R of the later sixteens; P U' with U' of these
constexpr uint32_t kT = 352;   // (DK columns) what is added to the state
constexpr uint32_t kColumns = 512;
// Columns of the products with tokens 16 kt .. 16 kt + 15, kt > 0, which reach the tokens from 16 kt on
__device__ __forceinline__ constexpr uint32_t later(int kt) { return kM + (kt > 1 ? 48 : 0) + (kt > 2 ? 32 : 0); }

template <int DK>
struct HeadSmem {
    alignas(128) char k[2][Tile<DK>::kBytes];
    char q[Tile<DK>::kBytes];
    char x[2 * kTri];
    char p[kTri];
    float vec[2][6 * C];  // kA ... kGamma, kSince, kPi
    char v[C * 2 * kDv];  // [token][value]
    char o[C * 2 * kDv];
    float most[4][kParts][kDv];  // largest elements of a row's parts
    uint64_t k_full[2], q_full, x_full, p_full;
    uint64_t done[5], last[2];  // MMAs: kKeys ...; all of the two warps that issue them
    uint32_t tmem;
    int abort, request;
    volatile int r, tokens, slot;  // the block's work (here, not in registers through the loop)
    volatile int asked[4];         // tiles asked for: K, Q, X, P
};
enum { kKeys, kQueries, kNew, kOutputs, kState };  // products

// Operand of 8 x 8 matrices in 128 bytes each: bytes from one to the next along K and along N
__device__ __forceinline__ uint64_t plain_desc(uint32_t addr, int along_k, int along_n) {
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>(along_k >> 4) << 16 |
           static_cast<uint64_t>(along_n >> 4) << 32 | 1ull << 46;
}

using tc::mul2;
__device__ __forceinline__ float2 mul2(float2 a, float b) { return mul2(a, make_float2(b, b)); }
__device__ __forceinline__ float largest(float most, float2 x) {  // of three absolute values
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(most), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return d;
}
// (an address whose descriptors are made where they are used, not kept in registers through the loop)
__device__ __forceinline__ uint32_t here(const void* p) {
    uint32_t x = tc::smem_addr(p);
    asm volatile("" : "+r"(x));
    return x;
}
__device__ __forceinline__ float2 pair_of(const float* x) { return make_float2(x[0], x[1]); }

// 8 consecutive 32-bit columns of this thread's TMEM lane (no wait)
__device__ __forceinline__ void tmem_st8_async(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// 16 consecutive fp32 columns of this thread's TMEM lane, with the wait
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}

// The same of two places at once
__device__ __forceinline__ void tmem_ld16_two(uint32_t a, uint32_t b, float* v, float* w) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%32];\n\ttcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31}, [%33];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(w[0]), "=f"(w[1]),
          "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7]), "=f"(w[8]), "=f"(w[9]), "=f"(w[10]),
          "=f"(w[11]), "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15])
        : "r"(a), "r"(b)
        : "memory");
}

// The sums of a product over the sixteens of tokens up to `part`, at the tokens of that sixteen: `first` is where the
// first sixteen's stands, `lanes` this warp's lanes
__device__ __forceinline__ void tmem_sum16(uint32_t lanes, uint32_t first, int part, float* v) {
    float w[16];
    auto add = [&]() {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 s = tc::add2(make_float2(v[i], v[i + 1]), make_float2(w[i], w[i + 1]));
            v[i] = s.x, v[i + 1] = s.y;
        }
    };
    if (part == 0) {
        tmem_ld16(lanes + first, v);
        return;
    }
    tmem_ld16_two(lanes + first + 16 * part, lanes + later(1) + 16 * (part - 1), v, w);
    add();
    if (part == 1) return;
    tmem_ld16(lanes + later(2) + 16 * (part - 2), w);
    add();
    if (part == 2) return;
    tmem_ld16(lanes + later(3), w);
    add();
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) delta_heads_kernel(const DeltaArgs a, const Scratch w) {
    extern __shared__ __align__(128) char raw[];
    using Smem = HeadSmem<DK>;
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    constexpr int N = DK / kParts, T = C / kParts;  // a thread's columns of the state, its tokens
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = warp / 4, row = tid % 128;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.k_full[i], 1);
        tc::mbar_init(&sm.q_full, 1);
        tc::mbar_init(&sm.x_full, 1);
        tc::mbar_init(&sm.p_full, 1);
        for (int i = 0; i < 5; ++i) tc::mbar_init(&sm.done[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.last[i], 1);
        sm.abort = 0;
        tc::fence_mbar_init();
    }
    pdl_wait();
    const int hv = blockIdx.x % a.Hv, r = longest_first(a, blockIdx.x / a.Hv, &sm.request);
    int tokens, slot;
    if (!delta_request(a, r, tid == 0 && hv == 0, tokens, slot)) return;
    if (tid == 0) {
        sm.r = r, sm.tokens = tokens, sm.slot = slot;
        for (int i = 0; i < 4; ++i) sm.asked[i] = 0;
    }
    if (warp == 0) {
        tc::tmem_alloc(&sm.tmem, kColumns);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // The next kernel may start once every block has its tensor memory: one that takes its own before it waits for this
    // kernel would otherwise keep a block from it for good.
    pdl_trigger();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16);  // this warp's lanes
    const int n_chunks = (tokens + C - 1) / C;

    // (after a wait that ran out the others end at once; the block leaves the loop together)
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
        bool there = tc::mbar_test_wait(bar, phase & 1);
        if (__all_sync(0xffffffffu, there)) return;
        if (!there)  // (two cycles a nanosecond: the SM clock stays below 2.1 GHz)
            there = tc::mbar_wait_cycles(bar, phase & 1, &sm.abort,
                                         static_cast<long long>(a.timeout_ns < (1ull << 61) ? 2 * a.timeout_ns : 1ull << 62));
        if (__all_sync(0xffffffffu, there)) return;
        ok = false;
        *const_cast<volatile int*>(&sm.abort) = 1;
    };

    // tiles, fetched by one warp as soon as their places are free
    const bool fetches = warp == 6;
    auto keys = [&](int c) {
        const int hk = static_cast<int>(blockIdx.x) % a.Hv / (a.Hv / a.Hk);
        return w.qk + ((1ll * sm.r * w.chunks + c) * a.Hk + hk) * 2 * Tile<DK>::kBytes;
    };
    auto head = [&](int c) { return w.heads + ((1ll * sm.r * w.chunks + c) * a.Hv + blockIdx.x % a.Hv) * kHeadBytes; };
    auto fetch_k = [&](int c) {
        if (!ok || lane) return;
        uint64_t* bar = &sm.k_full[c & 1];
        const char* from = head(c);
        tc::mbar_arrive_expect_tx(bar, Tile<DK>::kBytes + 6 * C * 4);
        bulk_load(tc::smem_addr(sm.k[c & 1]), keys(c), Tile<DK>::kBytes, bar);
        bulk_load(tc::smem_addr(sm.vec[c & 1]), from + 2 * kTri, 4 * C * 4, bar);
        bulk_load(tc::smem_addr(sm.vec[c & 1] + 4 * C), from + kXBytes + kTri, 2 * C * 4, bar);
        sm.asked[0] = c + 1;
    };
    auto fetch_one = [&](int which, int c, char* dst, const char* src, uint32_t bytes, uint64_t* bar) {
        if (!ok || lane) return;
        tc::mbar_arrive_expect_tx(bar, bytes);
        bulk_load(tc::smem_addr(dst), src, bytes, bar);
        sm.asked[which] = c + 1;
    };
    auto fetch_q = [&](int c) { fetch_one(1, c, sm.q, keys(c) + Tile<DK>::kBytes, Tile<DK>::kBytes, &sm.q_full); };
    auto fetch_x = [&](int c) { fetch_one(2, c, sm.x, head(c), 2 * kTri, &sm.x_full); };
    auto fetch_p = [&](int c) { fetch_one(3, c, sm.p, head(c) + kXBytes, kTri, &sm.p_full); };
    auto fetch_v = [&](int c) {  // (by all) zeros behind the request's tokens
        const int left = sm.tokens - c * C;
        const bf16* vp = static_cast<const bf16*>(a.v) + (1ll * sm.r * a.n + c * C) * a.v_ld + blockIdx.x % a.Hv * kDv + 8 * (tid % 16);
#pragma unroll
        for (int i = 0; i < C; i += kThreads / 16) {
            const int tok = i + tid / 16;
            cp16(tc::smem_addr(sm.v) + i * 2 * kDv + tid * 16, vp + (tok < left ? tok : 0) * a.v_ld, tok < left);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (fetches && n_chunks) {
        fetch_k(0);
        fetch_x(0);
        fetch_q(0);
        fetch_p(0);
        if (n_chunks > 1) fetch_k(1);
    }
    if (n_chunks) fetch_v(0);

    // S0 by rows in units of their own, powers of two that keep the largest element of a row within [2^9, 2^15)
    float S[N], up = 1.f, down = 1.f;
    auto place = [&]() { return ((1ll * sm.slot * a.Hv + blockIdx.x % a.Hv) * kDv + row) * DK + part * N; };
    {
        const long long state0 = place();
        const bool fresh = a.fresh && a.fresh[r];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 x = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(a.state + state0 + i);
            S[i] = x.x, S[i + 1] = x.y, S[i + 2] = x.z, S[i + 3] = x.w;
        }
    }

    // the largest element of a row from those of its parts (in the warps of the same lanes)
    auto all_parts = [&](int which, float most) {
        sm.most[which][part][row] = most;
        tc::named_bar_sync(1 + warp % 4, 32 * kParts);
#pragma unroll
        for (int i = 1; i < kParts; ++i) most = fmaxf(most, sm.most[which][(part + i) % kParts][row]);
        return most;
    };
    auto store_outputs = [&](int c) {
        const int left = sm.tokens - c * C;
        bf16* op = static_cast<bf16*>(a.out) + ((1ll * sm.r * a.n + c * C) * a.Hv + blockIdx.x % a.Hv) * kDv + 8 * (tid % 16);
#pragma unroll
        for (int i = 0; i < C; i += kThreads / 16) {
            const int tok = i + tid / 16;
            if (tok < left)
                *reinterpret_cast<uint4*>(op + 1ll * tok * a.Hv * kDv) = *reinterpret_cast<const uint4*>(sm.o + i * 2 * kDv + tid * 16);
        }
    };
    const uint32_t idesc64 = tc::idesc_f16(128, 64);

#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
        const float* vec = sm.vec[c & 1] + T * part;
        bool empty;
        {
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < N; i += 2) most = largest(most, pair_of(S + i));
            most = all_parts(0, most);
            empty = most == 0.f;
            // (a unit is changed only where the decay or the new tokens ask for it)
            const bool moved = !empty && (most < 0x1p9f || most >= 0x1p15f);
            if (__any_sync(0xffffffffu, moved)) {
                if (moved) {
                    const float f = scale_to(most, 12), now = fminf(fmaxf(up * f, 0x1p-126f), 0x1p126f), by = now * down;
#pragma unroll
                    for (int i = 0; i < N; ++i) S[i] *= by;
                    up = now;
                    down = inverse(now);
                }
            }
        }
        // as two f16 parts
#pragma unroll
        for (int i = 0; i < N; i += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split(S[i + 2 * j], S[i + 2 * j + 1], hi[j], lo[j]);
            tmem_st8_async(mine + kS + (part * N + i) / 2, hi);
            tmem_st8_async(mine + kL + (part * N + i) / 2, lo);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (__syncthreads_or(!ok)) break;
        // (the last chunk's keys, factors and P have been read, its outputs are there)
        if (fetches && c) {
            fetch_p(c);
            if (c + 1 < n_chunks) fetch_k(c + 1);
        }
        if (warp == 0) {
            tc::fence_after_sync();
            wait(&sm.k_full[c & 1], c >> 1);
            if (ok && tc::elect_one()) {
                const uint32_t k_at = here(sm.k[c & 1]);
#pragma unroll
                for (int kt = 0; kt < DK / 16; ++kt) {
                    const uint64_t b = plain_desc(k_at + kt * kCols16, 1024, 128);
                    tc::mma_f16_tmem_a(tmem + kR, tmem + kS + 8 * kt, b, idesc64, kt > 0);
                    tc::mma_f16_tmem_a(tmem + kR, tmem + kL + 8 * kt, b, idesc64, 1);
                }
                tc::mma_commit(&sm.done[kKeys]);
            }
            __syncwarp();
        }
        if (c) store_outputs(c - 1);
        // R = beta c (v - e^G c S0 k)
        float rdown;
        {
            float x[T];
            wait(&sm.k_full[c & 1], c >> 1);
            wait(&sm.done[kKeys], c);
            tc::fence_after_sync();
            if (warp == 1) {  // (while the other warps make R)
                wait(&sm.q_full, c);
                if (ok && tc::elect_one()) {
                    const uint32_t q_at = here(sm.q);
#pragma unroll
                    for (int kt = 0; kt < DK / 16; ++kt)
                        tc::mma_f16_tmem_a(tmem + kO, tmem + kS + 8 * kt, plain_desc(q_at + kt * kCols16, 1024, 128), idesc64, kt > 0);
                    tc::mma_commit(&sm.done[kQueries]);
                }
                __syncwarp();
            }
            tmem_ld16(mine + kR + T * part, x);
            const char* vp = sm.v + T * part * 2 * kDv + 2 * row;
            float most = 0.f;
#pragma unroll
            for (int t = 0; t < T; t += 4) {
                const float4 av = *reinterpret_cast<const float4*>(vec + kA * C + t);
                const float4 be = *reinterpret_cast<const float4*>(vec + kBeta * C + t);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const uint32_t v0 = *reinterpret_cast<const unsigned short*>(vp + (t + e) * 2 * kDv);
                    const uint32_t v1 = *reinterpret_cast<const unsigned short*>(vp + (t + e + 1) * 2 * kDv);
                    const float2 as = e ? make_float2(av.z, av.w) : make_float2(av.x, av.y);
                    const float2 bs = e ? make_float2(be.z, be.w) : make_float2(be.x, be.y);
                    const float2 old = mul2(pair_of(x + t + e), -down);
                    const float2 y = mul2(tc::fma2(as, old, make_float2(__uint_as_float(v0 << 16), __uint_as_float(v1 << 16))), bs);
                    most = largest(most, y);
                    x[t + e] = y.x, x[t + e + 1] = y.y;
                }
            }
            const float rup = scale_to(all_parts(1, most), 12);  // (and S0 K^T has been read)
            rdown = inverse(rup);
            uint32_t hi[T / 2], lo[T / 2];
#pragma unroll
            for (int t = 0; t < T; t += 2) {
                const float2 y = mul2(pair_of(x + t), rup);
                split(y.x, y.y, hi[t / 2], lo[t / 2]);
            }
            tmem_st8_async(mine + kR + T / 2 * part, hi);
            tmem_st8_async(mine + kR + 32 + T / 2 * part, lo);
            tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncthreads();
        if (c + 1 < n_chunks) fetch_v(c + 1);
        if (warp == 0) {
            tc::fence_after_sync();
            wait(&sm.x_full, c);
            if (ok && tc::elect_one()) {
                // U' = X R: token 16 kt and those behind it
                const uint32_t x_at = here(sm.x);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    const uint64_t b = plain_desc(x_at + tri(kt, kt), 128, 256), l = plain_desc(x_at + kTri + tri(kt, kt), 128, 256);
                    const uint32_t idesc = tc::idesc_f16(128, 64 - 16 * kt), d = tmem + (kt ? later(kt) : kL);
                    tc::mma_f16_tmem_a(d, tmem + kR + 8 * kt, b, idesc, 0);
                    tc::mma_f16_tmem_a(d, tmem + kR + 32 + 8 * kt, b, idesc, 1);
                    tc::mma_f16_tmem_a(d, tmem + kR + 8 * kt, l, idesc, 1);
                }
                tc::mma_commit(&sm.done[kNew]);
            }
            __syncwarp();
        }
        // U' and U' e^(G_C - G), each brought to 2^12
        float udown, dup, ddown, ratio;
        {
            float u[T];
            wait(&sm.done[kNew], c);
            tc::fence_after_sync();
            tmem_sum16(mine, kL, part, u);
            float umost = 0.f, dmost = 0.f;
#pragma unroll
            for (int t = 0; t < T; t += 4) {
                const float4 left = *reinterpret_cast<const float4*>(vec + kD * C + t);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 y = mul2(pair_of(u + t + e), rdown);
                    umost = largest(umost, y);
                    dmost = largest(dmost, mul2(y, e ? make_float2(left.z, left.w) : make_float2(left.x, left.y)));
                    u[t + e] = y.x, u[t + e + 1] = y.y;
                }
            }
            sm.most[3][part][row] = dmost;
            umost = all_parts(2, umost);  // (and U' has been read)
#pragma unroll
            for (int i = 1; i < kParts; ++i) dmost = fmaxf(dmost, sm.most[3][(part + i) % kParts][row]);
            // (U' is added to e^G S0 Q^T in its own unit: where S0's is more than 2^60 of that, in one that large)
            float uup = scale_to(umost, 12);
            if (!empty) uup = fminf(uup, up * 0x1p60f);
            udown = inverse(uup);
            ratio = empty ? 0.f : down * uup;
            dup = scale_to(dmost, 12);
            ddown = inverse(dup);
            uint32_t y[T / 2], hi[T / 2], lo[T / 2];
#pragma unroll
            for (int t = 0; t < T; t += 2) {
                const float2 z = mul2(pair_of(u + t), uup);
                y[t / 2] = pack(z.x, z.y);
            }
            tmem_st8_async(mine + kR + T / 2 * part, y);
#pragma unroll
            for (int t = 0; t < T; t += 4) {
                const float4 left = *reinterpret_cast<const float4*>(vec + kD * C + t);
                const float2 z0 = mul2(mul2(pair_of(u + t), make_float2(left.x, left.y)), dup);
                const float2 z1 = mul2(mul2(pair_of(u + t + 2), make_float2(left.z, left.w)), dup);
                split(z0.x, z0.y, hi[t / 2], lo[t / 2]);
                split(z1.x, z1.y, hi[t / 2 + 1], lo[t / 2 + 1]);
            }
            tmem_st8_async(mine + kL + T / 2 * part, hi);
            tmem_st8_async(mine + kL + 32 + T / 2 * part, lo);
        }
        {
            wait(&sm.done[kQueries], c);
            tc::fence_after_sync();
            float o[T];
            tmem_ld16(mine + kO + T * part, o);
            uint32_t y[T];
#pragma unroll
            for (int t = 0; t < T; t += 4) {
                const float4 since = *reinterpret_cast<const float4*>(vec + (4 + kSince) * C + t);
                const float2 z0 = mul2(pair_of(o + t), mul2(make_float2(since.x, since.y), ratio));
                const float2 z1 = mul2(pair_of(o + t + 2), mul2(make_float2(since.z, since.w), ratio));
                y[t] = __float_as_uint(z0.x), y[t + 1] = __float_as_uint(z0.y);
                y[t + 2] = __float_as_uint(z1.x), y[t + 3] = __float_as_uint(z1.y);
            }
            tc::tmem_st16_async(mine + kS + T * part, y);
            tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncthreads();
        if (fetches && c + 1 < n_chunks) {
            fetch_x(c + 1);
            fetch_q(c + 1);
        }
        if (warp == 0) {
            tc::fence_after_sync();
            wait(&sm.p_full, c);
            if (ok && tc::elect_one()) {
                const uint32_t p_at = here(sm.p);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    tc::mma_f16_tmem_a(tmem + (kt ? later(kt) : kS), tmem + kR + 8 * kt, plain_desc(p_at + tri(kt, kt), 128, 256),
                                       tc::idesc_f16(128, 64 - 16 * kt), kt == 0);
                tc::mma_commit(&sm.done[kOutputs]);
                const uint32_t k_at = here(sm.k[c & 1]), idesc = tc::idesc_f16(128, DK) | tc::kIdescTransposeB;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    const uint64_t b = plain_desc(k_at + kt * kRows16, 128, 1024);
                    tc::mma_f16_tmem_a(tmem + kT, tmem + kL + 8 * kt, b, idesc, kt > 0);
                    tc::mma_f16_tmem_a(tmem + kT, tmem + kL + 32 + 8 * kt, b, idesc, 1);
                }
                tc::mma_commit(&sm.done[kState]);
            }
            __syncwarp();
        }
        {
            wait(&sm.done[kOutputs], c);
            tc::fence_after_sync();
            float o[T];
            tmem_sum16(mine, kS, part, o);
            char* op = sm.o + T * part * 2 * kDv + 2 * row;
#pragma unroll
            for (int t = 0; t < T; t += 4) {
                const float4 pi = *reinterpret_cast<const float4*>(vec + (4 + kPi) * C + t);
                const float2 z0 = mul2(mul2(pair_of(o + t), udown), make_float2(pi.x, pi.y));
                const float2 z1 = mul2(mul2(pair_of(o + t + 2), udown), make_float2(pi.z, pi.w));
                const __nv_bfloat162 b0 = __floats2bfloat162_rn(z0.x, z0.y), b1 = __floats2bfloat162_rn(z1.x, z1.y);
                *reinterpret_cast<bf16*>(op + t * 2 * kDv) = b0.x;
                *reinterpret_cast<bf16*>(op + (t + 1) * 2 * kDv) = b0.y;
                *reinterpret_cast<bf16*>(op + (t + 2) * 2 * kDv) = b1.x;
                *reinterpret_cast<bf16*>(op + (t + 3) * 2 * kDv) = b1.y;
            }
        }
        // S = e^G_C S0 + U' e^(G_C - G) K
        {
            const float gamma = sm.vec[c & 1][kGamma * C];
            float step = ddown * up;
            if (!(step < 0x1p40f)) {  // the unit of what is added, where that is far larger
                const float by = dup * down;
#pragma unroll
                for (int i = 0; i < N; ++i) S[i] *= by;
                up = dup, down = ddown, step = 1.f;
            }
            wait(&sm.done[kState], c);
            tc::fence_after_sync();
#pragma unroll
            for (int i = 0; i < N; i += 16) {
                float d[16];
                tmem_ld16(mine + kT + part * N + i, d);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 y = tc::fma2(pair_of(S + i + j), make_float2(gamma, gamma), mul2(pair_of(d + j), step));
                    S[i + j] = y.x, S[i + j + 1] = y.y;
                }
            }
        }
    }
    tc::fence_before_sync();
    const bool failed = __syncthreads_or(!ok);
    tc::fence_after_sync();
    if (failed) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (lane == 0 && !ok) record_error(a.err, kErrTimeoutMma);
        int zero = 0;
        constexpr unsigned long long kLimit = 1000000000ull;
        if (fetches && lane == 0) {  // copies in flight
            for (int c = max(0, sm.asked[0] - 2); c < sm.asked[0]; ++c) tc::mbar_wait(&sm.k_full[c & 1], c >> 1 & 1, &zero, kLimit);
            if (sm.asked[1]) tc::mbar_wait(&sm.q_full, (sm.asked[1] - 1) & 1, &zero, kLimit);
            if (sm.asked[2]) tc::mbar_wait(&sm.x_full, (sm.asked[2] - 1) & 1, &zero, kLimit);
            if (sm.asked[3]) tc::mbar_wait(&sm.p_full, (sm.asked[3] - 1) & 1, &zero, kLimit);
        }
        if (warp < 2) {  // and MMAs
            if (tc::elect_one()) {
                tc::mma_commit(&sm.last[warp]);
                tc::mbar_wait(&sm.last[warp], 0, &zero, kLimit);
            }
            __syncwarp();
        }
    } else {
        if (n_chunks) store_outputs(n_chunks - 1);
        if (a.state_out) {
            const long long state0 = place();
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *reinterpret_cast<float4*>(a.state_out + state0 + i) = make_float4(S[i] * down, S[i + 1] * down, S[i + 2] * down, S[i + 3] * down);
        }
    }
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, kColumns);
}

template <int DK>
cudaError_t launch_dk(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    constexpr size_t bytes = sizeof(HeadSmem<DK>);
    static_assert(bytes <= 227 * 1024);
    static int done[64];
    const cudaError_t e = ensure_smem(delta_heads_kernel<DK>, bytes, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(delta_heads_kernel<DK>, dim3(static_cast<unsigned>(a.R * a.Hv)), dim3(kThreads), bytes, s, a, w);
}

}  // namespace

cudaError_t launch_delta_heads(const DeltaArgs& a, const Scratch& w, cudaStream_t s) {
    return a.Dk == 128 ? launch_dk<128>(a, w, s) : launch_dk<64>(a, w, s);
}

}  // namespace moestep
