// Attention over a paged bf16 or FP8 cache on tcgen05 tensor cores.
//
// One persistent CTA per SM takes an equal share of the key tiles (attn.cuh) and streams
// them once through shared memory, 128 keys at a time, with the running maximum and sum of
// the softmax.  The query rows of one (request, key-value head), n_q tokens x G heads, are
// the MMA's M = 128: S = Q K^T into tensor memory, P = 2^(S c - m) written back over S as
// bf16, O += P V with P read from tensor memory.
//
// Two streams run through each CTA, each with a softmax warpgroup, its S / P (128 columns) and
// its O (D columns), so that one stream's MMAs run under the other's exponentials:
//   more than 128 rows: the streams are two row tiles of 128 on the same keys;
//   else:               they take alternate key tiles of the same rows, each with its own (m, l, O).
// Where a lane has a whole row of the tile (65 rows and more) the tile passes in two halves of 64
// keys: the scores of the next tile's half are issued as soon as this half's weights have been
// multiplied, so a stream's MMAs also run under its own exponentials.
// Few rows would leave most of the 128 lanes idle and one lane with 128 exponentials a tile, so
// 32 (64) rows are held four (two) times, and warp w of a warpgroup computes only its quarter
// (half) of the tile's keys, the rest of its lanes' P being zero: each such copy is one more
// independent (m, l, O).  All of them meet in shared memory when a segment ends.
//
// The maximum m that the weights refer to moves only when a tile's maximum exceeds it by more
// than 8 (a factor 256, harmless in fp32 sums and bf16 weights): O is then rescaled in tensor
// memory by the softmax warps, which is rare after the first tiles (a known method).
//
// Weights are rounded to bf16 for P V, by 2^-8 at most, because that is the MMA's type; their sum l is of
// the unrounded ones.  S, m, l and O are fp32.
//
// FP8 cache.  Keys are multiplied as they are stored: a query row is scaled by a power of two and
// split into two E4M3 parts (4 significant bits each, the 8 of a bf16: see the staging), S is the
// sum of both parts' products, and the keys' powers of two come in with the softmax's scale.
// That halves the keys' way through shared memory and needs no conversion of them.  Weights have
// no such split, so values are turned into bf16 (code * 2^exp, exact) by eight converter warps.
//
// Warps: 0-7 softmax (two warpgroups), 8 and 11 TMA producers (keys, values), 9-10 MMA issuers (a
// stream each), with FP8 12-19 converters.
// Keys outside [lo, L) of the request reach no result: their scores are replaced by -inf, and
// their V rows, which a zero weight would still multiply (NaN), are zeroed in shared memory.
// Every wait is bounded (timeout -> error word, orderly teardown).
//
// What bounds it, measured with the join launch (16 query heads of 128 over 2, cold caches; in
// brackets the copy rate's time for the keys and values): single tokens of 16 ragged requests, up
// to 8192 positions, 26 us (12.1): starting up 4 us, the beginnings of two segments, eight tiles
// and the join; tensor pipe 21 % busy.  One token at 131072 FP8 positions 37 us (10.0): 13 tiles
// of 2700 cycles, issue slots 54 %.  32 tokens at 16384 positions 25 us (2.5): one beginning, two
// tiles, 128 KB of parts a CTA and their join.  16 such blocks, up to 32768 FP8 positions, 130 us
// (24.9; 43.6 by operations at the bf16 rate): 34 tiles of two row tiles, 4500 to 5000 cycles
// each, issue slots 60 %, tensor pipe 32 %: exponentials, conversions and staging share the issue
// slots.  (The compiler has 96 registers for all FP8 roles, what 640 threads leave at launch, and with
// heads of 128 spills 150 to 250 bytes.  By how it allocates them the batch takes 130 or 132 to 137 us, so
// what is added beside the softmax's loop is measured, not only counted.)
#include "attn.cuh"
#include "attn_tc.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

namespace moestep {
namespace {

constexpr int kKeys = 128;                        // keys of a tile
constexpr uint64_t kTeardown = 1000000000ull;     // limit for draining copies and MMAs in flight
constexpr uint64_t kAbortedTile = 1000000ull;     // for FP8 key tiles whose scales an aborted CTA did not write
constexpr int kStagger = 4;                       // key tiles of a share whose streams are put out of step (measured: D = 128)
constexpr float kSlack = 8.f;                     // how far a tile's maximum may pass m

// MODE 0, 1, 2: row tiles of 32, 64, 128 (one tile, streams on alternate keys); 3: of 256 (two tiles)
template <int D, int MODE, bool F8>
struct Cfg {
    static constexpr bool kTwo = MODE == 3;
    static constexpr int kRows = 32 << MODE;
    static constexpr int kRep = MODE == 0 ? 4 : MODE == 1 ? 2 : 1;
    static constexpr int kCols = kKeys / kRep;            // keys of a tile that a lane handles
    static constexpr int kHalves = kRep == 1 ? 2 : 1;     // turns in which a tile's keys pass through a stream
    static constexpr int kWide = kCols / kHalves;         // scores of a lane and turn: 32 or 64
    static constexpr int kConv = F8 ? 8 : 0;              // converter warps
    // FP8: 20 warps of 96 registers a thread, 61440 in all, redistributed: 256 softmax threads
    // x 136 (64 scores in registers) + 384 others x 64 = 59392
    static constexpr int kThreads = F8 ? 640 : 384;
    static constexpr int kSoftRegs = 136, kOtherRegs = 64;
    static_assert(!F8 || 256 * kSoftRegs + (kThreads - 256) * kOtherRegs <= kThreads * 96, "registers");
    static constexpr int kTile = kKeys * D * 2;           // bytes of a bf16 operand tile
    static constexpr int kKTile = F8 ? kKeys * D : kTile; // of keys, as they are multiplied
    static constexpr int kRaw = kKeys * D;                // of FP8 values
    static constexpr int kQ = 128 * D * 2;                // of queries (FP8: two E4M3 parts)
    // query tile(s); with one row tile also the merge buffer, once the segment's scores are done
    static constexpr int kFront = kTwo ? 2 * kQ : 32768;
    static constexpr int kMul = 128 / D;
    static constexpr int kNK = 3 * kMul;                               // key tiles
    static constexpr int kNV = (kTwo || F8 ? 2 : 3) * kMul;            // value tiles
    static constexpr int kNR = F8 ? (kTwo ? 2 : 4) * kMul : 0;         // FP8 value tiles as stored
    static constexpr int kNS = F8 ? kNK + 2 : 0;  // key tiles' scales: a turn's are read while the tiles two ahead land
    static constexpr int kMisc = 1024 + (F8 ? 1024 + (kNK + kNR) * kKeys + kNS * kKeys * 4 : 0);
    static constexpr int kSmem = 1024 + kFront + kNK * kKTile + kNV * kTile + kNR * kRaw + kMisc;
    static_assert(kSmem <= 232448, "shared memory");
};

// FP8 scores.  A product of codes is below 2^25 (D 448^2) and the keys' powers of two go up to 2^119, so
// the keys' factor is 2^(exp - 127) * 2^-17, finite wherever the score is, and the row's is 2^17 times the
// query's power.  Of a power above kBigQuery, which would take that factor past fp32's range, the rest
// comes in by a multiplication beside the masking of a partial tile (16 blocks of 32 tokens, up to 32768
// positions, 129.1 -> 129.8 us; as a branch of its own 134 to 137 us).  The scale's mantissa is among the
// keys' factors too: see unit_of.
constexpr float kKeyShift = 0x1p17f, kBigQuery = 0x1p32f;
__device__ __forceinline__ float key_scale(uint32_t e) {  // of an exponent byte
    return __uint_as_float(e > 17 ? (e - 17) << 23 : 1u << (e + 5));
}
// Scores beyond 2^30.  Fp32 holds multiples of 64 of them, so their softmax is one key's (or some equal
// ones'), and weights are 2^(S c - m), a fused product: with c of 24 bits it is off a maximum m that was
// rounded by up to half a step of it, which from 2^31 on takes the largest weight itself out of range.
// FP8: c is a power of two (the scale's mantissa is in the keys' factors), so that m is exact.  bf16: such
// a row's scores are counted in a unit that brings the maximum down to 2^30, a power of two that leaves
// neighbouring scores 32 apart.
__device__ __forceinline__ float unit_of(float top) {
    const uint32_t e = __float_as_uint(top) >> 23 & 255;
    return e > 127 + 30 && e < 255 ? __uint_as_float((2 * 127 + 30 - e) << 23) : 1.f;
}
__device__ __forceinline__ float ratio_pow2(float a, float b) {  // of two floats with the same mantissa
    return __uint_as_float(__float_as_uint(a) - __float_as_uint(b) + (127u << 23));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 32 columns of the output.  The FP8 converters leave every four columns of the values in the order
// 0, 2, 1, 3 (see there): they are put back.
template <bool F8>
__device__ __forceinline__ void load_output(uint32_t taddr, float* x) {
    tc::tmem_ld32(taddr, x);
    if (F8) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float t = x[i + 1];
            x[i + 1] = x[i + 2];
            x[i + 2] = t;
        }
    }
}

// A warp's bounded waits.  Lane 0 alone polls the barrier (a poll is served lane by lane: with all
// 32 a wait on a phase long complete took 300 cycles).  Once one gave up, the rest return at once.
struct Waits {
    volatile int* abort;
    long long limit;  // cycles
    bool ok;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
        if (ok) {
            int r = 1;
            if ((threadIdx.x & 31) == 0) r = tc::mbar_wait_cycles(bar, parity, abort, limit);
            ok = __shfl_sync(0xffffffffu, r, 0) != 0;
            __syncwarp();
        }
        return ok;
    }
    // two barriers, polled by two lanes
    __device__ __forceinline__ bool both(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1) {
        if (ok) {
            const int l = threadIdx.x & 31;
            int r = 1;
            if (l < 2) r = tc::mbar_wait_cycles(l ? bar1 : bar0, l ? parity1 : parity0, abort, limit);
            ok = __all_sync(0xffffffffu, r) != 0;
            __syncwarp();
        }
        return ok;
    }
};

// The buffers of a segment of n key tiles in the order in which the MMAs use them: number i of
// 2 n is the keys or the values of a tile.  Two row tiles: K0 V0 K1 V1 ..; else, with two key
// tiles in work, K0 K1 V0 K2 V1 K3 .. V(n-2) V(n-1).  (One loop over i at every place that goes
// through them: the code of all roles together has to stay small, or it runs at the speed of
// its instruction fetches.)
struct Buffer {
    bool v;
    int tile;
};
template <bool TWO>
__device__ __forceinline__ Buffer buffer_of(int i, int n) {
    if (TWO) return {(i & 1) != 0, i >> 1};
    if (i == 2 * n - 1) return {true, n - 1};
    if (i < 2) return {false, i};
    return {(i & 1) == 0, (i & 1) == 0 ? (i >> 1) - 1 : (i + 1) >> 1};
}

template <int D, int MODE, bool F8>
__global__ void __launch_bounds__(Cfg<D, MODE, F8>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const AttnArgs a) {
    using C = Cfg<D, MODE, F8>;
    constexpr int NK = C::kNK, NV = C::kNV, NR = F8 ? C::kNR : 1, NS = F8 ? C::kNS : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = sm;
    uint8_t* vring = sq + C::kFront;
    uint8_t* kring = vring + NV * C::kTile;
    uint8_t* raw = kring + NK * C::kKTile;
    float* kscale = reinterpret_cast<float*>(raw + C::kNR * C::kRaw);        // FP8 [NS][128]: factors of keys
    float* qscale = kscale + C::kNS * kKeys;                                 // FP8 [256]: powers of two of query rows
    uint8_t* kexps = reinterpret_cast<uint8_t*>(qscale + (F8 ? 256 : 0));    // FP8 [NK][128]
    uint8_t* exps = kexps + (F8 ? NK * kKeys : 0);                           // FP8 [NR][128] of values
    int* plan_sm = reinterpret_cast<int*>(exps + C::kNR * kKeys);            // 40
    uint64_t* kfull = reinterpret_cast<uint64_t*>(plan_sm + 40);
    uint64_t* kempty = kfull + NK;
    uint64_t* vfull = kempty + NK;
    uint64_t* vempty = vfull + NV;
    uint64_t* rfull = vempty + NV;   // FP8 values as stored
    uint64_t* rempty = rfull + C::kNR;
    uint64_t* xfull = rempty + C::kNR;  // FP8 keys' exponents
    uint64_t* s_full = xfull + (F8 ? NK : 0);
    uint64_t* p_full = s_full + 4;  // both [stream][half]
    uint64_t* o_full = p_full + 4;
    uint64_t* pv_done = o_full + 2;  // [stream] each product of weights and values
    uint64_t* q_full = pv_done + 2;
    uint64_t* fin = q_full + 1;
    uint64_t* go = fin + 1;  // the first stream has begun a segment (two row tiles)
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(go + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    int* zero_flag = abort_flag + 1;
    static_assert((3 * NK + 2 * NV + 2 * C::kNR + 15) * 8 + 12 + 160 <= 1024, "misc area");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            tc::mbar_init(&kfull[i], F8 ? 2 : 1);  // the copy, and the scales
            tc::mbar_init(&kempty[i], 2);          // both MMA issuers
            if (F8) tc::mbar_init(&xfull[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            tc::mbar_init(&vfull[i], F8 ? C::kConv : 1);
            tc::mbar_init(&vempty[i], 2);
        }
        for (int i = 0; i < C::kNR; ++i) {
            tc::mbar_init(&rfull[i], 1);
            tc::mbar_init(&rempty[i], C::kConv);
        }
        for (int g = 0; g < 2; ++g) {
            for (int q = 0; q < C::kHalves; ++q) {
                tc::mbar_init(&s_full[g * 2 + q], 1);
                tc::mbar_init(&p_full[g * 2 + q], 4);
            }
            tc::mbar_init(&o_full[g], 1);
            tc::mbar_init(&pv_done[g], 1);
        }
        tc::mbar_init(q_full, 8);
        tc::mbar_init(fin, 2);
        tc::mbar_init(go, 4);
        *abort_flag = 0;
        *zero_flag = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_holder, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // (from one lane, so that the compiler knows it for uniform: an MMA whose accumulator address is
    // not issues in 97 cycles instead of 67)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    pdl_trigger();
    pdl_wait();
    const AttnPlan plan = attn_plan<kKeys, C::kThreads>(a, plan_sm);
    // (two cycles a nanosecond: the SM clock stays below 2.1 GHz)
    Waits wait{abort_flag, static_cast<long long>(a.timeout_ns < (1ull << 61) ? 2 * a.timeout_ns : 1ull << 62), true};
    int err_bits = 0;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax and output
        if (F8) tc::more_registers<C::kSoftRegs>();
        const int g = warp >> 2, w = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        const uint32_t t_s = tmem + lanes + g * 128, t_o = tmem + lanes + 256 + g * 128;
        const int part = MODE == 0 ? w : MODE == 1 ? w >> 1 : 0;        // which of the tile's keys
        const int lrow = C::kTwo ? g * 128 + w * 32 + lane               // row within the row tile
                                 : (w * 32 + lane) & (C::kRows - 1);
        const int col0 = part * C::kCols;
        uint32_t tiles_g = 0, turns_g = 0, segs = 0, kt0 = 0;
        // The eight warps meet at a hardware barrier between the steps of a merge.  They pass it
        // equally often whatever happens: after a wait that gave up they go through the rest of
        // their segments without waiting (their results are then unspecified).
        auto sync8 = [&]() { tc::named_bar_sync(1, 256); };
        AttnWalk s = attn_begin<kKeys>(a, plan);
        while (attn_next<kKeys>(a, s)) {
            const int h = s.h, row0 = s.rt * C::kRows;
            const int nrows = min(C::kRows, a.rows - row0);
            {   // query rows into the swizzled operand tile(s), copies for lanes that repeat rows
                constexpr int kChunks = D / 8, NT = C::kTwo ? 128 : 256, kBatch = 128 * kChunks / NT;
                uint8_t* dst = sq + (C::kTwo ? g * C::kQ : 0);
                const int c = threadIdx.x % kChunks, m0 = (threadIdx.x & (NT - 1)) / kChunks;
                constexpr int kStep = NT / kChunks;  // rows apart
                // (all loads in flight at once, ahead of the key and value copies that follow)
                uint4 x[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int m = m0 + b * kStep, row = C::kTwo ? g * 128 + m : m & (C::kRows - 1);
                    x[b] = make_uint4(0, 0, 0, 0);
                    if (row < nrows) {
                        const int rr = row0 + row, qi = attn_query(a, rr);
                        x[b] = __ldg(reinterpret_cast<const uint4*>(
                            static_cast<const bf16*>(a.q) + (static_cast<long long>(s.r) * a.n_q + qi) * a.q_ld +
                            (h * a.G + rr - qi * a.G) * D + c * 8));
                    }
                }
                __syncwarp();
                // Two row tiles: the segment before left through the query tile, a part a warp, and
                // these rows go to all parts.  (One row tile: the merge ended with a barrier.)
                if (C::kTwo && s.k > 0) tc::named_bar_sync(2 + g, 128);
                // (four pieces of code in a loop, the loaded pieces moved up: unrolled in full, the
                // instructions alone took 7 us to arrive)
#pragma unroll 1
                for (int mb = m0; mb < 128; mb += 4 * kStep) {
                    uint4 y[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) y[u] = x[u];
#pragma unroll
                    for (int b = 0; b + 4 < kBatch; ++b) x[b] = x[b + 4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int m = mb + u * kStep;
                        const uint4 piece16 = y[u];
                        if (!F8) {
                            *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + m * 128 + (((c & 7) ^ (m & 7)) << 4)) = piece16;
                            continue;
                        }
                        // A row times a power of two that brings it to at most 448, as the sum of two E4M3
                        // parts: the first takes the leading 4 bits of a bf16's 8, the second the rest.
                        // Exact for elements of 1/4 and more; below that the second's smallest step,
                        // 2^-9, leaves an error of at most 2^-10, against a largest element above
                        // 224: 2^-17 of it (in rows below 2^-117, which no normal power brings there, 2^-136).
                        // An infinite row gives NaN scores.
                        const uint32_t w[4] = {piece16.x, piece16.y, piece16.z, piece16.w};
                        float amax = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
                        for (int o = kChunks / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        const uint32_t bits = __float_as_uint(amax);
                        int e = static_cast<int>(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u);  // 448 = 0.875 * 2^9
                        e = min(max(e, -126), 119);
                        const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                        if (c == 0)
                            qscale[(C::kTwo ? g * 128 : 0) + m] = bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                                                      : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                        uint32_t hi[2], lo[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t p[2], q[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float y0 = __uint_as_float(w[2 * i + j] << 16) * s, y1 = __uint_as_float(w[2 * i + j] & 0xffff0000u) * s;
                                p[j] = to_e4m3x2(y0, y1);
                                const uint32_t h2 = tc::e4m3x2_to_f16x2(p[j], 0);
                                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                                q[j] = to_e4m3x2(y0 - f.x, y1 - f.y);
                            }
                            hi[i] = p[0] | p[1] << 16;
                            lo[i] = q[0] | q[1] << 16;
                        }
                        const int piece = D == 128 ? (c >> 1) ^ (m & 7) : (c >> 1) ^ ((m >> 1) & 3);  // TMA's swizzles
                        uint8_t* d = dst + m * D + (piece << 4) + (c & 1) * 8;
                        *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(d + 128 * D) = make_uint2(lo[0], lo[1]);
                    }
                }
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(q_full);
            }
            const int2 see = attn_sees(a, s.L, attn_query(a, row0 + min(lrow, nrows - 1)));
            if (F8) __syncwarp();
            float scl = a.scale_log2;  // of this row's scores; FP8: read once the queries are staged; bf16: see unit_of
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            const int step = C::kTwo ? 1 : 2, first = s.tile + (C::kTwo ? 0 : g);
            int turn = 0;
            uint32_t kt = kt0 + first - s.tile;  // number of the key tile among all of the CTA's
            kt0 += s.tiles;
            for (int t = first; t < s.tile + s.tiles; t += step, ++tiles_g, kt += step)
#pragma unroll 1
            for (int half = 0; half < C::kHalves; ++half, ++turn) {  // (both loops' body)
                wait(&s_full[g * 2 + half], tiles_g & 1);
                tc::fence_after_sync();
                if (F8 && turn == 0) {
                    const float q = qscale[C::kTwo ? lrow : w * 32 + lane];
                    scl = a.scale_log2 * ((q > kBigQuery ? kBigQuery : q) * kKeyShift);
                }
                const uint32_t t_x = t_s + half * 64;  // this turn's scores, then its weights
                const int c0 = col0 + half * 64;
                const int lo = see.x - (t * kKeys + c0), hi = see.y - (t * kKeys + c0);
                const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < C::kWide ||  // or a big query's row
                                                                (F8 && scl >= a.scale_log2 * (kBigQuery * kKeyShift)));
                constexpr int kHold = C::kWide;  // scores held in registers between the two passes
                float v[kHold];
                float mx = -INFINITY;
                auto fetch = [&](int c) {  // kHold of the lane's scores, the hidden ones replaced
                    const uint32_t at = C::kRep == 1 ? t_x + c : t_s + col0 + c;
                    if constexpr (kHold == 64) tc::tmem_ld64(at, v);
                    else tc::tmem_ld32(at, v);
                    if (F8) {
                        const float* ks = kscale + (kt % NS) * kKeys + c0 + c;
#pragma unroll
                        for (int i = 0; i < kHold; i += 4) {
                            const float4 k4 = *reinterpret_cast<const float4*>(ks + i);
                            v[i] *= k4.x, v[i + 1] *= k4.y, v[i + 2] *= k4.z, v[i + 3] *= k4.w;
                        }
                    }
                    if (masked) {
                        if (F8) {
                            const float q = qscale[C::kTwo ? lrow : w * 32 + lane], x = q > kBigQuery ? q * (1.f / kBigQuery) : 1.f;
#pragma unroll
                            for (int i = 0; i < kHold; i += 2) {
                                const float2 y = tc::mul2(make_float2(v[i], v[i + 1]), make_float2(x, x));
                                v[i] = y.x, v[i + 1] = y.y;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kHold; ++i) v[i] = (c + i >= lo && c + i < hi) ? v[i] : -INFINITY;
                    }
                };
                fetch(0);
#pragma unroll
                for (int i = 0; i < kHold; i += 2) mx = fmaxf(mx, fmaxf(v[i], v[i + 1]));
                mx *= scl;
                const bool move = mx > m + kSlack || (m == -INFINITY && mx > m);
                if (__any_sync(0xffffffffu, move)) {
                    if (!F8 && move) {  // in units of 1, then of this maximum
                        const float up = ratio_pow2(a.scale_log2, scl);
                        m *= up, mx *= up;
                    }
                    const float f = move ? tc::exp2_fast(m - mx) : 1.f;  // 0 from m = -inf
                    if (move) m = mx;
                    if (!F8 && move) {
                        const float unit = unit_of(m);
                        scl = a.scale_log2 * unit;
                        m *= unit;
                    }
                    l2 = make_float2(l2.x * f, l2.y * f);
                    if (turn > 0) {
                        if (C::kHalves > 1) {  // the half before is multiplied meanwhile
                            wait(&pv_done[g], (turns_g + turn - 1) & 1);
                            tc::fence_after_sync();
                        }
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tc::tmem_ld32(t_o + c, o);
                            uint32_t u[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
                            tc::tmem_st16_async(t_o + c, u);
                            tc::tmem_st16_async(t_o + c + 16, u + 16);
                        }
                    }
                }
                const float ms = m == -INFINITY ? 0.f : m;
                if (C::kTwo && g == 0 && turn == 0 && lane == 0) tc::mbar_arrive(go);
                const float2 c2 = make_float2(scl, scl), m2 = make_float2(-ms, -ms);
#pragma unroll
                for (int j = 0; j < kHold; j += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = tc::fma2(make_float2(v[j + 2 * i], v[j + 2 * i + 1]), c2, m2);
                        x = make_float2(tc::exp2_fast(x.x), tc::exp2_fast(x.y));
                        l2 = tc::add2(l2, x);
                        p[i] = tc::pack_bf16(x.x, x.y);
                    }
                    tc::tmem_st16_async((C::kRep == 1 ? t_x : t_s + col0 / 2) + j / 2, p);
                }
                if (C::kRep > 1) {  // the other copies' keys (after the lane's own scores have been read)
                    const uint32_t z[16] = {};
#pragma unroll
                    for (int c = 0; c < kKeys / 2; c += 16)
                        if (c / (C::kCols / 2) != part) tc::tmem_st16_async(t_s + c, z);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_full[g * 2 + half]);
            }
            turns_g += turn;
            if (!F8) m *= ratio_pow2(a.scale_log2, scl);
            const float l = l2.x + l2.y;
            wait(&o_full[g], segs & 1);
            ++segs;
            tc::fence_after_sync();
            const int slot = 2 * blockIdx.x + (s.k > 0);
            // row `rr` of the row tile: where it goes
            auto where = [&](int rr) {
                const int row = row0 + rr, qi = attn_query(a, row);
                return (static_cast<size_t>(s.r) * a.n_q + qi) * a.Hq + h * a.G + row - qi * a.G;
            };
            if constexpr (C::kTwo) {
                // Each warp passes its 32 rows through its own part of the query tile, which is no
                // longer read, so that whole lines are written.
                const bool on = lrow < nrows;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                constexpr int kPart = 32 * D * 2;  // bytes: 32 rows of bf16, or half of their fp32 columns
                uint8_t* mine = sq + g * C::kQ + w * kPart;
                const int wrow0 = g * 128 + w * 32, wrows = min(32, nrows - wrow0);
                constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;  // lanes of a row, 16 bytes each
                const int sr = lane / kLanes, sc = lane % kLanes;
                const int halves = s.whole ? 1 : 2;
#pragma unroll 1
                for (int half = 0; half < halves; ++half) {
#pragma unroll 1
                    for (int c = 0; c < (s.whole ? D : D / 2); c += 32) {
                        float x[32];
                        __syncwarp();
                        load_output<F8>(t_o + half * (D / 2) + c, x);
                        uint8_t* r = mine + lane * D * 2;
                        if (s.whole) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4*>(r + (((c / 8 + i) ^ (lane & 7)) << 4)) =
                                    make_uint4(tc::pack_bf16(x[8 * i] * inv, x[8 * i + 1] * inv),
                                               tc::pack_bf16(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                                               tc::pack_bf16(x[8 * i + 4] * inv, x[8 * i + 5] * inv),
                                               tc::pack_bf16(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4*>(r + (((c / 4 + i) ^ (lane & 7)) << 4)) =
                                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        }
                    }
                    if (!s.whole) {  // as it stands, swizzle and all: one copy for the join to unravel
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tc::bulk_store(a.part_o + ((static_cast<size_t>(slot) * 2 + half) * 256 + wrow0) * (D / 2),
                                           mine, kPart);
                            tc::bulk_stores_read();
                        }
                        __syncwarp();
                        continue;
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = 0; i < 32; i += kRowsAtOnce) {
                        const int rr = i + sr;
                        if (rr >= wrows) continue;
                        *reinterpret_cast<uint4*>(static_cast<bf16*>(a.out) + where(wrow0 + rr) * D + sc * 8) =
                            *reinterpret_cast<const uint4*>(mine + rr * D * 2 + ((sc ^ (rr & 7)) << 4));
                    }
                }
                __syncwarp();
                if (on && s.whole && a.lse) a.lse[where(lrow)] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                if (on && !s.whole) a.part_ml[static_cast<size_t>(slot) * a.slot_rows + lrow] = make_float2(m, l);
            } else {
                // merge the row's (m, l, O): p = stream * copies + copy
                constexpr int kParts = 2 * C::kRep;
                const int p = g * C::kRep + part;
                float2* ml = reinterpret_cast<float2*>(sq);  // [parts][rows]
                sync8();  // neither stream reads the query tile any more
                ml[p * C::kRows + lrow] = make_float2(m, l);
                sync8();
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < kParts; ++i) M = fmaxf(M, ml[i * C::kRows + lrow].x);
                const float Ms = M == -INFINITY ? 0.f : M;
                const float f = tc::exp2_fast(m - Ms);
                // The buffer holds 32768 / (parts * rows * 4) columns of every part's valid rows, a
                // multiple of 32: all of D at once where rows are few.  Threads of a group of
                // 256 / rows put together a row's columns, four at a time.
                const int wide = C::kRows == 32 && nrows <= 8 ? min(D, 128) : C::kRows == 32 && nrows <= 16 ? 64 : 32;
                const int trow = C::kRows == 32 && nrows <= 8 ? 8 : C::kRows == 32 && nrows <= 16 ? 16 : C::kRows;
                const int tpr = 256 / trow, orow = threadIdx.x / tpr, ocol = (threadIdx.x % tpr) * 4;
                float OM = -INFINITY, ol = 0.f;
#pragma unroll
                for (int i = 0; i < kParts; ++i) OM = fmaxf(OM, ml[i * C::kRows + orow].x);
                const float OMs = OM == -INFINITY ? 0.f : OM;
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const float2 q = ml[i * C::kRows + orow];
                    ol += q.y * tc::exp2_fast(q.x - OMs);
                }
                const bool on = orow < nrows;
                const size_t o = on ? where(orow) : 0, at = static_cast<size_t>(slot) * a.slot_rows + orow;
                const float inv = ol == 0.f ? 0.f : 1.f / ol;
                float* buf = reinterpret_cast<float*>(sq);  // [parts][trow][wide], 16-byte pieces swizzled by row
                sync8();  // the statistics have been read
#pragma unroll 1
                for (int c = 0; c < D; c += wide) {
                    float* b = buf + (p * trow + lrow) * wide;
#pragma unroll 1
                    for (int cc = 0; cc < wide; cc += 32) {
                        float x[32];
                        __syncwarp();
                        if (turn > 0) {
                            load_output<F8>(t_o + c + cc, x);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = 0.f;
                        }
                        if (lrow < nrows) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4*>(b + cc + ((i ^ (lrow & 7)) << 2)) =
                                    make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
                        }
                    }
                    sync8();
                    if (on) {
                        for (int k = ocol; k < wide; k += 4 * tpr) {
                            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                            const int kk = (k & ~31) + ((((k & 31) >> 2) ^ (orow & 7)) << 2);
#pragma unroll
                            for (int i = 0; i < kParts; ++i) {
                                const float4 z = *reinterpret_cast<const float4*>(buf + (i * trow + orow) * wide + kk);
                                y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
                            }
                            if (s.whole)
                                *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + o * D + c + k) = make_uint2(
                                    tc::pack_bf16(y.x * inv, y.y * inv), tc::pack_bf16(y.z * inv, y.w * inv));
                            else
                                *reinterpret_cast<float4*>(a.part_o + at * D + c + k) = y;
                        }
                    }
                    sync8();  // the slice has been read
                }
                if (on && ocol == 0) {
                    if (!s.whole) a.part_ml[at] = make_float2(OM, ol);
                    else if (a.lse) a.lse[o] = ol == 0.f ? -INFINITY : (OM + log2f(ol)) * 0.69314718055994531f;
                }
            }
        }
        if (C::kTwo && lane == 0) tc::bulk_stores_done();
        if (!wait.ok) err_bits = kErrTimeoutEpilogue;
    } else {
    if (F8) tc::fewer_registers<C::kOtherRegs>();
    if (warp == 8 || warp == 11) {
        // ------------------------------------------------------------ TMA producers: keys, values
        const bool v = warp == 11;
        uint64_t* const bf = !v ? kfull : F8 ? rfull : vfull;
        uint64_t* const be = !v ? kempty : F8 ? rempty : vempty;
        const CUtensorMap* map = v ? &vmap : &kmap;
        uint8_t* const base = !v ? kring : F8 ? raw : vring;
        const int bytes = !v ? C::kKTile : F8 ? C::kRaw : C::kTile, N = v ? (F8 ? NR : NV) : NK;
        const uint8_t* const ex = v ? a.v_exp : a.k_exp;
        int b = 0;              // buffer
        uint32_t it = 0, ph = 0;  // buffers so far, times round the ring
        const int page = 1 << a.page_log2, pages = kKeys >> a.page_log2;
        AttnWalk s = attn_begin<kKeys>(a, plan);
        while (wait.ok && attn_next<kKeys>(a, s)) {
            const int h = s.h, lo = attn_lo(a, s.L);
            const int32_t* tab = a.table + static_cast<long long>(s.r) * a.max_pages;
            // Page numbers come 32 at a time, a lane each, the next 32 while these are used: a
            // table read behind the copies in flight takes as long as they do.
            const int pg0 = (s.tile * kKeys) >> a.page_log2, pg_lo = lo >> a.page_log2;
            const int pg_end = (min(s.L, (s.tile + s.tiles) * kKeys) + page - 1) >> a.page_log2;
            auto table = [&](int at) -> int {  // entries at .. at + 31
                const int pg = at + lane;
                return pg >= pg_lo && pg < pg_end ? __ldg(&tab[pg]) : -2;
            };
            int chunk = pg0, ids = table(chunk), ids_next = table(chunk + 32);
#pragma unroll 1
            for (int at = pg0; at < pg0 + s.tiles * pages; at += pages, ++it) {
                if (at >= chunk + 32) {
                    chunk += 32;
                    ids = ids_next;
                    ids_next = table(chunk + 32);
                }
                // lane l: page l of the tile, -2 for one that is not loaded
                const int id = __shfl_sync(0xffffffffu, ids, (at - chunk + lane) & 31);
                const bool here = lane < pages && id != -2;
                const bool good = here && static_cast<unsigned>(id) < static_cast<unsigned>(a.n_pages);
                if (here && !good) record_error(a.err, kErrBadInput);
                const unsigned on = __ballot_sync(0xffffffffu, good);
                const int y = good ? (id * a.Hkv + h) << a.page_log2 : 0;
                const int keys = __popc(on) * page;
                if (!wait(&be[b], ph ^ 1u)) break;
                uint64_t* ebar = F8 && !v ? &xfull[b] : &bf[b];  // what the exponents' copies report to
                if (lane == 0) {
                    if (F8 && !v) tc::mbar_arrive_expect_tx(ebar, keys);
                    tc::mbar_arrive_expect_tx(&bf[b], keys * (F8 ? D + v : 2 * D));
                }
                __syncwarp();
                uint8_t* dst = base + b * bytes;
                uint8_t* edst = (v ? exps : kexps) + b * kKeys;
#pragma unroll 1
                for (int p = 0; p < pages; ++p) {
                    const int yp = __shfl_sync(0xffffffffu, y, p);
                    if (!(on >> p & 1)) continue;
                    if (tc::elect_one()) {
                        if (F8) {
                            tc::tma_load_2d(dst + p * page * D, map, &bf[b], 0, yp);
                            tc::bulk_load(edst + p * page, ex + yp, page, ebar);
                        } else {
#pragma unroll
                            for (int half = 0; half < D / 64; ++half)
                                tc::tma_load_2d(dst + half * 16384 + p * page * 128, map, &bf[b], half * 64, yp);
                        }
                    }
                    __syncwarp();
                }
                if (++b == N) b = 0, ph ^= 1u;
            }
        }
        if (!wait.ok) err_bits = kErrTimeoutProducer;
        // copies in flight land before the CTA ends
        if (lane == 0) {
            for (uint32_t i = it > N ? it - N : 0; i < it; ++i) {
                const int w = i % N;
                const uint32_t parity = (i / N) & 1;
                // (a phase of FP8 keys also needs their scales, which an aborted CTA may not write)
                if (F8 && !v) tc::mbar_wait(&xfull[w], parity, zero_flag, kTeardown);
                tc::mbar_wait(&bf[w], parity, zero_flag, F8 && !v && !wait.ok ? kAbortedTile : kTeardown);
            }
        }
        __syncwarp();
    } else if (warp < 11) {
        // ------------------------------------------------------------ MMA issuers, one a stream
        // With two row tiles the second stream's first scores wait until the first stream's weights
        // are under way, so that one's MMAs run under the other's exponentials: in step with each
        // other both waited for both.  (Not in a short share, which would only end later by that
        // much: 32 tokens at 16384 positions, two tiles a CTA, 26.8 -> 25.6 us.)
        const int g = warp - 9;
        if (g == 1 && lane == 0) attn_describe_join<kKeys>(a, plan);
        __syncwarp();
        constexpr uint32_t idesc_s = F8 ? tc::idesc_e4m3(128, kKeys / C::kHalves) : tc::idesc_bf16(128, kKeys / C::kHalves);
        constexpr uint32_t idesc_o = tc::idesc_bf16(128, D) | tc::kIdescTransposeB;
        const uint32_t t_s = tmem + g * 128, t_o = tmem + 256 + g * 128;
        auto sdesc = [](const void* p) {
            return F8 && D == 64 ? tc::sdesc_k_sw64(tc::smem_addr(p)) : tc::sdesc_k_sw128(tc::smem_addr(p));
        };
        const uint64_t qd = sdesc(sq + (C::kTwo ? g * C::kQ : 0)), kd0 = sdesc(kring);
        const uint64_t vd0 = tc::sdesc_mn_sw128(tc::smem_addr(vring), 16384);
        // Every buffer is waited for and released in order, the other stream's too: a parity names
        // a phase only as long as nobody skips one or falls two behind.
        uint32_t ik = 0, iv = 0, segs = 0, turns = 0;
        auto ready = [&](bool v) -> bool {
            return v ? wait(&vfull[iv % NV], (iv / NV) & 1) : wait(&kfull[ik % NK], (ik / NK) & 1);
        };
        auto pass = [&](bool v) -> bool {  // a buffer of the other stream's
            if (!ready(v)) return false;
            if (lane == 0) tc::mbar_arrive(v ? &vempty[iv % NV] : &kempty[ik % NK]);
            if (v) ++iv;
            else ++ik;
            return true;
        };
        auto scores = [&](int half) {  // Q K^T of half the keys of buffer ik
            const int b = ik % NK;
            // (descriptors count in 16 bytes)
            const uint64_t kd = kd0 + b * (C::kKTile >> 4) + half * (F8 ? 4 * D : 512);
            tc::fence_after_sync();
            if (tc::elect_one()) {
                if (F8) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)  // of the queries
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            tc::mma_e4m3(t_s + half * 64, qd + part * (128 * D / 16) + k * 2, kd + k * 2, idesc_s,
                                         part > 0 || k > 0);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int off = (k >> 2) * 1024 + (k & 3) * 2;
                        tc::mma_bf16(t_s + half * 64, qd + off, kd + off, idesc_s, k > 0);
                    }
                }
                tc::mma_commit(&s_full[g * 2 + half]);
                if (half == C::kHalves - 1) tc::mma_commit(&kempty[b]);
            }
            __syncwarp();
        };
        AttnWalk s = attn_begin<kKeys>(a, plan);
        while (wait.ok && attn_next<kKeys>(a, s)) {
            const int lo = attn_lo(a, s.L), n = s.tiles;
            if (!wait(q_full, segs & 1)) break;
            if (C::kTwo && g == 1 && n >= kStagger && !wait(go, segs & 1)) break;
            ++segs;
            // A stream without a tile here reports at once: the softmax warps stage the next segment's
            // queries only once both issuers have taken these (q_full's parity names one of two phases).
            if (!C::kTwo && g >= n && lane == 0) tc::mbar_arrive(&o_full[g]);
            constexpr int kNext = C::kTwo ? 1 : 2;  // from one of the stream's key tiles to the next
            uint32_t begun = 0;
            // t = -kNext ..: the values of tile t, and the scores of the stream's next tile, each
            // half taking the place of the weights just used
#pragma unroll 1
            for (int t = -kNext; t < n && wait.ok; ++t) {
                const bool now = t >= 0, more = t + kNext < n;
                if (!C::kTwo && ((t ^ g) & 1)) {
                    if ((!now || pass(true)) && more) pass(false);
                    continue;
                }
                const int b = iv % NV;
                if (now && !ready(true)) break;
                const int j0 = (s.tile + t) * kKeys, za = max(lo - j0, 0), zb = min(s.L - j0, kKeys);
                // V's keys in steps of 16: those that some query sees, one step at least; the rows
                // of the first and last step that none sees are zeroed (by both streams alike)
                const int k0 = min(za >> 4, 7), k1 = max((zb + 15) >> 4, k0 + 1);
                if (!F8 && now && ((za & 15) != 0 || (zb & 15) != 0 || zb <= 0)) {
                    uint8_t* v = vring + b * C::kTile;
#pragma unroll 1
                    for (int i = lane; i < 2 * 16 * (D / 8); i += 32) {
                        const int r = (i >> 3) & 31, row = r < 16 ? k0 * 16 + r : k1 * 16 - 32 + r;
                        if (row < za || row >= zb)
                            *reinterpret_cast<uint4*>(v + (i >> 8) * 16384 + row * 128 + (i & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint64_t vd = vd0 + b * (C::kTile >> 4);
                constexpr int kPer = 8 / C::kHalves;
#pragma unroll 1
                for (int half = 0; half < C::kHalves; ++half) {
                    if (now) {
                        if (!wait(&p_full[g * 2 + half], turns & 1)) break;
                        tc::fence_after_sync();
                        const uint32_t tp = t_s + half * 64;
                        const uint64_t vh = vd + half * kPer * 128;
                        if (tc::elect_one()) {
#pragma unroll
                            for (int k = 0; k < kPer; ++k)
                                if (k >= k0 - half * kPer && k < k1 - half * kPer) {
                                    tc::mma_f16_tmem_a(t_o, tp + k * 8, vh + k * 128, idesc_o, begun);
                                    begun = 1;
                                }
                            if (C::kHalves > 1) tc::mma_commit(&pv_done[g]);
                            if (half == C::kHalves - 1) {
                                tc::mma_commit(&vempty[b]);
                                if (!more) tc::mma_commit(&o_full[g]);
                            }
                        }
                        __syncwarp();
                    }
                    if (more) {
                        if (half == 0 && !ready(false)) break;
                        scores(half);
                    }
                }
                if (now) ++turns, ++iv;
                if (more) ++ik;
            }
        }
        if (!wait.ok) err_bits = kErrTimeoutMma;
        __syncwarp();
        if (tc::elect_one()) {  // MMAs in flight complete before the tensor memory is freed
            tc::mma_commit(fin);
            tc::mbar_wait(fin, 0, zero_flag, kTeardown);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ FP8 converters
        // Eight lanes take 64 codes of a key, 8 each, and write the 16-byte piece of the 128-byte
        // swizzled bf16 tile that holds them; each lane does that twice a step (D = 128: the key's
        // other half, the halves in the other order for odd keys, so that two keys' lanes read
        // different banks; D = 64: four keys further on).
        // A code s eeee mmm placed as s 0000eeee mmm0000 is the bf16 value code * 2^-120,
        // subnormals included, so one exact multiplication by 2^(exp - 127 + 120) dequantises two
        // codes (two of them where that factor passes bf16's range).  The four codes of a word
        // are placed as bytes 0 and 2, then 1 and 3, which is the column order 0, 2, 1, 3.  The
        // conversion instruction would share its unit with the exponentials (2300 cycles a
        // tile instead of ~1000); NaN codes, which the placement does not keep, are rare and patched.
        const int cw = warp - 12;
        constexpr int kStepRows = D == 128 ? 4 : 8, kStepsC = 16 / kStepRows;  // of a warp's 16 keys
        const int lr = lane >> 3, lc = lane & 7;
        uint32_t ik = 0, iv = 0;
        AttnWalk s = attn_begin<kKeys>(a, plan);
        while (wait.ok && attn_next<kKeys>(a, s)) {
            const int lo = attn_lo(a, s.L);
#pragma unroll 1
            for (int i = 0; i < 2 * s.tiles; ++i) {
                const Buffer buf = buffer_of<C::kTwo>(i, s.tiles);
                // Keys: their scales, by one warp, always the same for a buffer: a warp that left out a
                // phase of xfull could take the one before for the one it waits for.
                static_assert(!F8 || NK <= C::kConv, "a converter warp for each key buffer");
                if (!buf.v) {
                    if (static_cast<int>(ik % NK) == cw) {
                        const int b = ik % NK;
                        if (!wait(&xfull[b], (ik / NK) & 1)) break;
                        const uint32_t w = reinterpret_cast<const uint32_t*>(kexps + b * kKeys)[lane];
                        float4 f;
                        f.x = key_scale(w & 255) * a.key_mul, f.y = key_scale(w >> 8 & 255) * a.key_mul;
                        f.z = key_scale(w >> 16 & 255) * a.key_mul, f.w = key_scale(w >> 24) * a.key_mul;
                        *reinterpret_cast<float4*>(kscale + (ik % NS) * kKeys + lane * 4) = f;
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&kfull[b]);
                    }
                    ++ik;
                    continue;
                }
                const int tt = buf.tile, rb = iv % NR, b = iv % NV;
                if (!wait.both(&rfull[rb], (iv / NR) & 1, &vempty[b], ((iv / NV) & 1) ^ 1u)) break;
                ++iv;
                const int j0 = (s.tile + tt) * kKeys;
                const int za = max(lo - j0, 0), zb = min(s.L - j0, kKeys);
                const bool partial = za > 0 || zb < kKeys;
#pragma unroll 1
                for (int base = cw * 16; base < kKeys; base += (F8 ? C::kConv : 1) * 16) {
                    uint2 x[2 * kStepsC];
                    uint32_t ex[2 * kStepsC];
                    auto row_of = [&](int i) { return base + (i >> 1) * kStepRows + lr + (D == 128 ? 0 : 4 * (i & 1)); };
                    auto half_of = [&](int i) { return D == 128 ? (i ^ lr) & 1 : 0; };
                    const uint8_t* src = raw + rb * C::kRaw + lc * 8;
                    const uint8_t* se = exps + rb * kKeys;
#pragma unroll
                    for (int i = 0; i < 2 * kStepsC; ++i) {
                        x[i] = *reinterpret_cast<const uint2*>(src + row_of(i) * D + half_of(i) * 64);
                        ex[i] = D == 128 && (i & 1) ? ex[i - 1] : se[row_of(i)];
                    }
                    uint8_t* dst = vring + b * C::kTile;
                    auto put = [&](int i, const uint32_t (&y)[4]) {
                        const int row = row_of(i);
                        const bool in = !partial || (row >= za && row < zb);
                        *reinterpret_cast<uint4*>(dst + half_of(i) * 16384 + row * 128 + ((lc ^ (row & 7)) << 4)) =
                            in ? make_uint4(y[0], y[1], y[2], y[3]) : make_uint4(0, 0, 0, 0);
                    };
                    uint32_t odd = 0;  // bit 7 of a byte: a NaN code among them; bit 0: a factor beyond bf16
#pragma unroll
                    for (int i = 0; i < 2 * kStepsC; ++i) {
                        const uint32_t s1 = min(ex[i] + 120u, 254u) * 0x00800080u;  // exponent field of the factor
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t w = k ? x[i].y : x[i].x;
                            y[2 * k] = mul_bf16x2(((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u), s1);
                            y[2 * k + 1] = mul_bf16x2((w & 0x80008000u) | ((w >> 4) & 0x07f007f0u), s1);
                            odd |= ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        }
                        odd |= ex[i] > 134u;
                        put(i, y);
                    }
                    if (odd) {  // again, with the patches
#pragma unroll 1
                        for (int i = 0; i < 2 * kStepsC; ++i) {
                            const uint2 xi = *reinterpret_cast<const uint2*>(src + row_of(i) * D + half_of(i) * 64);
                            const uint32_t e = se[row_of(i)];
                            const uint32_t s1 = min(e + 120u, 254u) * 0x00800080u, s2 = (e > 134u ? e - 7u : 127u) * 0x00800080u;
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t w = k < 2 ? xi.x : xi.y, c = w >> (8 * (k & 1));
                                const uint32_t t = k & 1 ? (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u)
                                                         : ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
                                y[k] = mul_bf16x2(mul_bf16x2(t, s1), s2);
                                if ((c & 0x7fu) == 0x7fu) y[k] |= 0x7fffu;
                                if ((c & 0x7f0000u) == 0x7f0000u) y[k] |= 0x7fff0000u;
                            }
                            put(i, y);
                        }
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&vfull[b]);
                    tc::mbar_arrive(&rempty[rb]);
                }
            }
        }
        if (!wait.ok) err_bits = kErrTimeoutProducer;
    }
    }
    if (err_bits) {
        *abort_flag = 1;
        if (lane == 0) record_error(a.err, err_bits);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, int MODE, bool F8>
cudaError_t launch_mode(const CUtensorMap& km, const CUtensorMap& vm, const AttnArgs& a, int grid, cudaStream_t s) {
    using C = Cfg<D, MODE, F8>;
    static int done[64] = {};
    cudaError_t e = ensure_smem(attn_tc_kernel<D, MODE, F8>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_tc_kernel<D, MODE, F8>, dim3(grid), dim3(C::kThreads), C::kSmem, s, km, vm, a);
}

template <int D, bool F8>
cudaError_t launch_rows(const CUtensorMap& km, const CUtensorMap& vm, const AttnArgs& a, int grid, cudaStream_t s) {
    switch (a.slot_rows) {
        case 32: return launch_mode<D, 0, F8>(km, vm, a, grid, s);
        case 64: return launch_mode<D, 1, F8>(km, vm, a, grid, s);
        case 128: return launch_mode<D, 2, F8>(km, vm, a, grid, s);
        default: return launch_mode<D, 3, F8>(km, vm, a, grid, s);
    }
}

}  // namespace

cudaError_t launch_attn_tc(int D, bool f8, const CUtensorMap& km, const CUtensorMap& vm, const AttnArgs& a, int grid,
                           cudaStream_t s) {
    if (D == 128) return f8 ? launch_rows<128, true>(km, vm, a, grid, s) : launch_rows<128, false>(km, vm, a, grid, s);
    return f8 ? launch_rows<64, true>(km, vm, a, grid, s) : launch_rows<64, false>(km, vm, a, grid, s);
}

}  // namespace moestep
