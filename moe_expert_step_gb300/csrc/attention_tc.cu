// Attention over a paged bf16 or FP8 cache on tcgen05 tensor cores.
//
// One persistent CTA per SM takes an equal share of the key tiles (attn.cuh) and streams
// them once through shared memory, 128 keys at a time, with the running maximum and sum of
// the softmax.  The query rows of one (request, key-value head), n_q tokens x G heads, are
// the MMA's M = 128: S = Q K^T into tensor memory, P = 2^(S c - m) written back over S as
// bf16, O += P V with P read from tensor memory.
//
// Two streams run through each CTA, each with a softmax warpgroup, its S / P (128 columns) and its O
// (D columns), so that one stream's MMAs run under the other's exponentials:
//   more than 128 rows: the streams are two row tiles of 128 on the same keys;
//   else:               they take alternate key tiles of the same rows, each with its own (m, l, O).
// Few rows would leave most of the 128 lanes idle and one lane with 128 exponentials a tile, so
// 32 (64) rows are held four (two) times, and warp w of a warpgroup computes only its quarter
// (half) of the tile's keys, the rest of its lanes' P being zero: each such copy is one more
// independent (m, l, O).  All of them meet in shared memory when a segment ends.
//
// The maximum m that the weights refer to moves only when a tile's maximum exceeds it by more
// than 8 (a factor 256, harmless in fp32 sums and bf16 weights): O is then rescaled in tensor
// memory by the softmax warps, which is rare after the first tiles.
//
// Warps: 0-7 softmax (two warpgroups), 8 TMA producer, 9 MMA issuer (one lane), and with FP8
// 10-13 converters (E4M3 code * 2^exp -> bf16, exact, into the swizzled operand buffers).
// Keys outside [lo, L) of the request reach no result: their scores are replaced by -inf, and
// their V rows, which a zero weight would still multiply (NaN), are zeroed in shared memory.
// Every wait is bounded (timeout -> error word, orderly teardown).
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
constexpr float kSlack = 8.f;                     // how far a tile's maximum may pass m

// MODE 0, 1, 2: row tiles of 32, 64, 128 (one tile, streams on alternate keys); 3: of 256 (two tiles)
template <int D, int MODE, bool F8>
struct Cfg {
    static constexpr bool kTwo = MODE == 3;
    static constexpr int kRows = 32 << MODE;
    static constexpr int kRep = MODE == 0 ? 4 : MODE == 1 ? 2 : 1;
    static constexpr int kCols = kKeys / kRep;            // keys of a tile that a lane handles
    static constexpr int kParts = kTwo ? 1 : 2 * kRep;    // (m, l, O) of a row
    static constexpr int kThreads = F8 ? 448 : 320;
    static constexpr int kTile = kKeys * D * 2;           // bytes of a bf16 operand tile
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kSide = kTwo ? kQ : 32768;       // second query tile, or the merge buffer
    static constexpr int kRaw = kKeys * D;                // bytes of an FP8 tile
    static constexpr int kBufs = F8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int kRaws = F8 ? (D == 128 ? 4 : 8) : 0;
    static constexpr int kMisc = 1024 + kRaws * kKeys;    // plan, barriers, exponents
    static constexpr int kSmem = 1024 + kQ + kSide + kBufs * kTile + kRaws * kRaw + kMisc;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Waits {
    volatile int* abort;
    uint64_t tmo;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return tc::mbar_wait(bar, parity, abort, tmo);
    }
};

// The buffers of a segment of n key tiles in the order in which the MMAs use them:
// f(is_v, tile) until it returns false.
template <bool TWO, typename F>
__device__ __forceinline__ bool each_buffer(int n, F f) {
    if (TWO) {
        for (int t = 0; t < n; ++t)
            if (!f(false, t) || !f(true, t)) return false;
        return true;
    }
    if (!f(false, 0)) return false;
    if (n > 1 && !f(false, 1)) return false;
    for (int t = 0; t < n; ++t) {
        if (!f(true, t)) return false;
        if (t + 2 < n && !f(false, t + 2)) return false;
    }
    return true;
}

template <int D, int MODE, bool F8>
__global__ void __launch_bounds__(Cfg<D, MODE, F8>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const AttnArgs a) {
    using C = Cfg<D, MODE, F8>;
    constexpr int NB = C::kBufs, NR = C::kRaws > 0 ? C::kRaws : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = sm;
    uint8_t* side = sq + C::kQ;
    uint8_t* ring = side + C::kSide;
    uint8_t* raw = ring + NB * C::kTile;
    uint8_t* exps = raw + C::kRaws * C::kRaw;              // [kRaws][128]
    long long* plan_sm = reinterpret_cast<long long*>(exps + C::kRaws * kKeys);  // 64 x 8 bytes
    uint64_t* full = reinterpret_cast<uint64_t*>(plan_sm + 64);
    uint64_t* empty = full + NB;
    uint64_t* rfull = empty + NB;
    uint64_t* rempty = rfull + C::kRaws;
    uint64_t* s_full = rempty + C::kRaws;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 2;
    uint64_t* q_full = o_full + 2;
    uint64_t* fin = q_full + 1;
    uint64_t* meet = fin + 1;  // the eight softmax warps, between the steps of a merge
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(meet + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
    int* zero_flag = abort_flag + 1;
    static_assert((2 * NB + 2 * C::kRaws + 9) * 8 + 12 + 512 <= 1024, "misc area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NB; ++i) {
            tc::mbar_init(&full[i], F8 ? 4 : 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kRaws; ++i) {
            tc::mbar_init(&rfull[i], 1);
            tc::mbar_init(&rempty[i], 4);
        }
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(&s_full[g], 1);
            tc::mbar_init(&p_full[g], 4);
            tc::mbar_init(&o_full[g], 1);
        }
        tc::mbar_init(q_full, 8);
        tc::mbar_init(fin, 1);
        tc::mbar_init(meet, 8);
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
    const uint32_t tmem = *tmem_holder;
    pdl_trigger();
    pdl_wait();
    const AttnPlan plan = attn_plan<kKeys, C::kThreads>(a, plan_sm);
    const Waits wait{abort_flag, a.timeout_ns};
    bool ok = true;
    int err_bits = 0;

    if (warp < 8) {
        // ------------------------------------------------------------ softmax and output
        const int g = warp >> 2, w = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        const uint32_t t_s = tmem + lanes + g * 128, t_o = tmem + lanes + 256 + g * 128;
        const int part = MODE == 0 ? w : MODE == 1 ? w >> 1 : 0;        // which of the tile's keys
        const int lrow = C::kTwo ? g * 128 + w * 32 + lane               // row within the row tile
                                 : (w * 32 + lane) & (C::kRows - 1);
        const int col0 = part * C::kCols;
        uint32_t turns = 0, segs_g = 0, meets = 0;
        auto sync8 = [&]() -> bool {  // all eight warps; false if the wait gave up
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(meet);
            return __all_sync(0xffffffffu, wait(meet, meets++ & 1));
        };
        AttnWalk s = attn_begin<kKeys>(plan);
        while (ok && attn_next<kKeys>(a, s)) {
            const int h = s.seg / a.row_tiles, row0 = (s.seg - h * a.row_tiles) * C::kRows;
            const int nrows = min(C::kRows, a.rows - row0);
            {   // query rows into the swizzled operand tile(s), copies for lanes that repeat rows
                constexpr int kChunks = D / 8, NT = C::kTwo ? 128 : 256;
                uint8_t* dst = C::kTwo ? (g == 0 ? sq : side) : sq;
                for (int i = (C::kTwo ? threadIdx.x & 127 : threadIdx.x); i < 128 * kChunks; i += NT) {
                    const int m = i / kChunks, c = i - m * kChunks;
                    const int row = C::kTwo ? g * 128 + m : m & (C::kRows - 1);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < nrows) {
                        const int rr = row0 + row, qi = rr / a.G;
                        x = __ldg(reinterpret_cast<const uint4*>(
                            static_cast<const bf16*>(a.q) + (static_cast<long long>(s.r) * a.n_q + qi) * a.q_ld +
                            (h * a.G + rr - qi * a.G) * D + c * 8));
                    }
                    *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + m * 128 + (((c & 7) ^ (m & 7)) << 4)) = x;
                }
                tc::fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(q_full);
            }
            const int2 see = attn_sees(a, s.L, (row0 + min(lrow, nrows - 1)) / a.G);
            float m = -INFINITY, l = 0.f;
            const int step = C::kTwo ? 1 : 2, first = s.tile + (C::kTwo ? 0 : g);
            int turn = 0;
            for (int t = first; t < s.tile + s.tiles; t += step, ++turn) {
                if (!__all_sync(0xffffffffu, wait(&s_full[g], turns & 1))) {
                    ok = false;
                    break;
                }
                ++turns;
                tc::fence_after_sync();
                const int lo = see.x - (t * kKeys + col0), hi = see.y - (t * kKeys + col0);
                const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < C::kCols);
                constexpr bool kKeep = C::kCols <= 64;  // scores held in registers between the two passes
                float v[kKeep ? C::kCols : 32];
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < C::kCols; c += 32) {
                    float* x = v + (kKeep ? c : 0);
                    tc::tmem_ld32(t_s + col0 + c, x);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = (c + i >= lo && c + i < hi) ? x[i] : -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[i]);
                }
                mx *= a.scale_log2;
                const bool move = mx > m + kSlack || (m == -INFINITY && mx > m);
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? tc::exp2_fast(m - mx) : 1.f;  // 0 from m = -inf
                    if (move) m = mx;
                    l *= f;
                    if (turn > 0) {
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
                if (C::kRep > 1) {  // the other copies' keys
                    const uint32_t z[16] = {};
#pragma unroll
                    for (int c = 0; c < kKeys / 2; c += 16)
                        if (c / (C::kCols / 2) != part) tc::tmem_st16_async(t_s + c, z);
                }
#pragma unroll
                for (int c = 0; c < C::kCols; c += 32) {
                    float* x = v + (kKeep ? c : 0);
                    if (!kKeep) {
                        tc::tmem_ld32(t_s + col0 + c, x);
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = (c + i >= lo && c + i < hi) ? x[i] : -INFINITY;
                        }
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = tc::exp2_fast(fmaf(x[2 * i], a.scale_log2, -ms));
                        const float p1 = tc::exp2_fast(fmaf(x[2 * i + 1], a.scale_log2, -ms));
                        l += p0 + p1;
                        p[i] = tc::pack_bf16(p0, p1);
                    }
                    tc::tmem_st16_async(t_s + (col0 + c) / 2, p);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_full[g]);
            }
            if (!ok) break;
            if (turn > 0) {
                if (!__all_sync(0xffffffffu, wait(&o_full[g], segs_g & 1))) {
                    ok = false;
                    break;
                }
                ++segs_g;
                tc::fence_after_sync();
            }
            const int slot = 2 * blockIdx.x + (s.k > 0);
            // row `rr` of the row tile: where it goes
            auto where = [&](int rr) {
                const int row = row0 + rr, qi = row / a.G;
                return (static_cast<size_t>(s.r) * a.n_q + qi) * a.Hq + h * a.G + row - qi * a.G;
            };
            if constexpr (C::kTwo) {
                const bool on = lrow < nrows;
                const size_t o = on ? where(lrow) : 0, at = static_cast<size_t>(slot) * a.slot_rows + lrow;
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    __syncwarp();
                    tc::tmem_ld32(t_o + c, x);
                    if (!on) continue;
                    if (s.whole) {
                        uint4* d = reinterpret_cast<uint4*>(static_cast<bf16*>(a.out) + o * D + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d[i] = make_uint4(tc::pack_bf16(x[8 * i] * inv, x[8 * i + 1] * inv),
                                              tc::pack_bf16(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                                              tc::pack_bf16(x[8 * i + 4] * inv, x[8 * i + 5] * inv),
                                              tc::pack_bf16(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
                    } else {
                        float4* d = reinterpret_cast<float4*>(a.part_o + at * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                }
                if (on && s.whole && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                if (on && !s.whole) a.part_ml[at] = make_float2(m, l);
            } else {
                // merge the row's parts: p = stream * copies + copy
                const int p = g * C::kRep + part;
                float2* ml = reinterpret_cast<float2*>(side);  // [parts][rows]
                ml[p * C::kRows + lrow] = make_float2(m, l);
                if (!sync8()) {
                    ok = false;
                    break;
                }
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < C::kParts; ++i) M = fmaxf(M, ml[i * C::kRows + lrow].x);
                const float Ms = M == -INFINITY ? 0.f : M;
                const float f = tc::exp2_fast(m - Ms);
                // the row that this thread puts together, and its sum
                constexpr int kPer = C::kRows * 32 / 256;  // columns of a 32-wide slice, a multiple of 4
                const int orow = threadIdx.x / (32 / kPer), ocol = (threadIdx.x % (32 / kPer)) * kPer;
                float OM = -INFINITY, ol = 0.f;
#pragma unroll
                for (int i = 0; i < C::kParts; ++i) OM = fmaxf(OM, ml[i * C::kRows + orow].x);
                const float OMs = OM == -INFINITY ? 0.f : OM;
#pragma unroll
                for (int i = 0; i < C::kParts; ++i) {
                    const float2 q = ml[i * C::kRows + orow];
                    ol += q.y * tc::exp2_fast(q.x - OMs);
                }
                const bool on = orow < nrows;
                const size_t o = on ? where(orow) : 0, at = static_cast<size_t>(slot) * a.slot_rows + orow;
                const float inv = ol == 0.f ? 0.f : 1.f / ol;
                float* buf = reinterpret_cast<float*>(side);  // [parts][rows][32], 16-byte pieces swizzled by row
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float x[32];
                    __syncwarp();
                    if (turn > 0) {
                        tc::tmem_ld32(t_o + c, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0.f;
                    }
                    if (!sync8()) {  // the statistics, or the slice before, have been read
                        ok = false;
                        break;
                    }
                    float* b = buf + (p * C::kRows + lrow) * 32;
                    if (lrow < nrows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4*>(b + ((i ^ (lrow & 7)) << 2)) =
                                make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
                    }
                    if (!sync8()) {
                        ok = false;
                        break;
                    }
                    if (!on) continue;
#pragma unroll
                    for (int k = 0; k < kPer; k += 4) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < C::kParts; ++i) {
                            const float4 z = *reinterpret_cast<const float4*>(
                                buf + (i * C::kRows + orow) * 32 + ((((ocol + k) >> 2) ^ (orow & 7)) << 2));
                            y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
                        }
                        if (s.whole)
                            *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + o * D + c + ocol + k) =
                                make_uint2(tc::pack_bf16(y.x * inv, y.y * inv), tc::pack_bf16(y.z * inv, y.w * inv));
                        else
                            *reinterpret_cast<float4*>(a.part_o + at * D + c + ocol + k) = y;
                    }
                }
                if (!ok) break;
                if (on && ocol == 0) {
                    if (!s.whole) a.part_ml[at] = make_float2(OM, ol);
                    else if (a.lse) a.lse[o] = ol == 0.f ? -INFINITY : (OM + log2f(ol)) * 0.69314718055994531f;
                }
                if (!sync8()) ok = false;  // the next segment's statistics reuse the buffer
            }
        }
        if (!ok) err_bits = kErrTimeoutEpilogue;
    } else if (warp == 8) {
        // ------------------------------------------------------------ TMA producer
        uint64_t* const bf = F8 ? rfull : full;
        uint64_t* const be = F8 ? rempty : empty;
        constexpr int N = F8 ? NR : NB;
        uint32_t it = 0;
        const int page = 1 << a.page_log2;
        AttnWalk s = attn_begin<kKeys>(plan);
        while (ok && attn_next<kKeys>(a, s)) {
            const int h = s.seg / a.row_tiles, lo = attn_lo(a, s.L);
            const int32_t* tab = a.table + static_cast<long long>(s.r) * a.max_pages;
            ok = each_buffer<C::kTwo>(s.tiles, [&](bool is_v, int tt) -> bool {
                const int p0 = (s.tile + tt) * kKeys + lane * page;  // this lane's page
                int id = -1;
                if (lane * page < kKeys && p0 < s.L && p0 + page > lo) {
                    id = __ldg(&tab[p0 >> a.page_log2]);
                    if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.n_pages)) {
                        id = -1;
                        record_error(a.err, kErrBadInput);
                    }
                }
                const int n = __popc(__ballot_sync(0xffffffffu, id >= 0));
                const int b = it % N;
                if (!__all_sync(0xffffffffu, wait(&be[b], ((it / N) & 1) ^ 1u))) return false;
                if (lane == 0) tc::mbar_arrive_expect_tx(&bf[b], n * page * (F8 ? D + 1 : 2 * D));
                __syncwarp();
                if (id >= 0) {
                    const int y = (id * a.Hkv + h) << a.page_log2;
                    const CUtensorMap* map = is_v ? &vmap : &kmap;
                    if (F8) {
                        tc::tma_load_2d(raw + b * C::kRaw + lane * page * D, map, &bf[b], 0, y);
                        tc::bulk_load(exps + b * kKeys + lane * page, (is_v ? a.v_exp : a.k_exp) + y, page, &bf[b]);
                    } else {
#pragma unroll
                        for (int half = 0; half < D / 64; ++half)
                            tc::tma_load_2d(ring + b * C::kTile + half * 16384 + lane * page * 128, map, &bf[b],
                                            half * 64, y);
                    }
                }
                ++it;
                return true;
            });
        }
        if (!ok) err_bits = kErrTimeoutProducer;
        // copies in flight land before the CTA ends
        for (uint32_t i = it > N ? it - N : 0; i < it; ++i) tc::mbar_wait(&bf[i % N], (i / N) & 1, zero_flag, kTeardown);
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc_s = tc::idesc_bf16(128, kKeys), idesc_o = tc::idesc_bf16(128, D) | tc::kIdescTransposeB;
        uint32_t it = 0, segs = 0, p_cnt[2] = {0, 0};
        int buf = 0;
        auto acquire = [&]() -> bool {  // the next buffer in the ring
            buf = it % NB;
            const bool got = __all_sync(0xffffffffu, wait(&full[buf], (it / NB) & 1));
            ++it;
            return got;
        };
        AttnWalk s = attn_begin<kKeys>(plan);
        while (ok && attn_next<kKeys>(a, s)) {
            const int N = C::kTwo ? 2 * s.tiles : s.tiles, lo = attn_lo(a, s.L);
            if (!__all_sync(0xffffffffu, wait(q_full, segs & 1))) {
                ok = false;
                break;
            }
            ++segs;
            int kb = 0, vb = 0;
            auto scores = [&](int n) -> bool {  // S of turn n
                const int g = n & 1;
                if (!C::kTwo || g == 0) {
                    if (!acquire()) return false;
                    kb = buf;
                }
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint32_t qa = tc::smem_addr(C::kTwo && g == 1 ? side : sq);
                    const uint32_t ka = tc::smem_addr(ring + kb * C::kTile);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
                        tc::mma_bf16(tmem + g * 128, tc::sdesc_k_sw128(qa + off), tc::sdesc_k_sw128(ka + off), idesc_s,
                                     k > 0);
                    }
                    tc::mma_commit(&s_full[g]);
                    if (!C::kTwo || g == 1) tc::mma_commit(&empty[kb]);
                }
                __syncwarp();
                return true;
            };
            ok = scores(0) && (N < 2 || scores(1));
            for (int n = 0; ok && n < N; ++n) {
                const int g = n & 1;
                if (!C::kTwo || g == 0) {
                    if (!acquire()) {
                        ok = false;
                        break;
                    }
                    vb = buf;
                    if (!F8) {  // V rows that no query sees
                        const int j0 = (s.tile + (C::kTwo ? n >> 1 : n)) * kKeys;
                        const int za = max(lo - j0, 0), zb = min(s.L - j0, kKeys);
                        if (za > 0 || zb < kKeys) {
                            uint8_t* v = ring + vb * C::kTile;
                            for (int i = lane; i < kKeys * (D / 8); i += 32) {
                                const int row = (i >> 3) & (kKeys - 1);
                                if (row < za || row >= zb)
                                    *reinterpret_cast<uint4*>(v + (i >> 10) * 16384 + row * 128 + (i & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                            }
                            tc::fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                }
                if (!__all_sync(0xffffffffu, wait(&p_full[g], p_cnt[g] & 1))) {
                    ok = false;
                    break;
                }
                ++p_cnt[g];
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint32_t va = tc::smem_addr(ring + vb * C::kTile);
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        tc::mma_f16_tmem_a(tmem + 256 + g * 128, tmem + g * 128 + k * 8,
                                           tc::sdesc_mn_sw128(va + k * 2048, 16384), idesc_o, n >= 2 || k > 0);
                    if (!C::kTwo || g == 1) tc::mma_commit(&empty[vb]);
                    if (n + 2 >= N) tc::mma_commit(&o_full[g]);
                }
                __syncwarp();
                if (n + 2 < N) ok = scores(n + 2);
            }
        }
        if (!ok) err_bits = kErrTimeoutMma;
        if (lane == 0) {  // MMAs in flight complete before the tensor memory is freed
            tc::mma_commit(fin);
            tc::mbar_wait(fin, 0, zero_flag, kTeardown);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ FP8 converters
        // Eight (D = 128) or four lanes take a key's codes, 16 each, and write 32 bytes of the
        // 128-byte swizzled bf16 tile; the lanes of the second 64-column box store their two
        // 16-byte pieces in the other order, so that no two of a row's lanes meet in a bank.
        const int cw = warp - 10;
        constexpr int L = D / 16, RPI = 32 / L;  // lanes a row, rows a step
        const int lr = lane / L, lc = lane % L;
        uint32_t it = 0;
        AttnWalk s = attn_begin<kKeys>(plan);
        while (ok && attn_next<kKeys>(a, s)) {
            const int lo = attn_lo(a, s.L);
            ok = each_buffer<C::kTwo>(s.tiles, [&](bool, int tt) -> bool {
                const int rb = it % NR, b = it % NB;
                if (!__all_sync(0xffffffffu, wait(&rfull[rb], (it / NR) & 1))) return false;
                if (!__all_sync(0xffffffffu, wait(&empty[b], ((it / NB) & 1) ^ 1u))) return false;
                const int j0 = (s.tile + tt) * kKeys;
                const int za = max(lo - j0, 0), zb = min(s.L - j0, kKeys);
                const uint8_t* src = raw + rb * C::kRaw;
                uint8_t* dst = ring + b * C::kTile + (lc >> 2) * 16384;
#pragma unroll 4
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int row = cw * 32 + i * RPI + lr;
                    uint4 x = *reinterpret_cast<const uint4*>(src + row * D + lc * 16);
                    const int e = exps[rb * kKeys + row];
                    const float sc = e > 0 ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 5.8774717541114375e-39f;
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t h2 = tc::e4m3x2_to_f16x2(in[k >> 1], 2 * (k & 1));
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                        y[k] = tc::pack_bf16(f.x * sc, f.y * sc);
                    }
                    if (row < za || row >= zb) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = 0;
                    }
                    uint8_t* d = dst + row * 128;
                    const int c = (lc & 3) * 2, sw = row & 7;
                    const uint4 y0 = make_uint4(y[0], y[1], y[2], y[3]), y1 = make_uint4(y[4], y[5], y[6], y[7]);
                    const bool flip = lc >= 4;
                    *reinterpret_cast<uint4*>(d + (((c + flip) ^ sw) << 4)) = flip ? y1 : y0;
                    *reinterpret_cast<uint4*>(d + (((c + !flip) ^ sw) << 4)) = flip ? y0 : y1;
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&full[b]);
                    tc::mbar_arrive(&rempty[rb]);
                }
                ++it;
                return true;
            });
        }
        if (!ok) err_bits = kErrTimeoutProducer;
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
