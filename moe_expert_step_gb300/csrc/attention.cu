// Attention of a block of new tokens over a paged key-value cache (see attn.cuh for how the
// work is divided): the CUDA-core kernel, the join of shared segments, and the C entry.
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

#include <cmath>

namespace moestep {
namespace {

// ---------------------------------------------------------------------------- CUDA cores
// Tiles of 16 query rows and 64 keys, 128 threads.  Each thread computes a 2 x 4 block of the
// tile's scores, the 16 rows' statistics are kept by 8 lanes each, and each thread accumulates
// 4 rows x (D / 32) columns of the output.  A tile's loads are in flight together, eight pieces a
// thread of keys and of values, the next tile's page numbers too (D = 128: 40 bytes spilled).  3 requests of 7 tokens, window
// 500, 8 heads of 64 over 4: 14 to 17 us, the latency of a tile, of starting up and of the join (0.5 us
// of bytes).
constexpr int kRT = 16, kKT = 64, kF32Threads = 128;
template <int D>
constexpr int f32_smem() {
    return (kRT * D + 2 * kKT * (D + 4) + kRT * (kKT + 4) + 3 * kRT) * 4;
}

template <int D>
__global__ void __launch_bounds__(kF32Threads) attn_f32_kernel(const AttnArgs a) {
    extern __shared__ float smf[];
    __shared__ int plan_sm[40], s_row[kKT];
    float* sq = smf;                       // [16][D]
    float* sk = sq + kRT * D;              // [64][D + 4]
    float* sv = sk + kKT * (D + 4);        // [64][D + 4]
    float* sp = sv + kKT * (D + 4);        // [16][68]: scores, then weights
    float* s_m = sp + kRT * (kKT + 4);     // [16] running maximum
    float* s_l = s_m + kRT;                // [16] running sum
    float* s_f = s_l + kRT;                // [16] factor of this tile's rescaling
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x;
    const AttnPlan plan = attn_plan<kKT, kF32Threads>(a, plan_sm);
    if (tid == 0) attn_describe_join<kKT>(a, plan);
    constexpr int CW = D / 32;             // output columns of a thread
    AttnWalk w = attn_begin<kKT>(a, plan);
    while (attn_next<kKT>(a, w)) {
        const int h = w.h, row0 = w.rt * kRT;
        const int nrows = min(kRT, a.rows - row0);
        // the queries and the first tile's pages are on their way together
        constexpr int kQ = kRT * (D / 4) / kF32Threads;  // pieces of a thread
        float4 qx[kQ];
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            const int i = tid + u * kF32Threads, rr = i / (D / 4), d = 4 * (i - rr * (D / 4)), row = row0 + rr;
            qx[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rr < nrows) {
                const int qi = attn_query(a, row), g = row - qi * a.G;
                qx[u] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                              (static_cast<long long>(w.r) * a.n_q + qi) * a.q_ld +
                                                              (h * a.G + g) * D + d));
            }
        }
        const int lo = attn_lo(a, w.L);
        auto page_of = [&](int t) {  // of key tid of a tile, -1: not to be read
            const int j = t * kKT + tid;
            return tid < kKT && j >= lo && j < w.L
                       ? __ldg(&a.table[static_cast<long long>(w.r) * a.max_pages + (j >> a.page_log2)]) : -1;
        };
        int page = page_of(w.tile);
        __syncthreads();  // the segment before is done with the queries
#pragma unroll
        for (int u = 0; u < kQ; ++u) *reinterpret_cast<float4*>(sq + 4 * (tid + u * kF32Threads)) = qx[u];
        if (tid < kRT) {
            s_m[tid] = -INFINITY;
            s_l[tid] = 0.f;
        }
        float acc[4][CW] = {};
        const int vr = tid >> 5, vc = tid & 31;  // output: rows 4 vr .., columns vc + 32 j
        for (int t = w.tile; t < w.tile + w.tiles; ++t) {
            const int j0 = t * kKT;
            if (tid < kKT) {  // each key's row in the pool, -1: not to be read
                const int j = j0 + tid;
                int row = -1;
                if (j >= lo && j < w.L) {
                    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
                        row = ((page * a.Hkv + h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
                    else
                        record_error(a.err, kErrBadInput);
                }
                s_row[tid] = row;
            }
            if (t + 1 < w.tile + w.tiles) page = page_of(t + 1);
            __syncthreads();
            constexpr int kPiece = D / 4, kBatch = 8;  // pieces of a row; loads of a thread in flight, twice
#pragma unroll 1
            for (int i0 = 0; i0 < kKT * kPiece; i0 += kBatch * kF32Threads) {
                float4 kx[kBatch], vx[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kF32Threads + tid, key = i / kPiece, row = s_row[key];
                    kx[u] = vx[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row >= 0) {
                        const long long at = static_cast<long long>(row) * D + 4 * (i - key * kPiece);
                        kx[u] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.k) + at));
                        vx[u] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.v) + at));
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kF32Threads + tid, key = i / kPiece, d = 4 * (i - key * kPiece);
                    *reinterpret_cast<float4*>(sk + key * (D + 4) + d) = kx[u];
                    *reinterpret_cast<float4*>(sv + key * (D + 4) + d) = vx[u];
                }
            }
            __syncthreads();
            {   // scores: rows 2 sr, 2 sr + 1; keys sc + 16 j
                const int sr = tid >> 4, sc = tid & 15;
                float s[2][4] = {};
#pragma unroll 4
                for (int d = 0; d < D; d += 4) {
                    const float4 q0 = *reinterpret_cast<const float4*>(sq + (2 * sr) * D + d);
                    const float4 q1 = *reinterpret_cast<const float4*>(sq + (2 * sr + 1) * D + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 kx = *reinterpret_cast<const float4*>(sk + (sc + 16 * j) * (D + 4) + d);
                        s[0][j] += q0.x * kx.x + q0.y * kx.y + q0.z * kx.z + q0.w * kx.w;
                        s[1][j] += q1.x * kx.x + q1.y * kx.y + q1.z * kx.z + q1.w * kx.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rr = 2 * sr + i;
                    const int2 see = attn_sees(a, w.L, attn_query(a, row0 + min(rr, nrows - 1)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int jj = j0 + sc + 16 * j;
                        sp[rr * (kKT + 4) + sc + 16 * j] =
                            (jj >= see.x && jj < see.y) ? s[i][j] * a.scale_log2 : -INFINITY;
                    }
                }
            }
            __syncthreads();
            {   // eight lanes a row: statistics and weights
                const int rr = tid >> 3, l8 = tid & 7;
                float* row = sp + rr * (kKT + 4) + l8 * 8;
                float mx = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) mx = fmaxf(mx, row[i]);  // passes over NaN, which the weights keep
#pragma unroll
                for (int o = 4; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m0 = s_m[rr], m1 = fmaxf(m0, mx), ms = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = exp2f(row[i] - ms);
                    row[i] = p;
                    sum += p;
                }
#pragma unroll
                for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                __syncwarp();
                if (l8 == 0) {
                    const float f = exp2f(m0 - ms);
                    s_f[rr] = f;
                    s_l[rr] = s_l[rr] * f + sum;
                    s_m[rr] = m1;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = s_f[4 * vr + i];
#pragma unroll
                for (int c = 0; c < CW; ++c) acc[i][c] *= f;
            }
#pragma unroll 4
            for (int key = 0; key < kKT; key += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (4 * vr + i) * (kKT + 4) + key);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        const float x = sv[(key + u) * (D + 4) + vc + 32 * c];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i][c] += (u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w) * x;
                    }
            }
        }
        __syncthreads();
        const int slot = 2 * blockIdx.x + (w.k > 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = 4 * vr + i;
            if (rr >= nrows) continue;
            const float m = s_m[rr], l = s_l[rr];
            if (w.whole) {
                const int row = row0 + rr, qi = attn_query(a, row), g = row - qi * a.G;
                const size_t o = (static_cast<size_t>(w.r) * a.n_q + qi) * a.Hq + h * a.G + g;
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int c = 0; c < CW; ++c) static_cast<float*>(a.out)[o * D + vc + 32 * c] = acc[i][c] * inv;
                if (a.lse && vc == 0) a.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            } else {
                const size_t at = static_cast<size_t>(slot) * a.slot_rows + rr;
#pragma unroll
                for (int c = 0; c < CW; ++c) a.part_o[at * D + vc + 32 * c] = acc[i][c];
                if (vc == 0) a.part_ml[at] = make_float2(m, l);
            }
        }
    }
}

// ---------------------------------------------------------------------------- join
// Rows of a shared segment: m = max m_c, l = sum l_c 2^(m_c - m), o = sum o_c 2^(m_c - m) / l over
// its CTAs c in order.  What is read is what the attention launch just left in L2, so the time
// is the latency of a row's parts: the launch's warps are spread over all rows of all joins, and
// where there are more warps than rows, up to eight share a row, each taking every eighth part.
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a, int ctas) {
    __shared__ int4 s_list[kAttnMaxCtas];  // the joins that there are
    __shared__ int s_cnt[8];
    __shared__ float s_f[8][(kAttnMaxCtas + 31) / 32 * 32];
    __shared__ float s_o[8][D];
    constexpr int W = D / 32, kBatch = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    int found = 0;
    for (int i0 = 0; i0 < ctas; i0 += kJoinThreads) {  // (once or twice)
        int4 j = make_int4(-1, 0, 0, 0);
        if (i0 + threadIdx.x < ctas) j = __ldcg(&a.joins[i0 + threadIdx.x]);
        const unsigned b = __ballot_sync(0xffffffffu, j.x >= 0);
        __syncthreads();
        if (lane == 0) s_cnt[warp] = __popc(b);
        __syncthreads();
        int at = found + __popc(b & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) at += s_cnt[w];
            found += s_cnt[w];
        }
        if (j.x >= 0) s_list[at] = j;
    }
    __syncthreads();
    const int rows = min(a.slot_rows, a.rows), work = found * rows;
    int wpr = 8;  // warps per row
    while (wpr > 1 && work * wpr > static_cast<int>(gridDim.x) * 8) wpr >>= 1;
    const int team = warp / wpr, part = warp % wpr, teams = 8 / wpr;
    for (int w0 = blockIdx.x * teams; w0 < work; w0 += gridDim.x * teams) {  // the same for the whole block
        const int w = w0 + team, seg = w / rows, rr = w - seg * rows;
        int4 j = make_int4(-1, 0, 0, 0);
        if (w < work) j = s_list[seg];
        const int h = j.y / a.row_tiles, row0 = (j.y - h * a.row_tiles) * a.slot_rows;
        const bool on = j.x >= 0 && row0 + rr < a.rows;
        const int c0 = j.z >> 1, n = on ? j.w - c0 + 1 : 0;
        auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? j.z : 2 * (c0 + i)) * a.slot_rows + rr; };
        auto load = [&](int i, float (&x)[W]) {
#pragma unroll
            for (int k = 0; k < W; ++k) x[k] = 0.f;
            if (i >= n) return;
            const float* p = a.part_o;
            if (a.slot_rows == 256) {  // halves of the columns, each row's 16-byte pieces swizzled (attention_tc.cu)
                const int col = lane * W, half = col / (D / 2), piece = (col - half * (D / 2)) / 4;
                const size_t s = static_cast<size_t>(i == 0 ? j.z : 2 * (c0 + i));
                p += ((s * 2 + half) * 256 + rr) * (D / 2) + ((piece ^ (rr & 7)) << 2) + (col & 3);
            } else {
                p += slot(i) * D + lane * W;
            }
            if constexpr (W == 4) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(p));
                x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
            } else {
                const float2 y = __ldcg(reinterpret_cast<const float2*>(p));
                x[0] = y.x, x[1] = y.y;
            }
        };
        float x[kBatch][W];  // the first parts are on their way while the statistics are joined
#pragma unroll
        for (int u = 0; u < kBatch; ++u) load(part + u * wpr, x[u]);
        constexpr int kStats = (kAttnMaxCtas + 31) / 32;
        float2 ml[kStats];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int u = 0; u < kStats; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            if (lane + 32 * u < n) ml[u] = __ldcg(&a.part_ml[slot(lane + 32 * u)]);
        }
#pragma unroll
        for (int u = 0; u < kStats; ++u) m = fmaxf(m, ml[u].x);
        m = warp_max(m);
        const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int u = 0; u < kStats; ++u) {
            if (32 * u >= n) break;
            const float f = exp2f(ml[u].x - ms);
            l += ml[u].y * f;
            s_f[warp][lane + 32 * u] = f;
        }
        l = warp_sum(l);
        __syncwarp();
        float acc[W] = {};
        for (int i = part;;) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (i + u * wpr < n) {
                    const float f = s_f[warp][i + u * wpr];
#pragma unroll
                    for (int k = 0; k < W; ++k) acc[k] += f * x[u][k];
                }
            }
            i += kBatch * wpr;
            if (i >= n) break;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) load(i + u * wpr, x[u]);
        }
        if (wpr > 1) {
#pragma unroll
            for (int i = 0; i < W; ++i) s_o[warp][lane * W + i] = acc[i];
            __syncthreads();
            if (part == 0)
                for (int k = 1; k < wpr; ++k)
#pragma unroll
                    for (int i = 0; i < W; ++i) acc[i] += s_o[warp + k][lane * W + i];
            __syncthreads();
        }
        __syncwarp();
        if (!on || part != 0) continue;
        const int row = row0 + rr, qi = attn_query(a, row), g = row - qi * a.G;
        const size_t o = (static_cast<size_t>(j.x) * a.n_q + qi) * a.Hq + h * a.G + g;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* out = static_cast<T*>(a.out) + o * D + lane * W;
#pragma unroll
        for (int i = 0; i < W; ++i) out[i] = from_f32<T>(acc[i] * inv);
        if (a.lse && lane == 0) a.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
}

template <int D>
cudaError_t launch_f32(const AttnArgs& a, int grid, cudaStream_t s) {
    static int done[64] = {};
    cudaError_t e = ensure_smem(attn_f32_kernel<D>, f32_smem<D>(), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_f32_kernel<D>, dim3(grid), dim3(kF32Threads), f32_smem<D>(), s, a);
}

template <typename T, int D>
cudaError_t launch_join(const AttnArgs& a, int ctas, int sms, cudaStream_t s) {
    // A block can take one row on its eight warps; no more are shared than there are segments, or
    // boundaries between CTAs.  (At most 8 blocks an SM, as many as its warps allow: 4 are a little
    // slower, 2 by 5 us where 256 rows are joined.)
    const long long segments = 1ll * a.R * a.Hkv * a.row_tiles;
    const long long work = (segments < ctas ? segments : ctas) * (a.slot_rows < a.rows ? a.slot_rows : a.rows);
    const int grid = work < 8ll * sms ? static_cast<int>(work) : 8 * sms;
    return launch_pdl(attn_join_kernel<T, D>, dim3(grid), dim3(kJoinThreads), 0, s, a, ctas);
}

// Row tile of the kernel that runs (attention_tc.cu), and the CTAs that it may have: rows that
// fit 32, 64 or 128 lanes, else two tiles of 128
int row_tile(const moestep_kv_dims& d, int n_q) {
    if (d.dtype == MOESTEP_F32) return kRT;
    const long long rows = 1ll * n_q * (d.Hq / d.Hkv);
    return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}
int max_ctas(const moestep_kv_dims& d) { return d.dtype == MOESTEP_F32 ? kAttnMaxCtas : kAttnMaxCtasTc; }

// Empty units of a segment (see attn.cuh) of 256 rows and of fewer.  Beginning one inside a CTA takes
// 12 (bf16) to 17 us (FP8) with 256 rows, a key tile 2 to 2.7.  Against no empty units: 16 blocks of
// 32 tokens, up to 32768 FP8 positions, 156 -> 131 us, 16 ragged single tokens 33 -> 26 us.  (Measured with
// heads of 128 and row tiles of 32 and 256; the others, and heads of 64, whose tiles cost less, take the same.)
constexpr int kAhead = 6, kAheadFew = 4;

struct KvLayout {
    size_t joins, ml, o, total;
    int slot_rows;
};
KvLayout kv_layout(const moestep_kv_dims& d, int n_q) {
    KvLayout L{};
    L.slot_rows = row_tile(d, n_q);
    const int ctas = max_ctas(d);
    size_t at = kKvHeader;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) / 256 * 256;
        return p;
    };
    L.joins = take(sizeof(int4) * ctas);
    L.ml = take(sizeof(float2) * 2 * ctas * L.slot_rows);
    L.o = take(sizeof(float) * 2 * ctas * L.slot_rows * d.D);
    L.total = at;
    return L;
}

int check_attn(const moestep_kv_dims* kd, int R, int n_q) {
    const int rc = check_kv_dims(kd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n_q <= 0) return MOESTEP_EINVAL;
    if (n_q > 1024 || R > (1 << 20)) return MOESTEP_EUNSUPPORTED;
    // units and rows are counted in 31 bits
    const long long row_tiles = (1ll * n_q * (kd->Hq / kd->Hkv) + kRT - 1) / kRT;
    const long long tiles = (1ll * kd->max_pages * kd->page + kKT - 1) / kKT + kAhead;
    if (tiles * kd->Hkv > ((1ll << 31) - 1) / row_tiles / R) return MOESTEP_EUNSUPPORTED;
    if (1ll * R * n_q > ((1ll << 31) - 1) / kd->Hq) return MOESTEP_EUNSUPPORTED;
    return MOESTEP_OK;
}

}  // namespace
}  // namespace moestep

extern "C" int moestep_kv_workspace_size(const moestep_kv_dims* kd, int R, int n_q, size_t* bytes) {
    using namespace moestep;
    const int rc = check_attn(kd, R, n_q);
    if (rc != MOESTEP_OK) return rc;
    if (bytes == nullptr) return MOESTEP_EINVAL;
    *bytes = kv_layout(*kd, n_q).total;
    return MOESTEP_OK;
}

extern "C" int block_attention(const moestep_kv_dims* kd, int R, int n_q, const void* q, long long q_ld,
                               const int32_t* kv_len, const moestep_kv_cache* cache, float scale, int causal,
                               int window, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    using namespace moestep;
    int rc = check_attn(kd, R, n_q);
    if (rc != MOESTEP_OK) return rc;
    if (!kv_len || !out || window < 0 || !std::isfinite(scale) || !(scale > 0.f)) return MOESTEP_EINVAL;
    if (window >= kd->max_pages * kd->page) window = 0;  // a window as long as the cache hides nothing
    if (window > (1ll << 31) - 1 - n_q) return MOESTEP_EUNSUPPORTED;  // (positions less a window stay in 32 bits)
    if ((rc = check_kv_cache(kd, cache)) != MOESTEP_OK) return rc;
    if ((rc = check_kv_rows(q, q_ld, 1ll * kd->Hq * kd->D, kd->dtype)) != MOESTEP_OK) return rc;
    if (!kv_aligned16(out)) return MOESTEP_EALIGN;
    const KvLayout L = kv_layout(*kd, n_q);
    if ((rc = check_kv_ws(ws, ws_bytes, L.total)) != MOESTEP_OK) return rc;
    int sms = 0;
    if ((rc = device_ok(&sms)) != MOESTEP_OK) return rc;
    char* w = static_cast<char*>(ws);
    AttnArgs a{};
    a.q = q;
    a.q_ld = q_ld;
    a.kv_len = kv_len;
    a.table = cache->table;
    a.k = cache->k;
    a.v = cache->v;
    a.k_exp = cache->k_exp;
    a.v_exp = cache->v_exp;
    a.out = out;
    a.lse = lse;
    a.joins = reinterpret_cast<int4*>(w + L.joins);
    a.part_ml = reinterpret_cast<float2*>(w + L.ml);
    a.part_o = reinterpret_cast<float*>(w + L.o);
    a.err = reinterpret_cast<int*>(w);
    a.R = R;
    a.n_q = n_q;
    a.Hq = kd->Hq;
    a.Hkv = kd->Hkv;
    a.G = kd->Hq / kd->Hkv;
    a.g_magic = a.G > 1 ? static_cast<uint32_t>(((1ull << 32) + a.G - 1) / a.G) : 0;
    a.rows = n_q * a.G;
    a.slot_rows = L.slot_rows;
    a.row_tiles = (a.rows + L.slot_rows - 1) / L.slot_rows;
    a.page_log2 = kd->page == 16 ? 4 : kd->page == 32 ? 5 : kd->page == 64 ? 6 : 7;
    a.max_pages = kd->max_pages;
    a.n_pages = kd->n_pages;
    const bool f32 = kd->dtype == MOESTEP_F32, f8 = kd->dtype == MOESTEP_FP8;
    a.causal = causal != 0;
    a.even = !f32 && L.slot_rows == 256 ? 4 : 0;
    a.ahead = f32 ? 0 : L.slot_rows == 256 ? kAhead : kAheadFew;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    if (f8) {
        int e = 0;
        a.key_mul = std::frexp(a.scale_log2, &e);
        a.scale_log2 = std::ldexp(1.f, e);
    }
    a.timeout_ns = wait_timeout_ns();
    const int want = f32 ? 2 * sms : sms, grid = want < max_ctas(*kd) ? want : max_ctas(*kd);
    CUtensorMap km, vm;
    if (!f32) {
        const uint64_t n = 1ull * kd->n_pages * kd->Hkv * kd->page;
        for (int i = 0; i < 2; ++i) {
            const void* p = i ? cache->v : cache->k;
            // FP8 keys are an operand as they are, FP8 values go through the converters
            rc = f8 ? encode_tile_map(i ? &vm : &km, 1, p, kd->D, n, kd->D, kd->page, i ? 0 : kd->D)
                    : encode_tile_map(i ? &vm : &km, 2, p, kd->D, n, 64, kd->page, 128);
            if (rc != MOESTEP_OK) return rc;
        }
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = kd->D == 128;
    prof_begin(8, s);
    cudaError_t e;
    if (f32)
        e = wide ? launch_f32<128>(a, grid, s) : launch_f32<64>(a, grid, s);
    else
        e = launch_attn_tc(kd->D, f8, km, vm, a, grid, s);
    prof_end(8, s);
    if (e == cudaSuccess) {
        count_launch();
        prof_begin(8, s);
        if (f32)
            e = wide ? launch_join<float, 128>(a, grid, sms, s) : launch_join<float, 64>(a, grid, sms, s);
        else
            e = wide ? launch_join<bf16, 128>(a, grid, sms, s) : launch_join<bf16, 64>(a, grid, sms, s);
        prof_end(8, s);
        if (e == cudaSuccess) count_launch();
    }
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    return MOESTEP_OK;
}
