// What the attention kernels share: the arguments, the division of the work among CTAs, and
// the rows a query sees.
//
// The work is a list of units: one tile of keys for one tile of query rows of one
// (request, key-value head).  Units are numbered request by request, then head, then row tile,
// then key tile, and every CTA takes the same number of them in a row (one more or less): it
// streams as many key tiles as any other whatever the requests' lengths are.  The lengths are on
// the device, so every CTA works the division out from kv_len itself (a block-wide scan over the
// requests; an empty request counts one key tile, whose only effect is to write its empty rows).
//
// The units of one (request, head, row tile) are a segment.  Beginning a segment inside a CTA costs
// about as much as some units (the last one is written out, queries are staged, the pipeline fills
// again), so each segment counts that many empty units (`ahead`) before its first key tile: CTAs in
// which segments end and begin get fewer tiles.
//
// Every row tile goes through all key tiles that some query of its request sees, also those that none of its
// own does.  With one row tile (32 tokens of 16 heads over 2) that is nothing; of a causal prompt in several it
// is up to half of the work, with a window much shorter than the prompt more: 1024 tokens, 8 row tiles,
// 39 us, with a window of 128, for which 2 or 3 of each row tile's 8 key tiles would do, 39 us too.
//
// A segment inside one CTA is written out directly; of one that CTAs share, each leaves its rows'
// (m, l, o) in a slot of the workspace (a CTA has at most two such: the one it begins in and the
// one it ends in) and the join launch adds them up in CTA order, so the result does not depend on
// timing.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "moestep.h"

namespace moestep {

constexpr int kAttnMaxCtas = 304;    // CTAs that the workspace has slots for: CUDA-core kernel,
constexpr int kAttnMaxCtasTc = 160;  // tensor-core kernel

struct AttnArgs {
    const void* q;
    long long q_ld;
    const int32_t* kv_len;
    const int32_t* table;
    const void* k;
    const void* v;
    const uint8_t* k_exp;
    const uint8_t* v_exp;
    void* out;
    float* lse;
    float* part_o;    // [2 * CTAs][slot_rows][D]; slot_rows = 256: [2 * CTAs][2][256][D / 2], swizzled
    float2* part_ml;  // [2 * CTAs][slot_rows]: maximum (times scale * log2 e), sum
    int4* joins;      // [CTAs]: {request or -1, head * row tiles + row tile, first CTA's slot, last CTA}
    int* err;
    int R, n_q, Hq, Hkv, G;
    uint32_t g_magic;  // ceil(2^32 / G); 0 for G = 1
    int rows;          // n_q * G: query rows of one (request, key-value head)
    int row_tiles;
    int slot_rows;
    int page_log2, max_pages, n_pages;
    int causal, window;
    int even;          // largest share (units a CTA) that is divided evenly
    int ahead;         // empty units of a segment
    float scale_log2;  // scale * log2(e): the kernels take exponentials to base 2
    float key_mul;     // FP8: scale_log2 is a power of two, this the rest of scale * log2(e) (1/2 .. 1)
    unsigned long long timeout_ns;
};

// Cached positions of a request (clamped; a bad length is recorded by CTA 0)
__device__ __forceinline__ int attn_len(const AttnArgs& a, int r) {
    const int L = __ldg(&a.kv_len[r]), most = a.max_pages << a.page_log2;
    return min(max(L, 0), most);
}

// Query of a row: row / G, exact while row * G < 2^32
__device__ __forceinline__ int attn_query(const AttnArgs& a, int row) {
    return a.g_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), a.g_magic)) : row;
}

// First position that some query of the request sees (the last is L - 1)
__device__ __forceinline__ int attn_lo(const AttnArgs& a, int L) {
    return a.window > 0 ? max(0, L - a.n_q - a.window + 1) : 0;
}

// Positions [lo, hi) that query i sees
__device__ __forceinline__ int2 attn_sees(const AttnArgs& a, int L, int i) {
    const int p = L - a.n_q + i;
    return make_int2(a.window > 0 ? max(0, p - a.window + 1) : 0, a.causal ? min(L, max(0, p + 1)) : L);
}

template <int KT>
__device__ __forceinline__ int2 attn_tiles(const AttnArgs& a, int L) {  // first tile, number of tiles
    const int t0 = attn_lo(a, L) / KT;
    return make_int2(t0, max(1, (L + KT - 1) / KT - t0));
}

// The division: of W units over A CTAs the first W % A take one more than the rest.  With few units
// a CTA (`even`), as many CTAs as have the same largest share: fewer parts to join for the same time.
struct AttnShare {
    int A, base, extra;
    __device__ __forceinline__ AttnShare(int W, int grid, int even) : A(min(W, grid)) {
        const int most = (W + A - 1) / A;
        if (most <= even) A = (W + most - 1) / most;
        base = W / A;
        extra = W - base * A;
    }
    __device__ __forceinline__ int first(int c) const { return c * base + min(c, extra); }  // of CTA c
    __device__ __forceinline__ int owner(int u) const {                                     // of unit u
        const int cut = extra * (base + 1);
        return u < cut ? u / (base + 1) : extra + (u - cut) / base;
    }
};

// One CTA's place in the list
struct AttnPlan {
    int W;        // units in all
    int first;    // the CTA's first unit
    int begin_r;  // that unit's request
    int begin_o;  // and its number within the request
    int begin_L;  // and the request's length
    int count;    // the CTA's units
};

// Executed by every thread of the block (NT threads); `sm`: 40 ints of shared memory.
template <int KT, int NT>
__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs& a, int* sm) {
    const int tid = threadIdx.x, per = (a.R + NT - 1) / NT, heads = a.Hkv * a.row_tiles;
    const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
        const int L = attn_len(a, r);
        if (blockIdx.x == 0 && L != __ldg(&a.kv_len[r])) record_error(a.err, kErrBadInput);
        mine += (a.ahead + attn_tiles<KT>(a, L).y) * heads;
    }
    int incl = mine;  // block-wide inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if ((tid & 31) >= o) incl += v;
    }
    if ((tid & 31) == 31) sm[tid >> 5] = incl;
    __syncthreads();
    int before = 0, W = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w == (tid >> 5)) before = W;
        W += sm[w];
    }
    incl += before;
    const AttnShare sh(W, gridDim.x, a.even);
    AttnPlan p;
    p.W = W;
    const int c = blockIdx.x;
    p.first = c < sh.A ? sh.first(c) : W;
    p.count = c < sh.A ? sh.first(c + 1) - p.first : 0;
    if (p.count > 0 && p.first >= incl - mine && p.first < incl) {
        int at = incl - mine;
        for (int r = r0; r < r1; ++r) {
            const int L = attn_len(a, r);
            const int2 t = attn_tiles<KT>(a, L);
            const int n = (a.ahead + t.y) * heads;
            if (p.first < at + n) {
                sm[32] = r;
                sm[33] = p.first - at;
                sm[34] = L;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    p.begin_r = p.count > 0 ? sm[32] : 0;
    p.begin_o = p.count > 0 ? sm[33] : 0;
    p.begin_L = p.count > 0 ? sm[34] : 0;
    return p;
}

// Executed by one thread: the join of a segment is described by the second CTA that works on it.
template <int KT>
__device__ __forceinline__ void attn_describe_join(const AttnArgs& a, const AttnPlan& p) {
    int4 j = make_int4(-1, 0, 0, 0);
    const int c = blockIdx.x;
    if (p.count > 0) {
        const int n = a.ahead + attn_tiles<KT>(a, p.begin_L).y, seg = p.begin_o / n, o = p.begin_o - seg * n;
        if (o > a.ahead) {
            const AttnShare sh(p.W, gridDim.x, a.even);
            const int start = p.first - o, c0 = sh.owner(start + a.ahead);  // who has the first key tile
            // the segment is the first one of CTA c0 (its slot 0) or not (slot 1)
            if (c0 == c - 1) j = make_int4(p.begin_r, seg, 2 * c0 + (sh.first(c0) < start), sh.owner(start + n - 1));
        }
    }
    a.joins[c] = j;
}

// A CTA's walk over its segments.
struct AttnWalk {
    int r, left, k;     // request, units left, segments done
    int h, rt;          // head and row tile of the current segment
    int L, t0, nt;      // its length, first key tile, key tiles
    int tile, tiles;    // its first key tile here and how many
    bool whole;
};
template <int KT>
__device__ __forceinline__ AttnWalk attn_begin(const AttnArgs& a, const AttnPlan& p) {
    AttnWalk w{};
    w.r = p.begin_r;
    w.left = p.count;
    w.k = -1;
    if (p.count > 0) {
        w.L = p.begin_L;
        const int2 t = attn_tiles<KT>(a, w.L);
        w.t0 = t.x;
        w.nt = t.y;
        const int seg = p.begin_o / (a.ahead + t.y), o = p.begin_o - seg * (a.ahead + t.y);
        w.tile = t.x + max(o - a.ahead, 0);
        w.left -= min(max(a.ahead - o, 0), w.left);
        w.h = seg / a.row_tiles;
        w.rt = seg - w.h * a.row_tiles;
    }
    return w;
}
template <int KT>
__device__ __forceinline__ bool attn_next(const AttnArgs& a, AttnWalk& w) {
    if (w.k >= 0) {
        w.left -= w.tiles + a.ahead;
        if (++w.rt == a.row_tiles) {
            w.rt = 0;
            if (++w.h == a.Hkv && w.left > 0) {
                w.h = 0;
                w.L = attn_len(a, ++w.r);
                const int2 t = attn_tiles<KT>(a, w.L);
                w.t0 = t.x;
                w.nt = t.y;
            }
        }
        w.tile = w.t0;
    }
    if (w.left <= 0) return false;
    w.tiles = min(w.t0 + w.nt - w.tile, w.left);
    w.whole = w.tiles == w.nt;
    ++w.k;
    return true;
}

// attention_tc.cu: bf16 or FP8 cache, row tiles of a.slot_rows (32, 64, 128 or 256)
cudaError_t launch_attn_tc(int D, bool f8, const CUtensorMap& km, const CUtensorMap& vm, const AttnArgs& a, int grid,
                           cudaStream_t s);

}  // namespace moestep
