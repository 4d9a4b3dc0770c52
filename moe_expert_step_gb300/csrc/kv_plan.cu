// Pages and positions of a batch's next tokens, given out on the GPU: requests take pages from
// the front of a ring of free pages or return them to its end, their page tables are extended,
// and every new token gets its position and its slot in the pool.
//
// A first-in-first-out ring, not a stack: pages taken are read from [first, first + count) and
// pages returned are written from first + count on, places that never meet while the pool's pages
// are distinct, so blocks need no order among themselves.  Where a request's pages begin in
// the ring is a sum over the requests before it.  Every block adds those up by itself (a few
// loads a thread from L2 for the batches of serving) instead of waiting for a launch that does.
// The header is written by one block: the last that has read it where it is updated in place (a ticket tells),
// else any.
//
// Bound by latency: header, lengths, sums, ring or table, slots are reads that depend on one another.  One request of 32
// new tokens takes 7 us on the device and the call of it 8.6; 256 requests of up to 4096 tokens (8.7 MB of positions and
// slots, 1.3 us at the copy rate) 8.6 us.  Divisions by the page size (a shift instead) and a header written by the last
// block only (by any, where it is not updated in place) cost the larger one 3.4 us.
#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

namespace moestep {
namespace {

constexpr int kThreads = 256;
constexpr int kTicket = 48;  // word of the workspace that counts the blocks that have read the ring's header (no other call's)

struct PlanArgs {
    const int32_t* kv_len;
    const int32_t* n_new;
    int32_t* ring;
    const int32_t* head;
    int32_t* head_out;
    int32_t* table;
    int32_t* new_len;
    int32_t* pos;
    int32_t* slots;
    int* err;
    int* ticket;
    int R, n, page_log2, n_pages, max_pages;
    int rows;      // requests of a block
    int segments;  // or, where that is 1, blocks of a request
    int wide;      // pos and slots can be written four at a time
    int in_place;  // head_out is head
};

// What a request asks for
struct Ask {
    int len, m, held, need;
    bool bad, fits;
    __device__ __forceinline__ int grow() const { return fits ? max(need - held, 0) : 0; }
    __device__ __forceinline__ int drop() const { return max(held - need, 0); }
};
__device__ __forceinline__ Ask ask_of(const PlanArgs& a, int r) {
    Ask q;
    q.len = __ldg(&a.kv_len[r]);
    q.m = __ldg(&a.n_new[r]);
    const int cap = a.max_pages << a.page_log2, up = (1 << a.page_log2) - 1;
    q.bad = q.len < 0 || q.len > cap || q.m > a.n || q.m < -q.len;
    if (q.bad) q.m = 0;
    const int len = q.bad ? 0 : q.len;
    q.held = (len + up) >> a.page_log2;
    q.fits = !q.bad && q.m <= cap - len;
    q.need = q.fits ? (len + q.m + up) >> a.page_log2 : q.held;
    return q;
}

struct Sums {
    long long grow, drop;
};

// Sums over the block, in all threads; `sm` is free again after the call's second barrier
__device__ __forceinline__ Sums block_sums(Sums v, Sums* sm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.grow += __shfl_xor_sync(0xffffffffu, v.grow, o);
        v.drop += __shfl_xor_sync(0xffffffffu, v.drop, o);
    }
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = v;
    __syncthreads();
    v = sm[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v.grow += sm[w].grow, v.drop += sm[w].drop;
    __syncthreads();
    return v;
}

// Sums over the threads before this one
__device__ __forceinline__ Sums block_before(Sums v, Sums* sm) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Sums run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long g = __shfl_up_sync(0xffffffffu, run.grow, o), d = __shfl_up_sync(0xffffffffu, run.drop, o);
        if (lane >= o) run.grow += g, run.drop += d;
    }
    if (lane == 31) sm[warp] = run;
    __syncthreads();
    Sums out{run.grow - v.grow, run.drop - v.drop};
    for (int w = 0; w < warp; ++w) out.grow += sm[w].grow, out.drop += sm[w].drop;
    __syncthreads();
    return out;
}

__device__ __forceinline__ Sums sums_of(const PlanArgs& a, int first, int last) {
    Sums s{0, 0};
    for (int r = first + threadIdx.x; r < last; r += kThreads) {
        const Ask q = ask_of(a, r);
        s.grow += q.grow();
        s.drop += q.drop();
    }
    return s;
}

struct Row {
    int len, m, held, need;
    long long take, back;  // pages that the requests before it take and return
    bool served;
};

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const PlanArgs a) {
    __shared__ Sums sm[kThreads / 32];
    __shared__ Row rows[kThreads];
    __shared__ bool writes;
    pdl_trigger();
    pdl_wait();
    int first = a.head[0], count = a.head[1];
    const bool broken = static_cast<unsigned>(first) >= static_cast<unsigned>(a.n_pages) ||
                        static_cast<unsigned>(count) > static_cast<unsigned>(a.n_pages);
    if (broken) first = 0, count = 0;
    if (broken && threadIdx.x == 0) record_error(a.err, kErrBadInput);

    const int r0 = blockIdx.x / a.segments * a.rows, segment = blockIdx.x % a.segments;
    const int n_rows = min(a.rows, a.R - r0);
    const Sums before = block_sums(sums_of(a, 0, r0), sm);
    // (behind the barriers of block_sums: every thread has read the header; the ticket wraps to 0 for the next call)
    if (threadIdx.x == 0) {
        writes = blockIdx.x == gridDim.x - 1;
        if (a.in_place && gridDim.x > 1) {
            __threadfence();
            writes = atomicInc(reinterpret_cast<unsigned*>(a.ticket), gridDim.x - 1) == gridDim.x - 1;
        }
    }
    {
        Ask q{};
        Sums mine{0, 0};
        const bool on = threadIdx.x < n_rows;
        if (on) {
            q = ask_of(a, r0 + threadIdx.x);
            mine = Sums{q.grow(), q.drop()};
        }
        const Sums ahead = block_before(mine, sm);
        if (on) {
            Row w{q.len, q.m, q.held, q.need, before.grow + ahead.grow, before.drop + ahead.drop, false};
            w.served = q.fits && (mine.grow == 0 || w.take + mine.grow <= count);
            if (broken) w.served = q.fits && q.need == q.held;
            if (!w.served) w.m = 0, w.need = w.held;
            rows[threadIdx.x] = w;
            if (segment == 0) {
                if (q.bad) record_error(a.err, kErrBadInput);
                a.new_len[r0 + threadIdx.x] = q.len + w.m;
            }
        }
    }
    __syncthreads();

    const unsigned ring = a.n_pages;
    auto around = [&](unsigned i) { return i >= ring ? i - ring : i; };  // (i < 2 n_pages < 2^32)
    auto page_at = [&](const Row& w, int i) {  // table entry i >= held of a served request
        const int id = a.ring[around(first + static_cast<unsigned>(w.take) + (i - w.held))];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.n_pages)) return id;
        record_error(a.err, kErrBadInput);
        return -1;
    };
    const int step = a.segments * kThreads;
    for (int j = 0; j < n_rows; ++j) {  // table entries that are new, pages that go back
        const Row& w = rows[j];
        int32_t* table = a.table + static_cast<long long>(r0 + j) * a.max_pages;
        const int t0 = segment * kThreads + threadIdx.x;
        for (int i = w.held + t0; i < w.need; i += step) table[i] = page_at(w, i);
        for (int i = w.need + t0; i < w.held; i += step) {
            const long long o = count + w.back + (i - w.need);  // (w.back may be a broken table's)
            const int id = table[i];
            if (o < ring) a.ring[around(first + static_cast<unsigned>(o))] = id;  // (else more pages than the pool has)
            if (o >= ring || static_cast<unsigned>(id) >= static_cast<unsigned>(a.n_pages))
                record_error(a.err, kErrBadInput);
        }
    }

    const int mask = (1 << a.page_log2) - 1;
    auto page_of = [&](const Row& w, const int32_t* table, int p) {  // first slot of the page of position p
        const int pg = p >> a.page_log2;
        const int id = pg < w.held ? __ldcg(&table[pg]) : page_at(w, pg);
        if (static_cast<unsigned>(id) < static_cast<unsigned>(a.n_pages)) return id << a.page_log2;
        record_error(a.err, kErrBadInput);
        return -1;
    };
    auto slot_at = [&](int page, int p) { return page < 0 ? -1 : page + (p & mask); };
    if (a.wide) {
        const int quads = a.n / 4, total = n_rows * quads;
#pragma unroll 4
        for (int k = segment * kThreads + threadIdx.x; k < total; k += step) {
            const int j = a.rows > 1 ? k / quads : 0, i = 4 * (k - j * quads);
            const Row& w = rows[j];
            const long long at = static_cast<long long>(r0 + j) * a.n + i;
            int4 p = make_int4(-1, -1, -1, -1), s = p;
            if (i < w.m) {
                const int32_t* table = a.table + static_cast<long long>(r0 + j) * a.max_pages;
                const int p0 = w.len + i, p3 = w.len + min(i + 3, w.m - 1);
                const int page = page_of(w, table, p0), after = p3 >> a.page_log2 == p0 >> a.page_log2 ? page : page_of(w, table, p3);
                auto slot = [&](int q) { return slot_at(q >> a.page_log2 == p0 >> a.page_log2 ? page : after, q); };
                p.x = p0, s.x = slot(p0);
                if (i + 1 < w.m) p.y = p0 + 1, s.y = slot(p0 + 1);
                if (i + 2 < w.m) p.z = p0 + 2, s.z = slot(p0 + 2);
                if (i + 3 < w.m) p.w = p0 + 3, s.w = slot(p0 + 3);
            }
            *reinterpret_cast<int4*>(a.pos + at) = p;
            if (a.slots) *reinterpret_cast<int4*>(a.slots + at) = s;
        }
    } else {
        const long long total = static_cast<long long>(n_rows) * a.n;
        for (long long k = segment * kThreads + threadIdx.x; k < total; k += step) {
            const int j = static_cast<int>(k / a.n), i = static_cast<int>(k - static_cast<long long>(j) * a.n);
            const Row& w = rows[j];
            const int p = i < w.m ? w.len + i : -1;
            const int s = p < 0 ? -1 : slot_at(page_of(w, a.table + static_cast<long long>(r0 + j) * a.max_pages, p), p);
            const long long at = static_cast<long long>(r0) * a.n + k;
            a.pos[at] = p;
            if (a.slots) a.slots[at] = s;
        }
    }

    // the header
    if (!writes) return;
    __syncthreads();
    Sums run{0, 0};
    long long taken = 0;
    for (int r = 0; r < a.R; r += kThreads) {
        Sums mine{0, 0};
        if (r + threadIdx.x < a.R) {
            const Ask q = ask_of(a, r + threadIdx.x);
            mine = Sums{q.grow(), q.drop()};
        }
        const Sums ahead = block_before(mine, sm);
        const long long upto = run.grow + ahead.grow + mine.grow;
        if (mine.grow > 0 && upto <= count) taken = upto;
        const Sums all = block_sums(mine, sm);
        run.grow += all.grow;
        run.drop += all.drop;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32].grow = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) taken = max(taken, sm[w].grow);
        if (broken) {
            a.head_out[0] = a.head[0];
            a.head_out[1] = a.head[1];
        } else {
            const long long most = static_cast<long long>(ring) - count;  // what did not fit was not written
            a.head_out[0] = static_cast<int>(around(first + static_cast<unsigned>(taken)));
            a.head_out[1] = static_cast<int>(count - taken + min(run.drop, most));
        }
    }
}

}  // namespace
}  // namespace moestep

extern "C" int kv_cache_plan(const moestep_kv_dims* kd, int R, int n, const int32_t* kv_len, const int32_t* n_new,
                             int32_t* ring, const int32_t* head, int32_t* head_out, int32_t* table, int32_t* new_len,
                             int32_t* pos, int32_t* slots, void* ws, size_t ws_bytes, void* stream) {
    using namespace moestep;
    int rc = check_kv_dims(kd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n <= 0) return MOESTEP_EINVAL;
    if (!kv_len || !n_new || !ring || !head || !head_out || !table || !new_len || !pos) return MOESTEP_EINVAL;
    // blocks read every request's lengths while others write theirs
    if (new_len == kv_len || new_len == n_new) return MOESTEP_EINVAL;
    for (const void* p : {static_cast<const void*>(kv_len), static_cast<const void*>(n_new),
                          static_cast<const void*>(ring), static_cast<const void*>(head),
                          static_cast<const void*>(head_out), static_cast<const void*>(table),
                          static_cast<const void*>(new_len), static_cast<const void*>(pos),
                          static_cast<const void*>(slots)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return MOESTEP_EALIGN;
    if (R > (1 << 20)) return MOESTEP_EUNSUPPORTED;
    if ((rc = check_kv_ws(ws, ws_bytes, kKvHeader)) != MOESTEP_OK) return rc;
    if ((rc = device_ok(nullptr)) != MOESTEP_OK) return rc;
    PlanArgs a{};
    a.kv_len = kv_len;
    a.n_new = n_new;
    a.ring = ring;
    a.head = head;
    a.head_out = head_out;
    a.table = table;
    a.new_len = new_len;
    a.pos = pos;
    a.slots = slots;
    a.err = static_cast<int*>(ws);
    a.ticket = static_cast<int*>(ws) + kTicket;
    a.R = R;
    a.n = n;
    a.page_log2 = kd->page == 16 ? 4 : kd->page == 32 ? 5 : kd->page == 64 ? 6 : 7;
    a.n_pages = kd->n_pages;
    a.max_pages = kd->max_pages;
    a.in_place = head_out == head;
    a.wide = n % 4 == 0 && kv_aligned16(pos) && (!slots || kv_aligned16(slots));
    // a block writes about 4096 positions
    constexpr int kEntries = 4096;
    a.rows = n >= kEntries ? 1 : kEntries / n < kThreads ? kEntries / n : kThreads;
    if (a.rows > R) a.rows = R;
    a.segments = a.rows > 1 ? 1 : static_cast<int>((n + kEntries - 1ll) / kEntries);
    const long long grid = 1ll * ((R + a.rows - 1) / a.rows) * a.segments;
    if (grid > (1ll << 31) - 1) return MOESTEP_EUNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    const cudaError_t e = launch_pdl(kv_plan_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, a);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}
