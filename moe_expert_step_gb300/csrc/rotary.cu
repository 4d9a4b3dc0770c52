// Rotary positions: the first `rot` elements of every query and key head are turned in pairs by
// position * frequency, x' = (x0 cos - x1 sin, x1 cos + x0 sin) * mscale.
//
// Angles.  A far position turns its fast pairs thousands of times, and 32-bit products keep nothing
// of the turn's fraction (position 10^6 at one radian a position: 0.06 radians off).  So a
// frequency is held as its fraction of a turn a position in 64-bit fixed point, 2^64 a turn:
// position * frequency modulo 2^64 is the fraction of the turn exactly, two integer
// multiplications.  Its upper 32 bits (2^-32 turns off at most), as a float of half-turns (another 2^-26 turns, 1.6 units of
// 2^-24 radians), go to sincospif.
//
// The kernel is a copy bound by memory.  A thread takes one 16-byte piece of the pairs of one
// token, computes its sines and cosines once, and turns that piece of several heads with them (four
// at most: their loads stand in registers before the first store.  32768 tokens of 18 heads of 128, 302 MB:
// 51.7 us, 5.75 TB/s, 85 % of the copy rate; with load and store by turns 77 us).  Few tokens are spread over more
// threads by heads: 32 tokens take 1.9 us of the device in a graph, the rest of their 16 us is the host.
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "kv.h"
#include "launch.cuh"

namespace moestep {
namespace {

struct RotaryArgs {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    long long q_ld, k_ld, qo_ld, ko_ld;
    const int32_t* pos;
    const uint64_t* freq;
    long long tokens;
    int Hq, Hkv, D, rot;
    int turned, items;  // pieces of a head that are turned, and all
    int groups;         // threads that share a token's piece, each with every groups-th head
    float mscale;
};

constexpr int kHeads = 4;  // of a thread, at most

// V elements of a 16-byte piece, or one
template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
    T v[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V == 1)
            v[0] = *p;
        else
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V == 1)
            *p = v[0];
        else
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    }
};

__device__ __forceinline__ void turn_of(int pos, uint64_t freq, float mscale, float& s, float& c) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * freq;
    // turns in [-1/2, 1/2): half-turns are sincospif's unit
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    s *= mscale;
    c *= mscale;
}

// PAIRS: neighbouring elements are turned together, else those half of `rot` apart
template <typename T, int V, bool PAIRS>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
    constexpr int N = PAIRS ? (V == 1 ? 1 : V / 2) : V;  // pairs of a piece
    pdl_trigger();
    const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int per = a.items * a.groups;
    const long long t = at >> 32 ? at / per : static_cast<unsigned>(at) / static_cast<unsigned>(per);
    const int in = static_cast<int>(at - t * per), group = in / a.items, item = in - group * a.items;
    pdl_wait();
    if (t >= a.tokens) return;
    const int pos = __ldg(&a.pos[t]);
    if (pos < 0) return;
    const bool turned = item < a.turned;
    float sn[N], cs[N];
    int lo, hi;  // first element of the piece, and of the other halves of its pairs
    if (turned) {
#pragma unroll
        for (int i = 0; i < N; ++i) turn_of(pos, __ldg(&a.freq[item * N + i]), a.mscale, sn[i], cs[i]);
        lo = PAIRS ? item * (V == 1 ? 2 : V) : item * V;
        hi = PAIRS ? lo + 1 : lo + a.rot / 2;  // (PAIRS: of the piece of one pair)
    } else {
        lo = hi = a.rot + (item - a.turned) * V;
    }
    // every load before the first store, which may go to the same rows
    const int heads = a.Hq + a.Hkv;
    Piece<T, V> x[kHeads], y[kHeads];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = group + u * a.groups;
        if (h >= heads) break;
        const bool key = h >= a.Hq;
        const T* src = static_cast<const T*>(key ? a.k : a.q) + t * (key ? a.k_ld : a.q_ld) + (key ? h - a.Hq : h) * a.D;
        x[u].load(src + lo);
        if (!(PAIRS && V > 1) && turned) y[u].load(src + hi);
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
        const int h = group + u * a.groups;
        if (h >= heads) break;
        const bool key = h >= a.Hq;
        T* dst = static_cast<T*>(key ? a.k_out : a.q_out) + t * (key ? a.ko_ld : a.qo_ld) + (key ? h - a.Hq : h) * a.D;
        if (!turned) {
            x[u].store(dst + lo);  // (of a row turned in place: what stands there)
            continue;
        }
        if constexpr (PAIRS && V > 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = to_f32(x[u].v[2 * i]), g = to_f32(x[u].v[2 * i + 1]);
                x[u].v[2 * i] = from_f32<T>(f * cs[i] - g * sn[i]);
                x[u].v[2 * i + 1] = from_f32<T>(g * cs[i] + f * sn[i]);
            }
            x[u].store(dst + lo);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = to_f32(x[u].v[i]), g = to_f32(y[u].v[i]);
                x[u].v[i] = from_f32<T>(f * cs[i] - g * sn[i]);
                y[u].v[i] = from_f32<T>(g * cs[i] + f * sn[i]);
            }
            x[u].store(dst + lo);
            y[u].store(dst + hi);
        }
    }
}

template <typename T, int V>
cudaError_t launch_rotary(RotaryArgs a, bool pairs, int sms, cudaStream_t s) {
    const int heads = a.Hq + a.Hkv;
    a.turned = pairs ? a.rot / (V == 1 ? 2 : V) : a.rot / 2 / V;
    const bool copies = (a.Hq && (a.q != a.q_out)) || (a.Hkv && (a.k != a.k_out));
    a.items = a.turned + (copies ? (a.D - a.rot) / V : 0);
    // kHeads heads a thread share its sines; where that leaves multiprocessors idle, fewer
    a.groups = (heads + kHeads - 1) / kHeads;
    while (a.groups < heads && a.tokens * a.items * a.groups < 4ll * sms * 256) a.groups = a.groups * 2 < heads ? a.groups * 2 : heads;
    const long long blocks = (a.tokens * a.items * a.groups + 255) / 256;
    if (blocks > (1ll << 31) - 1) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks));
    return pairs ? launch_pdl(rotary_kernel<T, V, true>, grid, dim3(256), 0, s, a)
                 : launch_pdl(rotary_kernel<T, V, false>, grid, dim3(256), 0, s, a);
}

struct FrequencyArgs {
    uint64_t* freq;
    int rot, scaling;
    double base, factor, original, low, high;
};

constexpr double kTwoPi = 6.283185307179586476925286766559;

__global__ void __launch_bounds__(128) frequency_kernel(const FrequencyArgs a) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * 128 + threadIdx.x;
    if (i >= a.rot / 2) return;
    double f = pow(a.base, -2.0 * i / a.rot);
    double keep = 1.0;  // share of the frequency that is not divided by the factor
    if (a.scaling == MOESTEP_ROTARY_LINEAR) {
        keep = 0.0;
    } else if (a.scaling == MOESTEP_ROTARY_ROTATIONS) {
        keep = (a.original * f / kTwoPi - a.low) / (a.high - a.low);
    } else if (a.scaling == MOESTEP_ROTARY_DIMENSIONS) {
        // index at which a pair turns `r` times within the original context
        const double per = a.rot / (2.0 * log(a.base)), all = log(a.original / kTwoPi);
        const double lo = fmax(floor(per * (all - log(a.high))), 0.0);
        const double hi = fmin(ceil(per * (all - log(a.low))), a.rot - 1.0);
        keep = 1.0 - (i - lo) / fmax(hi - lo, 0.001);
    }
    keep = fmin(fmax(keep, 0.0), 1.0);
    if (a.scaling != MOESTEP_ROTARY_PLAIN) f = f * keep + f / a.factor * (1.0 - keep);
    double turns = f / kTwoPi;
    turns -= floor(turns);  // whole turns a position do not show
    a.freq[i] = __double2ull_rn(turns * 0x1p64);  // (turns <= 1 - 2^-53)
}

int check_rotary_rows(const void* p, long long ld, long long width, int dtype) {
    if (!p || ld < width) return MOESTEP_EINVAL;
    if (reinterpret_cast<uintptr_t>(p) % kv_act_bytes(dtype)) return MOESTEP_EALIGN;
    return MOESTEP_OK;
}

}  // namespace
}  // namespace moestep

extern "C" int rotary_frequencies(int rot, double base, int scaling, double factor, double original, double low,
                                  double high, uint64_t* freq, void* stream) {
    using namespace moestep;
    if (rot <= 0 || rot % 2 || !freq) return MOESTEP_EINVAL;
    if (!std::isfinite(base) || !(base > 1.0)) return MOESTEP_EINVAL;
    if (scaling < MOESTEP_ROTARY_PLAIN || scaling > MOESTEP_ROTARY_DIMENSIONS) return MOESTEP_EINVAL;
    if (scaling != MOESTEP_ROTARY_PLAIN && (!std::isfinite(factor) || !(factor > 0.0))) return MOESTEP_EINVAL;
    if (scaling == MOESTEP_ROTARY_ROTATIONS || scaling == MOESTEP_ROTARY_DIMENSIONS) {
        if (!std::isfinite(original) || !(original > 0.0) || !std::isfinite(low) || !std::isfinite(high) ||
            !(low > 0.0) || !(high > low))
            return MOESTEP_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(freq) & 7u) return MOESTEP_EALIGN;
    if (rot > 4096) return MOESTEP_EUNSUPPORTED;
    int rc;
    if ((rc = device_ok(nullptr)) != MOESTEP_OK) return rc;
    const FrequencyArgs a{freq, rot, scaling, base, factor, original, low, high};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    const cudaError_t e = launch_pdl(frequency_kernel, dim3((rot / 2 + 127) / 128), dim3(128), 0, s, a);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}

extern "C" int block_rotary(const moestep_kv_dims* kd, int R, int n, const void* q, long long q_ld, const void* k,
                            long long k_ld, const int32_t* pos, const uint64_t* freq, int rot, int pairs,
                            float mscale, void* q_out, long long qo_ld, void* k_out, long long ko_ld, void* stream) {
    using namespace moestep;
    int rc = check_kv_dims(kd);
    if (rc != MOESTEP_OK) return rc;
    if (R <= 0 || n <= 0 || !pos || !freq || rot <= 0 || rot % 2 || !std::isfinite(mscale)) return MOESTEP_EINVAL;
    if ((!q && !k) || !q != !q_out || !k != !k_out) return MOESTEP_EINVAL;
    if (rot > kd->D) return MOESTEP_EINVAL;
    const long long wq = 1ll * kd->Hq * kd->D, wk = 1ll * kd->Hkv * kd->D;
    if (q && (rc = check_rotary_rows(q, q_ld, wq, kd->dtype)) != MOESTEP_OK) return rc;
    if (q && (rc = check_rotary_rows(q_out, qo_ld, wq, kd->dtype)) != MOESTEP_OK) return rc;
    if (k && (rc = check_rotary_rows(k, k_ld, wk, kd->dtype)) != MOESTEP_OK) return rc;
    if (k && (rc = check_rotary_rows(k_out, ko_ld, wk, kd->dtype)) != MOESTEP_OK) return rc;
    if ((q && q == q_out && q_ld != qo_ld) || (k && k == k_out && k_ld != ko_ld)) return MOESTEP_EINVAL;
    if (reinterpret_cast<uintptr_t>(pos) & 3u || reinterpret_cast<uintptr_t>(freq) & 7u) return MOESTEP_EALIGN;
    // (a thread an element and head at most)
    if (1ll * R * n > ((1ll << 31) - 1) * 256 / (1ll * kd->D * (kd->Hq + kd->Hkv))) return MOESTEP_EUNSUPPORTED;
    int sms = 0;
    if ((rc = device_ok(&sms)) != MOESTEP_OK) return rc;
    RotaryArgs a{};
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.qo_ld = qo_ld;
    a.ko_ld = ko_ld;
    a.pos = pos;
    a.freq = freq;
    a.tokens = 1ll * R * n;
    a.Hq = q ? kd->Hq : 0;
    a.Hkv = k ? kd->Hkv : 0;
    a.D = kd->D;
    a.rot = rot;
    a.mscale = mscale;
    // 16-byte pieces where every row and the boundaries of the rotated part allow them
    const int bytes = kv_act_bytes(kd->dtype), v = 16 / bytes;
    bool wide = pairs ? rot % v == 0 : rot / 2 % v == 0;
    for (const void* p : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)}) wide = wide && kv_aligned16(p);
    if (q) wide = wide && q_ld % v == 0 && qo_ld % v == 0;
    if (k) wide = wide && k_ld % v == 0 && ko_ld % v == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    prof_begin(8, s);
    cudaError_t e;
    if (kd->dtype == MOESTEP_F32)
        e = wide ? launch_rotary<float, 4>(a, pairs != 0, sms, s) : launch_rotary<float, 1>(a, pairs != 0, sms, s);
    else
        e = wide ? launch_rotary<bf16, 8>(a, pairs != 0, sms, s) : launch_rotary<bf16, 1>(a, pairs != 0, sms, s);
    prof_end(8, s);
    if (e != cudaSuccess) {
        set_last_cuda(static_cast<int>(e));
        return MOESTEP_ECUDA;
    }
    count_launch();
    return MOESTEP_OK;
}
