// Arguments and host-side checks shared by the two forms of the gated delta rule.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv.h"
#include "moestep.h"

namespace moestep {

struct DeltaArgs {
    const void* q;
    const void* k;
    const void* v;
    long long q_ld, k_ld, v_ld;
    const float* g;
    const float* beta;
    const int32_t* length;
    const int32_t* slot;
    const uint8_t* fresh;
    const float* state;
    float* state_out;
    void* out;
    int* err;
    int R, n, Hk, Hv, Dk, Dv, n_slots;
    float scale, eps;  // eps <= 0: queries and keys as they are
    unsigned long long timeout_ns;
};

inline int check_delta_dims(const moestep_delta_dims* d) {
    if (d == nullptr) return MOESTEP_EINVAL;
    if (d->Hk <= 0 || d->Hv <= 0 || d->Dk <= 0 || d->Dv <= 0 || d->n_slots <= 0) return MOESTEP_EINVAL;
    if (d->dtype != MOESTEP_BF16 && d->dtype != MOESTEP_F32) return MOESTEP_EINVAL;
    if (d->Hv % d->Hk || d->Hv > 1024) return MOESTEP_EUNSUPPORTED;
    if ((d->Dk != 64 && d->Dk != 128) || (d->Dv != 64 && d->Dv != 128)) return MOESTEP_EUNSUPPORTED;
    return MOESTEP_OK;
}

// e^g - 1 for |g| < 1/4 by its Taylor series up to g^7 (what is left out is below 2^-29 of the whole, 2^-31 of e^g).  1 + that, rounded
// once, for decays close to 1: they multiply a state hundreds of times, where errors of one direction add up (with expf 500
// tokens of g around -2e-4 leave states 2e-6 off, so 3e-7; expm1f cost one token of 128 requests 3 us of 80).
__device__ __forceinline__ float grown(float g) {
    float c = 1.f / 5040;
    c = fmaf(c, g, 1.f / 720);
    c = fmaf(c, g, 1.f / 120);
    c = fmaf(c, g, 1.f / 24);
    c = fmaf(c, g, 1.f / 6);
    c = fmaf(c, g, 0.5f);
    return fmaf(c, g, 1.f) * g;
}

// Request's tokens and slot; false: nothing to do (a negative slot), or bad values, recorded once
__device__ __forceinline__ bool delta_request(const DeltaArgs& a, int r, bool record, int& tokens, int& slot) {
    tokens = a.length ? __ldg(&a.length[r]) : a.n;
    slot = a.slot ? __ldg(&a.slot[r]) : r;
    if (slot < 0) return false;
    if (slot >= a.n_slots || tokens < 0 || tokens > a.n) {
        if (record) atomicOr(a.err, 1 << 8);
        return false;
    }
    return true;
}

// Workspace of the chunked form (bytes behind the header); 0 where the recurrent one is taken
bool delta_chunked(const moestep_delta_dims& d, int R, int n);
size_t delta_chunk_bytes(const moestep_delta_dims& d, int R, int n);
cudaError_t launch_delta_recurrent(const DeltaArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_delta_chunks(const DeltaArgs& a, void* scratch, int sms, cudaStream_t s);

}  // namespace moestep
