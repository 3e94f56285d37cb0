// abi_checks.h -- host-side argument checks shared by the C ABI layers
// (abi.cu, abi_selective.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssm.h"
#include "ssm_internal.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

Range range_of(const void *p, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}

bool overlap(Range a, Range b)
{
    if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

size_t dtype_size(int dt) { return dt == SSM_BF16 ? 2 : 4; }

bool valid_dtype(int dt) { return dt == SSM_F32 || dt == SSM_BF16; }

bool pow2_in(int v, int lo, int hi)
{
    return v >= lo && v <= hi && (v & (v - 1)) == 0;
}

// Device-side form of the optional dt transform.  Returns SSM_OK, or the
// status for a malformed one (misaligned bias, dt_min > dt_max, NaN bounds).
int read_dt_params(const ssm_dt_params *p, ssm::DtParams &out)
{
    out = ssm::DtParams{};
    if (!p) return SSM_OK;
    if (p->dt_bias && !aligned16(p->dt_bias)) return SSM_ERR_MISALIGNED;
    if (p->clamp && !(p->dt_min <= p->dt_max)) return SSM_ERR_INVALID_ARG;
    out.bias = p->dt_bias;
    out.softplus = p->softplus != 0;
    out.clamp = p->clamp != 0;
    out.lo = p->dt_min;
    out.hi = p->dt_max;
    return SSM_OK;
}

// Storage of a state pool: fp32, or fp16 with round-to-nearest (rounding
// NULL) or stochastic rounding.
int read_state_format(int state_dtype, const ssm_rounding *r, ssm::RoundParams &out)
{
    out = ssm::RoundParams{};
    if (state_dtype == SSM_F32) return SSM_OK;
    if (state_dtype != SSM_F16) return SSM_ERR_INVALID_ARG;
    out.f16 = 1;
    if (r) {
        if (r->philox_rounds < 1 || r->philox_rounds > 16) return SSM_ERR_INVALID_ARG;
        out.stochastic = 1;
        out.key0 = (uint32_t)r->seed;
        out.key1 = (uint32_t)(r->seed >> 32);
        out.off0 = (uint32_t)r->offset;
        out.off1 = (uint32_t)(r->offset >> 32);
        out.rounds = r->philox_rounds;
    }
    return SSM_OK;
}

}  // namespace
