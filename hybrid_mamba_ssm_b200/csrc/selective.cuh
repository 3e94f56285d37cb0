// selective.cuh -- device helpers of the per-channel selective scan kernels
// (selective_scan.cu, selective_scan_bwd.cu, selective_update.cu).
#pragma once

#include "common.cuh"
#include "ssm_internal.h"

namespace ssm {

// Two fp32 lanes in one 64-bit register.  The packed operations run the same
// fp32 arithmetic as the scalar ones at the same rate of lanes, but take one
// issue slot for two of them (measured on this part: 16 packed fma beside 8
// ex2 hide completely under the ex2; 32 scalar ones do not).
struct f32x2 {
    uint64_t v;
};
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(f32x2 a) {
    return __uint_as_float((uint32_t)a.v);
}
__device__ __forceinline__ float hi2(f32x2 a) {
    return __uint_as_float((uint32_t)(a.v >> 32));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 a) { return lo2(a) + hi2(a); }
__device__ __forceinline__ f32x2 ex2_pair(f32x2 a) {
    return pack2(ex2_approx(lo2(a)), ex2_approx(hi2(a)));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// NV consecutive fp32 values of shared memory (16-byte aligned for NV >= 4,
// 8-byte for NV == 2) as packed pairs.
template <int NP2>
__device__ __forceinline__ void lds_pairs(const float *p, f32x2 (&v)[NP2]) {
    if constexpr (NP2 % 2 == 0) {
#pragma unroll
        for (int i = 0; i < NP2 / 2; ++i) {
            const ulonglong2 q = reinterpret_cast<const ulonglong2 *>(p)[i];
            v[2 * i].v = q.x;
            v[2 * i + 1].v = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP2; ++i) v[i].v = reinterpret_cast<const unsigned long long *>(p)[i];
    }
}

// Sum of v[i] over groups of S lanes (lane bits kLow*1 .. kLow*S/2, i.e. lanes
// that differ in log2(S) bits starting at bit value kLow), for TG (a power of
// two) independent values at once.  Each exchange halves the values a lane
// still carries, so TG values cost TG/2 + TG/4 + ... shuffles rather than
// TG log2(S).  On return v[0 .. reduce_left(TG, S)-1] hold the sums of values
// first_value .. first_value + reduce_left - 1 (first_value depends on the
// lane).  When S > TG every value ends in S / TG lanes.
constexpr int reduce_left(int tg, int s) { return tg > s ? tg / s : 1; }

template <int TG, int S, int kLow>
__device__ __forceinline__ int reduce_lanes(float (&v)[TG], int lane) {
    int first = 0, n = TG;
#pragma unroll
    for (int o = kLow * S / 2; o >= kLow; o >>= 1) {
        if (n > 1) {
            const int half = n / 2;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < TG / 2; ++i) {
                if (i < half) {
                    const float send = up ? v[i] : v[i + half];
                    const float keep = up ? v[i + half] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
            first += up ? half : 0;
            n = half;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return first;
}

// dt after the optional transform, and the derivative of that transform with
// respect to the raw dt: sigmoid of the biased value for the softplus (1
// above 20, where log1p(e^v) equals v in fp32), 0 where the clamp is active.
// expf rather than the faster __expf: a step size enters every decay of its
// token, so its relative error is felt over the whole memory of a state.
__device__ __forceinline__ float dt_value(const DtParams &p, float raw, float bias) {
    float v = raw + bias;
    if (p.softplus) v = v > 20.f ? v : log1pf(expf(v));
    if (p.clamp) v = fminf(fmaxf(v, p.lo), p.hi);
    return v;
}
__device__ __forceinline__ float dt_slope(const DtParams &p, float raw, float bias) {
    float v = raw + bias, d = 1.f;
    if (p.softplus && v <= 20.f) {
        const float e = expf(v);
        d = __fdividef(e, 1.f + e);
        v = log1pf(e);
    }
    if (p.clamp && (v < p.lo || v > p.hi)) d = 0.f;
    return d;
}

// An activation value as loaded, and its fp32 value.  Loads keep the raw bits
// so that many can be in flight before the first is converted.
template <typename T>
__device__ __forceinline__ uint32_t raw_load(const void *p, long i) {
    if constexpr (sizeof(T) == 2) return static_cast<const unsigned short *>(p)[i];
    else return static_cast<const uint32_t *>(p)[i];
}
template <typename T>
__device__ __forceinline__ float raw_value(uint32_t r) {
    return __uint_as_float(sizeof(T) == 2 ? r << 16 : r);
}
template <typename T>
__device__ __forceinline__ float ld_as(const void *p, long i) {
    return raw_value<T>(raw_load<T>(p, i));
}

// Element i of an output row in either storage type.
__device__ __forceinline__ void st_act(void *p, long i, float v, int bf16) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// Token range [lo, hi) of sequence s in the packed stream; false (and a
// status) where the offsets are inconsistent, so that nothing outside the
// stream is touched.
__device__ __forceinline__ bool seq_range(const SelScanArgs &a, long T, int s, long &lo, long &hi) {
    if (!a.cu_seqlens) {
        lo = (long)s * a.seqlen;
        hi = lo + a.seqlen;
        return true;
    }
    lo = a.cu_seqlens[s];
    hi = a.cu_seqlens[s + 1];
    return lo >= 0 && hi >= lo && hi <= T && (s > 0 || lo == 0) && (s < a.nseq - 1 || hi == T);
}

}  // namespace ssm
