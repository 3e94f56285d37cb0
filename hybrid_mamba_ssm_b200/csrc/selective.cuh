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

// Decays 2^(v A) (A in units of log2 e).  ex2.approx is 2e-8 of its value low
// on average between 2^-0.5 and 2^-0.003 (measured here), which a long memory
// adds up: a state that lasts 300 tokens would come out 6e-6 small.  kEx2Bias in
// the exponent takes the average out, at no cost (an fma for a product); it
// rounds away where the decay is exactly 1.
constexpr float kEx2Bias = 2.9e-8f;
__device__ __forceinline__ f32x2 decay2(f32x2 v, f32x2 A) {
    return ex2_pair(fma2(v, A, pack2(kEx2Bias, kEx2Bias)));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Decay rates in units of log2 e, kept finite: a token with a step size of 0
// (the tokens that fill up a tile among them) has the decay 2^(0 A) = 1
// whatever A is, and 0 * -inf would be NaN.
__device__ __forceinline__ f32x2 decay_rate2(f32x2 A) {
    const f32x2 r = mul2(A, pack2(kLog2e, kLog2e));
    return pack2(max_nan(lo2(r), -3.402823466e38f), max_nan(hi2(r), -3.402823466e38f));
}

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

// e^-a for a >= 0 to about an ulp: 2^t with the rounding of t = -a log2 e
// carried as a first-order correction.
__device__ __forceinline__ float exp_neg(float a) {
    const float t = a * -kLog2e, lost = fmaf(a, -kLog2e, -t) - a * 1.9259629911e-8f;
    const float e = ex2_approx(t);
    return fmaf(e, lost * kLn2, e);
}

// log(1 + e^v) = max(v, 0) + log1p(e) with e = e^-|v| in [0, 1]; log1p(e) / e
// is interpolated at ten Chebyshev nodes of [0, 1] (error 1.4e-8).  A step
// size enters every decay of its token, so it is kept to about an ulp.
__device__ constexpr float kLog1p[10] = {
    1.f, -0.49999892711639404f, 0.33329710364341736f, -0.24951615929603577f, 0.1966327428817749f,
    -0.1526966691017151f, 0.10543623566627502f, -0.056373611092567444f, 0.019542526453733444f,
    -0.0031760570127516985f};
__device__ __forceinline__ float log1p_unit(float e) {
    float q = kLog1p[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) q = fmaf(q, e, kLog1p[i]);
    return q * e;
}

// dt after the optional transform, and the derivative of that transform with
// respect to the raw dt: the sigmoid of the biased value for the softplus, 0
// where the clamp is active.  exp_neg's argument is capped where the result
// has long been 0 (infinities would meet in its correction).
__device__ __forceinline__ float dt_value(const DtParams &p, float raw, float bias) {
    float v = raw + bias;
    if (p.softplus) v = fmaxf(v, 0.f) + log1p_unit(exp_neg(min_nan(fabsf(v), 120.f)));
    if (p.clamp) v = clamp_nan(v, p.lo, p.hi);
    return v;
}
__device__ __forceinline__ float dt_slope(const DtParams &p, float raw, float bias) {
    float v = raw + bias, d = 1.f;
    if (p.softplus) {
        const float e = ex2_approx(min_nan(fabsf(v), 120.f) * -kLog2e), r = rcp_approx(1.f + e);
        d = v >= 0.f ? r : e * r;
    }
    if (p.clamp) {
        if (p.softplus) v = fmaxf(v, 0.f) + log1p_unit(exp_neg(min_nan(fabsf(v), 120.f)));
        if (v < p.lo || v > p.hi) d = 0.f;
    }
    return d;
}

// dt_value of two channels at once (packed).
__device__ __forceinline__ f32x2 dt_value2(const DtParams &p, f32x2 raw, f32x2 bias) {
    f32x2 v = add2(raw, bias);
    if (p.softplus) {
        const f32x2 a = pack2(min_nan(fabsf(lo2(v)), 120.f), min_nan(fabsf(hi2(v)), 120.f));
        const f32x2 t = mul2(a, pack2(-kLog2e, -kLog2e));
        const f32x2 lost = fma2(a, pack2(1.9259629911e-8f, 1.9259629911e-8f), fma2(a, pack2(kLog2e, kLog2e), t));
        f32x2 e = ex2_pair(t);
        e = fma2(e, mul2(lost, pack2(-kLn2, -kLn2)), e);
        f32x2 q = pack2(kLog1p[9], kLog1p[9]);
#pragma unroll
        for (int i = 8; i >= 0; --i) q = fma2(q, e, pack2(kLog1p[i], kLog1p[i]));
        v = fma2(q, e, pack2(fmaxf(lo2(v), 0.f), fmaxf(hi2(v), 0.f)));
    }
    if (p.clamp) v = pack2(clamp_nan(lo2(v), p.lo, p.hi), clamp_nan(hi2(v), p.lo, p.hi));
    return v;
}
__device__ __forceinline__ f32x2 dt_slope2(const DtParams &p, f32x2 raw, f32x2 bias) {
    if (p.clamp)   // rare: one by one
        return pack2(dt_slope(p, lo2(raw), lo2(bias)), dt_slope(p, hi2(raw), hi2(bias)));
    if (!p.softplus) return pack2(1.f, 1.f);
    const f32x2 v = add2(raw, bias);
    const f32x2 a = pack2(min_nan(fabsf(lo2(v)), 120.f), min_nan(fabsf(hi2(v)), 120.f));
    const f32x2 e = ex2_pair(mul2(a, pack2(-kLog2e, -kLog2e))), d = add2(e, pack2(1.f, 1.f));
    const float r0 = rcp_approx(lo2(d)), r1 = rcp_approx(hi2(d));
    return pack2(lo2(v) >= 0.f ? r0 : lo2(e) * r0, hi2(v) >= 0.f ? r1 : hi2(e) * r1);
}
__device__ __forceinline__ f32x2 silu2(f32x2 z) {
    const f32x2 d = add2(ex2_pair(mul2(z, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f));
    return mul2(z, pack2(rcp_approx(lo2(d)), rcp_approx(hi2(d))));
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
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
}

// Two adjacent values as loaded.  kPacked: they are one aligned access, so a
// bf16 pair is one register.
template <typename T, bool kPacked>
struct RawPair {
    uint32_t r[sizeof(T) == 2 && kPacked ? 1 : 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(r) / 4); ++i) r[i] = 0u;
    }
    // values p[i], p[i + 1]; p + i is aligned to both
    __device__ __forceinline__ void load(const T *p, int i) {
        static_assert(kPacked, "");
        if constexpr (sizeof(T) == 2) {
            r[0] = *reinterpret_cast<const uint32_t *>(p + i);
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(p + i);
            r[0] = q.x;
            r[1] = q.y;
        }
    }
    // one by one; ok1 without ok0 does not happen
    __device__ __forceinline__ void load(const T *p, int i, bool ok0, bool ok1) {
        if constexpr (sizeof(r) == 4) {
            r[0] = ok0 ? (uint32_t)raw_load<T>(p, i) | (ok1 ? (uint32_t)raw_load<T>(p, i + 1) << 16 : 0u) : 0u;
        } else {
            r[0] = ok0 ? raw_load<T>(p, i) : 0u;
            r[1] = ok1 ? raw_load<T>(p, i + 1) : 0u;
        }
    }
    __device__ __forceinline__ f32x2 value() const {
        if constexpr (sizeof(r) == 4) return pack2(__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u));
        else return pack2(raw_value<T>(r[0]), raw_value<T>(r[1]));
    }
};

// Stores v[0], and v[1] when `both`: as one aligned access when `aligned`.
template <typename T>
__device__ __forceinline__ void store_pair(T *p, f32x2 v, bool aligned, bool both) {
    if (aligned) {
        if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(lo2(v), hi2(v));
        else *reinterpret_cast<float2 *>(p) = make_float2(lo2(v), hi2(v));
    } else {
        store_out(p, lo2(v));
        if (both) store_out(p + 1, hi2(v));
    }
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

// Units of work: a sequence, or a segment of `span` tokens of one (span: a
// multiple of kSavedEvery; 0: whole sequences).  Segment k of sequence s is
// unit start(s) / span + s + k of start(end) / span + nseq: sequences never
// share a unit (see saved_row), and some units have no tokens.
struct Unit {
    int s, k;
    long lo, hi;   // the sequence
    long b, e;     // the unit's tokens
    long base;     // the sequence's segment 0
};
__device__ __forceinline__ bool find_unit(const SelScanArgs &a, long T, int u, Unit &q) {
    auto base = [&](int s) { return (a.cu_seqlens ? (long)a.cu_seqlens[s] : (long)s * a.seqlen) / a.span + s; };
    q.s = u;
    q.k = 0;
    q.base = u;
    if (a.span) {
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (base(mid) <= u) lo = mid; else hi = mid - 1;
        }
        q.s = lo;
        q.base = base(lo);
        if (q.base > u) return false;
        q.k = (int)(u - q.base);
    }
    if (!seq_range(a, T, q.s, q.lo, q.hi)) {
        report_status(a.status_dev, kStatusDeviceInput);
        return false;
    }
    q.b = a.span ? q.lo + (long)q.k * a.span : q.lo;
    q.e = a.span ? min(q.b + a.span, q.hi) : q.hi;
    return q.k == 0 || q.b < q.hi;
}

// With segments, a unit is found by searching the offsets, which inconsistent
// ones can lead past a sequence: one CTA looks at them all, to report them.
__device__ __forceinline__ void check_offsets(const SelScanArgs &a, long T) {
    if (!a.span || blockIdx.x || !a.cu_seqlens) return;
    long lo, hi;
    for (int s = threadIdx.x; s < a.nseq; s += blockDim.x)
        if (!seq_range(a, T, s, lo, hi)) report_status(a.status_dev, kStatusDeviceInput);
}

// The sequence with the u-th longest range (ties by index): packed batches run
// longest first, so that the last CTAs to start are short.  Every thread of
// the CTA takes part; nseq is at most blockDim.x.
__device__ __forceinline__ int longest_first(const SelScanArgs &a, int u, int *shared) {
    const int i = threadIdx.x;
    if (i < a.nseq) {
        const int len = a.cu_seqlens[i + 1] - a.cu_seqlens[i];
        int rank = 0;
        for (int k = 0; k < a.nseq; ++k) {
            const int other = a.cu_seqlens[k + 1] - a.cu_seqlens[k];
            rank += other > len || (other == len && k < i);
        }
        if (rank == u) *shared = i;
    }
    __syncthreads();
    return *shared;
}
}  // namespace ssm
