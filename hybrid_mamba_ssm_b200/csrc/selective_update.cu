// selective_update.cu -- one token per batch row of the per-channel selective
// scan, in place on the row's fp32 state [dim][d_state]:
//
//   h[d][n] <- exp(v A[d][n]) h[d][n] + v x[d] B[g][n]
//   y[d]     = (sum_n h[d][n] C[g][n] + D[d] x[d]) silu(z[d])
//
// Bound by HBM: every state element is read and written once.  A CTA takes
// kSets * 128 / L adjacent channels of one row (8 KB of state at d_state 16:
// one long run of addresses).  A thread owns four states (one 16-byte access) of
// kSets channels, whose loads are all issued before any arithmetic, and reads
// its B and C once for all of them.  The L lanes of a channel share the scalar
// work: a lane transforms the step size of its own set(s) of channels and hands
// v and v x to the others by shuffles, and the sums over n end in that same lane
// (reduce_lanes), which writes that y.  256 rows of 8192 channels, 16 states:
// 59 us, 4.8 TB/s (the loads' latency: 40 % occupancy by registers).  Four rows
// of 64 channels a CTA, which share a read of A, took 72 us: 4 KB runs from four
// places, and four sets of B and C.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kUpThreads = 128;
constexpr int kSets = 4;

template <typename TIn, typename TDt, int L, bool kVec>
__global__ void __launch_bounds__(kUpThreads, 7)
selective_update_kernel(SelUpdateArgs a, int ctiles)
{
    constexpr int CT = kUpThreads / L;                 // channels of a set
    constexpr int kOwn = reduce_left(kSets, L);        // sets whose scalar work is this lane's
    __shared__ __align__(16) float s_B[256], s_C[256];
    const int tid = threadIdx.x, lane = tid & 31, j = tid % L, N = a.d_state;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CT * kSets - 1) / (CT * kSets);
    const int ct = (int)(blockIdx.x % ctiles), g = ct / gtiles;
    const long b = blockIdx.x / ctiles;
    const int d0 = g * gdim + (ct - g * gtiles) * CT * kSets + tid / L, dend = (g + 1) * gdim;   // channel of set s: d0 + s CT

    long slot = b;
    if (a.slot_idx) {
        slot = a.slot_idx[b];
        if (slot >= a.max_slots) report_status(a.status_dev, kStatusDeviceInput);
        if (slot < 0 || slot >= a.max_slots) return;   // padding, or reported: the whole CTA
    }
    float *row = a.state + (slot * a.dim + d0) * (long)N;
    const float *Arow = a.A + (long)d0 * N;
    const int step = CT * N;                           // elements between the sets
    auto load4 = [&](const float *p, int n, bool stream, float (&v)[4]) {
        if (kVec) {
            const float4 q = stream ? __ldcs(reinterpret_cast<const float4 *>(p + n)) : __ldg(reinterpret_cast<const float4 *>(p + n));
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = n + i < N ? (stream ? __ldcs(p + n + i) : __ldg(p + n + i)) : 0.f;
        }
    };
    float h[kSets][4];
#pragma unroll
    for (int s = 0; s < kSets; ++s)
        if (d0 + s * CT < dend && j * 4 < N) load4(row + (long)s * step, j * 4, true, h[s]);

    // sets of this lane: as reduce_lanes leaves them
    const int first = L >= kSets ? j / (L / kSets) : j * kOwn;
    float x[kOwn], z[kOwn], v[kOwn], u[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int d = d0 + (first + i) * CT;
        const bool ok = d < dend;
        x[i] = ok ? ld_as<TIn>(a.x, b * a.x_stride + d) : 0.f;
        v[i] = ok ? ld_as<TDt>(a.dt, b * a.dt_stride + d) : 0.f;
        z[i] = ok && a.z ? ld_as<TIn>(a.z, b * a.z_stride + d) : 0.f;
    }
    for (int e = tid; e < N; e += kUpThreads) {
        s_B[e] = ld_as<TIn>(a.B, b * a.B_stride + g * N + e);
        s_C[e] = ld_as<TIn>(a.C, b * a.C_stride + g * N + e);
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int d = d0 + (first + i) * CT;
        v[i] = dt_value(a.dtp, v[i], a.dtp.bias && d < dend ? __ldg(a.dtp.bias + d) : 0.f);
        u[i] = v[i] * x[i];
    }
    float vs[kSets], us[kSets];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        constexpr int kLanes = L >= kSets ? L / kSets : 1;
        const int owner = (lane & ~(L - 1)) | (L >= kSets ? s * kLanes : s / kOwn);
        vs[s] = __shfl_sync(0xffffffffu, v[s % kOwn], owner);
        us[s] = __shfl_sync(0xffffffffu, u[s % kOwn], owner);
    }
    __syncthreads();

    float acc[kSets] = {};
    for (int n = j * 4; n < N; n += L * 4) {
        float B[4], C[4];
        if (kVec) {
            const float4 p = *reinterpret_cast<const float4 *>(&s_B[n]), q = *reinterpret_cast<const float4 *>(&s_C[n]);
            B[0] = p.x; B[1] = p.y; B[2] = p.z; B[3] = p.w;
            C[0] = q.x; C[1] = q.y; C[2] = q.z; C[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                B[i] = n + i < N ? s_B[n + i] : 0.f;
                C[i] = n + i < N ? s_C[n + i] : 0.f;
            }
        }
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            if (d0 + s * CT >= dend) break;
            float A[4];
            load4(Arow + (long)s * step, n, false, A);
            if (n != j * 4) load4(row + (long)s * step, n, true, h[s]);   // d_state above 128
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[s][i] = fmaf(ex2_approx(fmaf(vs[s] * kLog2e, A[i], kEx2Bias)), h[s][i], us[s] * B[i]);
                acc[s] = fmaf(h[s][i], C[i], acc[s]);
            }
            float *p = row + (long)s * step + n;
            if (kVec) {
                __stcs(reinterpret_cast<float4 *>(p), make_float4(h[s][0], h[s][1], h[s][2], h[s][3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < N) __stcs(p + i, h[s][i]);
            }
        }
    }
    reduce_lanes<kSets, L, 1>(acc, lane);
    if (L > kSets && j % (L > kSets ? L / kSets : 1)) return;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int d = d0 + (first + i) * CT;
        if (d >= dend) break;
        float y = fmaf(a.D ? __ldg(a.D + d) : 0.f, x[i], acc[i]);
        if (a.z) y *= silu_approx(z[i]);
        st_act(a.y, b * a.dim + d, y, a.y_bf16);
    }
}

template <typename TIn, typename TDt, int L>
cudaError_t launch_l(const SelUpdateArgs &a, cudaStream_t stream)
{
    constexpr int CT = kUpThreads / L;
    const int gdim = a.dim / a.ngroups, ctiles = (gdim + CT * kSets - 1) / (CT * kSets) * a.ngroups;
    const long long blocks = (long long)ctiles * a.batch;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.d_state % 4 == 0)
        selective_update_kernel<TIn, TDt, L, true><<<(unsigned)blocks, kUpThreads, 0, stream>>>(a, ctiles);
    else
        selective_update_kernel<TIn, TDt, L, false><<<(unsigned)blocks, kUpThreads, 0, stream>>>(a, ctiles);
    return cudaGetLastError();
}

template <typename TIn, typename TDt>
cudaError_t launch_types(const SelUpdateArgs &a, cudaStream_t stream)
{
    const int N = a.d_state;
    if (N <= 4) return launch_l<TIn, TDt, 1>(a, stream);
    if (N <= 8) return launch_l<TIn, TDt, 2>(a, stream);
    if (N <= 16) return launch_l<TIn, TDt, 4>(a, stream);
    if (N <= 32) return launch_l<TIn, TDt, 8>(a, stream);
    if (N <= 64) return launch_l<TIn, TDt, 16>(a, stream);
    return launch_l<TIn, TDt, 32>(a, stream);
}

}  // namespace

cudaError_t launch_selective_update(const SelUpdateArgs &a, cudaStream_t stream)
{
    if (!a.in_bf16) return launch_types<float, float>(a, stream);
    if (a.dt_bf16) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return launch_types<__nv_bfloat16, float>(a, stream);
}

}  // namespace ssm
