// selective_update.cu -- one token per batch row of the per-channel selective
// scan, in place on the row's fp32 state [dim][d_state]:
//
//   h[d][n] <- exp(v A[d][n]) h[d][n] + v x[d] B[g][n]
//   y[d]     = (sum_n h[d][n] C[g][n] + D[d] x[d]) silu(z[d])
//
// Bound by HBM: every state element is read and written once.  A thread owns
// four states of one channel (one 16-byte access) for kRows batch rows: A is
// as large as one row's state, so reading it for every row would double the
// reads that reach the SM; kRows rows share one read, and their loads are all
// issued before any arithmetic.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kUpThreads = 256;
constexpr int kRows = 4;

template <typename TIn, typename TDt, int L, bool kVec>
__global__ void __launch_bounds__(kUpThreads)
selective_update_kernel(SelUpdateArgs a, int ctiles)
{
    constexpr int CT = kUpThreads / L;
    const int tid = threadIdx.x, j = tid % L;
    const int ct = (int)(blockIdx.x % ctiles);
    const long b0 = (long)(blockIdx.x / ctiles) * kRows;
    const int d = ct * CT + tid / L, N = a.d_state;
    const bool live = d < a.dim;
    const int dd = live ? d : a.dim - 1;               // lanes behind dim only take part in the shuffles
    const int g = dd / (a.dim / a.ngroups);

    // states n0 + 128 q .. + 3 for q = 0, 1 (d_state above 128 only)
    float *row[kRows];
    bool on[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const long b = b0 + r;
        on[r] = false;
        row[r] = nullptr;
        if (b >= a.batch) continue;
        long slot = b;
        if (a.slot_idx) {
            slot = a.slot_idx[b];
            if (slot < 0) continue;
            if (slot >= a.max_slots) {
                report_status(a.status_dev, kStatusDeviceInput);
                continue;
            }
        }
        on[r] = true;
        row[r] = a.state + (slot * a.dim + dd) * (long)N;
    }
    const float bias = a.dtp.bias ? __ldg(a.dtp.bias + dd) : 0.f;
    const float skip = a.D ? __ldg(a.D + dd) : 0.f;
    float acc[kRows] = {}, v[kRows], x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        v[r] = x[r] = 0.f;
        if (on[r]) {
            x[r] = ld_as<TIn>(a.x, (b0 + r) * a.x_stride + dd);
            v[r] = ld_as<TDt>(a.dt, (b0 + r) * a.dt_stride + dd);
        }
    }
    for (int n = j * 4; n < N; n += L * 4) {
        float h[kRows][4], A[4];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (kVec) {
                const float4 q = on[r] && live ? __ldcs(reinterpret_cast<const float4 *>(row[r] + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
                h[r][0] = q.x; h[r][1] = q.y; h[r][2] = q.z; h[r][3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[r][i] = on[r] && live && n + i < N ? __ldcs(row[r] + n + i) : 0.f;
            }
        }
        if (kVec) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(a.A + (long)dd * N + n));
            A[0] = q.x * kLog2e; A[1] = q.y * kLog2e; A[2] = q.z * kLog2e; A[3] = q.w * kLog2e;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = n + i < N ? __ldg(a.A + (long)dd * N + n + i) * kLog2e : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (!on[r]) continue;
            const long b = b0 + r;
            const float vv = dt_value(a.dtp, v[r], bias), u = vv * x[r];
            float B[4], C[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                B[i] = n + i < N ? ld_as<TIn>(a.B, b * a.B_stride + (long)g * N + n + i) : 0.f;
                C[i] = n + i < N ? ld_as<TIn>(a.C, b * a.C_stride + (long)g * N + n + i) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(ex2_approx(vv * A[i]), h[r][i], u * B[i]);
                acc[r] = fmaf(h[r][i], C[i], acc[r]);
            }
            if (!live) continue;
            if (kVec) {
                __stcs(reinterpret_cast<float4 *>(row[r] + n), make_float4(h[r][0], h[r][1], h[r][2], h[r][3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < N) __stcs(row[r] + n + i, h[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        if (on[r] && live && j == 0) {
            const long b = b0 + r;
            float y = fmaf(skip, x[r], acc[r]);
            if (a.z) y *= silu_approx(ld_as<TIn>(a.z, b * a.z_stride + d));
            st_act(a.y, b * a.dim + d, y, a.y_bf16);
        }
    }
}

template <typename TIn, typename TDt, int L>
cudaError_t launch_l(const SelUpdateArgs &a, cudaStream_t stream)
{
    constexpr int CT = kUpThreads / L;
    const int ctiles = (a.dim + CT - 1) / CT;
    const long long blocks = (long long)ctiles * ((a.batch + kRows - 1) / kRows);
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
