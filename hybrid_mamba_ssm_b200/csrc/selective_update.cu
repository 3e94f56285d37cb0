// selective_update.cu -- one token per batch row of the per-channel selective
// scan, in place on the row's fp32 state [dim][d_state]:
//
//   h[d][n] <- exp(v A[d][n]) h[d][n] + v x[d] B[g][n]
//   y[d]     = (sum_n h[d][n] C[g][n] + D[d] x[d]) silu(z[d])
//
// Bound by HBM: every state element is read and written once.  A thread owns
// four states of one channel (one 16-byte access) in kRows batch rows, whose
// loads are all issued before any arithmetic; the kRows rows also share one
// read of A, which is as large as a row's state.  The L lanes of a channel
// share the rows' scalar work: a lane transforms the step size of its own
// row(s) and hands v and v x to the others by shuffles, and the sums over n
// end in that same lane (reduce_lanes), which writes its row's y.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kUpThreads = 256;
constexpr int kRows = 4;

template <typename TIn, typename TDt, int L, bool kVec>
__global__ void __launch_bounds__(kUpThreads, 4)
selective_update_kernel(SelUpdateArgs a, int ctiles)
{
    constexpr int CT = kUpThreads / L;
    constexpr int kOwn = reduce_left(kRows, L);        // rows whose scalar work is this lane's
    __shared__ __align__(16) float s_B[kRows][256], s_C[kRows][256];
    const int tid = threadIdx.x, lane = tid & 31, j = tid % L, N = a.d_state;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CT - 1) / CT;
    const int ct = (int)(blockIdx.x % ctiles), g = ct / gtiles;
    const long b0 = (long)(blockIdx.x / ctiles) * kRows;
    const int d = g * gdim + (ct - g * gtiles) * CT + tid / L;
    const bool live = d < (g + 1) * gdim;

    float *row[kRows];
    bool on[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const long b = b0 + r;
        long slot = b < a.batch ? b : -1;
        if (a.slot_idx && b < a.batch) {
            slot = a.slot_idx[b];
            if (slot >= a.max_slots) {
                report_status(a.status_dev, kStatusDeviceInput);
                slot = -1;
            }
        }
        on[r] = slot >= 0;
        row[r] = a.state + (slot * a.dim + d) * (long)N;
    }
    auto load4s = [&](int n, float (&h)[kRows][4]) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool ok = on[r] && live;
            if (kVec) {
                const float4 q = ok && n < N ? __ldcs(reinterpret_cast<const float4 *>(row[r] + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
                h[r][0] = q.x; h[r][1] = q.y; h[r][2] = q.z; h[r][3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[r][i] = ok && n + i < N ? __ldcs(row[r] + n + i) : 0.f;
            }
        }
    };
    float h[kRows][4];
    load4s(j * 4, h);

    // rows of this lane: as reduce_lanes leaves them
    const int first = L >= kRows ? j / (L / kRows) : j * kOwn;
    float x[kOwn], z[kOwn], v[kOwn], u[kOwn];
    const float bias = live && a.dtp.bias ? __ldg(a.dtp.bias + d) : 0.f, skip = live && a.D ? __ldg(a.D + d) : 0.f;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const long b = b0 + first + i;
        const bool ok = live && b < a.batch;
        x[i] = ok ? ld_as<TIn>(a.x, b * a.x_stride + d) : 0.f;
        v[i] = ok ? ld_as<TDt>(a.dt, b * a.dt_stride + d) : 0.f;
        z[i] = ok && a.z ? ld_as<TIn>(a.z, b * a.z_stride + d) : 0.f;
    }
    for (int e = tid; e < kRows * N; e += kUpThreads) {
        const int r = e / N, n = e - r * N;
        const bool ok = b0 + r < a.batch;
        s_B[r][n] = ok ? ld_as<TIn>(a.B, (b0 + r) * a.B_stride + (long)g * N + n) : 0.f;
        s_C[r][n] = ok ? ld_as<TIn>(a.C, (b0 + r) * a.C_stride + (long)g * N + n) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        v[i] = dt_value(a.dtp, v[i], bias);
        u[i] = v[i] * x[i];
    }
    float vr[kRows], ur[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        constexpr int kLanes = L >= kRows ? L / kRows : 1;
        const int owner = (lane & ~(L - 1)) | (L >= kRows ? r * kLanes : r / kOwn);
        vr[r] = __shfl_sync(0xffffffffu, v[r % kOwn], owner);
        ur[r] = __shfl_sync(0xffffffffu, u[r % kOwn], owner);
    }
    __syncthreads();

    float acc[kRows] = {};
    for (int n = j * 4; n < N; n += L * 4) {
        if (n != j * 4) load4s(n, h);                  // d_state above 128
        float A[4];
        if (kVec) {
            const float4 q = live ? __ldg(reinterpret_cast<const float4 *>(a.A + (long)d * N + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
            A[0] = q.x; A[1] = q.y; A[2] = q.z; A[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = live && n + i < N ? __ldg(a.A + (long)d * N + n + i) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] *= kLog2e;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float B[4], C[4];
            if (kVec) {
                const float4 p = *reinterpret_cast<const float4 *>(&s_B[r][n]), q = *reinterpret_cast<const float4 *>(&s_C[r][n]);
                B[0] = p.x; B[1] = p.y; B[2] = p.z; B[3] = p.w;
                C[0] = q.x; C[1] = q.y; C[2] = q.z; C[3] = q.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    B[i] = n + i < N ? s_B[r][n + i] : 0.f;
                    C[i] = n + i < N ? s_C[r][n + i] : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(ex2_approx(vr[r] * A[i]), h[r][i], ur[r] * B[i]);
                acc[r] = fmaf(h[r][i], C[i], acc[r]);
            }
            if (!on[r] || !live) continue;
            if (kVec) {
                __stcs(reinterpret_cast<float4 *>(row[r] + n), make_float4(h[r][0], h[r][1], h[r][2], h[r][3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < N) __stcs(row[r] + n + i, h[r][i]);
            }
        }
    }
    reduce_lanes<kRows, L, 1>(acc, lane);
    if (!live || (L > kRows && j % (L / kRows))) return;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const long b = b0 + first + i;
        bool mine = false;
#pragma unroll
        for (int r = 0; r < kRows; ++r) mine |= on[r] && r == first + i;
        if (!mine) continue;
        float y = fmaf(skip, x[i], acc[i]);
        if (a.z) y *= silu_approx(z[i]);
        st_act(a.y, b * a.dim + d, y, a.y_bf16);
    }
}

template <typename TIn, typename TDt, int L>
cudaError_t launch_l(const SelUpdateArgs &a, cudaStream_t stream)
{
    constexpr int CT = kUpThreads / L;
    const int gdim = a.dim / a.ngroups, ctiles = (gdim + CT - 1) / CT * a.ngroups;
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
