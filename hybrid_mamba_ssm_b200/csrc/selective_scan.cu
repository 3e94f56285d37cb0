// selective_scan.cu -- the per-channel selective scan over whole sequences:
// for channel d (group g = d / (dim / ngroups)), state index n and token t,
//
//   v       = clamp(softplus(dt[t][d] + dt_bias[d]))
//   h[d][n] = exp(v A[d][n]) h[d][n] + v x[t][d] B[t][g][n]
//   y[t][d] = (sum_n h[d][n] C[t][g][n] + D[d] x[t][d]) silu(z[t][d])
//
// Unlike the per-head scan of scan_tc.cu the decay differs in every (d, n), so
// a chunk's token-to-token products do not factor into matrix products over d
// or n: the state is advanced token by token.  Per (token, channel, n) that is
// one exponential and four fp32 multiply-adds.
//
// Layout of the work: L lanes of a warp share a channel, each keeping R of its
// states in registers as packed pairs; a CTA of 128 threads takes 128 / L
// channels of one group.  Tokens go through shared memory in tiles: each
// (token, channel) is loaded, its step size transformed and multiplied by x
// exactly once, then read by the channel's L lanes, while the next tile's
// global loads are in flight.  The sums over n of a few tokens are exchanged
// together (reduce_lanes), so they cost about one shuffle per token and lane.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 128;

constexpr int min3(int a, int b, int c) { return a < b ? (a < c ? a : c) : (b < c ? b : c); }

template <int R, int L>
struct ScanShape {
    static constexpr int CT = kThreads / L;                      // channels per CTA
    static constexpr int NP = R * L;                             // states, zero padded
    static constexpr int KT = min3(32, 1024 / NP, 1024 / CT);    // tokens per tile
    static constexpr int TG = KT < 4 ? KT : 4;                   // tokens summed together
    static constexpr int RS = kThreads / CT;                     // tokens per staging step
    static constexpr int E = (KT + RS - 1) / RS;                 // staged values per thread
    static constexpr int EB = (KT * NP + kThreads - 1) / kThreads;
};

// States of one channel: R values from index j * R on, zero behind d_state.
template <int R>
__device__ __forceinline__ void load_states(const float *row, int j, int N, f32x2 (&h)[R / 2]) {
    if (R % 4 == 0 && N % 4 == 0) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const int n = j * R + r;
            const float4 q = n < N ? *reinterpret_cast<const float4 *>(row + n) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[r / 2] = pack2(q.x, q.y);
            h[r / 2 + 1] = pack2(q.z, q.w);
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            const int n = j * R + r;
            h[r / 2] = pack2(n < N ? row[n] : 0.f, n + 1 < N ? row[n + 1] : 0.f);
        }
    }
}
template <int R>
__device__ __forceinline__ void store_states(float *row, int j, int N, const f32x2 (&h)[R / 2]) {
    if (R % 4 == 0 && N % 4 == 0) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const int n = j * R + r;
            if (n < N)
                *reinterpret_cast<float4 *>(row + n) =
                    make_float4(lo2(h[r / 2]), hi2(h[r / 2]), lo2(h[r / 2 + 1]), hi2(h[r / 2 + 1]));
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            const int n = j * R + r;
            if (n < N) row[n] = lo2(h[r / 2]);
            if (n + 1 < N) row[n + 1] = hi2(h[r / 2]);
        }
    }
}

// Sequence that holds token t (t < T): the last s with start <= t.
__device__ __forceinline__ int seq_of(const SelScanArgs &a, long t) {
    if (!a.cu_seqlens) return (int)(t / a.seqlen);
    int lo = 0, hi = a.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

enum { kWhole = 0, kRangeState = 1, kRangeOut = 2 };

// kWhole: one CTA per (sequence, channel tile).
// kRangeState / kRangeOut: one CTA per (range of the token stream, channel
// tile), two launches.  The first leaves, for every range whose last sequence
// goes on behind it, the state that the range's own tokens build from zero (or
// from the sequence's initial state, where it starts inside the range) and the
// sum of its step sizes: the range multiplies the state that enters it by
// exp(A sum v).  It also copies the initial state of a sequence that goes on
// behind the range.  The second folds the ranges before its own and runs its
// tokens from the state that enters.
template <typename TIn, typename TDt, int R, int L, int kMode>
__global__ void __launch_bounds__(kThreads)
selective_scan_kernel(SelScanArgs a)
{
    using S = ScanShape<R, L>;
    constexpr int CT = S::CT, NP = S::NP, KT = S::KT, TG = S::TG, RS = S::RS, E = S::E, EB = S::EB;
    constexpr int P = R / 2;
    __shared__ __align__(16) float s_v[KT * CT];
    __shared__ __align__(16) float s_u[KT * CT];
    __shared__ __align__(16) float s_y[kMode == kRangeState ? 1 : KT * CT];
    __shared__ __align__(16) float s_B[KT * NP];
    __shared__ __align__(16) float s_C[kMode == kRangeState ? 4 : KT * NP];

    const int tid = threadIdx.x, lane = tid & 31;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CT - 1) / CT, tiles = gtiles * a.ngroups;
    const int unit = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x - (unsigned)unit * tiles);
    const int g = tile / gtiles, c0 = g * gdim + (tile - g * gtiles) * CT, cend = min(c0 + CT, (g + 1) * gdim);
    const int N = a.d_state;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;

    const int j = tid % L, ch = tid / L, d = c0 + ch;      // scanning: lane j of channel d
    const int sc = tid % CT, st = tid / CT, ds = c0 + sc;  // staging: channel ds
    const bool live = d < cend, slive = ds < cend;
    const float bias = slive && a.dtp.bias ? a.dtp.bias[ds] : 0.f;
    const float skip = slive && a.D ? a.D[ds] : 0.f;

    f32x2 A[P], h[P];
#pragma unroll
    for (int p = 0; p < P; ++p) A[p] = pack2(0.f, 0.f);
    if (live) load_states<R>(a.A + (long)d * N, j, N, A);
#pragma unroll
    for (int p = 0; p < P; ++p) A[p] = mul2(A[p], pack2(kLog2e, kLog2e));

    float vsum = 0.f;
    uint32_t xr[E], vr[E], Br[EB], Cr[EB];      // raw values of the next tile

    // Raw values of the tile at t (tokens up to te), zero elsewhere.
    auto fetch = [&](long t, long te) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const long tt = t + st + i * RS;
            const bool ok = slive && tt < te && st + i * RS < KT;
            xr[i] = ok ? raw_load<TIn>(a.x, tt * a.x_stride + ds) : 0u;
            vr[i] = ok ? raw_load<TDt>(a.dt, tt * a.dt_stride + ds) : 0u;
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            const int e = tid + i * kThreads, n = e % NP;
            const long tt = t + e / NP;
            const bool ok = n < N && tt < te && e < KT * NP;
            Br[i] = ok ? raw_load<TIn>(a.B, tt * a.B_stride + (long)g * N + n) : 0u;
            if (kMode != kRangeState)
                Cr[i] = ok ? raw_load<TIn>(a.C, tt * a.C_stride + (long)g * N + n) : 0u;
        }
    };

    // Tokens [t, te) of a sequence that starts at token lo.
    auto run = [&](long t, long te, long lo, long save0) {
        auto tile_end = [&](long t0) {   // tiles end on multiples of KT of the sequence
            return min(te, t0 + KT - (t0 - lo) % KT);
        };
        long t1 = tile_end(t);
        fetch(t, t1);
        while (t < te) {
            float xc[E];
            uint32_t zc[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int k = st + i * RS;
                xc[i] = raw_value<TIn>(xr[i]);
                if (k < KT) {
                    const float v = slive && t + k < t1 ? dt_value(a.dtp, raw_value<TDt>(vr[i]), bias) : 0.f;
                    s_v[k * CT + sc] = v;
                    s_u[k * CT + sc] = v * xc[i];
                }
            }
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int e = tid + i * kThreads;
                if (e < KT * NP) {
                    s_B[e] = raw_value<TIn>(Br[i]);
                    if (kMode != kRangeState) s_C[e] = raw_value<TIn>(Cr[i]);
                }
            }
            __syncthreads();
            const long t2 = t1 < te ? tile_end(t1) : t1;
            if (t1 < te) fetch(t1, t2);
            if (kMode != kRangeState && a.z) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int k = st + i * RS;
                    zc[i] = slive && k < KT && t + k < t1 ? raw_load<TIn>(a.z, (t + k) * a.z_stride + ds) : 0u;
                }
            }
            if (kMode != kRangeState && a.saved && (t - lo) % kSavedEvery == 0 && live)
                store_states<R>(a.saved + ((save0 + (t - lo) / kSavedEvery) * a.dim + d) * N, j, N, h);

#pragma unroll 1
            for (int k0 = 0; k0 < KT && t + k0 < t1; k0 += TG) {
                float yv[TG];
#pragma unroll
                for (int k = 0; k < TG; ++k) {
                    const float v = s_v[(k0 + k) * CT + ch], u = s_u[(k0 + k) * CT + ch];
                    const f32x2 vv = pack2(v, v), uu = pack2(u, u);
                    f32x2 B[P], C[P], acc = pack2(0.f, 0.f);
                    lds_pairs(s_B + (k0 + k) * NP + j * R, B);
                    if (kMode != kRangeState) lds_pairs(s_C + (k0 + k) * NP + j * R, C);
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        h[p] = fma2(ex2_pair(mul2(vv, A[p])), h[p], mul2(uu, B[p]));
                        if (kMode != kRangeState) acc = fma2(h[p], C[p], acc);
                    }
                    yv[k] = sum2(acc);
                    if (kMode == kRangeState) vsum += v;
                }
                if (kMode != kRangeState) {
                    const int first = reduce_lanes<TG, L, 1>(yv, lane);
                    constexpr int kLeft = reduce_left(TG, L);
                    constexpr int kSame = L > TG ? L / TG : 1;   // lanes that end with the same sum
                    if (j % kSame == 0) {
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) s_y[(k0 + first + i) * CT + ch] = yv[i];
                    }
                }
            }
            __syncthreads();
            if (kMode != kRangeState) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int k = st + i * RS;
                    if (slive && k < KT && t + k < t1) {
                        float y = fmaf(skip, xc[i], s_y[k * CT + sc]);
                        if (a.z) y *= silu_approx(raw_value<TIn>(zc[i]));
                        st_act(a.y, (t + k) * a.dim + ds, y, a.y_bf16);
                    }
                }
            }
            t = t1;
            t1 = t2;
        }
    };

    // Row of the sequence's state, -1 for a bad slot; whether it is read.
    auto state_row = [&](int s, bool &init) -> long {
        init = a.initial && !(a.has_initial && a.has_initial[s] == 0);
        if (!a.slot_idx) return s;
        const int slot = a.slot_idx[s];
        if (slot >= 0 && slot < a.max_slots) return slot;
        report_status(a.status_dev, kStatusDeviceInput);
        return -1;
    };
    auto load_initial = [&](long row, bool init) {
#pragma unroll
        for (int p = 0; p < P; ++p) h[p] = pack2(0.f, 0.f);
        if (init && live) load_states<R>(a.initial + (row * a.dim + d) * N, j, N, h);
    };
    auto one_sequence = [&](int s, long r0, long r1) {   // its tokens within [r0, r1)
        long lo, hi;
        if (!seq_range(a, T, s, lo, hi)) {
            report_status(a.status_dev, kStatusDeviceInput);
            return;
        }
        if (lo < r0 && hi <= r0) return;                  // ended in an earlier range
        bool init;
        const long row = state_row(s, init);
        if (row < 0) return;
        if (kMode == kRangeOut && lo < r0) {
            // the state entering this range: the ranges since the sequence's start, folded
            const int first = (int)(lo / a.span), own = (int)(r0 / a.span);
#pragma unroll
            for (int p = 0; p < P; ++p) h[p] = pack2(0.f, 0.f);
            for (int q = first; q < own && live; ++q) {
                f32x2 e[P];
                load_states<R>(a.range_state + ((long)q * a.dim + d) * N, j, N, e);
                const float v = a.range_dt[(long)q * a.dim + d];
#pragma unroll
                for (int p = 0; p < P; ++p) h[p] = q == first ? e[p] : fma2(ex2_pair(mul2(pack2(v, v), A[p])), h[p], e[p]);
            }
        } else if (kMode == kRangeOut && hi > r1) {
            // its row may be written (in place) by the range it ends in: the copy is read
#pragma unroll
            for (int p = 0; p < P; ++p) h[p] = pack2(0.f, 0.f);
            if (live) load_states<R>(a.range_initial + ((r0 / a.span) * a.dim + d) * N, j, N, h);
        } else {
            load_initial(row, init);
        }
        const long b = max(lo, r0), e = min(hi, r1);
        if (b < e) run(b, e, lo, lo / kSavedEvery + s);
        if (hi <= r1 && a.final && live && (lo < hi || a.final != a.initial || !init))
            store_states<R>(a.final + (row * a.dim + d) * N, j, N, h);
    };

    if (kMode == kWhole) {
        one_sequence(unit, 0, T);
    } else if (kMode == kRangeState) {
        const long r0 = (long)unit * a.span, r1 = r0 + a.span;   // never the last range: r1 < T
        const int s = seq_of(a, r1 - 1);
        long lo, hi;
        bool init;
        if (!seq_range(a, T, s, lo, hi) || lo >= r1 || hi <= r1) return;
        const long row = state_row(s, init);
        if (row < 0) return;
        load_initial(row, init && lo >= r0);
        if (lo >= r0 && live) store_states<R>(a.range_initial + ((long)unit * a.dim + d) * N, j, N, h);
        run(max(lo, r0), r1, lo, 0);
        if (!live) return;
        store_states<R>(a.range_state + ((long)unit * a.dim + d) * N, j, N, h);
        if (j == 0) a.range_dt[(long)unit * a.dim + d] = vsum;
    } else {
        const long r0 = (long)unit * a.span, r1 = min(r0 + a.span, T);
        int s = seq_of(a, r0);
        // empty sequences that lie at r0, before the one that holds it
        while (a.cu_seqlens && s > 0 && a.cu_seqlens[s - 1] >= r0) --s;
        for (; s < a.nseq; ++s) {
            const long lo = a.cu_seqlens ? (long)a.cu_seqlens[s] : (long)s * a.seqlen;
            if (lo >= r1 && r1 < T) break;
            one_sequence(s, r0, r1);
        }
    }
}

template <typename TIn, typename TDt, int R, int L>
cudaError_t launch_shape(const SelScanArgs &a, cudaStream_t stream)
{
    const int gdim = a.dim / a.ngroups, CT = ScanShape<R, L>::CT;
    const long long tiles = (long long)((gdim + CT - 1) / CT) * a.ngroups;
    if (tiles * (a.ranges ? a.ranges : a.nseq) > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (!a.ranges) {
        selective_scan_kernel<TIn, TDt, R, L, kWhole><<<(unsigned)(tiles * a.nseq), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    if (a.ranges > 1)
        selective_scan_kernel<TIn, TDt, R, L, kRangeState><<<(unsigned)(tiles * (a.ranges - 1)), kThreads, 0, stream>>>(a);
    selective_scan_kernel<TIn, TDt, R, L, kRangeOut><<<(unsigned)(tiles * a.ranges), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename TIn, typename TDt>
cudaError_t launch_types(const SelScanArgs &a, cudaStream_t stream)
{
    const int N = a.d_state;
    if (N <= 4) return launch_shape<TIn, TDt, 4, 1>(a, stream);
    if (N <= 8) return launch_shape<TIn, TDt, 4, 2>(a, stream);
    if (N <= 16) return launch_shape<TIn, TDt, 4, 4>(a, stream);
    if (N <= 32) return launch_shape<TIn, TDt, 4, 8>(a, stream);
    if (N <= 64) return launch_shape<TIn, TDt, 4, 16>(a, stream);
    if (N <= 128) return launch_shape<TIn, TDt, 4, 32>(a, stream);
    return launch_shape<TIn, TDt, 8, 32>(a, stream);
}

}  // namespace

int selective_scan_ranges(int nseq, long T, int dim, int d_state, int ngroups, int *span)
{
    *span = 0;
    return 0;
}

cudaError_t launch_selective_scan(const SelScanArgs &a, cudaStream_t stream)
{
    if (!a.in_bf16) return launch_types<float, float>(a, stream);
    if (a.dt_bf16) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return launch_types<__nv_bfloat16, float>(a, stream);
}

}  // namespace ssm
