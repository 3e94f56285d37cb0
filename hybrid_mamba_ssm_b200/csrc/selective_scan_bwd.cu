// selective_scan_bwd.cu -- gradient of the per-channel selective scan
// (selective_scan.cu).  With a = exp(v A), dyg = dy silu(z) and dh the
// gradient of the state behind token t, walking the tokens backwards:
//
//   dh   = C dyg + (a dh of the token behind; the final state's gradient at the end)
//   dC[n] += h dyg              dB[n] += dh v x          (summed over the channels of a group)
//   q    = (a dh) h_before      dA    += q v             (summed over the tokens)
//   w    = sum_n dh B           dx     = w v + D dyg
//   dv   = sum_n q A + w x      ddt    = dv (slope of the step-size transform)
//   dz   = dy (sum_n h C + D x) silu'(z),   dD = sum dyg x
//
// The states are recomputed, not stored: the forward pass left the state of
// every kSavedEvery-th token.  A CTA goes over a sequence's chunks of that
// length from the last to the first.  In a chunk it first runs forward from
// the saved state, leaving the state of every kSub-th token in shared memory
// (a thread reads back only what it wrote), then takes the sub-tiles in
// reverse: decays and states of kSub tokens are recomputed into registers and
// the recurrence above runs back over them.  That is two exponentials per
// (token, channel, n).
//
// L lanes share a channel, each with R states in packed pairs; a warp holds
// 32 / L channels at a time and takes CS such sets one after another, adding
// their dB and dC in registers before they are summed over its channels by
// shuffles (the sums over n, three per token and channel, go over the L lanes
// of a channel).  Per sub-tile the CTA's warps are added up through shared
// memory and the sum is written as one part per channel tile; a second launch
// adds the parts, in a fixed order, so results do not depend on the schedule.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kSub = 4;                          // tokens of a sub-tile
constexpr int kSubs = kSavedEvery / kSub;        // sub-tiles of a chunk
constexpr int kWarps = 4;
constexpr int kBwdThreads = 32 * kWarps;
constexpr int kMaxUnits = 64;                    // sequences are dealt to at most this many CTAs per tile

template <int R, int L, int CS>
struct BwdShape {
    static constexpr int CL = 32 / L;            // channels of a warp at a time
    static constexpr int CW = CL * CS;           // channels of a warp
    static constexpr int CB = CW * kWarps;       // channels of a CTA
    static constexpr int NP = R * L;
    static constexpr int kRow = kSavedEvery * CB;
    // floats of shared memory: v, u, g; B, C; sub-tile states; parts of dB, dC (two buffers)
    static constexpr int kStates = kSubs * CS * kBwdThreads * R;
    static constexpr int kParts = 2 * 2 * kWarps * kSub * NP;
    static constexpr size_t kBytes = sizeof(float) * (3 * kRow + 2 * kSavedEvery * NP + kStates + kParts);
    static_assert(kBwdThreads % CB == 0, "a staging thread keeps its channel");
};

template <int R>
__device__ __forceinline__ void load_row(const float *row, int j, int N, f32x2 (&h)[R / 2]) {
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
__device__ __forceinline__ void store_row(float *row, int j, int N, const f32x2 (&h)[R / 2]) {
#pragma unroll
    for (int r = 0; r < R; r += 2) {
        const int n = j * R + r;
        if (n < N) row[n] = lo2(h[r / 2]);
        if (n + 1 < N) row[n + 1] = hi2(h[r / 2]);
    }
}

template <typename TIn, typename TDt, int R, int L, int CS>
__global__ void __launch_bounds__(kBwdThreads)
selective_scan_bwd_kernel(SelScanBwdArgs b, int units)
{
    using S = BwdShape<R, L, CS>;
    constexpr int CB = S::CB, NP = S::NP, P = R / 2, KC = kSavedEvery;
    constexpr int RS = kBwdThreads / CB;         // tokens per staging step
    extern __shared__ __align__(16) float smem[];
    float *s_v = smem, *s_u = s_v + S::kRow, *s_g = s_u + S::kRow;
    float *s_B = s_g + S::kRow, *s_C = s_B + KC * NP;
    float *s_h = s_C + KC * NP, *s_part = s_h + S::kStates;
    const SelScanArgs &a = b.f;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CB - 1) / CB, tiles = gtiles * a.ngroups;
    const int unit = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x - (unsigned)unit * tiles);
    const int grp = tile / gtiles, gtile = tile - grp * gtiles;
    const int c0 = grp * gdim + gtile * CB, cend = min(c0 + CB, (grp + 1) * gdim);
    const int N = a.d_state;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;

    const int j = lane % L;
    const int ch0 = warp * S::CW + lane / L;     // channel of set q: ch0 + q * CL
    const int sc = tid % CB, st = tid / CB, ds = c0 + sc;
    const bool slive = ds < cend;
    const float bias = slive && a.dtp.bias ? a.dtp.bias[ds] : 0.f;
    const float skip = slive && a.D ? a.D[ds] : 0.f;

    f32x2 A[CS][P], G[CS][P], dA[CS][P];
#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = c0 + ch0 + q * S::CL;
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = dA[q][p] = pack2(0.f, 0.f);
        if (d < cend) load_row<R>(a.A + (long)d * N, j, N, A[q]);
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = mul2(A[q][p], pack2(kLog2e, kLog2e));
    }
    float sum_D = 0.f, sum_bias = 0.f;

    for (int s = unit; s < a.nseq; s += units) {
        long lo, hi;
        if (!seq_range(a, T, s, lo, hi)) {
            report_status(a.status_dev, kStatusDeviceInput);
            continue;
        }
        const long save0 = lo / KC + s;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
            const int d = c0 + ch0 + q * S::CL;
#pragma unroll
            for (int p = 0; p < P; ++p) G[q][p] = pack2(0.f, 0.f);
            if (b.dfinal && d < cend) load_row<R>(b.dfinal + ((long)s * a.dim + d) * N, j, N, G[q]);
        }

        for (long chunk = (hi - lo + KC - 1) / KC - 1; chunk >= 0; --chunk) {
            const long t0 = lo + chunk * KC;
            const int n_tok = (int)min((long)KC, hi - t0);
            // stage: step sizes, v x, gated dy; B, C; zero behind the sequence's end
            constexpr int kStep = 4;             // tokens whose loads are in flight together
            for (int k0 = st; k0 < KC; k0 += RS * kStep) {
                uint32_t rv[kStep], rx[kStep], rg[kStep], rz[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    const long t = t0 + k;
                    const bool ok = slive && k < n_tok;
                    rv[i] = ok ? raw_load<TDt>(a.dt, t * a.dt_stride + ds) : 0u;
                    rx[i] = ok ? raw_load<TIn>(a.x, t * a.x_stride + ds) : 0u;
                    rg[i] = ok ? raw_load<TIn>(b.dy, t * b.dy_stride + ds) : 0u;
                    rz[i] = ok && a.z ? raw_load<TIn>(a.z, t * a.z_stride + ds) : 0u;
                }
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    if (k >= KC) break;
                    const float v = slive && k < n_tok ? dt_value(a.dtp, raw_value<TDt>(rv[i]), bias) : 0.f;
                    float g = raw_value<TIn>(rg[i]);
                    if (a.z) g *= silu_approx(raw_value<TIn>(rz[i]));
                    s_v[k * CB + sc] = v;
                    s_u[k * CB + sc] = v * raw_value<TIn>(rx[i]);
                    s_g[k * CB + sc] = g;
                }
            }
#pragma unroll 4
            for (int e = tid; e < KC * NP; e += kBwdThreads) {
                const int k = e / NP, n = e % NP;
                const bool ok = k < n_tok && n < N;
                s_B[e] = ok ? ld_as<TIn>(a.B, (t0 + k) * a.B_stride + (long)grp * N + n) : 0.f;
                s_C[e] = ok ? ld_as<TIn>(a.C, (t0 + k) * a.C_stride + (long)grp * N + n) : 0.f;
            }
            f32x2 h[CS][P];
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = c0 + ch0 + q * S::CL;
#pragma unroll
                for (int p = 0; p < P; ++p) h[q][p] = pack2(0.f, 0.f);
                if (d < cend) load_row<R>(a.saved + ((save0 + chunk) * a.dim + d) * N, j, N, h[q]);
            }
            __syncthreads();

            const int last = (n_tok - 1) / kSub;
            // forward: the state in front of every sub-tile
            for (int sub = 0; sub <= last; ++sub) {
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    float *slot = s_h + ((sub * CS + q) * kBwdThreads + tid) * R;
#pragma unroll
                    for (int p = 0; p < P; ++p) reinterpret_cast<unsigned long long *>(slot)[p] = h[q][p].v;
                }
                if (sub == last) break;
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    const int t = sub * kSub + k;
                    f32x2 B[P];
                    lds_pairs(s_B + t * NP + j * R, B);
#pragma unroll
                    for (int q = 0; q < CS; ++q) {
                        const float v = s_v[t * CB + ch0 + q * S::CL], u = s_u[t * CB + ch0 + q * S::CL];
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            h[q][p] = fma2(ex2_pair(mul2(pack2(v, v), A[q][p])), h[q][p], mul2(pack2(u, u), B[p]));
                    }
                }
            }

            for (int sub = last; sub >= 0; --sub) {
                f32x2 dB[kSub][P], dC[kSub][P];
#pragma unroll
                for (int k = 0; k < kSub; ++k)
#pragma unroll
                    for (int p = 0; p < P; ++p) dB[k][p] = dC[k][p] = pack2(0.f, 0.f);
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    const int ch = ch0 + q * S::CL;
                    f32x2 hh[kSub + 1][P], aa[kSub][P];
                    lds_pairs(s_h + ((sub * CS + q) * kBwdThreads + tid) * R, hh[0]);
#pragma unroll
                    for (int k = 0; k < kSub; ++k) {
                        const int t = sub * kSub + k;
                        const float v = s_v[t * CB + ch], u = s_u[t * CB + ch];
                        f32x2 B[P];
                        lds_pairs(s_B + t * NP + j * R, B);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            aa[k][p] = ex2_pair(mul2(pack2(v, v), A[q][p]));
                            hh[k + 1][p] = fma2(aa[k][p], hh[k][p], mul2(pack2(u, u), B[p]));
                        }
                    }
                    float yv[kSub], wv[kSub], qv[kSub];
#pragma unroll
                    for (int k = kSub - 1; k >= 0; --k) {
                        const int t = sub * kSub + k;
                        const float v = s_v[t * CB + ch], u = s_u[t * CB + ch], g = s_g[t * CB + ch];
                        const f32x2 vv = pack2(v, v), uu = pack2(u, u), gg = pack2(g, g);
                        f32x2 B[P], C[P], ya = pack2(0.f, 0.f), wa = ya, qa = ya;
                        lds_pairs(s_B + t * NP + j * R, B);
                        lds_pairs(s_C + t * NP + j * R, C);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const f32x2 dh = fma2(gg, C[p], G[q][p]);
                            ya = fma2(hh[k + 1][p], C[p], ya);
                            dC[k][p] = fma2(hh[k + 1][p], gg, dC[k][p]);
                            dB[k][p] = fma2(dh, uu, dB[k][p]);
                            wa = fma2(dh, B[p], wa);
                            G[q][p] = mul2(aa[k][p], dh);
                            const f32x2 qq = mul2(G[q][p], hh[k][p]);
                            qa = fma2(qq, A[q][p], qa);
                            dA[q][p] = fma2(qq, vv, dA[q][p]);
                        }
                        yv[k] = sum2(ya);
                        wv[k] = sum2(wa);
                        qv[k] = sum2(qa);
                    }
                    const int first = reduce_lanes<kSub, L, 1>(yv, lane);
                    reduce_lanes<kSub, L, 1>(wv, lane);
                    reduce_lanes<kSub, L, 1>(qv, lane);
                    constexpr int kLeft = reduce_left(kSub, L), kSame = L > kSub ? L / kSub : 1;
                    __syncwarp();
                    // the channel's lanes have read v, u, g of these tokens: the sums take their place
                    if (j % kSame == 0) {
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) {
                            const int t = sub * kSub + first + i;
                            s_v[t * CB + ch] = qv[i];
                            s_u[t * CB + ch] = wv[i];
                            s_g[t * CB + ch] = yv[i];
                        }
                    }
                }
                // dB, dC of the sub-tile: over the warp's channels, then the CTA's warps
                float *part = s_part + (sub & 1) * (2 * kWarps * kSub * NP);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float f[kSub * R];
#pragma unroll
                    for (int k = 0; k < kSub; ++k)
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            f[k * R + 2 * p] = w ? lo2(dC[k][p]) : lo2(dB[k][p]);
                            f[k * R + 2 * p + 1] = w ? hi2(dC[k][p]) : hi2(dB[k][p]);
                        }
                    const int first = reduce_lanes<kSub * R, S::CL, L>(f, lane);
                    constexpr int kLeft = reduce_left(kSub * R, S::CL);
                    constexpr int kSame = S::CL > kSub * R ? S::CL / (kSub * R) : 1;
                    if ((lane / L) % kSame == 0) {
#pragma unroll
                        for (int i = 0; i < kLeft; ++i) {
                            const int k = (first + i) / R, r = (first + i) % R;
                            part[((w * kWarps + warp) * kSub + k) * NP + j * R + r] = f[i];
                        }
                    }
                }
                __syncthreads();
                for (int e = tid; e < 2 * kSub * NP; e += kBwdThreads) {
                    const int w = e / (kSub * NP), k = (e / NP) % kSub, n = e % NP;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) sum += part[((w * kWarps + i) * kSub + k) * NP + n];
                    const int t = sub * kSub + k;
                    if (t < n_tok && n < N)
                        (w ? b.part_C : b.part_B)[(((long)gtile * T + t0 + t) * a.ngroups + grp) * N + n] = sum;
                }
            }
            __syncthreads();
            // per (token, channel) outputs, from the sums over n and the inputs again
            for (int k0 = st; k0 < n_tok && slive; k0 += RS * kStep) {
                uint32_t rv[kStep], rx[kStep], rg[kStep], rz[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const long t = t0 + min(k0 + i * RS, n_tok - 1);
                    rv[i] = raw_load<TDt>(a.dt, t * a.dt_stride + ds);
                    rx[i] = raw_load<TIn>(a.x, t * a.x_stride + ds);
                    rg[i] = raw_load<TIn>(b.dy, t * b.dy_stride + ds);
                    rz[i] = a.z ? raw_load<TIn>(a.z, t * a.z_stride + ds) : 0u;
                }
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    if (k >= n_tok) break;
                    const long t = t0 + k;
                    const float raw = raw_value<TDt>(rv[i]), x = raw_value<TIn>(rx[i]);
                    const float v = dt_value(a.dtp, raw, bias), w = s_u[k * CB + sc];
                    float dy = raw_value<TIn>(rg[i]);
                    if (a.z) {
                        const float z = raw_value<TIn>(rz[i]);
                        const float sg = rcp_approx(1.f + ex2_approx(-z * kLog2e));
                        store_out(static_cast<TIn *>(b.dz) + t * a.dim + ds,
                                  dy * fmaf(skip, x, s_g[k * CB + sc]) * sg * fmaf(z, 1.f - sg, 1.f));
                        dy *= z * sg;
                    }
                    const float ddt = fmaf(s_v[k * CB + sc], kLn2, w * x) * dt_slope(a.dtp, raw, bias);
                    store_out(static_cast<TIn *>(b.dx) + t * a.dim + ds, fmaf(w, v, skip * dy));
                    store_out(static_cast<TDt *>(b.ddt) + t * a.dim + ds, ddt);
                    sum_D = fmaf(dy, x, sum_D);
                    sum_bias += ddt;
                }
            }
            __syncthreads();
        }
        if (b.dinitial) {
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = c0 + ch0 + q * S::CL;
                if (d < cend) store_row<R>(b.dinitial + ((long)s * a.dim + d) * N, j, N, G[q]);
            }
        }
    }

#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = c0 + ch0 + q * S::CL;
        if (d < cend) store_row<R>(b.part_A + ((long)unit * a.dim + d) * N, j, N, dA[q]);
    }
    s_v[tid] = sum_D;
    s_u[tid] = sum_bias;
    __syncthreads();
    if (st == 0 && slive) {
        for (int i = 1; i < RS; ++i) {
            sum_D += s_v[i * CB + sc];
            sum_bias += s_u[i * CB + sc];
        }
        b.part_D[(long)unit * a.dim + ds] = sum_D;
        b.part_bias[(long)unit * a.dim + ds] = sum_bias;
    }
}

// Sums of the parts: dB and dC over the channel tiles of a group, dA, dD and
// ddt_bias over the units.
__global__ void __launch_bounds__(256)
selective_scan_bwd_sum_kernel(SelScanBwdArgs b, int gtiles, int units, long nB, long nA)
{
    const SelScanArgs &a = b.f;
    long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < 2 * nB) {
        const bool c = i >= nB;
        if (c) i -= nB;
        const float *p = (c ? b.part_C : b.part_B) + i;
        float s = 0.f;
        for (int q = 0; q < gtiles; ++q) s += p[q * nB];
        st_act(c ? b.dC : b.dB, i, s, a.in_bf16);
        return;
    }
    i -= 2 * nB;
    const float *p;
    float *out;
    long n = a.dim;
    if (i < nA) {
        n = nA;
        p = b.part_A;
        out = b.dA;
    } else if (i < nA + a.dim) {
        i -= nA;
        p = b.part_D;
        out = b.dD;
    } else if (i < nA + 2L * a.dim) {
        i -= nA + a.dim;
        p = b.part_bias;
        out = b.ddt_bias;
    } else {
        return;
    }
    if (!out) return;
    float s = 0.f;
    for (int q = 0; q < units; ++q) s += p[q * n + i];
    out[i] = s;
}

struct BwdPlan {
    int cs, cb, units, gtiles;
    long tokens;
    size_t bytes_B, bytes_A, bytes_D;
};

template <typename TIn, typename TDt, int R, int L, int CS>
cudaError_t launch_shape(SelScanBwdArgs b, const BwdPlan &p, cudaStream_t stream)
{
    using S = BwdShape<R, L, CS>;
    const cudaError_t e = cudaFuncSetAttribute(selective_scan_bwd_kernel<TIn, TDt, R, L, CS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
    if (e) return e;
    const long long blocks = (long long)p.gtiles * b.f.ngroups * p.units;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    selective_scan_bwd_kernel<TIn, TDt, R, L, CS><<<(unsigned)blocks, kBwdThreads, S::kBytes, stream>>>(b, p.units);
    return cudaGetLastError();
}

// Lanes per channel for d_state (R = 4 states a lane, 8 above 128).
int lanes_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

BwdPlan make_plan(int nseq, long T, int dim, int d_state, int ngroups)
{
    BwdPlan p{};
    const int L = lanes_for(d_state);
    p.tokens = T;
    p.units = nseq < kMaxUnits ? nseq : kMaxUnits;
    p.cs = L == 1 || d_state > 128 ? 1 : 2;
    p.cb = 32 / L * p.cs * kWarps;
    p.gtiles = (dim / ngroups + p.cb - 1) / p.cb;
    auto up = [](size_t v) { return (v + 15) / 16 * 16; };
    p.bytes_B = up((size_t)p.gtiles * T * ngroups * d_state * sizeof(float));
    p.bytes_A = up((size_t)p.units * dim * d_state * sizeof(float));
    p.bytes_D = up((size_t)p.units * dim * sizeof(float));
    return p;
}

template <typename TIn, typename TDt>
cudaError_t launch_types(const SelScanBwdArgs &b, const BwdPlan &p, cudaStream_t stream)
{
    const int N = b.f.d_state;
    if (N <= 4) return launch_shape<TIn, TDt, 4, 1, 1>(b, p, stream);
    if (N <= 8) return launch_shape<TIn, TDt, 4, 2, 2>(b, p, stream);
    if (N <= 16) return launch_shape<TIn, TDt, 4, 4, 2>(b, p, stream);
    if (N <= 32) return launch_shape<TIn, TDt, 4, 8, 2>(b, p, stream);
    if (N <= 64) return launch_shape<TIn, TDt, 4, 16, 2>(b, p, stream);
    if (N <= 128) return launch_shape<TIn, TDt, 4, 32, 2>(b, p, stream);
    return launch_shape<TIn, TDt, 8, 32, 1>(b, p, stream);
}

}  // namespace

size_t selective_scan_bwd_workspace(int nseq, long T, int dim, int d_state, int ngroups)
{
    const BwdPlan p = make_plan(nseq, T, dim, d_state, ngroups);
    return 2 * p.bytes_B + p.bytes_A + 2 * p.bytes_D;
}

cudaError_t launch_selective_scan_bwd(SelScanBwdArgs b, void *workspace, cudaStream_t stream)
{
    const SelScanArgs &a = b.f;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const int N = a.d_state;
    const BwdPlan p = make_plan(a.nseq, T, a.dim, N, a.ngroups);
    char *w = static_cast<char *>(workspace);
    b.part_B = reinterpret_cast<float *>(w);
    b.part_C = reinterpret_cast<float *>(w + p.bytes_B);
    b.part_A = reinterpret_cast<float *>(w + 2 * p.bytes_B);
    b.part_D = reinterpret_cast<float *>(w + 2 * p.bytes_B + p.bytes_A);
    b.part_bias = reinterpret_cast<float *>(w + 2 * p.bytes_B + p.bytes_A + p.bytes_D);
    const cudaError_t e = !a.in_bf16 ? launch_types<float, float>(b, p, stream)
        : a.dt_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(b, p, stream)
                    : launch_types<__nv_bfloat16, float>(b, p, stream);
    if (e) return e;
    const long nB = T * a.ngroups * N, nA = (long)a.dim * N;
    const long long blocks = (2 * nB + nA + 2L * a.dim + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    selective_scan_bwd_sum_kernel<<<(unsigned)blocks, 256, 0, stream>>>(b, p.gtiles, p.units, nB, nA);
    return cudaGetLastError();
}

}  // namespace ssm
