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
// shuffles.  The sums over n (three per token and channel) go over the L lanes
// of a channel and end with the sub-tile's tokens spread over those lanes:
// each lane then finishes its tokens' dx, ddt and dz from the inputs, which it
// loaded when the sub-tile began.  Per sub-tile the CTA's warps are added up
// through shared memory and the sum is written as one part per channel tile; a
// second launch adds the parts, in a fixed order, so results do not depend on
// the schedule.
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
    // floats of shared memory: v and v x, gated dy; B, C; sub-tile states; parts of dB, dC (two buffers)
    static constexpr int kRow = kSavedEvery * CB;
    static constexpr int kStates = kSubs * CS * kBwdThreads * R;
    static constexpr int kParts = 2 * 2 * kWarps * kSub * NP;
    static constexpr size_t kBytes = sizeof(float) * (3 * kRow + 2 * kSavedEvery * NP + kStates + kParts);
    static_assert(CB % 2 == 0 && kBwdThreads % (CB / 2) == 0, "a staging thread keeps its two channels");
};

// First value that reduce_lanes<TG, S, kLow> leaves in this lane.
template <int TG, int S, int kLow>
__device__ __forceinline__ int reduced_first(int lane) {
    int first = 0, n = TG;
#pragma unroll
    for (int o = kLow * S / 2; o >= kLow; o >>= 1)
        if (n > 1) {
            n /= 2;
            if (lane & o) first += n;
        }
    return first;
}

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
__global__ void __launch_bounds__(kBwdThreads, R == 4 ? 3 : 1)
selective_scan_bwd_kernel(SelScanBwdArgs b, int units)
{
    using S = BwdShape<R, L, CS>;
    constexpr int CB = S::CB, CL = S::CL, NP = S::NP, P = R / 2, KC = kSavedEvery;
    constexpr int RS = kBwdThreads / (CB / 2);       // tokens per staging step (a thread: two channels)
    constexpr int kLeft = reduce_left(kSub, L);      // tokens of a sub-tile that a lane finishes
    constexpr int kSame = L > kSub ? L / kSub : 1;   // lanes that end with the same sums
    extern __shared__ __align__(16) float smem[];
    float2 *s_vu = reinterpret_cast<float2 *>(smem);
    float *s_g = smem + 2 * S::kRow, *s_B = s_g + S::kRow, *s_C = s_B + KC * NP;
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
    const int ch0 = warp * S::CW + lane / L;         // channel of set q: c0 + ch0 + q * CL
    const int first = reduced_first<kSub, L, 1>(lane);
    const int sc = 2 * (tid % (CB / 2)), st = tid / (CB / 2), ds = c0 + sc;   // staging: channels ds, ds + 1
    const bool slive0 = ds < cend, slive1 = ds + 1 < cend;
    const f32x2 bias2 = pack2(a.dtp.bias && slive0 ? a.dtp.bias[ds] : 0.f, a.dtp.bias && slive1 ? a.dtp.bias[ds + 1] : 0.f);
    const int xs = (int)a.x_stride, vs = (int)a.dt_stride, ys = (int)b.dy_stride, zs = (int)a.z_stride;
    const int Bs = (int)a.B_stride, Cs = (int)a.C_stride;
    const bool whole_rows = a.pairs && cend - c0 == CB && N == NP;

    f32x2 A[CS][P], G[CS][P], dA[CS][P];
    float sum_D[CS], sum_bias[CS];
#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = c0 + ch0 + q * CL;
        sum_D[q] = sum_bias[q] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = dA[q][p] = pack2(0.f, 0.f);
        if (d < cend) load_row<R>(a.A + (long)d * N, j, N, A[q]);
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = mul2(A[q][p], pack2(kLog2e, kLog2e));
    }

    for (int s = unit; s < a.nseq; s += units) {
        long lo, hi;
        if (!seq_range(a, T, s, lo, hi)) {
            report_status(a.status_dev, kStatusDeviceInput);
            continue;
        }
        const long save0 = lo / KC + s;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
            const int d = c0 + ch0 + q * CL;
#pragma unroll
            for (int p = 0; p < P; ++p) G[q][p] = pack2(0.f, 0.f);
            if (b.dfinal && d < cend) load_row<R>(b.dfinal + ((long)s * a.dim + d) * N, j, N, G[q]);
        }

        for (long chunk = (hi - lo + KC - 1) / KC - 1; chunk >= 0; --chunk) {
            const long t0 = lo + chunk * KC;
            const int n_tok = (int)min((long)KC, hi - t0);
            // rows of the chunk's first token; everything below is a 32-bit offset from them
            const TIn *xt = static_cast<const TIn *>(a.x) + t0 * xs + c0, *yt = static_cast<const TIn *>(b.dy) + t0 * ys + c0;
            const TIn *zt = static_cast<const TIn *>(a.z) + t0 * zs + c0;
            const TDt *vt = static_cast<const TDt *>(a.dt) + t0 * vs + c0;
            const TIn *Bt = static_cast<const TIn *>(a.B) + t0 * Bs + grp * N, *Ct = static_cast<const TIn *>(a.C) + t0 * Cs + grp * N;
            const bool full = whole_rows && n_tok == KC;

            f32x2 h[CS][P];
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = c0 + ch0 + q * CL;
#pragma unroll
                for (int p = 0; p < P; ++p) h[q][p] = pack2(0.f, 0.f);
                if (d < cend) load_row<R>(a.saved + ((save0 + chunk) * a.dim + d) * N, j, N, h[q]);
            }
            // stage: step sizes, v x, gated dy; B, C; zero behind the sequence's end
            constexpr int kStep = KC / RS < 4 ? (KC / RS < 1 ? 1 : KC / RS) : 4;   // tokens whose loads are in flight together
#pragma unroll 1
            for (int k0 = st; k0 < KC; k0 += RS * kStep) {
                uint32_t rv[kStep][2], rx[kStep][2], rg[kStep][2], rz[kStep][2];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    if (full) {
                        pair_load(vt, k * vs + sc, rv[i]);
                        pair_load(xt, k * xs + sc, rx[i]);
                        pair_load(yt, k * ys + sc, rg[i]);
                        if (a.z) pair_load(zt, k * zs + sc, rz[i]);
                    } else {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const bool ok = k < n_tok && (w ? slive1 : slive0);
                            rv[i][w] = ok ? raw_load<TDt>(vt, k * vs + sc + w) : 0u;
                            rx[i][w] = ok ? raw_load<TIn>(xt, k * xs + sc + w) : 0u;
                            rg[i][w] = ok ? raw_load<TIn>(yt, k * ys + sc + w) : 0u;
                            rz[i][w] = ok && a.z ? raw_load<TIn>(zt, k * zs + sc + w) : 0u;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    f32x2 v = dt_value2(a.dtp, pair_value<TDt>(rv[i]), bias2);
                    if (k >= n_tok) v = pack2(0.f, 0.f);
                    const f32x2 u = mul2(v, pair_value<TIn>(rx[i]));
                    f32x2 g = pair_value<TIn>(rg[i]);
                    if (a.z) g = mul2(g, silu2(pair_value<TIn>(rz[i])));
                    if (KC % (RS * kStep) && k >= KC) break;
                    *reinterpret_cast<float4 *>(&s_vu[k * CB + sc]) = make_float4(lo2(v), lo2(u), hi2(v), hi2(u));
                    *reinterpret_cast<float2 *>(&s_g[k * CB + sc]) = make_float2(lo2(g), hi2(g));
                }
            }
#pragma unroll 4
            for (int e = tid; e < KC * NP; e += kBwdThreads) {
                const int k = e / NP, n = e % NP;
                const bool ok = k < n_tok && n < N;
                s_B[e] = ok ? ld_as<TIn>(Bt, k * Bs + n) : 0.f;
                s_C[e] = ok ? ld_as<TIn>(Ct, k * Cs + n) : 0.f;
            }
            __syncthreads();

            const int last = (n_tok - 1) / kSub;
            // forward: the state in front of every sub-tile
#pragma unroll 1
            for (int sub = 0; sub <= last; ++sub) {
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    float *slot = s_h + ((sub * CS + q) * kBwdThreads + tid) * R;
#pragma unroll
                    for (int p = 0; p < P; p += 2)
                        *reinterpret_cast<ulonglong2 *>(slot + 2 * p) = make_ulonglong2(h[q][p].v, h[q][p + 1].v);
                }
                if (sub == last) break;
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    const int t = sub * kSub + k;
                    f32x2 B[P];
                    lds_pairs(s_B + t * NP + j * R, B);
#pragma unroll
                    for (int q = 0; q < CS; ++q) {
                        const float2 vu = s_vu[t * CB + ch0 + q * CL];
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            h[q][p] = fma2(ex2_pair(mul2(pack2(vu.x, vu.x), A[q][p])), h[q][p], mul2(pack2(vu.y, vu.y), B[p]));
                    }
                }
            }

#pragma unroll 1
            for (int sub = last; sub >= 0; --sub) {
                f32x2 dB[kSub][P], dC[kSub][P], B[kSub][P], C[kSub][P];
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    lds_pairs(s_B + (sub * kSub + k) * NP + j * R, B[k]);
                    lds_pairs(s_C + (sub * kSub + k) * NP + j * R, C[k]);
                }
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    const int ch = ch0 + q * CL, d = c0 + ch;
                    // inputs of the tokens that this lane finishes
                    uint32_t rv[kLeft], rx[kLeft], rg[kLeft], rz[kLeft];
                    bool mine[kLeft];
#pragma unroll
                    for (int i = 0; i < kLeft; ++i) {
                        const int t = sub * kSub + first + i;
                        mine[i] = t < n_tok && d < cend && j % kSame == 0;
                        rv[i] = rx[i] = rg[i] = rz[i] = 0u;
                        if (mine[i]) {
                            rv[i] = raw_load<TDt>(vt, t * vs + ch);
                            rx[i] = raw_load<TIn>(xt, t * xs + ch);
                            if (a.z) {
                                rg[i] = raw_load<TIn>(yt, t * ys + ch);
                                rz[i] = raw_load<TIn>(zt, t * zs + ch);
                            }
                        }
                    }
                    f32x2 hh[kSub + 1][P], aa[kSub][P];
                    lds_pairs(s_h + ((sub * CS + q) * kBwdThreads + tid) * R, hh[0]);
                    float2 vu[kSub];
#pragma unroll
                    for (int k = 0; k < kSub; ++k) {
                        vu[k] = s_vu[(sub * kSub + k) * CB + ch];
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            aa[k][p] = ex2_pair(mul2(pack2(vu[k].x, vu[k].x), A[q][p]));
                            hh[k + 1][p] = fma2(aa[k][p], hh[k][p], mul2(pack2(vu[k].y, vu[k].y), B[k][p]));
                        }
                    }
                    float yv[kSub], wv[kSub], qv[kSub];
#pragma unroll
                    for (int k = kSub - 1; k >= 0; --k) {
                        const float g = s_g[(sub * kSub + k) * CB + ch];
                        const f32x2 vv = pack2(vu[k].x, vu[k].x), uu = pack2(vu[k].y, vu[k].y), gg = pack2(g, g);
                        f32x2 ya, wa, qa;
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const f32x2 dh = fma2(gg, C[k][p], G[q][p]);
                            G[q][p] = mul2(aa[k][p], dh);
                            const f32x2 qq = mul2(G[q][p], hh[k][p]);
                            dA[q][p] = fma2(qq, vv, dA[q][p]);
                            ya = p ? fma2(hh[k + 1][p], C[k][p], ya) : mul2(hh[k + 1][p], C[k][p]);
                            wa = p ? fma2(dh, B[k][p], wa) : mul2(dh, B[k][p]);
                            qa = p ? fma2(qq, A[q][p], qa) : mul2(qq, A[q][p]);
                            dC[k][p] = q ? fma2(hh[k + 1][p], gg, dC[k][p]) : mul2(hh[k + 1][p], gg);
                            dB[k][p] = q ? fma2(dh, uu, dB[k][p]) : mul2(dh, uu);
                        }
                        yv[k] = sum2(ya);
                        wv[k] = sum2(wa);
                        qv[k] = sum2(qa);
                    }
                    reduce_lanes<kSub, L, 1>(yv, lane);
                    reduce_lanes<kSub, L, 1>(wv, lane);
                    reduce_lanes<kSub, L, 1>(qv, lane);
                    const float bias = a.dtp.bias && d < cend ? __ldg(a.dtp.bias + d) : 0.f;
                    const float skip = a.D && d < cend ? __ldg(a.D + d) : 0.f;
#pragma unroll
                    for (int i = 0; i < kLeft; ++i) {
                        if (!mine[i]) continue;
                        const int t = sub * kSub + first + i;
                        const long o = t0 * a.dim + c0;
                        const int oo = t * a.dim + ch;
                        const float x = raw_value<TIn>(rx[i]), v = s_vu[t * CB + ch].x, g = s_g[t * CB + ch];
                        if (a.z) {
                            const float z = raw_value<TIn>(rz[i]);
                            const float sg = rcp_approx(1.f + ex2_approx(-z * kLog2e));
                            store_out(static_cast<TIn *>(b.dz) + o + oo,
                                      raw_value<TIn>(rg[i]) * fmaf(skip, x, yv[i]) * sg * fmaf(z, 1.f - sg, 1.f));
                        }
                        const float ddt = fmaf(qv[i], kLn2, wv[i] * x) * dt_slope(a.dtp, raw_value<TDt>(rv[i]), bias);
                        store_out(static_cast<TIn *>(b.dx) + o + oo, fmaf(wv[i], v, skip * g));
                        store_out(static_cast<TDt *>(b.ddt) + o + oo, ddt);
                        sum_D[q] = fmaf(g, x, sum_D[q]);
                        sum_bias[q] += ddt;
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
                    const int f0 = reduce_lanes<kSub * R, CL, L>(f, lane);
                    constexpr int kVals = reduce_left(kSub * R, CL);
                    constexpr int kCopies = CL > kSub * R ? CL / (kSub * R) : 1;
                    if ((lane / L) % kCopies == 0) {
#pragma unroll
                        for (int i = 0; i < kVals; ++i) {
                            const int k = (f0 + i) / R, r = (f0 + i) % R;
                            part[((w * kWarps + warp) * kSub + k) * NP + j * R + r] = f[i];
                        }
                    }
                }
                __syncthreads();
                float *oB = b.part_B + (((long)gtile * T + t0 + sub * kSub) * a.ngroups + grp) * N;
                float *oC = b.part_C + (((long)gtile * T + t0 + sub * kSub) * a.ngroups + grp) * N;
                for (int e = tid; e < 2 * kSub * NP; e += kBwdThreads) {
                    const int w = e / (kSub * NP), k = (e / NP) % kSub, n = e % NP;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) sum += part[((w * kWarps + i) * kSub + k) * NP + n];
                    if (sub * kSub + k < n_tok && n < N) (w ? oC : oB)[k * a.ngroups * N + n] = sum;
                }
            }
            // the last sub-tile's barrier lies behind every read of the staged chunk: the next may be staged
        }
        if (b.dinitial) {
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = c0 + ch0 + q * CL;
                if (d < cend) store_row<R>(b.dinitial + ((long)s * a.dim + d) * N, j, N, G[q]);
            }
        }
    }

#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = c0 + ch0 + q * CL;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            sum_D[q] += __shfl_xor_sync(0xffffffffu, sum_D[q], o);
            sum_bias[q] += __shfl_xor_sync(0xffffffffu, sum_bias[q], o);
        }
        if (d >= cend) continue;
        store_row<R>(b.part_A + ((long)unit * a.dim + d) * N, j, N, dA[q]);
        if (j == 0) {
            b.part_D[(long)unit * a.dim + d] = sum_D[q];
            b.part_bias[(long)unit * a.dim + d] = sum_bias[q];
        }
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
