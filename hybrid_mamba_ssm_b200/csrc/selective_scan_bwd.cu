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
//
// The parts of dB and dC are one copy of both per channel tile, written and read
// again; a tile is 4 to 128 channels, the fewer the more states, so above 32
// states they are what the workspace holds and most of the HBM traffic (8192
// tokens of 8192 channels: 0.14 GiB at 16 states, 2.0 at 64, 8.0 at 128).
//
// What bounds it (ncu, 16 x 128 tokens of 8192 channels, 16 states, bf16): no
// one unit.  29 instructions an element (element: one (token, channel, n)) leave
// issue slots at 53 %, the shared-memory pipe at 52 %, the special-function unit
// at 35 % (two exponentials an element and six a (token, channel)), HBM at 8 %;
// 168 registers and 75 KB a CTA allow 12 warps an SM, whose latencies are not
// all hidden.  16 x 512 tokens take 1.60 ms, 4 x 2048 2.0 ms (2.11 as whole
// sequences, for a second round of CTAs), 1 x 4096 of 2048 channels with 128 states 2.50 ms.
// Steps that paid: lanes finishing their own tokens instead of a second pass
// over the chunk (2.9 -> 2.4 ms at 4 x 2048 with the next one), the sums over
// channels by 16-byte accesses to shared memory instead of shuffles (36 -> 31
// instructions an element), bf16 pairs in one register (1.79 -> 1.60 ms at 16 x
// 512).  Interleaving the two sets of channels by hand was slower (1.99 ms).
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kSub = 4;                          // tokens of a sub-tile
constexpr int kSubs = kSavedEvery / kSub;        // sub-tiles of a chunk
constexpr int kWarps = 4;
constexpr int kBwdThreads = 32 * kWarps;
constexpr int kMaxCtas = 64;                     // whole sequences are dealt to at most this many CTAs per tile

template <int R, int L, int CS>
struct BwdShape {
    static constexpr int CL = 32 / L;            // channels of a warp at a time
    static constexpr int CW = CL * CS;           // channels of a warp
    static constexpr int CB = CW * kWarps;       // channels of a CTA
    static constexpr int NP = R * L;
    // floats of shared memory: v and v x, gated dy; B, C; states in front of all
    // sub-tiles but the last (which is still in registers); every thread's dB, dC
    // of a sub-tile, 4 floats apart more so that eight 16-byte accesses of a warp
    // fall into different banks
    static constexpr int kRow = kSavedEvery * CB;
    static constexpr int kStates = (kSubs - 1) * CS * kBwdThreads * R;
    static constexpr int kVals = 2 * kSub * R, kPitch = kVals + 4;
    static constexpr size_t kStaged = sizeof(float) * (3 * kRow + 2 * kSavedEvery * NP);
    static constexpr size_t kBytes = kStaged + sizeof(float) * (kStates + kBwdThreads * kPitch);
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

// CTAs of an SM: 168 registers a thread with two sets of channels, 128 with one.
// For 9 to 64 states shared memory (kBytes) has room for as many; for fewer and
// for 65 to 128 it has room for one or two less, so the registers are bounded
// more tightly there than they need to be.
template <int R, int CS>
constexpr int kCtasPerSm = R > 4 ? 1 : CS == 2 ? 3 : 4;

// One CTA per (unit, channel tile); with more units than CTAs per tile, a CTA
// takes every `ctas`-th.  kCarry: the pass before, where sequences are cut
// into segments.  It leaves the gradient of the state in front of a segment as
// the segment's own tokens give it (the last one of a sequence: from the final
// state's gradient), and the sum of its step sizes; the main pass folds the
// segments behind its own.
template <typename TIn, typename TDt, int R, int L, int CS, bool kCarry, bool kPacked>
__global__ void __launch_bounds__(kBwdThreads, kCtasPerSm<R, CS>)
selective_scan_bwd_kernel(SelScanBwdArgs b, int ctas)
{
    using S = BwdShape<R, L, CS>;
    constexpr int CB = S::CB, CL = S::CL, NP = S::NP, P = R / 2, KC = kSavedEvery;
    constexpr int RS = kBwdThreads / (CB / 2);       // tokens per staging step (a thread: two channels)
    constexpr int kLeft = reduce_left(kSub, L);      // tokens of a sub-tile that a lane finishes
    constexpr int kSame = L > kSub ? L / kSub : 1;   // lanes that end with the same sums
    extern __shared__ __align__(16) float smem[];
    float2 *s_vu = reinterpret_cast<float2 *>(smem);
    float *s_g = smem + 2 * S::kRow, *s_B = s_g + S::kRow, *s_C = s_B + KC * NP;
    float *s_h = s_C + KC * NP, *s_red = s_h + S::kStates;
    const SelScanArgs &a = b.f;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CB - 1) / CB, tiles = gtiles * a.ngroups;
    const int unit = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x - (unsigned)unit * tiles);
    const int grp = tile / gtiles, gtile = tile - grp * gtiles;
    const int c0 = grp * gdim + gtile * CB, cend = min(c0 + CB, (grp + 1) * gdim);
    const int N = a.d_state;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;

    const int j = lane % L;
    const int ch0 = warp * S::CW + CS * (lane / L);  // channel of set q: c0 + ch0 + q
    const int dc = c0 + ch0;
    const int first = reduced_first<kSub, L, 1>(lane);
    const int sc = 2 * (tid % (CB / 2)), st = tid / (CB / 2), ds = c0 + sc;   // staging: channels ds, ds + 1
    const bool slive0 = ds < cend, slive1 = ds + 1 < cend;
    const f32x2 bias2 = pack2(a.dtp.bias && slive0 ? a.dtp.bias[ds] : 0.f, a.dtp.bias && slive1 ? a.dtp.bias[ds + 1] : 0.f);
    const int xs = (int)a.x_stride, vs = (int)a.dt_stride, ys = (int)b.dy_stride, zs = (int)a.z_stride;
    const int Bs = (int)a.B_stride, Cs = (int)a.C_stride;
    // this lane's own two channels as one access (loads, and stores into rows of dim values)
    const bool pair_in = CS == 2 && kPacked && dc + 1 < cend, pair_out = CS == 2 && gdim % 2 == 0 && dc + 1 < cend;
    const f32x2 own_bias = pack2(a.dtp.bias && dc < cend ? a.dtp.bias[dc] : 0.f, a.dtp.bias && CS == 2 && dc + 1 < cend ? a.dtp.bias[dc + 1] : 0.f);
    const f32x2 own_skip = pack2(a.D && dc < cend ? a.D[dc] : 0.f, a.D && CS == 2 && dc + 1 < cend ? a.D[dc + 1] : 0.f);
    const bool whole_rows = kPacked && cend - c0 == CB && N == NP;

    f32x2 A[CS][P], G[CS][P], dA[CS][P];
    f32x2 sum_D = pack2(0.f, 0.f), sum_bias = sum_D;  // of this lane's channel(s)
#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = dc + q;
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = dA[q][p] = pack2(0.f, 0.f);
        if (d < cend) load_row<R>(a.A + (long)d * N, j, N, A[q]);
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = decay_rate2(A[q][p]);
    }

    __shared__ int s_seq;
    if (kCarry) check_offsets(a, T);
    const bool ranked = !a.span && a.cu_seqlens && a.nseq > 1 && a.nseq <= kMaxRanked && ctas == a.nseq;
    for (int u = unit; u < a.units; u += ctas) {
        Unit w;
        if (!find_unit(a, T, ranked ? longest_first(a, u, &s_seq) : u, w)) continue;
        if (kCarry && w.k == 0) continue;
        const int s = w.s;
        const long lo = w.lo, hi = w.hi, save0 = lo / KC + s;
#pragma unroll
        for (int q = 0; q < CS; ++q) {
            const int d = dc + q;
#pragma unroll
            for (int p = 0; p < P; ++p) G[q][p] = pack2(0.f, 0.f);
            if (w.e == hi && b.dfinal && d < cend) load_row<R>(b.dfinal + ((long)s * a.dim + d) * N, j, N, G[q]);
        }
        if (!kCarry && w.e < hi) {               // the gradient that enters from the segments behind
#pragma unroll 4
            for (int m = (int)((hi - lo - 1) / a.span); m > w.k; --m) {
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    const int d = dc + q;
                    if (d >= cend) continue;
                    f32x2 own[P];
                    load_row<R>(a.range_state + ((w.base + m) * a.dim + d) * N, j, N, own);
                    const float v = a.range_dt[(w.base + m) * a.dim + d];
#pragma unroll
                    for (int p = 0; p < P; ++p) G[q][p] = fma2(decay2(pack2(v, v), A[q][p]), G[q][p], own[p]);
                }
            }
        }
        float vsum[CS];
#pragma unroll
        for (int q = 0; q < CS; ++q) vsum[q] = 0.f;

        const long chunk0 = (w.b - lo) / KC;
        for (long chunk = (w.e - lo + KC - 1) / KC - 1; chunk >= chunk0; --chunk) {
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
                const int d = dc + q;
#pragma unroll
                for (int p = 0; p < P; ++p) h[q][p] = pack2(0.f, 0.f);
                if (!kCarry && d < cend) load_row<R>(a.saved + ((save0 + chunk) * a.dim + d) * N, j, N, h[q]);
            }
            // stage: step sizes, v x, gated dy; B, C; zero behind the sequence's end
            constexpr int kStep = KC / RS < 4 ? (KC / RS < 1 ? 1 : KC / RS) : 4;   // tokens whose loads are in flight together
#pragma unroll 1
            for (int k0 = st; k0 < KC; k0 += RS * kStep) {
                RawPair<TDt, kPacked> rv[kStep];
                RawPair<TIn, kPacked> rx[kStep], rg[kStep], rz[kStep];
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    if (full) {
                        if constexpr (kPacked) {
                            rv[i].load(vt, k * vs + sc);
                            rx[i].load(xt, k * xs + sc);
                            rg[i].load(yt, k * ys + sc);
                            if (a.z) rz[i].load(zt, k * zs + sc);
                        }
                    } else {
                        const bool ok0 = slive0 && k < n_tok, ok1 = slive1 && ok0;
                        rv[i].load(vt, k * vs + sc, ok0, ok1);
                        rx[i].load(xt, k * xs + sc, ok0, ok1);
                        rg[i].load(yt, k * ys + sc, ok0, ok1);
                        rz[i].load(zt, k * zs + sc, ok0 && a.z, ok1 && a.z);
                    }
                }
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int k = k0 + i * RS;
                    f32x2 v = dt_value2(a.dtp, rv[i].value(), bias2);
                    if (k >= n_tok) v = pack2(0.f, 0.f);
                    const f32x2 u = mul2(v, rx[i].value());
                    f32x2 g = rg[i].value();
                    if (a.z) g = mul2(g, silu2(rz[i].value()));
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
            // the chunk that comes next, into L2: its rows of x, dt, dy and z (a line each), and its saved state
            if (chunk > chunk0) {
                constexpr int kLine = 128;
                const char *px = reinterpret_cast<const char *>(xt - (long)KC * xs), *pv = reinterpret_cast<const char *>(vt - (long)KC * vs);
                const char *py = reinterpret_cast<const char *>(yt - (long)KC * ys), *pz = reinterpret_cast<const char *>(zt - (long)KC * zs);
                const int row = tid % KC, which = tid / KC;     // kBwdThreads = 4 KC
                const char *p = which == 0 ? px + (long)row * xs * (int)sizeof(TIn) : which == 1 ? pv + (long)row * vs * (int)sizeof(TDt)
                              : which == 2 ? py + (long)row * ys * (int)sizeof(TIn) : pz + (long)row * zs * (int)sizeof(TIn);
                if (which < 3 || a.z) prefetch_l2(p);
                const char *ps = reinterpret_cast<const char *>(a.saved + ((save0 + chunk - 1) * a.dim + c0) * N);
                if ((long)tid * kLine < (long)(cend - c0) * N * (long)sizeof(float)) prefetch_l2(ps + tid * kLine);
            }
            __syncthreads();

            const int last = (n_tok - 1) / kSub;
            // step sizes v and v x of token t for this lane's channels
            auto load_vu = [&](int t, float (&v)[CS], float (&u)[CS]) {
                if constexpr (CS == 2) {
                    const float4 q = *reinterpret_cast<const float4 *>(&s_vu[t * CB + ch0]);
                    v[0] = q.x; u[0] = q.y; v[1] = q.z; u[1] = q.w;
                } else {
                    const float2 q = s_vu[t * CB + ch0];
                    v[0] = q.x; u[0] = q.y;
                }
            };
            auto load_g = [&](int t, float (&g)[CS]) {
                if constexpr (CS == 2) {
                    const float2 q = *reinterpret_cast<const float2 *>(&s_g[t * CB + ch0]);
                    g[0] = q.x; g[1] = q.y;
                } else {
                    g[0] = s_g[t * CB + ch0];
                }
            };
            if constexpr (kCarry) {
#pragma unroll 4
                for (int t = n_tok - 1; t >= 0; --t) {
                    f32x2 C[P];
                    float v[CS], u[CS], g[CS];
                    lds_pairs(s_C + t * NP + j * R, C);
                    load_vu(t, v, u);
                    load_g(t, g);
#pragma unroll
                    for (int q = 0; q < CS; ++q) {
                        vsum[q] += v[q];
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            G[q][p] = mul2(decay2(pack2(v[q], v[q]), A[q][p]), fma2(pack2(g[q], g[q]), C[p], G[q][p]));
                    }
                }
                __syncthreads();
                continue;
            }
            // forward: the state in front of every sub-tile
#pragma unroll 1
            for (int sub = 0; sub < last; ++sub) {
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    float *slot = s_h + ((sub * CS + q) * kBwdThreads + tid) * R;
#pragma unroll
                    for (int p = 0; p < P; p += 2)
                        *reinterpret_cast<ulonglong2 *>(slot + 2 * p) = make_ulonglong2(h[q][p].v, h[q][p + 1].v);
                }
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    const int t = sub * kSub + k;
                    f32x2 B[P];
                    float v[CS], u[CS];
                    lds_pairs(s_B + t * NP + j * R, B);
                    load_vu(t, v, u);
#pragma unroll
                    for (int q = 0; q < CS; ++q)
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            h[q][p] = fma2(decay2(pack2(v[q], v[q]), A[q][p]), h[q][p], mul2(pack2(u[q], u[q]), B[p]));
                }
            }

#pragma unroll 1
            for (int sub = last; sub >= 0; --sub) {
                // inputs of the tokens that this lane finishes
                RawPair<TDt, kPacked> rv[kLeft];
                RawPair<TIn, kPacked> rx[kLeft], rg[kLeft], rz[kLeft];
                bool mine[kLeft];
#pragma unroll
                for (int i = 0; i < kLeft; ++i) {
                    const int t = sub * kSub + first + i;
                    mine[i] = t < n_tok && dc < cend && j % kSame == 0;
                    rv[i].zero();
                    rx[i].zero();
                    rg[i].zero();
                    rz[i].zero();
                    if (!mine[i]) continue;
                    if (pair_in) {
                        if constexpr (kPacked) {
                            rv[i].load(vt, t * vs + ch0);
                            rx[i].load(xt, t * xs + ch0);
                            if (a.z) {
                                rg[i].load(yt, t * ys + ch0);
                                rz[i].load(zt, t * zs + ch0);
                            }
                        }
                    } else {
                        const bool two = CS == 2 && dc + 1 < cend;
                        rv[i].load(vt, t * vs + ch0, true, two);
                        rx[i].load(xt, t * xs + ch0, true, two);
                        if (a.z) {
                            rg[i].load(yt, t * ys + ch0, true, two);
                            rz[i].load(zt, t * zs + ch0, true, two);
                        }
                    }
                }
                f32x2 dB[kSub][P], dC[kSub][P], B[kSub][P], C[kSub][P];
                float v[kSub][CS], u[kSub][CS], g[kSub][CS];
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
                    lds_pairs(s_B + (sub * kSub + k) * NP + j * R, B[k]);
                    lds_pairs(s_C + (sub * kSub + k) * NP + j * R, C[k]);
                    load_vu(sub * kSub + k, v[k], u[k]);
                    load_g(sub * kSub + k, g[k]);
                }
                float ys_[CS][kSub], ws_[CS][kSub], qs_[CS][kSub];
#pragma unroll
                for (int q = 0; q < CS; ++q) {
                    f32x2 hh[kSub + 1][P], aa[kSub][P];
                    if (sub == last) {
#pragma unroll
                        for (int p = 0; p < P; ++p) hh[0][p] = h[q][p];
                    } else {
                        lds_pairs(s_h + ((sub * CS + q) * kBwdThreads + tid) * R, hh[0]);
                    }
#pragma unroll
                    for (int k = 0; k < kSub; ++k)
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            aa[k][p] = decay2(pack2(v[k][q], v[k][q]), A[q][p]);
                            hh[k + 1][p] = fma2(aa[k][p], hh[k][p], mul2(pack2(u[k][q], u[k][q]), B[k][p]));
                        }
#pragma unroll
                    for (int k = kSub - 1; k >= 0; --k) {
                        const f32x2 vv = pack2(v[k][q], v[k][q]), uu = pack2(u[k][q], u[k][q]), gg = pack2(g[k][q], g[k][q]);
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
                        ys_[q][k] = sum2(ya);
                        ws_[q][k] = sum2(wa);
                        qs_[q][k] = sum2(qa);
                    }
                    reduce_lanes<kSub, L, 1>(ys_[q], lane);
                    reduce_lanes<kSub, L, 1>(ws_[q], lane);
                    reduce_lanes<kSub, L, 1>(qs_[q], lane);
                }
#pragma unroll
                for (int i = 0; i < kLeft; ++i) {
                    if (!mine[i]) continue;
                    constexpr int q1 = CS - 1;                 // CS == 1: the second half repeats the first and is not stored
                    const int t = sub * kSub + first + i;
                    float tv[CS], tu[CS], tg[CS];
                    load_vu(t, tv, tu);
                    load_g(t, tg);
                    const f32x2 x = rx[i].value(), vv = pack2(tv[0], tv[q1]), gg = pack2(tg[0], tg[q1]);
                    const f32x2 w = pack2(ws_[0][i], ws_[q1][i]), y = pack2(ys_[0][i], ys_[q1][i]), qq = pack2(qs_[0][i], qs_[q1][i]);
                    const long o = (t0 + t) * a.dim + dc;
                    const f32x2 dx = fma2(w, vv, mul2(own_skip, gg));
                    const f32x2 ddt = mul2(fma2(qq, pack2(kLn2, kLn2), mul2(w, x)), dt_slope2(a.dtp, rv[i].value(), own_bias));
                    store_pair(static_cast<TIn *>(b.dx) + o, dx, pair_out, CS == 2 && dc + 1 < cend);
                    store_pair(static_cast<TDt *>(b.ddt) + o, ddt, pair_out, CS == 2 && dc + 1 < cend);
                    if (a.z) {
                        const f32x2 z = rz[i].value(), one = pack2(1.f, 1.f);
                        const f32x2 e = add2(ex2_pair(mul2(z, pack2(-kLog2e, -kLog2e))), one);
                        const f32x2 sg = pack2(rcp_approx(lo2(e)), rcp_approx(hi2(e)));
                        const f32x2 slope = mul2(sg, fma2(z, fma2(sg, pack2(-1.f, -1.f), one), one));
                        store_pair(static_cast<TIn *>(b.dz) + o, mul2(mul2(rg[i].value(), fma2(own_skip, x, y)), slope),
                                   pair_out, CS == 2 && dc + 1 < cend);
                    }
                    sum_D = fma2(gg, x, sum_D);
                    sum_bias = add2(sum_bias, ddt);
                }
                // dB, dC of the sub-tile, summed over the CTA's channels: every thread leaves its own, and
                // thread (warp k, lane: state group j, which of dB and dC, part) adds those of token k from
                // the threads of its part; the parts are added by shuffles
                if (sub != last) __syncthreads();              // the sums of the sub-tile before have been read
                float *mine_red = s_red + tid * S::kPitch;
#pragma unroll
                for (int k = 0; k < kSub; ++k)
#pragma unroll
                    for (int p = 0; p < P; p += 2) {
                        *reinterpret_cast<ulonglong2 *>(mine_red + k * R + 2 * p) = make_ulonglong2(dB[k][p].v, dB[k][p + 1].v);
                        *reinterpret_cast<ulonglong2 *>(mine_red + (kSub + k) * R + 2 * p) = make_ulonglong2(dC[k][p].v, dC[k][p + 1].v);
                    }
                __syncthreads();
                constexpr int kPartsN = L < 16 ? 16 / L : 1, kFrom = kBwdThreads / L / kPartsN;
                static_assert(kWarps == kSub, "a warp adds one token of the sub-tile");
#pragma unroll
                for (int it = 0; it < (L == 32 ? 2 : 1) * (R / 4); ++it) {
                    const int combo = L == 32 ? lane + 32 * (it % 2) : lane % (2 * L), r4 = 4 * (L == 32 ? it / 2 : it);
                    const int cj = combo % L, w = combo / L, part = L == 32 ? 0 : lane / (2 * L);
                    f32x2 s01 = pack2(0.f, 0.f), s23 = s01;
#pragma unroll
                    for (int i = 0; i < kFrom; ++i) {
                        const int m = part * kFrom + i, from = m / CL * 32 + m % CL * L + cj;
                        f32x2 f[2];
                        lds_pairs(s_red + from * S::kPitch + (w * kSub + warp) * R + r4, f);
                        s01 = add2(s01, f[0]);
                        s23 = add2(s23, f[1]);
                    }
                    float f[4] = {lo2(s01), hi2(s01), lo2(s23), hi2(s23)};
                    const int f0 = reduce_lanes<4, kPartsN, (L < 16 ? 2 * L : 32)>(f, lane);
                    constexpr int kOut = reduce_left(4, kPartsN), kDup = kPartsN > 4 ? kPartsN / 4 : 1;
                    const int t = sub * kSub + warp;
                    if (t >= n_tok || part % kDup) continue;
                    float *out = (w ? b.part_C : b.part_B) + (((long)gtile * T + t0 + t) * a.ngroups + grp) * N + cj * R + r4 + f0;
#pragma unroll
                    for (int i = 0; i < kOut; ++i)
                        if (cj * R + r4 + f0 + i < N) out[i] = f[i];
                }
            }
            // the last sub-tile's second barrier lies behind every read of the staged chunk, so the next may be
            // staged; its sums are read before the barrier that follows the staging
        }
        if (kCarry) {
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = dc + q;
                if (d >= cend) continue;
                store_row<R>(a.range_state + ((long)u * a.dim + d) * N, j, N, G[q]);
                if (j == 0) a.range_dt[(long)u * a.dim + d] = vsum[q];
            }
        } else if (b.dinitial && w.k == 0) {
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                const int d = dc + q;
                if (d < cend) store_row<R>(b.dinitial + ((long)s * a.dim + d) * N, j, N, G[q]);
            }
        }
    }

    if (kCarry) return;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        sum_D = add2(sum_D, pack2(__shfl_xor_sync(0xffffffffu, lo2(sum_D), o), __shfl_xor_sync(0xffffffffu, hi2(sum_D), o)));
        sum_bias = add2(sum_bias, pack2(__shfl_xor_sync(0xffffffffu, lo2(sum_bias), o), __shfl_xor_sync(0xffffffffu, hi2(sum_bias), o)));
    }
#pragma unroll
    for (int q = 0; q < CS; ++q) {
        const int d = dc + q;
        if (d >= cend) continue;
        store_row<R>(b.part_A + ((long)unit * a.dim + d) * N, j, N, dA[q]);
        if (j == 0) {
            b.part_D[(long)unit * a.dim + d] = q ? hi2(sum_D) : lo2(sum_D);
            b.part_bias[(long)unit * a.dim + d] = q ? hi2(sum_bias) : lo2(sum_bias);
        }
    }
}

// Sums of the parts: dB and dC over the channel tiles of a group, dA, dD and
// ddt_bias over the CTAs of a tile.
__global__ void __launch_bounds__(256)
selective_scan_bwd_sum_kernel(SelScanBwdArgs b, int gtiles, int ctas, long nB, long nA)
{
    const SelScanArgs &a = b.f;
    long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < 2 * nB) {
        const bool c = i >= nB;
        if (c) i -= nB;
        const float *p = (c ? b.part_C : b.part_B) + i;
        float s = 0.f;
#pragma unroll 8
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
#pragma unroll 8
    for (int q = 0; q < ctas; ++q) s += p[q * n + i];
    out[i] = s;
}

struct BwdPlan {
    int cs, gtiles, ctas, units, span;
    size_t bytes_B, bytes_A, bytes_D, bytes_carry;
    size_t bytes() const { return 2 * bytes_B + bytes_A + 2 * bytes_D + bytes_carry; }
};

template <typename TIn, typename TDt, int R, int L, int CS, bool kPacked>
cudaError_t launch_packed(const SelScanBwdArgs &b, const BwdPlan &p, cudaStream_t stream)
{
    using S = BwdShape<R, L, CS>;
    const auto main = selective_scan_bwd_kernel<TIn, TDt, R, L, CS, false, kPacked>;
    const auto carry = selective_scan_bwd_kernel<TIn, TDt, R, L, CS, true, kPacked>;
    const long long tiles = (long long)p.gtiles * b.f.ngroups;
    if (tiles * p.units > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (const cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes)) return e;
    if (p.span) {
        if (const cudaError_t e = cudaFuncSetAttribute(carry, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kStaged)) return e;
        carry<<<(unsigned)(tiles * p.units), kBwdThreads, S::kStaged, stream>>>(b, p.units);
    }
    main<<<(unsigned)(tiles * p.ctas), kBwdThreads, S::kBytes, stream>>>(b, p.ctas);
    return cudaGetLastError();
}

template <typename TIn, typename TDt, int R, int L, int CS>
cudaError_t launch_shape(const SelScanBwdArgs &b, const BwdPlan &p, cudaStream_t stream)
{
    return b.f.pairs ? launch_packed<TIn, TDt, R, L, CS, true>(b, p, stream)
                     : launch_packed<TIn, TDt, R, L, CS, false>(b, p, stream);
}

// Lanes per channel for d_state (R = 4 states a lane, 8 above 128).
int lanes_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 148;
    }
    return sms;
}

// Time of `ctas` equal CTAs, `per` to an SM, in rounds: a last round with fewer
// to an SM runs faster, but not in proportion (share[k]: k CTAs an SM against a
// full one).
double rounds(long long ctas, int sms, int per, const double *share)
{
    const long long full = ctas / ((long long)sms * per), rest = ctas - full * sms * per;
    return (double)full + share[(rest + sms - 1) / sms];
}

BwdPlan make_plan(int nseq, long T, int dim, int d_state, int ngroups)
{
    BwdPlan p{};
    const int L = lanes_for(d_state), gdim = dim / ngroups, sms = sm_count();
    auto tiles_of = [&](int cs) { const int cb = 32 / L * cs * kWarps; return (gdim + cb - 1) / cb; };
    // Segments, where one-set CTAs of whole sequences would fill less than half of the device: as many as fill
    // it, of at least 32 tokens; and the long sequences of a ragged batch that fills it (segment_span).  The pass
    // before costs about a quarter of the cut sequences' work again.  Measured, training steps: 701 tokens in 5
    // sequences of 1002 channels 129 us whole, 87 cut; 4000 in 4 of 2048 channels 1005 and 543 us.
    const double fill = (double)tiles_of(1) * ngroups * nseq / (4. * sms);
    p.units = nseq;
    p.span = segment_span(nseq, T, fill, true);
    if (p.span) p.units = (int)(T / p.span + nseq);
    p.ctas = p.span || p.units < kMaxCtas ? p.units : kMaxCtas;
    // One or two sets of channels a warp: two share the loads of B and C and the sums over the channels, one
    // makes twice as many CTAs.  Measured: 4 x 2048 tokens of 8192 channels with 16 states, 2.32 ms with one set
    // (1024 CTAs, 1.7 rounds), 2.11 with two (512, 1.15 rounds); 16 x 512 tokens, 1.60 ms with two (2.16 with
    // one); 5 x 140 tokens of 1002 channels, 0.076 ms with one (160 CTAs), 0.100 with two (80).
    p.cs = 1;
    if (L > 1 && d_state <= 128) {
        static const double share1[] = {0., 0.45, 0.55, 0.8, 1.}, share2[] = {0., 0.6, 0.75, 1.};
        const double one = rounds((long long)tiles_of(1) * ngroups * p.ctas, sms, 4, share1);
        const double two = 1.06 * rounds((long long)tiles_of(2) * ngroups * p.ctas, sms, 3, share2);
        if (two < 0.95 * one) p.cs = 2;
    }
    p.gtiles = tiles_of(p.cs);
    auto up = [](size_t v) { return (v + 15) / 16 * 16; };
    const size_t row = (size_t)dim * sizeof(float);
    p.bytes_B = up((size_t)p.gtiles * T * ngroups * d_state * sizeof(float));
    p.bytes_A = up(p.ctas * row * d_state);
    p.bytes_D = up(p.ctas * row);
    p.bytes_carry = p.span ? p.units * row * d_state + up(p.units * row) : 0;
    return p;
}

template <typename TIn, typename TDt, int R, int L>
cudaError_t launch_sets(const SelScanBwdArgs &b, const BwdPlan &p, cudaStream_t stream)
{
    if constexpr (R == 4 && L > 1)
        if (p.cs == 2) return launch_shape<TIn, TDt, R, L, 2>(b, p, stream);
    return launch_shape<TIn, TDt, R, L, 1>(b, p, stream);
}

template <typename TIn, typename TDt>
cudaError_t launch_types(const SelScanBwdArgs &b, const BwdPlan &p, cudaStream_t stream)
{
    const int N = b.f.d_state;
    if (N <= 4) return launch_sets<TIn, TDt, 4, 1>(b, p, stream);
    if (N <= 8) return launch_sets<TIn, TDt, 4, 2>(b, p, stream);
    if (N <= 16) return launch_sets<TIn, TDt, 4, 4>(b, p, stream);
    if (N <= 32) return launch_sets<TIn, TDt, 4, 8>(b, p, stream);
    if (N <= 64) return launch_sets<TIn, TDt, 4, 16>(b, p, stream);
    if (N <= 128) return launch_sets<TIn, TDt, 4, 32>(b, p, stream);
    return launch_sets<TIn, TDt, 8, 32>(b, p, stream);
}

// The plan that a call runs: the one that sized the workspace, but without its cuts where equal lengths leave
// nothing to cut.
BwdPlan launch_plan(int nseq, int seqlen, bool packed, int dim, int d_state, int ngroups)
{
    BwdPlan p = make_plan(nseq, packed ? (long)seqlen : (long)nseq * seqlen, dim, d_state, ngroups);
    if (p.span && !packed && p.span >= seqlen) {
        p.span = 0;
        p.ctas = p.units = nseq;
    }
    return p;
}

}  // namespace

int selective_scan_bwd_rows(int nseq, int seqlen, bool packed, int dim, int d_state, int ngroups, int *held)
{
    *held = make_plan(nseq, packed ? (long)seqlen : (long)nseq * seqlen, dim, d_state, ngroups).ctas;
    return launch_plan(nseq, seqlen, packed, dim, d_state, ngroups).ctas;
}

size_t selective_scan_bwd_workspace(int nseq, long T, int dim, int d_state, int ngroups)
{
    return make_plan(nseq, T, dim, d_state, ngroups).bytes();
}

cudaError_t launch_selective_scan_bwd(SelScanBwdArgs b, void *workspace, cudaStream_t stream)
{
    SelScanArgs &a = b.f;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const int N = a.d_state;
    const BwdPlan p = launch_plan(a.nseq, a.seqlen, a.cu_seqlens != nullptr, a.dim, N, a.ngroups);
    char *w = static_cast<char *>(workspace);
    auto take = [&](size_t bytes) {
        float *f = reinterpret_cast<float *>(w);
        w += bytes;
        return f;
    };
    b.part_B = take(p.bytes_B);
    b.part_C = take(p.bytes_B);
    b.part_A = take(p.bytes_A);
    b.part_D = take(p.bytes_D);
    b.part_bias = take(p.bytes_D);
    a.span = p.span;
    a.units = p.units;
    a.range_state = p.span ? take((size_t)p.units * a.dim * N * sizeof(float)) : nullptr;
    a.range_dt = p.span ? take(0) : nullptr;
    const cudaError_t e = !a.in_bf16 ? launch_types<float, float>(b, p, stream)
        : a.dt_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(b, p, stream)
                    : launch_types<__nv_bfloat16, float>(b, p, stream);
    if (e) return e;
    const long nB = T * a.ngroups * N, nA = (long)a.dim * N;
    const long long blocks = (2 * nB + nA + 2L * a.dim + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    selective_scan_bwd_sum_kernel<<<(unsigned)blocks, 256, 0, stream>>>(b, p.gtiles, p.ctas, nB, nA);
    return cudaGetLastError();
}

}  // namespace ssm
