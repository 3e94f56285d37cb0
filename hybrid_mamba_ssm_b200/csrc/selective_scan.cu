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
// states in registers as packed pairs, of Q channels; a CTA of 128 threads takes
// Q 128 / L channels of one group.  Tokens go through shared memory in tiles:
// each (token, channel) is loaded, its step size transformed and multiplied by x
// exactly once, then read by the channel's L lanes, while the next tile's global
// loads are in flight.  Up to four partial sums over n a (token, channel) are
// left to the step that writes y.
//
// What bounds it (ncu, 4096 tokens of 8192 channels, 16 states, bf16): the
// shared-memory pipe at 77 % of its cycles, of which B and C, read by every
// lane for its own states, are two thirds; the special-function unit at 53 %
// (one exponential an element and three a (token, channel): 0.28 ms for 4 x
// 2048 tokens if it were the bound); issue slots at 58 %; HBM at 11 %.  4 x 2048
// tokens take 0.53 ms, 1 x 32768 of 2048 channels 0.90 ms.
// Q = 2 halves the reads of B and C but also the warps: 0.62 ms against 0.53 at
// 16 states, where seven CTAs an SM hide the latencies, but 0.48 against 0.63 ms
// at 32 states (4 x 2048 x 4096), 0.40 against 0.49 at 64 (4 x 1024 x 4096) and
// 0.92 against 1.92 at 256 (4 x 1024 x 2048), where few channels share a tile of
// B and C.  Q = 4 is slower at all of them.
#include <type_traits>

#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kThreads = 128;

constexpr int min3(int a, int b, int c) { return a < b ? (a < c ? a : c) : (b < c ? b : c); }

template <int R, int L, int Q>
struct ScanShape {
    static constexpr int CS = kThreads / L;                      // channels of a set
    static constexpr int CT = CS * Q;                            // channels per CTA
    static constexpr int NP = R * L;                             // states, zero padded
    static constexpr int KT = min3(32, 1024 / NP, 512 / CT);     // tokens per tile
    static constexpr int TG = 4;                                 // tokens per step of the scan
    static constexpr int RS = kThreads / (CT / 2);               // tokens per staging step (a thread: two channels)
    static constexpr int E = (KT + RS - 1) / RS;                 // staged pairs per thread
    static constexpr int EB = (KT * NP + kThreads - 1) / kThreads;
    static constexpr int YP = L < 4 ? L : 4;                     // partial sums over n left to the output step
    // two buffers of v and v x, of B and C, and of the partial sums of y
    static constexpr size_t bytes(bool out) { return sizeof(float) * (4 * KT * CT + 4 * KT * NP + (out ? 2 * KT * CT * YP : 0)); }
    static_assert(KT % TG == 0 && CT % 2 == 0, "");
};

// CTAs that an SM must hold at once: registers are the limit (a thread keeps
// 4 R Q of them for the states and decay rates).
template <int R, int Q>
constexpr int kMinBlocks = R * Q <= 4 ? 7 : 4;

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

enum { kWhole = 0, kRangeState = 1, kRangeOut = 2 };

// kWhole: one CTA per (sequence, channel tile).
// kRangeState / kRangeOut: one CTA per (segment of a sequence, channel tile),
// two launches.  The first leaves, for every segment but a sequence's last, the
// state that its own tokens build from zero (the first one: from the initial
// state) and the sum of its step sizes: the segment multiplies the state that
// enters it by exp(A sum v).  It also copies the initial state.  The second
// folds the segments before its own and runs its tokens from the state that
// enters.
template <typename TIn, typename TDt, int R, int L, int Q, int kMode, bool kPacked>
__global__ void __launch_bounds__(kThreads, kMinBlocks<R, Q>)
selective_scan_kernel(SelScanArgs a)
{
    using S = ScanShape<R, L, Q>;
    constexpr int CS = S::CS, CT = S::CT, NP = S::NP, KT = S::KT, TG = S::TG, RS = S::RS, E = S::E, EB = S::EB;
    constexpr int P = R / 2, YP = S::YP;
    constexpr bool kOut = kMode != kRangeState;
    // two buffers each: a tile is staged while the one before is still read
    extern __shared__ __align__(16) float smem[];
    auto s_vu = reinterpret_cast<float2 (*)[KT * CT]>(smem);     // step size, step size times x
    auto s_B = reinterpret_cast<float (*)[KT * NP]>(smem + 4 * KT * CT);
    auto s_C = reinterpret_cast<float (*)[KT * NP]>(smem + 4 * KT * CT + 2 * KT * NP);
    auto s_y = reinterpret_cast<float (*)[KT * CT * YP]>(smem + 4 * KT * CT + 4 * KT * NP);

    const int tid = threadIdx.x, lane = tid & 31;
    const int gdim = a.dim / a.ngroups, gtiles = (gdim + CT - 1) / CT, tiles = gtiles * a.ngroups;
    const int unit = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x - (unsigned)unit * tiles);
    const int g = tile / gtiles, c0 = g * gdim + (tile - g * gtiles) * CT, cend = min(c0 + CT, (g + 1) * gdim);
    const int N = a.d_state;
    const long T = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;

    const int j = tid % L, ch = tid / L, d0 = c0 + ch;     // scanning: lane j of channels d0 + q CS
    const int sc = 2 * (tid % (CT / 2)), st = tid / (CT / 2), ds = c0 + sc;   // staging: channels ds, ds + 1
    const bool slive0 = ds < cend, slive1 = ds + 1 < cend;
    auto per_channel = [&](const float *p) {
        return pack2(p && slive0 ? p[ds] : 0.f, p && slive1 ? p[ds + 1] : 0.f);
    };
    const f32x2 bias = per_channel(a.dtp.bias), skip = per_channel(a.D);
    auto live = [&](int q) { return d0 + q * CS < cend; };
    auto row_of = [&](const float *p, long row, int q) { return p + (row * a.dim + d0 + q * CS) * N; };

    f32x2 A[Q][P], h[Q][P];
    float vsum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        vsum[q] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = pack2(0.f, 0.f);
        if (live(q)) load_states<R>(row_of(a.A, 0, q), j, N, A[q]);
#pragma unroll
        for (int p = 0; p < P; ++p) A[q][p] = decay_rate2(A[q][p]);
    }
    // Raw values of the next tile; x and z of the one whose output is due.
    RawPair<TIn, kPacked> xr[E], zr[E], xc[E], zc[E];
    RawPair<TDt, kPacked> vr[E];
    uint32_t Br[EB], Cr[EB];

    // Pointers to this thread's values of the tile to fetch, moved on tile by
    // tile (the address arithmetic of the loads was a quarter of all
    // instructions when it started from the operands' bases).
    const bool whole_rows = kPacked && cend - c0 == CT && N == NP;   // no channel or state of the tile is padding
    constexpr int BR = NP <= kThreads ? kThreads / NP : 1;           // tokens per staging step of B and C
    const int bn = NP <= kThreads ? tid % NP : tid, bk = NP <= kThreads ? tid / NP : 0;
    const TIn *px, *pz, *pB, *pC;
    const TDt *pv;
    auto seek = [&](long t) {
        px = static_cast<const TIn *>(a.x) + (t + st) * a.x_stride + ds;
        pv = static_cast<const TDt *>(a.dt) + (t + st) * a.dt_stride + ds;
        pz = static_cast<const TIn *>(a.z) + (t + st) * a.z_stride + ds;
        pB = static_cast<const TIn *>(a.B) + (t + bk) * a.B_stride + g * N + bn;
        pC = static_cast<const TIn *>(a.C) + (t + bk) * a.C_stride + g * N + bn;
    };
    // Strides are at most 2^24 and a tile has at most 32 tokens: 32-bit offsets within it.
    const int xs = (int)a.x_stride, vs = (int)a.dt_stride, Bs = (int)a.B_stride, Cs = (int)a.C_stride, zs = (int)a.z_stride;

    // Raw values of the next n tokens, zero behind them.
    auto fetch = [&](int n) {
        if (n == KT && whole_rows) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (KT % RS && st + i * RS >= KT) break;
                if constexpr (kPacked) {
                    xr[i].load(px, i * RS * xs);
                    vr[i].load(pv, i * RS * vs);
                    if (kOut && a.z) zr[i].load(pz, i * RS * zs);
                }
            }
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                if (NP <= kThreads) {
                    if (KT % BR && bk + i * BR >= KT) break;
                    Br[i] = raw_load<TIn>(pB, i * BR * Bs);
                    if (kOut) Cr[i] = raw_load<TIn>(pC, i * BR * Cs);
                } else {                       // a row takes two steps
                    Br[i] = raw_load<TIn>(pB, i / 2 * Bs + i % 2 * kThreads);
                    if (kOut) Cr[i] = raw_load<TIn>(pC, i / 2 * Cs + i % 2 * kThreads);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const bool ok0 = slive0 && st + i * RS < n, ok1 = slive1 && ok0;
                xr[i].load(px, i * RS * xs, ok0, ok1);
                vr[i].load(pv, i * RS * vs, ok0, ok1);
                if (kOut) zr[i].load(pz, i * RS * zs, ok0 && a.z, ok1 && a.z);
            }
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int k = NP <= kThreads ? bk + i * BR : i / 2, add = NP <= kThreads ? 0 : i % 2 * kThreads;
                const int from = NP <= kThreads ? i * BR : i / 2;
                const bool ok = bn + add < N && k < n;
                Br[i] = ok ? raw_load<TIn>(pB, from * Bs + add) : 0u;
                if (kOut) Cr[i] = ok ? raw_load<TIn>(pC, from * Cs + add) : 0u;
            }
        }
        px += (long)n * xs;
        pv += (long)n * vs;
        pz += (long)n * zs;
        pB += (long)n * Bs;
        pC += (long)n * Cs;
    };
    // Step sizes, B and C of the fetched tile of n tokens into buffer b.
    auto stage = [&](int n, int b) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int k = st + i * RS;
            if (KT % RS && k >= KT) break;
            f32x2 v = dt_value2(a.dtp, vr[i].value(), bias);
            if (n < KT && k >= n) v = pack2(0.f, 0.f);   // tokens behind the tile leave the state as it is
            const f32x2 u = mul2(v, xr[i].value());
            *reinterpret_cast<float4 *>(&s_vu[b][k * CT + sc]) = make_float4(lo2(v), lo2(u), hi2(v), hi2(u));
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            const int e = tid + i * kThreads;
            if (KT * NP % kThreads && e >= KT * NP) break;
            s_B[b][e] = raw_value<TIn>(Br[i]);
            if (kOut) s_C[b][e] = raw_value<TIn>(Cr[i]);
        }
    };
    // y of a tile of n tokens, from the partial sums of buffer b; this thread's first is element `first`.
    auto output = [&](long first, int n, int b) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int k = st + i * RS;
            if (k >= n || !slive0) break;
            float f[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x2 part[(YP + 1) / 2];
                if constexpr (YP == 1) {
                    f[q] = s_y[b][k * CT + sc + q];
                } else {
                    lds_pairs(&s_y[b][(k * CT + sc + q) * YP], part);
                    f[q] = sum2(YP == 4 ? add2(part[0], part[YP / 2 - 1]) : part[0]);
                }
            }
            f32x2 y = fma2(skip, xc[i].value(), pack2(f[0], f[1]));
            if (a.z) y = mul2(y, silu2(zc[i].value()));
            const int o = i * RS * a.dim;
            if (a.y_bf16) {
                __nv_bfloat16 *yp = static_cast<__nv_bfloat16 *>(a.y) + first + o;
                if (slive1 && gdim % 2 == 0) {      // the even channel of a pair is even in y too
                    *reinterpret_cast<__nv_bfloat162 *>(yp) = __floats2bfloat162_rn(lo2(y), hi2(y));
                } else {
                    store_out(yp, lo2(y));
                    if (slive1) store_out(yp + 1, hi2(y));
                }
            } else {
                float *yp = static_cast<float *>(a.y) + first + o;
                store_out(yp, lo2(y));
                if (slive1) store_out(yp + 1, hi2(y));
            }
        }
    };

    // Tokens [t, te) of a sequence that starts at token lo.  One barrier per
    // tile: the output of the tile before and the scan of this one follow it.
    auto run = [&](long t, long te, long lo, long save0) {
        int rel = (int)(t - lo), left = (int)(te - t), before = 0, b = 0;
        int n = min(left, KT - rel % KT);          // tiles end on multiples of KT of the sequence
        seek(t);
        fetch(n);
        long out = (t + st) * a.dim + ds;          // y of the tile before, at this thread's first token
        while (left > 0) {
            stage(n, b);
            __syncthreads();
            if (kOut) {
                if (before) output(out, before, b ^ 1);
                out += (long)before * a.dim;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    xc[i] = xr[i];
                    zc[i] = zr[i];
                }
            }
            const int n2 = min(left - n, KT);
            if (n2 > 0) fetch(n2);
            if (kOut && a.saved && rel % kSavedEvery == 0) {
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    if (live(q)) store_states<R>(const_cast<float *>(row_of(a.saved, save0 + rel / kSavedEvery, q)), j, N, h[q]);
            }
#pragma unroll 1
            for (int k0 = 0; k0 < n; k0 += TG) {
                float yv[Q][TG];
#pragma unroll
                for (int k = 0; k < TG; ++k) {
                    f32x2 B[P], C[P];
                    lds_pairs(&s_B[b][(k0 + k) * NP + j * R], B);
                    if (kOut) lds_pairs(&s_C[b][(k0 + k) * NP + j * R], C);
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const float2 vu = s_vu[b][(k0 + k) * CT + ch + q * CS];
                        const f32x2 vv = pack2(vu.x, vu.x), uu = pack2(vu.y, vu.y);
                        f32x2 acc;
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            h[q][p] = fma2(decay2(vv, A[q][p]), h[q][p], mul2(uu, B[p]));
                            if (kOut) acc = p ? fma2(h[q][p], C[p], acc) : mul2(h[q][p], C[p]);
                        }
                        if (kOut) {
                            yv[q][k] = sum2(acc);
                            if (L <= 4) s_y[b][((k0 + k) * CT + ch + q * CS) * YP + j] = yv[q][k];
                        } else {
                            vsum[q] += vu.x;
                        }
                    }
                }
                if (kOut && L > 4) {
                    // four partial sums are left to the output step: lanes that differ in the upper bits are added
                    constexpr int kUp = L > 4 ? L / 4 : 1, kLeft = reduce_left(TG, kUp), kSame = kUp > TG ? kUp / TG : 1;
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int first = reduce_lanes<TG, kUp, 4>(yv[q], lane);
                        if ((j / 4) % kSame == 0) {
#pragma unroll
                            for (int i = 0; i < kLeft; ++i)
                                s_y[b][((k0 + first + i) * CT + ch + q * CS) * YP + j % 4] = yv[q][i];
                        }
                    }
                }
            }
            rel += n;
            left -= n;
            before = n;
            n = n2;
            b ^= 1;
        }
        __syncthreads();
        if (kOut) output(out, before, b ^ 1);
        __syncthreads();                           // the next sequence stages into either buffer
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
    // Every channel's states from rows[row] (or zero).
    auto load_all = [&](const float *rows, long row, f32x2 (&to)[Q][P]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int p = 0; p < P; ++p) to[q][p] = pack2(0.f, 0.f);
            if (rows && live(q)) load_states<R>(row_of(rows, row, q), j, N, to[q]);
        }
    };
    auto store_all = [&](float *rows, long row) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (live(q)) store_states<R>(const_cast<float *>(row_of(rows, row, q)), j, N, h[q]);
    };
    __shared__ int s_seq;
    Unit w;
    if (!find_unit(a, T, kMode == kWhole && a.cu_seqlens && a.nseq > 1 && a.nseq <= kMaxRanked ? longest_first(a, unit, &s_seq) : unit, w)) {
        check_offsets(a, T);
        return;
    }
    check_offsets(a, T);
    bool init;
    const long row = state_row(w.s, init);
    if (row < 0) return;
    if (kMode == kRangeState) {
        if (w.e == w.hi) return;                           // the last segment: nothing follows it
        load_all(init && w.k == 0 ? a.initial : nullptr, row, h);
        if (w.k == 0) store_all(a.range_initial, w.s);
        run(w.b, w.e, w.lo, 0);
        store_all(a.range_state, unit);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (j == 0 && live(q)) a.range_dt[(long)unit * a.dim + d0 + q * CS] = vsum[q];
        return;
    }
    if (kMode == kRangeOut && w.k > 0) {
        load_all(a.range_state, w.base, h);
#pragma unroll 4
        for (int i = 1; i < w.k; ++i) {                    // (loads of four segments in flight)
            f32x2 e[Q][P];
            load_all(a.range_state, w.base + i, e);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float v = live(q) ? a.range_dt[(w.base + i) * a.dim + d0 + q * CS] : 0.f;
#pragma unroll
                for (int p = 0; p < P; ++p)
                    h[q][p] = fma2(decay2(pack2(v, v), A[q][p]), h[q][p], e[q][p]);
            }
        }
    } else if (kMode == kRangeOut && w.e < w.hi) {
        // its row may be written (in place) by the segment it ends in: the copy is read
        load_all(a.range_initial, w.s, h);
    } else {
        load_all(init ? a.initial : nullptr, row, h);
    }
    if (w.b < w.e) run(w.b, w.e, w.lo, w.lo / kSavedEvery + w.s);
    if (w.e == w.hi && a.final && (w.lo < w.hi || a.final != a.initial || !init)) store_all(a.final, row);
}

template <typename TIn, typename TDt, int R, int L, int Q, int kMode, bool kPacked>
cudaError_t launch_mode(const SelScanArgs &a, unsigned blocks, cudaStream_t stream)
{
    constexpr size_t bytes = ScanShape<R, L, Q>::bytes(kMode != kRangeState);
    if (bytes > 48 * 1024)
        if (const cudaError_t e = cudaFuncSetAttribute(selective_scan_kernel<TIn, TDt, R, L, Q, kMode, kPacked>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) return e;
    selective_scan_kernel<TIn, TDt, R, L, Q, kMode, kPacked><<<blocks, kThreads, bytes, stream>>>(a);
    return cudaGetLastError();
}

template <typename TIn, typename TDt, int R, int L, int Q>
cudaError_t launch_shape(const SelScanArgs &a, cudaStream_t stream)
{
    const int gdim = a.dim / a.ngroups, CT = ScanShape<R, L, Q>::CT;
    const long long tiles = (long long)((gdim + CT - 1) / CT) * a.ngroups;
    if (tiles * a.units > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)(tiles * a.units);
    auto run = [&](auto packed) -> cudaError_t {
        constexpr bool kPacked = decltype(packed)::value;
        if (!a.span) return launch_mode<TIn, TDt, R, L, Q, kWhole, kPacked>(a, blocks, stream);
        if (const cudaError_t e = launch_mode<TIn, TDt, R, L, Q, kRangeState, kPacked>(a, blocks, stream)) return e;
        return launch_mode<TIn, TDt, R, L, Q, kRangeOut, kPacked>(a, blocks, stream);
    };
    return a.pairs ? run(std::true_type{}) : run(std::false_type{});
}

template <typename TIn, typename TDt>
cudaError_t launch_types(const SelScanArgs &a, cudaStream_t stream)
{
    const int N = a.d_state;
    if (N <= 4) return launch_shape<TIn, TDt, 4, 1, 1>(a, stream);
    if (N <= 8) return launch_shape<TIn, TDt, 4, 2, 1>(a, stream);
    if (N <= 16) return launch_shape<TIn, TDt, 4, 4, 1>(a, stream);
    if (N <= 32) return launch_shape<TIn, TDt, 4, 8, 2>(a, stream);
    if (N <= 64) return launch_shape<TIn, TDt, 4, 16, 2>(a, stream);
    if (N <= 128) return launch_shape<TIn, TDt, 4, 32, 2>(a, stream);
    return launch_shape<TIn, TDt, 8, 32, 2>(a, stream);
}

}  // namespace

// Lanes of a warp that share a channel.
static int lanes_for(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

// Tokens of a segment (0: sequences stay whole), for kernels whose CTAs of whole
// sequences would fill `fill` of the device.  Below a half: as many segments as
// fill it, of at least kSavedEvery tokens, if that is half as many again as
// there are sequences.  With `ragged`, up to three times the device: segments of
// 5/16 of the mean sequence, so that neither a long sequence's chain nor a last
// round of few CTAs is the time of all.  (The gradient does: 16884 tokens in 14
// sequences of 1276 channels 1.83 ms with segments of 5/4 of the mean, 1.36 with
// 5/8, 1.34 with 5/16, 1.30 with 5/32; 4 x 2048 tokens of 8192 channels 2.66,
// 2.54, 2.57, 2.58 with the forward pass.  Up to six times the device it loses:
// 8 x 2048 tokens 4.42 ms whole, 4.91 cut.  The forward pass pays 0.6 of the cut
// work and does not: 5 sequences, 8000 tokens, 4096 channels 0.46 to 0.73 ms
// whole, 0.54 to 0.62 cut, the same on average.)
int segment_span(int nseq, long T, double fill, bool ragged)
{
    if (nseq < 1) return 0;
    if (fill < 0.5) {
        long segments = (long)(nseq / fill);
        if (segments > T / kSavedEvery) segments = T / kSavedEvery;
        if (segments > 256) segments = 256;
        if (segments >= 2 && segments > nseq + nseq / 2) {
            const long n = (T / segments + kSavedEvery / 2) / kSavedEvery * kSavedEvery;
            return (int)(n < kSavedEvery ? kSavedEvery : n);
        }
    }
    const long mean = T / nseq;
    if (ragged && fill < 3. && nseq > 1 && nseq <= kMaxRanked && mean >= 128)
        return (int)((mean * 5 / 16 + kSavedEvery - 1) / kSavedEvery * kSavedEvery);
    return 0;
}

// A sequence is a chain of its tokens: nseq * dim channels give
// nseq * dim * lanes / 32 warps, however long it is.  Cutting sequences costs
// the first pass over the segments, about 0.6 of their work again (1 x 32768
// tokens, 2048 channels of 16 states: 2.8 ms as one chain, 0.9 ms cut; 600
// tokens in 4 sequences of 700 channels: 82 and 31 us).  Returns the number of
// units, 0 for whole sequences.
int selective_scan_segments(int nseq, long T, int dim, int d_state, int ngroups, int *span)
{
    *span = 0;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 0;
    }
    const double warps = (double)dim * lanes_for(d_state) / 32;
    *span = segment_span(nseq, T, warps * nseq / (28. * sms), false);
    return *span ? (int)(T / *span + nseq) : 0;
}

cudaError_t launch_selective_scan(const SelScanArgs &a, cudaStream_t stream)
{
    if (!a.in_bf16) return launch_types<float, float>(a, stream);
    if (a.dt_bf16) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, stream);
    return launch_types<__nv_bfloat16, float>(a, stream);
}

}  // namespace ssm
