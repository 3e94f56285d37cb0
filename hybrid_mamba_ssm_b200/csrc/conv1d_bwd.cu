// conv1d_bwd.cu -- gradient of the causal depthwise conv1d (conv1d.cu).  For
// channel c, width K, token t of a sequence, with in[] the sequence's inputs
// behind its K-1 history entries:
//
//   pre[t]     = bias + sum_k w[k] in[t-(K-1)+k]
//   dpre[t]    = dy[t] act'(pre[t])        act' = s (1 + pre (1 - s)), s = sigmoid(pre)
//   din[t]     = sum_k w[k] dpre[t+(K-1)-k]     (tokens of the same sequence)
//   dweight[k] = sum_t dpre[t] in[t-(K-1)+k],   dbias = sum_t dpre[t]
//
// din of the history entries is the gradient of the initial conv state; the
// gradient of the final conv state (copies of the last K-1 inputs) adds to
// the inputs it copies.
//
// A thread owns two adjacent channels (packed fp32 arithmetic) and a tile of
// tokens, which it walks in groups of kGroup: the group's inputs and dy are
// loaded together, one group ahead, so that 2 kGroup loads are in flight while
// a group is computed.  pre comes from a register window of inputs; a second
// window holds dpre, so din of token t is complete K-1 tokens later.  The
// tile's first K-1 and last K-1 tokens depend on its neighbours: the walk
// starts with the inputs of the K-1 tokens before the tile and runs K-1 tokens
// past its end, recomputing their dpre (2 (K-1) tokens of a tile are read
// twice, from L2).  Weight and bias sums stay in registers over
// the tile and are added up over the tiles by a second launch, in a fixed
// order.  Bound by HBM: x and dy read once, dx written once.  16384 tokens of
// 10240 bf16 channels, width 4: 0.23 ms (4.3 TB/s of the bytes above, two launches;
// issue slots at 53 %).  One
// token at a time, without groups: 0.61 ms.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kBwdThreads = 128;
constexpr int kGroup = 8;

// Tokens of a tile: a walk inside one sequence is `walk` tokens, K - 1 of them
// behind the tile.  256 where that leaves eight CTAs an SM (16384 tokens of
// 10240 channels 233 us, 239 with 128: fewer parts to add), 128 down to two, else
// 32 (a walk is a chain of its groups: 701 tokens of 1002 channels take 22 us in
// 24 CTAs of 128, 8 us in 88 of 32).
__host__ __device__ __forceinline__ int tile_tokens(int walk, int K) { return walk - (K - 1); }
inline int walk_tokens(long T, int dim)
{
    const long strip = 148L * 2 * kBwdThreads;       // channels of one CTA an SM
    return T * dim >= 8 * strip * 256 ? 256 : T * dim >= 2 * strip * 128 ? 128 : 32;
}

// Raw values of channels c, c + 1 of a row (the second only where it exists).
template <typename T, bool kPair>
__device__ __forceinline__ void load_two(const T *row, int c, bool both, RawPair<T, kPair> &r) {
    if constexpr (kPair) r.load(row, c);
    else r.load(row, c, true, both);
}
template <typename T, bool kPair>
__device__ __forceinline__ void store_two(T *row, int c, bool both, f32x2 v) {
    if constexpr (kPair && sizeof(T) == 2) {
        *reinterpret_cast<__nv_bfloat162 *>(row + c) = __floats2bfloat162_rn(lo2(v), hi2(v));
    } else if constexpr (kPair) {
        *reinterpret_cast<float2 *>(row + c) = make_float2(lo2(v), hi2(v));
    } else {
        store_out(row + c, lo2(v));
        if (both) store_out(row + c + 1, hi2(v));
    }
}

// kPair: dim is even, so two channels are one aligned access.
template <typename T, int K, bool kPair>
__global__ void __launch_bounds__(kBwdThreads, K <= 4 ? 4 : 2)
conv1d_bwd_kernel(ConvBwdArgs a, int ctiles, int walk)
{
    constexpr int H = K - 1;                  // history entries
    const int c = ((int)(blockIdx.x % ctiles) * kBwdThreads + threadIdx.x) * 2;
    const long tile = blockIdx.x / ctiles;
    const long total = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const int len = tile_tokens(walk, K);
    const long t0 = tile * len, t1 = min(t0 + len, total);
    if (c >= a.dim) return;
    const bool both = kPair || c + 1 < a.dim;
    const int c1 = both ? c + 1 : c;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    const T *init = static_cast<const T *>(a.initial), *dfin = static_cast<const T *>(a.dfinal);
    T *dx = static_cast<T *>(a.dx), *dinit = static_cast<T *>(a.dinitial);

    f32x2 w[K], dw[K], db = pack2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = pack2(a.weight[(long)c * K + k], a.weight[(long)c1 * K + k]);
        dw[k] = db;
    }
    const f32x2 bias = a.bias ? pack2(a.bias[c], a.bias[c1]) : db, one = pack2(1.f, 1.f);
    // history entry h of sequence s
    auto history = [&](const T *p, int s, long h) {
        return pack2(load_f32(p + ((long)s * a.dim + c) * H + h), load_f32(p + ((long)s * a.dim + c1) * H + h));
    };

    // sequence of the first token (the last s that starts at or before it)
    int s = 0;
    if (a.cu_seqlens) {
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_seqlens[mid] <= t0) lo = mid; else hi = mid - 1;
        }
        s = lo;
    } else {
        s = (int)(t0 / a.seqlen);
    }

    for (long t = t0; t < t1;) {
        if (s >= a.nseq) {
            report_status(a.status_dev, kStatusDeviceInput);
            break;
        }
        long lo = (long)s * a.seqlen, hi = lo + a.seqlen;
        if (a.cu_seqlens) {
            lo = a.cu_seqlens[s];
            hi = a.cu_seqlens[s + 1];
            if (lo < 0 || lo > t || hi < lo || hi > total) {
                report_status(a.status_dev, kStatusDeviceInput);
                break;
            }
        }
        const long end = min(hi, t1);
        if (end <= t) {
            ++s;
            continue;
        }
        const int nend = (int)(end - t);                        // tokens of this walk
        const int npast = (int)(min(hi, end + H) - t);          // tokens whose dpre it needs
        const int start = t == lo ? -H : 0;                     // first entry that this walk completes
        const int copied = dfin ? (int)min(hi - H - t, (long)nend) : nend;   // entries from here on are in the final state
        const T *xt = x + t * a.dim, *gt = dy + t * a.dim;
        T *ot = dx + t * a.dim;
        // win[H + i], dp[H + i]: input and dpre of token i of the group; the first H are the tokens before
        f32x2 win[H + kGroup], dp[H + kGroup];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            dp[k] = pack2(0.f, 0.f);
            const long i = t - H + k;
            RawPair<T, kPair> r;
            r.zero();
            if (i >= lo) load_two<T, kPair>(x + i * a.dim, c, both, r);
            win[k] = r.value();
            if (i < lo && init && i >= lo - H) win[k] = history(init, s, i - lo + H);
        }
        RawPair<T, kPair> rx[kGroup], rg[kGroup];
        auto fetch = [&](int i0) {                              // 32-bit offsets from the walk's first row
            if (i0 + kGroup <= npast) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    load_two<T, kPair>(xt, (i0 + i) * a.dim + c, both, rx[i]);
                    load_two<T, kPair>(gt, (i0 + i) * a.dim + c, both, rg[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    rx[i].zero();
                    rg[i].zero();
                    if (i0 + i < npast) {
                        load_two<T, kPair>(xt, (i0 + i) * a.dim + c, both, rx[i]);
                        load_two<T, kPair>(gt, (i0 + i) * a.dim + c, both, rg[i]);
                    }
                }
            }
        };
        // gradient through the activation, for the group's tokens
        auto group_dpre = [&](f32x2 (&g)[kGroup]) {
            if (!a.activation) return;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                f32x2 pre = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) pre = fma2(w[k], win[i + k], pre);
                const f32x2 d = add2(ex2_pair(mul2(pre, pack2(-kLog2e, -kLog2e))), one);
                const f32x2 sg = pack2(rcp_approx(lo2(d)), rcp_approx(hi2(d)));
                g[i] = mul2(mul2(g[i], sg), fma2(pre, fma2(sg, pack2(-1.f, -1.f), one), one));
            }
        };
        auto add_weight = [&](int i) {                          // token i of the group in the sums
            db = add2(db, dp[H + i]);
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k] = fma2(dp[H + i], win[i + k], dw[k]);
        };
        auto taps = [&](int i) {                                // din of the entry H tokens before it
            f32x2 din = mul2(w[K - 1], dp[i]);
#pragma unroll
            for (int k = 1; k < K; ++k) din = fma2(w[K - 1 - k], dp[i + k], din);
            return din;
        };
        fetch(0);
        for (int i0 = 0; i0 < nend + H; i0 += kGroup) {
            f32x2 g[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                win[H + i] = rx[i].value();
                g[i] = rg[i].value();
            }
            if (i0 + kGroup < npast) fetch(i0 + kGroup);
            group_dpre(g);
            if (i0 >= H && i0 + kGroup <= nend && i0 + kGroup - H <= copied) {   // all inside: no conditions
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    dp[H + i] = g[i];
                    add_weight(i);
                    store_two<T, kPair>(ot, (i0 + i - H) * a.dim + c, both, taps(i));
                }
            } else {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    // tokens behind the sequence have no dpre (their pre need not be finite)
                    dp[H + i] = i0 + i < npast ? g[i] : pack2(0.f, 0.f);
                    if (i0 + i < nend) add_weight(i);
                    const int e = i0 + i - H;
                    if (e >= nend || e < start) continue;       // another walk completes it
                    f32x2 din = taps(i);
                    if (e >= copied) din = add2(din, history(dfin, s, t + e - hi + H));
                    if (e >= 0) {
                        store_two<T, kPair>(ot, e * a.dim + c, both, din);
                    } else if (dinit) {
                        store_out(dinit + ((long)s * a.dim + c) * H + (e + H), lo2(din));
                        if (both) store_out(dinit + ((long)s * a.dim + c1) * H + (e + H), hi2(din));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < H; ++k) {
                win[k] = win[kGroup + k];
                dp[k] = dp[kGroup + k];
            }
        }
        t = end;
    }

    float *part = a.part + tile * (K + 1) * a.dim;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        const f32x2 v = k < K ? dw[k < K ? k : 0] : db;
        part[(long)k * a.dim + c] = lo2(v);
        if (both) part[(long)k * a.dim + c1] = hi2(v);
    }
}

// Empty sequences: their final conv state is the initial one.
template <typename T>
__global__ void conv1d_bwd_empty_kernel(ConvBwdArgs a)
{
    const int s = blockIdx.x, H = a.width - 1;
    if (a.cu_seqlens ? a.cu_seqlens[s] != a.cu_seqlens[s + 1] : a.seqlen != 0) return;
    const long n = (long)a.dim * H;
    T *out = static_cast<T *>(a.dinitial) + s * n;
    const T *in = static_cast<const T *>(a.dfinal);
    for (long i = threadIdx.x; i < n; i += blockDim.x) store_out(out + i, in ? load_f32(in + s * n + i) : 0.f);
}

// dweight / dbias: sums of the tiles' parts, 64 channels x 4 tile lanes a CTA.
// Lane sums are added in a fixed order, so the result does not depend on the
// order in which CTAs ran.
__global__ void __launch_bounds__(256)
conv1d_bwd_sum_kernel(ConvBwdArgs a, int tiles)
{
    __shared__ float red[4][64];
    const int cx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + cx, k = blockIdx.y, K = a.width;
    float v = 0.f;
    if (c < a.dim) {
        const float *p = a.part + (long)k * a.dim + c;
#pragma unroll 8
        for (int i = ty; i < tiles; i += 4) v += p[(long)i * (K + 1) * a.dim];
    }
    red[ty][cx] = v;
    __syncthreads();
    if (ty || c >= a.dim) return;
    v = (red[0][cx] + red[1][cx]) + (red[2][cx] + red[3][cx]);
    if (k < K) a.dweight[(long)c * K + k] = v;
    else if (a.dbias) a.dbias[c] = v;
}

template <typename T, int K>
cudaError_t launch_k(const ConvBwdArgs &a, cudaStream_t stream)
{
    const long total = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const int walk = walk_tokens(total, a.dim), len = tile_tokens(walk, K);
    const long tiles = (total + len - 1) / len;
    if (tiles > 0) {
        const int ctiles = (a.dim + 2 * kBwdThreads - 1) / (2 * kBwdThreads);
        if (tiles * ctiles > 0x7fffffffL) return cudaErrorInvalidValue;
        const unsigned blocks = (unsigned)(tiles * ctiles);
        if (a.dim % 2 == 0) conv1d_bwd_kernel<T, K, true><<<blocks, kBwdThreads, 0, stream>>>(a, ctiles, walk);
        else conv1d_bwd_kernel<T, K, false><<<blocks, kBwdThreads, 0, stream>>>(a, ctiles, walk);
    }
    if (a.dinitial && K > 1) conv1d_bwd_empty_kernel<T><<<(unsigned)a.nseq, 256, 0, stream>>>(a);
    conv1d_bwd_sum_kernel<<<dim3((unsigned)((a.dim + 63) / 64), (unsigned)(K + 1)), 256, 0, stream>>>(a, (int)tiles);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ConvBwdArgs &a, cudaStream_t stream)
{
    switch (a.width) {
    case 1: return launch_k<T, 1>(a, stream);
    case 2: return launch_k<T, 2>(a, stream);
    case 3: return launch_k<T, 3>(a, stream);
    case 4: return launch_k<T, 4>(a, stream);
    case 5: return launch_k<T, 5>(a, stream);
    case 6: return launch_k<T, 6>(a, stream);
    case 7: return launch_k<T, 7>(a, stream);
    default: return launch_k<T, 8>(a, stream);
    }
}

}  // namespace

size_t conv1d_bwd_workspace(long T, int dim, int width)
{
    const long n = tile_tokens(walk_tokens(T, dim), width);
    return (size_t)((T + n - 1) / n) * (width + 1) * dim * sizeof(float);
}

cudaError_t launch_conv1d_bwd(const ConvBwdArgs &a, cudaStream_t stream)
{
    return a.in_bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace ssm
