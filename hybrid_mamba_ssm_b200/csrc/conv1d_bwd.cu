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
// A thread owns kCh adjacent channels and a tile of tokens.  It walks the tile
// forward, recomputing pre from a register window of inputs; a second window
// holds the last K-1 dpre, so din of token t is complete K-1 tokens later.
// The tile's first K-1 and last K-1 tokens depend on its neighbours: the walk
// starts with the inputs of the K-1 tokens before the tile and runs K-1 tokens
// past its end, recomputing their dpre (2 (K-1) of `kTile` tokens are read
// twice, from L2).  Weight and bias sums stay in registers over the tile and
// are added up over the tiles by a second launch, in a fixed order.
// Bound by HBM: x and dy read once, dx written once.
#include "selective.cuh"

namespace ssm {

namespace {

constexpr int kBwdThreads = 128;
constexpr int kTile = 128;

// Loads and stores of kCh adjacent channels.
template <typename T, int kCh>
__device__ __forceinline__ void load_ch(const T *p, float (&v)[kCh]) {
    if constexpr (kCh == 1) {
        v[0] = load_f32(p);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(p));
        v[0] = __uint_as_float(q << 16);
        v[1] = __uint_as_float(q & 0xffff0000u);
    } else {
        const float2 q = __ldg(reinterpret_cast<const float2 *>(p));
        v[0] = q.x;
        v[1] = q.y;
    }
}
template <typename T, int kCh>
__device__ __forceinline__ void store_ch(T *p, const float (&v)[kCh]) {
    if constexpr (kCh == 1) {
        store_out(p, v[0]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
    } else {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    }
}

template <typename T, int K, int kCh>
__global__ void __launch_bounds__(kBwdThreads)
conv1d_bwd_kernel(ConvBwdArgs a, int ctiles)
{
    constexpr int H = K - 1;                  // history entries
    const int c = ((int)(blockIdx.x % ctiles) * kBwdThreads + threadIdx.x) * kCh;
    const long tile = blockIdx.x / ctiles;
    const long total = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const long t0 = tile * kTile, t1 = min(t0 + kTile, total);
    if (c >= a.dim) return;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    const T *init = static_cast<const T *>(a.initial), *dfin = static_cast<const T *>(a.dfinal);
    T *dx = static_cast<T *>(a.dx), *dinit = static_cast<T *>(a.dinitial);

    float w[K][kCh], bias[kCh], dw[K][kCh], db[kCh];
#pragma unroll
    for (int q = 0; q < kCh; ++q) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            w[k][q] = a.weight[(long)(c + q) * K + k];
            dw[k][q] = 0.f;
        }
        bias[q] = a.bias ? a.bias[c + q] : 0.f;
        db[q] = 0.f;
    }

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
        // win[k]: input of tap k of the current token (win[K-1] its own);
        // dp[k]: dpre of token t-(K-1)+k
        float win[K][kCh], dp[K][kCh];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int q = 0; q < kCh; ++q) win[k][q] = dp[k][q] = 0.f;
        // entry i of the sequence's line: a token, or one of the H history entries before it
        auto entry = [&](long i, float (&v)[kCh]) {
            if (i >= lo) {
                load_ch<T, kCh>(x + i * a.dim + c, v);
            } else {
#pragma unroll
                for (int q = 0; q < kCh; ++q)
                    v[q] = init && i >= lo - H ? load_f32(init + ((long)s * a.dim + c + q) * H + (i - lo + H)) : 0.f;
            }
        };
#pragma unroll
        for (int k = 1; k < K; ++k) entry(t - K + k, win[k]);
        const long past = min(hi, end + H);     // dpre is needed for H tokens past the end
        for (long i = t; i < end + H; ++i) {
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int q = 0; q < kCh; ++q) {
                    win[k][q] = win[k + 1][q];
                    dp[k][q] = dp[k + 1][q];
                }
#pragma unroll
            for (int q = 0; q < kCh; ++q) dp[K - 1][q] = 0.f;
            if (i < past) {
                float g[kCh];
                load_ch<T, kCh>(x + i * a.dim + c, win[K - 1]);
                load_ch<T, kCh>(dy + i * a.dim + c, g);
#pragma unroll
                for (int q = 0; q < kCh; ++q) {
                    if (a.activation) {
                        float pre = bias[q];
#pragma unroll
                        for (int k = 0; k < K; ++k) pre = fmaf(w[k][q], win[k][q], pre);
                        const float sg = rcp_approx(1.f + ex2_approx(-pre * kLog2e));
                        g[q] *= sg * fmaf(pre, 1.f - sg, 1.f);
                    }
                    dp[K - 1][q] = g[q];
                }
                if (i < end) {
#pragma unroll
                    for (int q = 0; q < kCh; ++q) {
                        db[q] += g[q];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][q] = fmaf(g[q], win[k][q], dw[k][q]);
                    }
                }
            }
            // entry i - H of the line is complete: taps K-1 .. 0 read it at tokens i-H .. i
            const long e = i - H;
            if (e < t && !(t == lo)) continue;      // the tile before writes it
            float din[kCh];
#pragma unroll
            for (int q = 0; q < kCh; ++q) {
                din[q] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) din[q] = fmaf(w[K - 1 - k][q], dp[k][q], din[q]);
            }
            if (dfin && e >= hi - H) {              // the final conv state is a copy of it
#pragma unroll
                for (int q = 0; q < kCh; ++q)
                    din[q] += load_f32(dfin + ((long)s * a.dim + c + q) * H + (e - hi + H));
            }
            if (e >= lo) {
                store_ch<T, kCh>(dx + e * a.dim + c, din);
            } else if (dinit) {
#pragma unroll
                for (int q = 0; q < kCh; ++q)
                    store_out(dinit + ((long)s * a.dim + c + q) * H + (e - lo + H), din[q]);
            }
        }
        t = end;
    }

    if (!a.part) return;
    float *part = a.part + tile * (K + 1) * a.dim + c;
#pragma unroll
    for (int q = 0; q < kCh; ++q) {
#pragma unroll
        for (int k = 0; k < K; ++k) part[(long)k * a.dim + q] = dw[k][q];
        part[(long)K * a.dim + q] = db[q];
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

// dweight / dbias: sums of the tiles' parts.  32 channels x 32 tile lanes a
// CTA; lane sums are added in a fixed tree, so the result does not depend on
// the order in which CTAs ran.
__global__ void __launch_bounds__(1024)
conv1d_bwd_sum_kernel(ConvBwdArgs a, long tiles)
{
    __shared__ float red[32][33];
    const int cx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx, k = blockIdx.y, K = a.width;
    float v = 0.f;
    if (c < a.dim)
        for (long i = ty; i < tiles; i += 32) v += a.part[(i * (K + 1) + k) * a.dim + c];
    red[ty][cx] = v;
    __syncthreads();
    v = red[cx][ty];                            // tile lane cx of channel ty
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int co = blockIdx.x * 32 + ty;
    if (cx == 0 && co < a.dim) {
        if (k < K) a.dweight[(long)co * K + k] = v;
        else if (a.dbias) a.dbias[co] = v;
    }
}

template <typename T, int K>
cudaError_t launch_k(const ConvBwdArgs &a, cudaStream_t stream)
{
    const long T_ = a.cu_seqlens ? (long)a.seqlen : (long)a.nseq * a.seqlen;
    const long tiles = (T_ + kTile - 1) / kTile;
    if (tiles > 0) {
        // pairs of channels need an even row length for aligned pair accesses
        const int ch = a.dim % 2 == 0 ? 2 : 1;
        const int ctiles = (a.dim + kBwdThreads * ch - 1) / (kBwdThreads * ch);
        if (tiles * ctiles > 0x7fffffffL) return cudaErrorInvalidValue;
        const unsigned blocks = (unsigned)(tiles * ctiles);
        if (ch == 2) conv1d_bwd_kernel<T, K, 2><<<blocks, kBwdThreads, 0, stream>>>(a, ctiles);
        else conv1d_bwd_kernel<T, K, 1><<<blocks, kBwdThreads, 0, stream>>>(a, ctiles);
    }
    if (a.dinitial && K > 1) conv1d_bwd_empty_kernel<T><<<(unsigned)a.nseq, 256, 0, stream>>>(a);
    conv1d_bwd_sum_kernel<<<dim3((unsigned)((a.dim + 31) / 32), (unsigned)(K + 1)), 1024, 0, stream>>>(a, tiles);
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
    return (size_t)((T + kTile - 1) / kTile) * (width + 1) * dim * sizeof(float);
}

cudaError_t launch_conv1d_bwd(const ConvBwdArgs &a, cudaStream_t stream)
{
    return a.in_bf16 ? launch_t<__nv_bfloat16>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace ssm
