// state_pool.cu -- rows of state pools copied (forked), zeroed (freed) and
// compacted, in any number of pools (one per layer and kind of state) by one
// launch.
//
// Every thread owns one column of a pool: the same 16 bytes (or 8 .. 1, by
// that pool's alignment) of every row.  It applies the list of row copies to
// its column in order, so the list has the meaning of a loop over it whatever
// rows it repeats or chains, without an ordering between threads.  kBatch
// copies are loaded before any is stored, unless one of them reads a row that
// an earlier one of the batch writes.  Bound by HBM: 12 rows of 48 pools (24
// layers, 280 KB a layer and row) in 21 us, 40 rows of 140 KB zeroed in 23 us
// (5.9 TB/s).
#include "common.cuh"
#include "ssm_internal.h"

namespace ssm {

namespace {

constexpr int kPoolThreads = 256;
constexpr int kBatch = 8;
constexpr int kPoolsPerLaunch = 64;

struct PoolList {
    char *base[kPoolsPerLaunch];
    long stride[kPoolsPerLaunch];
    long cols[kPoolsPerLaunch];                  // columns of a row
    uint8_t width[kPoolsPerLaunch];              // bytes of a column
    unsigned first_block[kPoolsPerLaunch + 1];   // blocks of pool p: [first_block[p], first_block[p + 1])
};

__device__ __forceinline__ int pool_of(const PoolList &l, int npools, unsigned block) {
    int lo = 0, hi = npools - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first_block[mid] <= block) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <typename U>
__device__ __forceinline__ U *cell(char *base, long stride, int row) {
    return reinterpret_cast<U *>(base + (long)row * stride);
}

// Calls f(a value of the column's type, the column's address in row 0, the row stride).
template <typename F>
__device__ __forceinline__ void for_column(const PoolList &l, int npools, F f) {
    const int p = pool_of(l, npools, blockIdx.x), width = l.width[p];
    const long col = (long)(blockIdx.x - l.first_block[p]) * kPoolThreads + threadIdx.x;
    if (col >= l.cols[p]) return;
    char *base = l.base[p] + col * width;
    if (width == 16) f(uint4{}, base, l.stride[p]);
    else if (width == 8) f(uint2{}, base, l.stride[p]);
    else if (width == 4) f(uint32_t{}, base, l.stride[p]);
    else if (width == 2) f(uint16_t{}, base, l.stride[p]);
    else f(uint8_t{}, base, l.stride[p]);
}

template <typename U>
__device__ __forceinline__ void copy_rows(char *base, long stride, int max_slots, int n, const int32_t *src,
                                          const int32_t *dst, int *status)
{
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        int s[kBatch], d[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            s[i] = i0 + i < n ? __ldg(src + i0 + i) : -1;
            d[i] = i0 + i < n ? __ldg(dst + i0 + i) : -1;
            if (s[i] < 0 || d[i] < 0 || s[i] >= max_slots || d[i] >= max_slots) {
                if (s[i] >= max_slots || d[i] >= max_slots) report_status(status, kStatusDeviceInput);
                s[i] = d[i] = -1;
            }
        }
        bool chained = false;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int k = 0; k < i; ++k) chained |= s[i] >= 0 && s[i] == d[k];
        if (!chained) {
            U v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s[i] >= 0) v[i] = *cell<U>(base, stride, s[i]);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s[i] >= 0) *cell<U>(base, stride, d[i]) = v[i];
        } else {
#pragma unroll 1
            for (int i = 0; i < kBatch; ++i) {
                const int a = i0 + i < n ? src[i0 + i] : -1, b = i0 + i < n ? dst[i0 + i] : -1;
                if (a < 0 || b < 0 || a >= max_slots || b >= max_slots) continue;
                *cell<U>(base, stride, b) = *cell<U>(base, stride, a);
            }
        }
    }
}

__global__ void __launch_bounds__(kPoolThreads)
pool_copy_kernel(const __grid_constant__ PoolList l, int npools, int max_slots, int n, const int32_t *src,
                 const int32_t *dst, const int32_t *count, int *status)
{
    if (count) n = min(n, *count);
    for_column(l, npools, [&](auto u, char *base, long stride) {
        copy_rows<decltype(u)>(base, stride, max_slots, n, src, dst, status);
    });
}

__global__ void __launch_bounds__(kPoolThreads)
pool_zero_kernel(const __grid_constant__ PoolList l, int npools, int max_slots, int n, const int32_t *rows,
                 int *status)
{
    for_column(l, npools, [&](auto u, char *base, long stride) {
        for (int i = 0; i < n; ++i) {
            const int r = __ldg(rows + i);
            if (r < 0) continue;
            if (r >= max_slots) report_status(status, kStatusDeviceInput);
            else *cell<decltype(u)>(base, stride, r) = u;
        }
    });
}

// Plan of a compaction, one CTA.  The distinct live rows are counted (n); the
// live rows >= n, ascending, move into the free rows < n, ascending.  table is
// rewritten.  map: [max_slots] scratch; src / dst: [min(nrows, max_slots)].
__global__ void __launch_bounds__(1024)
pool_plan_kernel(int32_t *table, int nrows, int max_slots, int32_t *map, int32_t *src, int32_t *dst,
                 int32_t *moves, int32_t *live, int *status)
{
    __shared__ int warp_a[32], warp_b[32], s_n, s_a, s_b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_n = s_a = s_b = 0;
    for (int i = tid; i < max_slots; i += 1024) map[i] = 0;
    __syncthreads();
    for (int b = tid; b < nrows; b += 1024) {
        const int r = table[b];
        if (r >= max_slots) report_status(status, kStatusDeviceInput);
        else if (r >= 0) map[r] = 1;
    }
    __syncthreads();
    int mine = 0;
    for (int i = tid; i < max_slots; i += 1024) mine += map[i];
    atomicAdd(&s_n, mine);              // integers: the order does not matter
    __syncthreads();
    const int n = s_n;
    for (int i0 = 0; i0 < max_slots; i0 += 1024) {
        const int i = i0 + tid;
        const bool on = i < max_slots && map[i] != 0;
        const bool mover = on && i >= n, hole = i < n && i < max_slots && !on;
        const unsigned ma = __ballot_sync(0xffffffffu, mover), mb = __ballot_sync(0xffffffffu, hole);
        if (lane == 0) {
            warp_a[warp] = __popc(ma);
            warp_b[warp] = __popc(mb);
        }
        __syncthreads();
        int ra = s_a, rb = s_b;
        for (int w = 0; w < warp; ++w) {
            ra += warp_a[w];
            rb += warp_b[w];
        }
        const unsigned below = (1u << lane) - 1u;
        if (mover) src[ra + __popc(ma & below)] = i;
        if (hole) dst[rb + __popc(mb & below)] = i;
        __syncthreads();
        if (tid == 1023) {
            s_a = ra + warp_a[31];
            s_b = rb + warp_b[31];
        }
        __syncthreads();
    }
    const int m = s_a;                  // = s_b: n live rows, n rows below n
    for (int i = tid; i < max_slots; i += 1024) map[i] = i;
    __syncthreads();
    for (int i = tid; i < m; i += 1024) map[src[i]] = dst[i];
    __syncthreads();
    for (int b = tid; b < nrows; b += 1024) {
        const int r = table[b];
        if (r >= 0 && r < max_slots) table[b] = map[r];
    }
    if (tid == 0) {
        *moves = m;
        if (live) *live = n;
    }
}

// Widest column that the pool's rows split into.
int column_bytes(const PoolRows &r)
{
    const uintptr_t bits = reinterpret_cast<uintptr_t>(r.base) | (uintptr_t)r.row_bytes | (uintptr_t)r.stride;
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
}

// Calls f(list, pools of the list, blocks) for lists of at most kPoolsPerLaunch pools.
template <typename F>
cudaError_t for_lists(const PoolArgs &a, F f)
{
    for (int p0 = 0; p0 < a.npools; p0 += kPoolsPerLaunch) {
        PoolList l;
        const int m = a.npools - p0 < kPoolsPerLaunch ? a.npools - p0 : kPoolsPerLaunch;
        unsigned long long blocks = 0;
        for (int p = 0; p < m; ++p) {
            const PoolRows &r = a.pools[p0 + p];
            l.base[p] = r.base;
            l.stride[p] = r.stride;
            l.width[p] = (uint8_t)column_bytes(r);
            l.cols[p] = r.row_bytes / l.width[p];
            l.first_block[p] = (unsigned)blocks;
            blocks += (unsigned long long)((l.cols[p] + kPoolThreads - 1) / kPoolThreads);
            if (blocks > 0x7fffffffULL) return cudaErrorInvalidValue;
        }
        l.first_block[m] = (unsigned)blocks;
        if (blocks) f(l, m, (unsigned)blocks);
        if (const cudaError_t e = cudaGetLastError()) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_pool_copy(const PoolArgs &a, cudaStream_t stream)
{
    return for_lists(a, [&](const PoolList &l, int m, unsigned blocks) {
        pool_copy_kernel<<<blocks, kPoolThreads, 0, stream>>>(l, m, a.max_slots, a.n, a.src, a.dst, a.count, a.status_dev);
    });
}

cudaError_t launch_pool_zero(const PoolArgs &a, cudaStream_t stream)
{
    return for_lists(a, [&](const PoolList &l, int m, unsigned blocks) {
        pool_zero_kernel<<<blocks, kPoolThreads, 0, stream>>>(l, m, a.max_slots, a.n, a.dst, a.status_dev);
    });
}

// map [max_slots], src and dst [min(nrows, max_slots)], the number of moves.
size_t pool_compact_workspace(int max_slots, int nrows)
{
    const size_t m = nrows < max_slots ? nrows : max_slots;
    return ((size_t)max_slots + 2 * m + 1) * sizeof(int32_t);
}

cudaError_t launch_pool_compact(const PoolArgs &a, int32_t *table, int nrows, int32_t *live, void *workspace,
                                cudaStream_t stream)
{
    const int m = nrows < a.max_slots ? nrows : a.max_slots;
    int32_t *map = static_cast<int32_t *>(workspace), *src = map + a.max_slots, *dst = src + m, *moves = dst + m;
    pool_plan_kernel<<<1, 1024, 0, stream>>>(table, nrows, a.max_slots, map, src, dst, moves, live, a.status_dev);
    if (const cudaError_t e = cudaGetLastError()) return e;
    PoolArgs c = a;
    c.n = m;
    c.src = src;
    c.dst = dst;
    c.count = moves;
    return launch_pool_copy(c, stream);
}

}  // namespace ssm
