// abi_selective.cu -- the extern "C" entry points of the per-channel selective
// scan, its gradient and decode update, the conv1d gradient and the state-pool
// row operations: host-side validation of every argument, then launches on the
// caller's stream.  Nothing here allocates, synchronises or keeps state
// between calls.
#include "abi_checks.h"

#include "../../include/ssm_testing.h"

namespace {

// One activation operand: rows of `width` elements, `stride` elements apart.
struct Rows {
    const void *p;
    int64_t stride;
    long long width;
    int dtype;
};

// The kernels address a tile of up to 32 tokens by 32-bit offsets.
constexpr int64_t kMaxRow = 1 << 24;

size_t rows_bytes(const Rows &r, long long T)
{
    return T > 0 ? (size_t)(((T - 1) * r.stride + r.width) * (long long)dtype_size(r.dtype)) : 0;
}

// SSM_OK, or the status of a bad operand: rows that overlap, or a base that is
// not aligned to its element.
int check_rows(const Rows &r, long long T)
{
    if (!r.p) return T > 0 ? SSM_ERR_INVALID_ARG : SSM_OK;
    if (T > 1 && r.stride < r.width) return SSM_ERR_INVALID_ARG;
    if (r.stride < 0) return SSM_ERR_INVALID_ARG;
    if (r.stride > kMaxRow || r.width > kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(r.p) % dtype_size(r.dtype)) return SSM_ERR_MISALIGNED;
    return SSM_OK;
}

// Whether channels 2i and 2i + 1 of every token are one aligned access.
bool paired(const Rows &r)
{
    return !r.p || (r.stride % 2 == 0 && reinterpret_cast<uintptr_t>(r.p) % (2 * dtype_size(r.dtype)) == 0);
}

// No output overlaps an input or another output.
int check_disjoint(const Range *outs, int nout, const Range *ins, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int k = 0; k < nin; ++k)
            if (overlap(outs[i], ins[k])) return SSM_ERR_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (overlap(outs[i], outs[k])) return SSM_ERR_INVALID_ARG;
    }
    return SSM_OK;
}

Range f32_range(const float *p, long long n) { return range_of(p, p ? (size_t)n * sizeof(float) : 0); }
Range i32_range(const int32_t *p, long long n) { return range_of(p, p ? (size_t)n * sizeof(int32_t) : 0); }

bool scan_shape_ok(int nseq, int seqlen, const int32_t *cu, int dim, int d_state, int ngroups)
{
    if (nseq < 0 || seqlen < 0 || dim <= 0 || d_state <= 0 || ngroups <= 0 || dim % ngroups) return false;
    return !(cu && nseq == 0 && seqlen != 0);
}

long long tokens_of(int nseq, int seqlen, const int32_t *cu) { return cu ? seqlen : (long long)nseq * seqlen; }

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

}  // namespace

extern "C" {

size_t selective_scan_saved_size(int nseq, long long ntokens, int dim, int d_state)
{
    if (nseq <= 0 || ntokens < 0 || dim <= 0 || d_state <= 0) return 0;
    return (size_t)ssm::saved_rows(ntokens, nseq) * dim * d_state * sizeof(float);
}

size_t selective_scan_workspace_size(int nseq, long long ntokens, int dim, int d_state, int ngroups)
{
    if (nseq <= 0 || ntokens <= 0 || dim <= 0 || d_state <= 0 || d_state > 256 || ngroups <= 0 || dim % ngroups)
        return 0;
    int span;
    const int units = ssm::selective_scan_segments(nseq, ntokens, dim, d_state, ngroups, &span);
    const size_t row = (size_t)dim * d_state * sizeof(float);
    return units ? up16(units * row) + up16(nseq * row) + (size_t)units * dim * sizeof(float) : 0;
}

int selective_scan_fwd(int nseq, int seqlen, const int32_t *cu_seqlens, int dim, int d_state, int ngroups,
                       int in_dtype, const void *x, int64_t x_stride,
                       int dt_dtype, const void *dt, int64_t dt_stride, const float *A,
                       const void *B, int64_t B_stride, const void *C, int64_t C_stride,
                       const float *D, const void *z, int64_t z_stride, const ssm_dt_params *dt_params,
                       const float *initial_state, float *final_state, int max_slots,
                       const int32_t *slot_idx, const int32_t *has_initial_state,
                       int y_dtype, void *y, float *saved_states, void *workspace, size_t workspace_bytes,
                       int *status_dev, cudaStream_t stream)
{
    if (!scan_shape_ok(nseq, seqlen, cu_seqlens, dim, d_state, ngroups)) return SSM_ERR_INVALID_ARG;
    if (!valid_dtype(in_dtype) || !valid_dtype(dt_dtype) || !valid_dtype(y_dtype)) return SSM_ERR_INVALID_ARG;
    if (d_state > 256 || (in_dtype == SSM_F32 && dt_dtype == SSM_BF16)) return SSM_ERR_UNSUPPORTED;
    if (nseq == 0) return SSM_OK;
    const long long T = tokens_of(nseq, seqlen, cu_seqlens);
    if (T > 0x7fffffffLL || nseq > 0x7fffffff / 2) return SSM_ERR_UNSUPPORTED;
    if (slot_idx && (max_slots <= 0 || (!initial_state && !final_state))) return SSM_ERR_INVALID_ARG;
    if (!A || (T > 0 && !y)) return SSM_ERR_INVALID_ARG;
    if (T == 0 && !final_state) return SSM_OK;
    const long long bc = (long long)ngroups * d_state;
    const Rows rows[] = {{x, x_stride, dim, in_dtype}, {dt, dt_stride, dim, dt_dtype}, {B, B_stride, bc, in_dtype},
                         {C, C_stride, bc, in_dtype}, {z, z_stride, dim, in_dtype}};
    for (int i = 0; i < (z ? 5 : 4); ++i)
        if (const int st = check_rows(rows[i], T)) return st;
    ssm::DtParams dtp;
    if (const int st = read_dt_params(dt_params, dtp)) return st;
    const void *ptrs[] = {cu_seqlens, A, D, initial_state, final_state, slot_idx, has_initial_state, y,
                          saved_states, workspace, status_dev};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_MISALIGNED;

    const long long srow = (long long)dim * d_state, nrows = slot_idx ? max_slots : nseq;
    const size_t need = selective_scan_workspace_size(nseq, T, dim, d_state, ngroups);
    const bool cut = need && workspace && workspace_bytes >= need;
    const Range outs[] = {range_of(y, (size_t)T * dim * dtype_size(y_dtype)), f32_range(final_state, nrows * srow),
                          range_of(saved_states, saved_states ? selective_scan_saved_size(nseq, T, dim, d_state) : 0),
                          range_of(workspace, workspace ? workspace_bytes : 0)};
    const Range init = f32_range(initial_state, nrows * srow);
    const Range ins[] = {range_of(x, rows_bytes(rows[0], T)), range_of(dt, rows_bytes(rows[1], T)),
                         range_of(B, rows_bytes(rows[2], T)), range_of(C, rows_bytes(rows[3], T)),
                         range_of(z, z ? rows_bytes(rows[4], T) : 0), f32_range(A, srow), f32_range(D, dim),
                         f32_range(dtp.bias, dim), i32_range(cu_seqlens, nseq + 1LL), i32_range(slot_idx, nseq),
                         i32_range(has_initial_state, nseq)};
    if (const int st = check_disjoint(outs, 4, ins, 11)) return st;
    // the final states may be written over the initial ones, row for row
    for (int i = 0; i < 4; ++i)
        if (!(i == 1 && final_state == initial_state) && overlap(outs[i], init)) return SSM_ERR_INVALID_ARG;

    ssm::SelScanArgs a{};
    a.nseq = nseq; a.seqlen = seqlen; a.cu_seqlens = cu_seqlens;
    a.dim = dim; a.d_state = d_state; a.ngroups = ngroups;
    a.in_bf16 = in_dtype == SSM_BF16; a.dt_bf16 = dt_dtype == SSM_BF16; a.y_bf16 = y_dtype == SSM_BF16;
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.z = z;
    a.x_stride = x_stride; a.dt_stride = dt_stride; a.B_stride = B_stride; a.C_stride = C_stride; a.z_stride = z_stride;
    a.A = A; a.D = D; a.dtp = dtp;
    a.initial = initial_state; a.final = final_state;
    a.slot_idx = slot_idx; a.has_initial = has_initial_state; a.max_slots = max_slots;
    a.y = y; a.saved = saved_states; a.status_dev = status_dev;
    a.pairs = dim / ngroups % 2 == 0 && paired(rows[0]) && paired(rows[1]) && paired(rows[4]);
    a.units = nseq;
    if (cut) {
        a.units = ssm::selective_scan_segments(nseq, T, dim, d_state, ngroups, &a.span);
        const size_t n = up16((size_t)a.units * srow * sizeof(float));
        char *w = static_cast<char *>(workspace);
        a.range_state = reinterpret_cast<float *>(w);
        a.range_initial = reinterpret_cast<float *>(w + n);
        a.range_dt = reinterpret_cast<float *>(w + n + up16((size_t)nseq * srow * sizeof(float)));
    }
    return ssm::launch_selective_scan(a, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

size_t selective_scan_bwd_workspace_size(int nseq, long long ntokens, int dim, int d_state, int ngroups)
{
    if (nseq <= 0 || ntokens < 0 || dim <= 0 || d_state <= 0 || d_state > 256 || ngroups <= 0 || dim % ngroups)
        return 0;
    return ssm::selective_scan_bwd_workspace(nseq, ntokens, dim, d_state, ngroups);
}

int selective_scan_bwd(int nseq, int seqlen, const int32_t *cu_seqlens, int dim, int d_state, int ngroups,
                       int in_dtype, const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                       int dt_dtype, const void *dt, int64_t dt_stride, const float *A,
                       const void *B, int64_t B_stride, const void *C, int64_t C_stride,
                       const float *D, const void *z, int64_t z_stride, const ssm_dt_params *dt_params,
                       const float *saved_states, const float *dfinal_state,
                       void *dx, void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz,
                       float *ddt_bias, float *dinitial_state, void *workspace, size_t workspace_bytes,
                       int *status_dev, cudaStream_t stream)
{
    if (!scan_shape_ok(nseq, seqlen, cu_seqlens, dim, d_state, ngroups)) return SSM_ERR_INVALID_ARG;
    if (!valid_dtype(in_dtype) || !valid_dtype(dt_dtype)) return SSM_ERR_INVALID_ARG;
    if (d_state > 256 || (in_dtype == SSM_F32 && dt_dtype == SSM_BF16)) return SSM_ERR_UNSUPPORTED;
    if (nseq == 0) return SSM_OK;
    const long long T = tokens_of(nseq, seqlen, cu_seqlens);
    if (T > 0x7fffffffLL || nseq > 0x7fffffff / 2) return SSM_ERR_UNSUPPORTED;
    if (!A || !dA || !saved_states || !workspace) return SSM_ERR_INVALID_ARG;
    if (T > 0 && (!dx || !ddt || !dB || !dC || (z && !dz))) return SSM_ERR_INVALID_ARG;
    if (!z && dz) return SSM_ERR_INVALID_ARG;
    const long long bc = (long long)ngroups * d_state, srow = (long long)dim * d_state;
    const Rows rows[] = {{x, x_stride, dim, in_dtype}, {dt, dt_stride, dim, dt_dtype}, {B, B_stride, bc, in_dtype},
                         {C, C_stride, bc, in_dtype}, {dy, dy_stride, dim, in_dtype}, {z, z_stride, dim, in_dtype}};
    for (int i = 0; i < (z ? 6 : 5); ++i)
        if (const int st = check_rows(rows[i], T)) return st;
    ssm::DtParams dtp;
    if (const int st = read_dt_params(dt_params, dtp)) return st;
    if (workspace_bytes < selective_scan_bwd_workspace_size(nseq, T, dim, d_state, ngroups)) return SSM_ERR_INVALID_ARG;
    const void *ptrs[] = {cu_seqlens, A, D, saved_states, dfinal_state, dx, ddt, dA, dB, dC, dD, dz, ddt_bias,
                          dinitial_state, workspace, status_dev};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_MISALIGNED;
    const size_t es = dtype_size(in_dtype);
    const Range outs[] = {range_of(dx, (size_t)T * dim * es), range_of(ddt, (size_t)T * dim * dtype_size(dt_dtype)),
                          f32_range(dA, srow), range_of(dB, (size_t)T * bc * es), range_of(dC, (size_t)T * bc * es),
                          f32_range(dD, dim), range_of(dz, dz ? (size_t)T * dim * es : 0), f32_range(ddt_bias, dim),
                          f32_range(dinitial_state, nseq * srow), range_of(workspace, workspace_bytes)};
    const Range ins[] = {range_of(x, rows_bytes(rows[0], T)), range_of(dt, rows_bytes(rows[1], T)),
                         range_of(B, rows_bytes(rows[2], T)), range_of(C, rows_bytes(rows[3], T)),
                         range_of(dy, rows_bytes(rows[4], T)), range_of(z, z ? rows_bytes(rows[5], T) : 0),
                         f32_range(A, srow), f32_range(D, dim), f32_range(dtp.bias, dim),
                         i32_range(cu_seqlens, nseq + 1LL), f32_range(dfinal_state, nseq * srow),
                         range_of(saved_states, selective_scan_saved_size(nseq, T, dim, d_state))};
    if (const int st = check_disjoint(outs, 10, ins, 12)) return st;

    ssm::SelScanBwdArgs b{};
    ssm::SelScanArgs &a = b.f;
    a.nseq = nseq; a.seqlen = seqlen; a.cu_seqlens = cu_seqlens;
    a.dim = dim; a.d_state = d_state; a.ngroups = ngroups;
    a.in_bf16 = in_dtype == SSM_BF16; a.dt_bf16 = dt_dtype == SSM_BF16;
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.z = z;
    a.x_stride = x_stride; a.dt_stride = dt_stride; a.B_stride = B_stride; a.C_stride = C_stride; a.z_stride = z_stride;
    a.A = A; a.D = D; a.dtp = dtp;
    a.saved = const_cast<float *>(saved_states);
    a.pairs = dim / ngroups % 2 == 0 && paired(rows[0]) && paired(rows[1]) && paired(rows[4]) && paired(rows[5]);
    a.status_dev = status_dev;
    b.dy = dy; b.dy_stride = dy_stride; b.dfinal = dfinal_state;
    b.dx = dx; b.ddt = ddt; b.dA = dA; b.dB = dB; b.dC = dC; b.dD = dD; b.dz = dz;
    b.ddt_bias = ddt_bias; b.dinitial = dinitial_state;
    return ssm::launch_selective_scan_bwd(b, workspace, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

int selective_state_update(int batch, int dim, int d_state, int ngroups, float *state, int max_slots,
                           const int32_t *slot_idx, int in_dtype, const void *x, int64_t x_stride,
                           int dt_dtype, const void *dt, int64_t dt_stride, const float *A,
                           const void *B, int64_t B_stride, const void *C, int64_t C_stride,
                           const float *D, const void *z, int64_t z_stride, const ssm_dt_params *dt_params,
                           int y_dtype, void *y, int *status_dev, cudaStream_t stream)
{
    if (batch < 0 || dim <= 0 || d_state <= 0 || ngroups <= 0 || dim % ngroups) return SSM_ERR_INVALID_ARG;
    if (!valid_dtype(in_dtype) || !valid_dtype(dt_dtype) || !valid_dtype(y_dtype)) return SSM_ERR_INVALID_ARG;
    if (d_state > 256 || (in_dtype == SSM_F32 && dt_dtype == SSM_BF16)) return SSM_ERR_UNSUPPORTED;
    if (batch == 0) return SSM_OK;
    if (!state || !A || !y || (slot_idx && max_slots <= 0)) return SSM_ERR_INVALID_ARG;
    const long long bc = (long long)ngroups * d_state, srow = (long long)dim * d_state;
    const Rows rows[] = {{x, x_stride, dim, in_dtype}, {dt, dt_stride, dim, dt_dtype}, {B, B_stride, bc, in_dtype},
                         {C, C_stride, bc, in_dtype}, {z, z_stride, dim, in_dtype}};
    for (int i = 0; i < (z ? 5 : 4); ++i)
        if (const int st = check_rows(rows[i], batch)) return st;
    ssm::DtParams dtp;
    if (const int st = read_dt_params(dt_params, dtp)) return st;
    const void *ptrs[] = {state, slot_idx, A, D, y, status_dev};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_MISALIGNED;
    const Range outs[] = {range_of(y, (size_t)batch * dim * dtype_size(y_dtype)),
                          f32_range(state, (slot_idx ? max_slots : batch) * srow)};
    const Range ins[] = {range_of(x, rows_bytes(rows[0], batch)), range_of(dt, rows_bytes(rows[1], batch)),
                         range_of(B, rows_bytes(rows[2], batch)), range_of(C, rows_bytes(rows[3], batch)),
                         range_of(z, z ? rows_bytes(rows[4], batch) : 0), f32_range(A, srow), f32_range(D, dim),
                         f32_range(dtp.bias, dim), i32_range(slot_idx, batch)};
    if (const int st = check_disjoint(outs, 2, ins, 9)) return st;

    ssm::SelUpdateArgs a{};
    a.batch = batch; a.dim = dim; a.d_state = d_state; a.ngroups = ngroups;
    a.in_bf16 = in_dtype == SSM_BF16; a.dt_bf16 = dt_dtype == SSM_BF16; a.y_bf16 = y_dtype == SSM_BF16;
    a.state = state; a.slot_idx = slot_idx; a.max_slots = max_slots;
    a.x = x; a.dt = dt; a.B = B; a.C = C; a.z = z;
    a.x_stride = x_stride; a.dt_stride = dt_stride; a.B_stride = B_stride; a.C_stride = C_stride; a.z_stride = z_stride;
    a.A = A; a.D = D; a.dtp = dtp; a.y = y; a.status_dev = status_dev;
    return ssm::launch_selective_update(a, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

int ssm_testing_selective_bwd_rows(int nseq, int seqlen, int packed, int dim, int d_state, int ngroups, int *held)
{
    if (!held || nseq <= 0 || seqlen < 0 || dim <= 0 || d_state <= 0 || d_state > 256 || ngroups <= 0 || dim % ngroups)
        return -1;
    return ssm::selective_scan_bwd_rows(nseq, seqlen, packed != 0, dim, d_state, ngroups, held);
}

size_t causal_conv1d_bwd_workspace_size(long long ntokens, int dim, int width)
{
    if (ntokens < 0 || dim <= 0 || width <= 0 || width > 8) return 0;
    return ssm::conv1d_bwd_workspace(ntokens, dim, width);
}

int causal_conv1d_bwd(int nseq, int seqlen, const int32_t *cu_seqlens, int dim, int width, int in_dtype,
                      const void *dy, const void *x, const float *weight, const float *bias, int activation,
                      const void *initial_state, const void *dfinal_state, void *dx, float *dweight,
                      float *dbias, void *dinitial_state, void *workspace, size_t workspace_bytes,
                      int *status_dev, cudaStream_t stream)
{
    if (nseq < 0 || seqlen < 0 || dim <= 0 || width < 1) return SSM_ERR_INVALID_ARG;
    if (!valid_dtype(in_dtype) || (activation != 0 && activation != 1)) return SSM_ERR_INVALID_ARG;
    if (width > 8 || nseq > 0x7fffffff / 2 || dim > kMaxRow / 2) return SSM_ERR_UNSUPPORTED;
    if (cu_seqlens && nseq == 0 && seqlen != 0) return SSM_ERR_INVALID_ARG;
    const long long T = tokens_of(nseq, seqlen, cu_seqlens);
    if (T > 0x7fffffffLL) return SSM_ERR_UNSUPPORTED;
    if (!weight || !dweight || (T > 0 && (!x || !dy || !dx || !workspace))) return SSM_ERR_INVALID_ARG;
    const void *ptrs[] = {cu_seqlens, dy, x, weight, bias, initial_state, dfinal_state, dx, dweight, dbias,
                          dinitial_state, workspace, status_dev};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_MISALIGNED;
    if (workspace_bytes < causal_conv1d_bwd_workspace_size(T, dim, width)) return SSM_ERR_INVALID_ARG;
    const size_t es = dtype_size(in_dtype), line = (size_t)T * dim * es, st = (size_t)nseq * dim * (width - 1) * es;
    const Range outs[] = {range_of(dx, line), f32_range(dweight, (long long)dim * width), f32_range(dbias, dim),
                          range_of(dinitial_state, dinitial_state ? st : 0),
                          range_of(workspace, workspace ? workspace_bytes : 0)};
    const Range ins[] = {range_of(dy, line), range_of(x, line), f32_range(weight, (long long)dim * width),
                         f32_range(bias, dim), range_of(initial_state, initial_state ? st : 0),
                         range_of(dfinal_state, dfinal_state ? st : 0), i32_range(cu_seqlens, nseq + 1LL)};
    if (const int e = check_disjoint(outs, 5, ins, 7)) return e;
    ssm::ConvBwdArgs a{};
    a.nseq = nseq; a.seqlen = seqlen; a.cu_seqlens = cu_seqlens;
    a.dim = dim; a.width = width; a.activation = activation; a.in_bf16 = in_dtype == SSM_BF16;
    a.x = x; a.dy = dy; a.weight = weight; a.bias = bias;
    a.initial = width > 1 ? initial_state : nullptr;
    a.dfinal = width > 1 ? dfinal_state : nullptr;
    a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.dinitial = width > 1 && nseq > 0 ? dinitial_state : nullptr;
    a.part = static_cast<float *>(workspace); a.status_dev = status_dev;
    return ssm::launch_conv1d_bwd(a, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // extern "C"

namespace {

// Slots of a pool and entries of an index list: the kernels step through both with 32-bit counters.
constexpr int kMaxRows = 1 << 30;

// Pools of a row operation, checked: no row overlaps the next, none overlaps
// the index lists (lists[0 .. nlists)), no pool is listed twice.
int read_pools(int npools, const ssm_pool *pools, int max_slots, const Range *lists, int nlists,
               ssm::PoolRows *out)
{
    for (int p = 0; p < npools; ++p) {
        const ssm_pool &q = pools[p];
        if (!q.base || q.row_bytes <= 0 || q.row_stride < q.row_bytes) return SSM_ERR_INVALID_ARG;
        if (q.row_stride > (1LL << 40)) return SSM_ERR_UNSUPPORTED;
        const Range r = range_of(q.base, (size_t)((max_slots - 1LL) * q.row_stride + q.row_bytes));
        for (int i = 0; i < nlists; ++i)
            if (overlap(r, lists[i])) return SSM_ERR_INVALID_ARG;
        for (int k = 0; k < p; ++k)
            if (pools[k].base == q.base) return SSM_ERR_INVALID_ARG;
        out[p] = ssm::PoolRows{static_cast<char *>(q.base), (long)q.row_bytes, (long)q.row_stride};
    }
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_pool_copy(int npools, const ssm_pool *pools, int max_slots, int npairs, const int32_t *src_idx,
                  const int32_t *dst_idx, int *status_dev, cudaStream_t stream)
{
    if (npools < 0 || npairs < 0 || max_slots <= 0) return SSM_ERR_INVALID_ARG;
    if (npools > SSM_MAX_POOLS || max_slots > kMaxRows || npairs > kMaxRows) return SSM_ERR_UNSUPPORTED;
    if (npools == 0 || npairs == 0) return SSM_OK;
    if (!pools || !src_idx || !dst_idx) return SSM_ERR_INVALID_ARG;
    if (!aligned16(src_idx) || !aligned16(dst_idx) || !aligned16(status_dev)) return SSM_ERR_MISALIGNED;
    ssm::PoolRows rows[SSM_MAX_POOLS];
    const Range lists[] = {i32_range(src_idx, npairs), i32_range(dst_idx, npairs)};
    if (const int st = read_pools(npools, pools, max_slots, lists, 2, rows)) return st;
    ssm::PoolArgs a{npools, rows, max_slots, npairs, src_idx, dst_idx, nullptr, status_dev};
    return ssm::launch_pool_copy(a, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

int ssm_pool_zero(int npools, const ssm_pool *pools, int max_slots, int nrows, const int32_t *row_idx,
                  int *status_dev, cudaStream_t stream)
{
    if (npools < 0 || nrows < 0 || max_slots <= 0) return SSM_ERR_INVALID_ARG;
    if (npools > SSM_MAX_POOLS || max_slots > kMaxRows || nrows > kMaxRows) return SSM_ERR_UNSUPPORTED;
    if (npools == 0 || nrows == 0) return SSM_OK;
    if (!pools || !row_idx) return SSM_ERR_INVALID_ARG;
    if (!aligned16(row_idx) || !aligned16(status_dev)) return SSM_ERR_MISALIGNED;
    ssm::PoolRows rows[SSM_MAX_POOLS];
    const Range lists[] = {i32_range(row_idx, nrows)};
    if (const int st = read_pools(npools, pools, max_slots, lists, 1, rows)) return st;
    ssm::PoolArgs a{npools, rows, max_slots, nrows, nullptr, row_idx, nullptr, status_dev};
    return ssm::launch_pool_zero(a, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

size_t ssm_pool_compact_workspace_size(int max_slots, int nrows)
{
    return max_slots > 0 && nrows >= 0 ? ssm::pool_compact_workspace(max_slots, nrows) : 0;
}

int ssm_pool_compact(int npools, const ssm_pool *pools, int max_slots, int nrows, int32_t *slot_idx,
                     int32_t *nlive, void *workspace, size_t workspace_bytes, int *status_dev,
                     cudaStream_t stream)
{
    if (npools < 0 || nrows < 0 || max_slots <= 0) return SSM_ERR_INVALID_ARG;
    if (npools > SSM_MAX_POOLS || max_slots > kMaxRows || nrows > kMaxRows) return SSM_ERR_UNSUPPORTED;
    if ((npools && !pools) || (nrows && !slot_idx) || !workspace) return SSM_ERR_INVALID_ARG;
    if (!aligned16(slot_idx) || !aligned16(nlive) || !aligned16(workspace) || !aligned16(status_dev))
        return SSM_ERR_MISALIGNED;
    if (workspace_bytes < ssm_pool_compact_workspace_size(max_slots, nrows)) return SSM_ERR_INVALID_ARG;
    ssm::PoolRows rows[SSM_MAX_POOLS];
    const Range lists[] = {i32_range(slot_idx, nrows), i32_range(nlive, 1), range_of(workspace, workspace_bytes)};
    if (const int st = check_disjoint(lists, 3, nullptr, 0)) return st;
    if (const int st = read_pools(npools, pools, max_slots, lists, 3, rows)) return st;
    ssm::PoolArgs a{npools, rows, max_slots, 0, nullptr, nullptr, nullptr, status_dev};
    return ssm::launch_pool_compact(a, slot_idx, nrows, nlive, workspace, stream) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // extern "C"
