// C ABI entries of the linear layer: argument checks, workspace plan, and the
// passes of the backward call.
//
//   forward   Y = act(X W^T + b) + R            (Z = X W^T + b kept if asked)
//   backward  dZ = dY * act'(Z),  dX = dZ W,  dW = dZ^T X,  db = sum_m dZ
// X is M x K, W is N x K, Y is M x N, all with rows of contiguous elements.
#include "linear.cuh"

namespace symar {

// ---------------------------------------------------------------- dZ and db
//
// One pass over dY (and Z): writes dZ rounded to the inputs' type (the tensor
// cores' operand type; the products that follow sum in 32 bits) and sums its
// columns unrounded in 32 bits.  A block takes 256 columns of a strip of rows;
// the strips' sums are added in order by a second launch.

constexpr int kDzThreads = 256, kDzCols = 256, kDzVec = 8;

struct DzArgs {
    const void* dy;
    size_t ldy;
    const void* pre;
    size_t ldp;
    void* dz;              // null: not wanted
    size_t ldz;
    float* partial;        // [strips][N]; null: not wanted
    size_t M, N, strip;
    int act;
};

template <class X>
__global__ void __launch_bounds__(kDzThreads) k_linear_dz(DzArgs a) {
    constexpr int LANES = kDzCols / kDzVec, ROWS = kDzThreads / LANES;
    __shared__ float red[ROWS][kDzCols];
    const int tx = threadIdx.x % LANES, ty = threadIdx.x / LANES;
    const size_t j0 = (size_t)blockIdx.x * kDzCols + tx * kDzVec;
    const size_t r0 = (size_t)blockIdx.y * a.strip, r1 = min(r0 + a.strip, a.M);
    float s[kDzVec] = {};
    for (size_t i = r0 + ty; i < r1; i += ROWS) {
#pragma unroll
        for (int e = 0; e < kDzVec; ++e) {
            const size_t j = j0 + e;
            if (j >= a.N) break;
            float d = load_f<X>(a.dy, i * a.ldy + j);
            if (a.pre) d *= act_slope(load_f<X>(a.pre, i * a.ldp + j), a.act);
            s[e] += d;
            if (a.dz) store_f<X>(a.dz, i * a.ldz + j, d);
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int e = 0; e < kDzVec; ++e) red[ty][tx * kDzVec + e] = s[e];
    __syncthreads();
    const size_t j = (size_t)blockIdx.x * kDzCols + threadIdx.x;
    if (j >= a.N) return;
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) t += red[r][threadIdx.x];
    a.partial[(size_t)blockIdx.y * a.N + j] = t;
}

template <class O>
__global__ void __launch_bounds__(kDzThreads) k_linear_db(const float* partial, size_t strips, size_t N, void* db,
                                                          bool accumulate) {
    const size_t j = (size_t)blockIdx.x * kDzThreads + threadIdx.x;
    if (j >= N) return;
    float t = accumulate ? load_f<O>(db, j) : 0.f;
    for (size_t s = 0; s < strips; ++s) t += partial[s * N + j];
    store_f<O>(db, j, t);
}

// Rows per strip: about four blocks per SM over all strips, at least 32 rows each.
static size_t dz_strip(size_t M, size_t N) {
    const size_t cols = ceil_div(N, (size_t)kDzCols);
    const size_t strips = std::max<size_t>(1, std::min<size_t>(ceil_div((size_t)608, cols), ceil_div(M, (size_t)32)));
    return std::max<size_t>(1, ceil_div(M, strips));
}

// ---------------------------------------------------------------- unaligned operands
//
// The tiled copies need rows on 16-byte boundaries.  An operand whose rows are not (an odd width, a
// view at an odd element) is first copied to rows that are, in the caller's workspace: one more pass
// over the operand, against products that read it from L2 many times.

static bool rows_aligned(const void* p, size_t rows, size_t ld) {
    return (uintptr_t)p % 16 == 0 && (rows < 2 || ld % 8 == 0);
}

static size_t padded(size_t cols) { return ceil_div(cols, (size_t)8) * 8; }

static size_t align_bytes(const void* p, size_t rows, size_t cols, size_t ld, sym_dtype_t t) {
    if (t == SYM_F32 || rows == 0 || cols == 0 || rows_aligned(p, rows, ld)) return 0;
    return ceil_div(rows * padded(cols) * 2, (size_t)256) * 256;
}

// 16-bit elements; a warp per row piece of 256, 8 a thread, so stores are 16 bytes and loads coalesced.
__global__ void __launch_bounds__(256) k_align_rows(const uint16_t* src, size_t ld, size_t rows, size_t cols,
                                                    uint16_t* dst, size_t ldd) {
    const size_t row = (size_t)blockIdx.x * 8 + threadIdx.x / 32;
    const size_t c0 = (size_t)blockIdx.y * 256 + (threadIdx.x % 32) * 8;
    if (row >= rows || c0 >= ldd) return;
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e < cols ? src[row * ld + c0 + e] : 0;
    uint4 o;
    o.x = v[0] | (uint32_t)v[1] << 16, o.y = v[2] | (uint32_t)v[3] << 16;
    o.z = v[4] | (uint32_t)v[5] << 16, o.w = v[6] | (uint32_t)v[7] << 16;
    *reinterpret_cast<uint4*>(dst + row * ldd + c0) = o;
}

// Points `p`, `ld` at an aligned copy of the operand if it is not aligned; `ws` moves past it.
static sym_status_t align_operand(const void*& p, size_t& ld, size_t rows, size_t cols, sym_dtype_t t, char*& ws,
                                  cudaStream_t st) {
    const size_t bytes = align_bytes(p, rows, cols, ld, t);
    if (!bytes) return SYM_OK;
    const size_t ldd = padded(cols);
    const size_t gx = ceil_div(rows, (size_t)8), gy = ceil_div(ldd, (size_t)256);
    if (gy > 65535) return SYM_ERR_UNSUPPORTED;
    k_align_rows<<<dim3((unsigned)gx, (unsigned)gy), 256, 0, st>>>((const uint16_t*)p, ld, rows, cols, (uint16_t*)ws,
                                                                   ldd);
    count_launch();
    SYM_CUDA(cudaGetLastError());
    p = ws;
    ld = ldd;
    ws += bytes;
    return SYM_OK;
}

struct BackwardPlan {
    size_t strip, strips, ldz, dz_off, partial_off, align_off, bytes;
};

static BackwardPlan backward_plan(size_t M, size_t N, size_t es, int act, size_t aligned) {
    BackwardPlan p{};
    p.strip = dz_strip(M, N);
    p.strips = std::max<size_t>(1, ceil_div(M, p.strip));
    p.ldz = ceil_div(N, (size_t)8) * 8;
    const size_t dz = act == SYM_ACT_NONE ? 0 : ceil_div(M * p.ldz * es, (size_t)256) * 256;
    p.partial_off = p.dz_off + dz;
    p.align_off = p.partial_off + ceil_div(p.strips * N * sizeof(float), (size_t)256) * 256;
    p.bytes = p.align_off + aligned;
    return p;
}

static bool good_act(int act) { return act >= SYM_ACT_NONE && act <= SYM_ACT_SILU; }

// Rows of `n` elements, `rows` of them `ld` apart: the bytes [first, past) they lie in.
struct Span {
    uintptr_t a, b;
};
static Span span(const void* p, size_t rows, size_t n, size_t ld, size_t es) {
    if (!p || !rows || !n) return {0, 0};
    return {(uintptr_t)p, (uintptr_t)p + ((rows - 1) * ld + n) * es};
}
static bool meet(Span x, Span y) { return x.a < y.b && y.a < x.b; }

// out = a b^T on the units of its type.  a_mn, b_mn: which index the operands are contiguous along
// (matmul_tc_bf16).  Without terms (kk = 0) the FMA kernel writes the epilogue of zero.
static sym_status_t matmul(const MatmulArgs& m, sym_dtype_t in, sym_dtype_t out, bool a_mn, bool b_mn,
                           cudaStream_t st) {
    if (in == SYM_F32 || m.kk == 0) return matmul_simt(m, in, out, st);
    int nt = 256;
    if (b_mn) nt = m.m <= 128 ? 128 : 256;
    else while (nt > 16 && m.m <= (size_t)nt / 2) nt /= 2;
    const uint32_t splits = 1;
    return in == SYM_BF16 ? matmul_tc_bf16(m, out, a_mn, b_mn, nt, splits, st)
                          : matmul_tc_f16(m, out, a_mn, b_mn, nt, splits, st);
}

}  // namespace symar

using namespace symar;

extern "C" {

size_t sym_linear_workspace(const void* x, size_t ldx, const void* w, size_t ldw, size_t M, size_t N, size_t K,
                            sym_dtype_t dtype) {
    return align_bytes(x, M, K, ldx, dtype) + align_bytes(w, N, K, ldw, dtype);
}

sym_status_t sym_linear(const void* x, size_t ldx, const void* w, size_t ldw, const void* bias, const void* residual,
                        size_t ldr, void* y, size_t ldy, void* pre, size_t ldp, size_t M, size_t N, size_t K,
                        sym_dtype_t dtype, sym_act_t act, void* workspace, size_t workspace_bytes,
                        sym_stream_t stream) {
    const size_t es = dtype_size(dtype);
    if (!es || !good_act(act)) return SYM_ERR_INVALID_ARG;
    if (M >= (1ull << 31) || N >= (1ull << 31) || K >= (1ull << 31)) return SYM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SYM_OK;
    if (!y || (K && (!x || !w))) return SYM_ERR_INVALID_ARG;
    if (ldx < K || ldw < K || ldy < N || (residual && ldr < N) || (pre && ldp < N)) return SYM_ERR_INVALID_ARG;
    for (const void* p : {x, w, bias, residual, (const void*)y, (const void*)pre})
        if ((uintptr_t)p % es) return SYM_ERR_INVALID_ARG;
    const Span sy = span(y, M, N, ldy, es), sp = span(pre, M, N, ldp, es);
    for (Span in : {span(x, M, K, ldx, es), span(w, N, K, ldw, es), span(bias, 1, N, N, es)})
        if (meet(sy, in) || meet(sp, in)) {
            set_last_error("sym_linear: an output overlaps an input");
            return SYM_ERR_INVALID_ARG;
        }
    const Span sr = span(residual, M, N, ldr, es);
    // y may be the residual itself (each element is read by the thread that writes it)
    if (meet(sy, sp) || meet(sp, sr) || (meet(sy, sr) && !(y == residual && ldy == ldr))) {
        set_last_error("sym_linear: y, pre and residual overlap");
        return SYM_ERR_INVALID_ARG;
    }
    const size_t need = sym_linear_workspace(x, ldx, w, ldw, M, N, K, dtype);
    if (workspace_bytes < need || (!workspace && workspace_bytes) || (uintptr_t)workspace % 256) {
        set_last_error("sym_linear: workspace missing, too small or not 256-byte aligned");
        return SYM_ERR_INVALID_ARG;
    }
    const Span sw = span(workspace, 1, need, need, 1);
    for (Span o : {sy, sp, sr, span(x, M, K, ldx, es), span(w, N, K, ldw, es), span(bias, 1, N, N, es)})
        if (meet(sw, o)) {
            set_last_error("sym_linear: the workspace overlaps a tensor");
            return SYM_ERR_INVALID_ARG;
        }
    cudaStream_t st = (cudaStream_t)stream;
    char* ws = (char*)workspace;
    sym_status_t s = align_operand(x, ldx, M, K, dtype, ws, st);
    if (s == SYM_OK) s = align_operand(w, ldw, N, K, dtype, ws, st);
    if (s != SYM_OK) return s;
    MatmulArgs m{x, w, ldx, 1, ldw, 1, M, N, K, bias, residual, ldr, pre, ldp, y, ldy, (int)act, false};
    return matmul(m, dtype, dtype, false, false, st);
}

size_t sym_linear_backward_workspace(const void* dy, size_t lddy, const void* x, size_t ldx, const void* w, size_t ldw,
                                     size_t M, size_t N, size_t K, sym_dtype_t dtype, sym_act_t act) {
    const size_t aligned = (act == SYM_ACT_NONE ? align_bytes(dy, M, N, lddy, dtype) : 0) +
                           align_bytes(x, M, K, ldx, dtype) + align_bytes(w, N, K, ldw, dtype);
    return backward_plan(M, N, dtype_size(dtype), act, aligned).bytes;
}

sym_status_t sym_linear_backward(const void* dy, size_t lddy, const void* x, size_t ldx, const void* w, size_t ldw,
                                 const void* pre, size_t ldp, void* dx, size_t lddx, void* dw, size_t lddw,
                                 void* dbias, size_t M, size_t N, size_t K, sym_dtype_t dtype,
                                 sym_dtype_t grad_dtype, sym_act_t act, int accumulate, void* workspace,
                                 size_t workspace_bytes, sym_stream_t stream) {
    const size_t es = dtype_size(dtype), gs = dtype_size(grad_dtype);
    if (!es || !gs || !good_act(act) || (grad_dtype != dtype && grad_dtype != SYM_F32)) return SYM_ERR_INVALID_ARG;
    if (M >= (1ull << 31) || N >= (1ull << 31) || K >= (1ull << 31)) return SYM_ERR_UNSUPPORTED;
    if (!dx && !dw && !dbias) return SYM_OK;
    if (M && N && (!dy || (act != SYM_ACT_NONE && !pre))) return SYM_ERR_INVALID_ARG;
    if ((dx && M && N && K && !w) || (dw && M && N && K && !x)) return SYM_ERR_INVALID_ARG;
    if ((dy && lddy < N) || (x && ldx < K) || (w && ldw < K) || (pre && ldp < N) || (dx && lddx < K) ||
        (dw && lddw < K))
        return SYM_ERR_INVALID_ARG;
    for (const void* p : {dy, x, w, pre, (const void*)dx})
        if ((uintptr_t)p % es) return SYM_ERR_INVALID_ARG;
    if ((uintptr_t)dw % gs || (uintptr_t)dbias % gs) return SYM_ERR_INVALID_ARG;
    const BackwardPlan bp =
        backward_plan(M, N, es, act,
                      sym_linear_backward_workspace(dy, lddy, x, ldx, w, ldw, M, N, K, dtype, act) -
                          backward_plan(M, N, es, act, 0).bytes);
    if (workspace_bytes < bp.bytes || (!workspace && bp.bytes) || (uintptr_t)workspace % 256) {
        set_last_error("sym_linear_backward: workspace missing, too small or not 256-byte aligned");
        return SYM_ERR_INVALID_ARG;
    }
    const Span outs[] = {span(dx, M, K, lddx, es), span(dw, N, K, lddw, gs), span(dbias, 1, N, N, gs),
                         span(workspace, 1, bp.bytes, bp.bytes, 1)};
    const Span ins[] = {span(dy, M, N, lddy, es), span(x, M, K, ldx, es), span(w, N, K, ldw, es),
                        span(pre, M, N, ldp, es)};
    for (int i = 0; i < 4; ++i) {
        for (Span in : ins)
            if (meet(outs[i], in)) {
                set_last_error("sym_linear_backward: an output overlaps an input");
                return SYM_ERR_INVALID_ARG;
            }
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) {
                set_last_error("sym_linear_backward: two outputs overlap");
                return SYM_ERR_INVALID_ARG;
            }
    }
    cudaStream_t st = (cudaStream_t)stream;
    char* ws = (char*)workspace;
    const void* dz = dy;
    size_t lddz = lddy;
    if (N && M && (act != SYM_ACT_NONE || dbias)) {
        DzArgs d{dy, lddy, act == SYM_ACT_NONE ? nullptr : pre, ldp, nullptr, 0, nullptr, M, N, bp.strip, (int)act};
        if (act != SYM_ACT_NONE && (dx || dw)) {
            d.dz = ws + bp.dz_off;
            d.ldz = bp.ldz;
            dz = d.dz;
            lddz = bp.ldz;
        }
        if (dbias) d.partial = (float*)(ws + bp.partial_off);
        const dim3 grid((unsigned)ceil_div(N, (size_t)kDzCols), (unsigned)bp.strips);
        switch (dtype) {
            case SYM_F32: k_linear_dz<float><<<grid, kDzThreads, 0, st>>>(d); break;
            case SYM_BF16: k_linear_dz<__nv_bfloat16><<<grid, kDzThreads, 0, st>>>(d); break;
            case SYM_F16: k_linear_dz<__half><<<grid, kDzThreads, 0, st>>>(d); break;
        }
        count_launch();
        SYM_CUDA(cudaGetLastError());
    }
    if (dbias && N) {
        const unsigned grid = (unsigned)ceil_div(N, (size_t)kDzThreads);
        const float* partial = (const float*)(ws + bp.partial_off);
        const size_t strips = M ? bp.strips : 0;
        switch (grad_dtype) {
            case SYM_F32:
                k_linear_db<float><<<grid, kDzThreads, 0, st>>>(partial, strips, N, dbias, accumulate != 0);
                break;
            case SYM_BF16:
                k_linear_db<__nv_bfloat16><<<grid, kDzThreads, 0, st>>>(partial, strips, N, dbias, accumulate != 0);
                break;
            case SYM_F16:
                k_linear_db<__half><<<grid, kDzThreads, 0, st>>>(partial, strips, N, dbias, accumulate != 0);
                break;
        }
        count_launch();
        SYM_CUDA(cudaGetLastError());
    }
    char* at = ws + bp.align_off;
    if ((dx && M && K) || (dw && N && K)) {
        sym_status_t s = SYM_OK;
        if (N && M && dz == dy) s = align_operand(dz, lddz, M, N, dtype, at, st);
        if (s == SYM_OK && dw && N && M) s = align_operand(x, ldx, M, K, dtype, at, st);
        if (s == SYM_OK && dx && N && M) s = align_operand(w, ldw, N, K, dtype, at, st);
        if (s != SYM_OK) return s;
    }
    if (dx && M && K) {
        // dX(m,k) = sum_n dZ(m,n) W(n,k)
        MatmulArgs m{dz, w, lddz, 1, 1, ldw, M, K, N, nullptr, nullptr, 0, nullptr, 0, dx, lddx, SYM_ACT_NONE, false};
        sym_status_t s = matmul(m, dtype, dtype, true, false, st);
        if (s != SYM_OK) return s;
    }
    if (dw && N && K) {
        // dW(n,k) = sum_m dZ(m,n) X(m,k)
        MatmulArgs m{dz, x, 1, lddz, 1, ldx, N, K, M, nullptr, nullptr, 0, nullptr, 0, dw, lddw, SYM_ACT_NONE,
                     accumulate != 0};
        sym_status_t s = matmul(m, dtype, grad_dtype, true, true, st);
        if (s != SYM_OK) return s;
    }
    return SYM_OK;
}

}  // extern "C"
