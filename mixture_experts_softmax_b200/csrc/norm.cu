// norm.cu -- RMSNorm and LayerNorm of rows, and their gradients with the reductions of the gain's
// and the bias's gradient.
//
//   y  = (x - m) r g + b        m = mean(x) (0 for RMSNorm), r = 1 / sqrt(mean((x - m)^2) + eps)
//   dx = r (h - mean(h) - xh mean(h xh)),   h = dy g,  xh = (x - m) r   (no mean(h) for RMSNorm)
//   dg = sum over rows of dy xh,   db = sum over rows of dy
//
// Both directions are bound by memory traffic (forward: x in, y out; backward: x and dy in, dx out).
// A row is held in registers from its load to its store, so it is read once: by one warp where
// it fits into the lanes' registers, else by a block.  The variance is taken around the mean, not as
// a difference of squares.  The backward pass runs a fixed number of blocks that walk over the rows
// and keep the columns' sums of dg and db in registers; each block leaves one row of partial sums
// and a second, short kernel adds those in block order, so results do not depend on scheduling.
// Rows too wide for the registers are read again from the caches instead, and their columns' sums
// taken by a kernel of their own.
#include "ops_common.cuh"

namespace moe {

namespace {

struct NormArgs {
    int T, d;
    const void *x, *gain, *bias;
    float eps;
    void *y;
    float *stats;               // [T, 2] mean, r; forward: written or nullptr, backward: read
    const void *dy;
    void *dx;
    float *part;                // [parts, 2, d] partial sums of dg and db
    float *dgain, *dbias;
};

constexpr int kRowWarps = 4;    // rows per block where a warp takes a row

// sum over the block's (or, WARP, the warp's) threads; buf: 32 floats, one per call between barriers
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *buf)
{
    v = warp_sum(v);
    if constexpr (WARP) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < (static_cast<int>(blockDim.x) >> 5) ? buf[lane] : 0.f);
}

template <class T, int N, int NV, bool LAYER, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 1024) norm_kernel(NormArgs a)
{
    __shared__ float buf[2][32];
    const int nt = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int row = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.T) return;
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.d;
    Vec<T, N> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * nt + tid) * N < a.d) v[i] = ld_vec<T, N>(x + (i * nt + tid) * N);
    float mean = 0.f;
    if constexpr (LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * nt + tid) * N < a.d) {
#pragma unroll
                for (int e = 0; e < N; ++e) s += to_f32(v[i].v[e]);
            }
        mean = row_sum<WARP>(s, buf[0]) / static_cast<float>(a.d);
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * nt + tid) * N < a.d) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float c = to_f32(v[i].v[e]) - mean;
                q = fmaf(c, c, q);
            }
        }
    const float r = 1.f / sqrtf(row_sum<WARP>(q, buf[1]) / static_cast<float>(a.d) + a.eps);
    if (tid == 0 && a.stats) *reinterpret_cast<float2 *>(a.stats + 2 * static_cast<size_t>(row)) = make_float2(mean, r);
    T *y = static_cast<T *>(a.y) + static_cast<size_t>(row) * a.d;
    const T *gain = static_cast<const T *>(a.gain), *bias = static_cast<const T *>(a.bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + tid) * N;
        if (c >= a.d) continue;
        Vec<T, N> g, b, o;
        if (gain) g = ld_vec<T, N>(gain + c);
        if (LAYER && bias) b = ld_vec<T, N>(bias + c);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            float h = (to_f32(v[i].v[e]) - mean) * r;
            if (gain) h *= to_f32(g.v[e]);
            if (LAYER && bias) h += to_f32(b.v[e]);
            o.v[e] = from_f32<T>(h);
        }
        st_vec<T, N>(y + c, o);
    }
}

// rows too wide for a block's registers: three passes, the second and third from the L2 cache
template <class T, bool LAYER>
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormArgs a)
{
    __shared__ float buf[2][32];
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(blockIdx.x) * a.d;
    T *y = static_cast<T *>(a.y) + static_cast<size_t>(blockIdx.x) * a.d;
    const T *gain = static_cast<const T *>(a.gain), *bias = static_cast<const T *>(a.bias);
    float mean = 0.f, s = 0.f;
    if constexpr (LAYER) {
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) s += to_f32(x[c]);
        mean = row_sum<false>(s, buf[0]) / static_cast<float>(a.d);
    }
    float q = 0.f;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        const float z = to_f32(x[c]) - mean;
        q = fmaf(z, z, q);
    }
    const float r = 1.f / sqrtf(row_sum<false>(q, buf[1]) / static_cast<float>(a.d) + a.eps);
    if (threadIdx.x == 0 && a.stats) {
        a.stats[2 * static_cast<size_t>(blockIdx.x)] = mean;
        a.stats[2 * static_cast<size_t>(blockIdx.x) + 1] = r;
    }
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        float h = (to_f32(x[c]) - mean) * r;
        if (gain) h *= to_f32(gain[c]);
        if (LAYER && bias) h += to_f32(bias[c]);
        y[c] = from_f32<T>(h);
    }
}

// ---- backward ------------------------------------------------------------------------

// the two row means of the gradient at once: one barrier a row (buffers by turns)
template <bool LAYER, bool WARP>
__device__ __forceinline__ float2 row_sums(float s0, float s1, float2 *buf)
{
    s1 = warp_sum(s1);
    if constexpr (LAYER) s0 = warp_sum(s0);
    if constexpr (WARP) return make_float2(s0, s1);
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(s0, s1);
    __syncthreads();
    const float2 w = lane < (static_cast<int>(blockDim.x) >> 5) ? buf[lane] : make_float2(0.f, 0.f);
    return make_float2(LAYER ? warp_sum(w.x) : 0.f, warp_sum(w.y));
}

template <class T, int N, int NV, bool LAYER, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 512) norm_grad_kernel(NormArgs a)
{
    __shared__ float2 buf[2][32];
    griddep_launch_dependents();   // the reduction's blocks wait for this kernel's end by themselves
    const int nt = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int rows = WARP ? kRowWarps : 1;
    const T *gain = static_cast<const T *>(a.gain);
    const float inv = 1.f / static_cast<float>(a.d);
    float dg[NV][N], db[LAYER ? NV : 1][LAYER ? N : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            dg[i][e] = 0.f;
            if constexpr (LAYER) db[i][e] = 0.f;
        }
    int parity = 0;
    for (int row = blockIdx.x * rows + (WARP ? threadIdx.x >> 5 : 0); row < a.T; row += gridDim.x * rows) {
        const size_t at = static_cast<size_t>(row) * a.d;
        const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
        T *dx = static_cast<T *>(a.dx) + at;
        Vec<T, N> xv[NV], dv[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * nt + tid) * N < a.d) {
                xv[i] = ld_vec<T, N>(x + (i * nt + tid) * N);
                dv[i] = ld_vec<T, N>(dy + (i * nt + tid) * N);
            }
        const float2 st = __ldg(reinterpret_cast<const float2 *>(a.stats) + row);
        const float mean = LAYER ? st.x : 0.f, r = st.y;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + tid) * N;
            if (c >= a.d) continue;
            Vec<T, N> g;
            if (gain) g = ld_vec<T, N>(gain + c);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float dyv = to_f32(dv[i].v[e]), xh = (to_f32(xv[i].v[e]) - mean) * r;
                const float h = gain ? dyv * to_f32(g.v[e]) : dyv;
                s1 = fmaf(h, xh, s1);
                dg[i][e] = fmaf(dyv, xh, dg[i][e]);
                if constexpr (LAYER) {
                    s0 += h;
                    db[i][e] += dyv;
                }
            }
        }
        const float2 s = row_sums<LAYER, WARP>(s0, s1, buf[parity]);
        parity ^= 1;
        const float m0 = s.x * inv, m1 = s.y * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + tid) * N;
            if (c >= a.d) continue;
            Vec<T, N> g, o;
            if (gain) g = ld_vec<T, N>(gain + c);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float xh = (to_f32(xv[i].v[e]) - mean) * r;
                float h = to_f32(dv[i].v[e]);
                if (gain) h *= to_f32(g.v[e]);
                o.v[e] = from_f32<T>(r * (fmaf(-xh, m1, h) - m0));
            }
            st_vec<T, N>(dx + c, o);
        }
    }
    // the block's sums, one row of [2, d]; a warp per row: the warps' sums joined in order first
    float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
    if constexpr (WARP) {
        __shared__ float sum[LAYER ? 2 : 1][32 * NV * N];
        for (int w = 0; w < kRowWarps; ++w) {
            if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const int c = (i * 32 + tid) * N + e;
                        sum[0][c] = w ? sum[0][c] + dg[i][e] : dg[i][e];
                        if constexpr (LAYER) sum[1][c] = w ? sum[1][c] + db[i][e] : db[i][e];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
            part[c] = sum[0][c];
            if constexpr (LAYER) part[a.d + c] = sum[1][c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + tid) * N;
            if (c >= a.d) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                part[c + e] = dg[i][e];
                if constexpr (LAYER) part[a.d + c + e] = db[i][e];
            }
        }
    }
}

// dx of rows too wide for the registers
template <class T, bool LAYER>
__global__ void __launch_bounds__(1024) norm_grad_wide_kernel(NormArgs a)
{
    __shared__ float2 buf[32];
    const size_t at = static_cast<size_t>(blockIdx.x) * a.d;
    const T *x = static_cast<const T *>(a.x) + at, *dy = static_cast<const T *>(a.dy) + at;
    const T *gain = static_cast<const T *>(a.gain);
    T *dx = static_cast<T *>(a.dx) + at;
    const float mean = LAYER ? a.stats[2 * static_cast<size_t>(blockIdx.x)] : 0.f;
    const float r = a.stats[2 * static_cast<size_t>(blockIdx.x) + 1];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        const float h = gain ? to_f32(dy[c]) * to_f32(gain[c]) : to_f32(dy[c]);
        s0 += h;
        s1 = fmaf(h, (to_f32(x[c]) - mean) * r, s1);
    }
    const float2 s = row_sums<LAYER, false>(s0, s1, buf);
    const float inv = 1.f / static_cast<float>(a.d), m0 = s.x * inv, m1 = s.y * inv;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        const float h = gain ? to_f32(dy[c]) * to_f32(gain[c]) : to_f32(dy[c]);
        dx[c] = from_f32<T>(r * (fmaf(-(to_f32(x[c]) - mean) * r, m1, h) - m0));
    }
}

// partial column sums of those rows: a block takes 32 columns of every gridDim.y-th group of 8 rows
template <class T, bool LAYER>
__global__ void __launch_bounds__(256) norm_grad_columns_kernel(NormArgs a)
{
    __shared__ float red[2][8][32];
    griddep_launch_dependents();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float g = 0.f, b = 0.f;
    if (c < a.d)
        for (int row = blockIdx.y * 8 + threadIdx.y; row < a.T; row += gridDim.y * 8) {
            const size_t at = static_cast<size_t>(row) * a.d + c;
            const float dyv = to_f32(static_cast<const T *>(a.dy)[at]);
            const float mean = LAYER ? a.stats[2 * static_cast<size_t>(row)] : 0.f;
            g = fmaf(dyv, (to_f32(static_cast<const T *>(a.x)[at]) - mean) * a.stats[2 * static_cast<size_t>(row) + 1], g);
            b += dyv;
        }
    red[0][threadIdx.y][threadIdx.x] = g;
    red[1][threadIdx.y][threadIdx.x] = b;
    __syncthreads();
    if (threadIdx.y >= (LAYER ? 2 : 1) || c >= a.d) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[threadIdx.y][w][threadIdx.x];
    a.part[(static_cast<size_t>(blockIdx.y) * 2 + threadIdx.y) * a.d + c] = s;
}

// dgain / dbias = the sum of the blocks' partial rows, in block order within each of 8 strands
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float *part, int parts, int d, float *dgain, float *dbias)
{
    __shared__ float red[8][32];
    griddep_wait();
    float *out = blockIdx.y ? dbias : dgain;
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (!out) return;   // the whole block
    float s = 0.f;
    if (c < d) {
        const float *p = part + static_cast<size_t>(blockIdx.y) * d + c;
#pragma unroll 8
        for (int i = threadIdx.y; i < parts; i += 8) s += __ldcg(p + static_cast<size_t>(i) * 2 * d);
    }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= d) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += red[w][threadIdx.x];
    out[c] = t;
}

// ---- host -------------------------------------------------------------------------------

// most rows of partial sums a backward call keeps: the blocks of the widest launch
int most_parts(int d) { return d <= 4096 ? 4 * kSms : d <= 16384 ? 2 * kSms : 64; }

int parts_for(int T, int d)
{
    const int most = most_parts(d);
    return T < most ? T : most;
}

int round32(int v) { return (v + 31) / 32 * 32; }

template <class T, int N, bool LAYER>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t s)
{
    constexpr int NW = N > 2 ? 4 : 8;                 // vectors a thread, by their size
    const int nvec = a.d / N;
    if (nvec <= 32 * NW)
        return op_launch(norm_kernel<T, N, NW, LAYER, true>, dim3((a.T + kRowWarps - 1) / kRowWarps), dim3(kRowWarps * 32), 0,
                         s, false, 1, a);
    if (nvec <= 1024 * NW)
        return op_launch(norm_kernel<T, N, NW, LAYER, false>, dim3(a.T), dim3(round32((nvec + NW - 1) / NW)), 0, s, false, 1,
                         a);
    if constexpr (N > 2) {
        if (nvec <= 1024 * 8)
            return op_launch(norm_kernel<T, N, 8, LAYER, false>, dim3(a.T), dim3(round32((nvec + 7) / 8)), 0, s, false, 1, a);
    }
    return op_launch(norm_wide_kernel<T, LAYER>, dim3(a.T), dim3(1024), 0, s, false, 1, a);
}

template <class T, int N, bool LAYER>
cudaError_t launch_norm_grad(const NormArgs &a, cudaStream_t s)
{
    constexpr int NW = N > 2 ? 4 : 8;
    const int nvec = a.d / N;
    int parts = parts_for(a.T, a.d);
    cudaError_t e;
    if (nvec <= 32 * NW) {
        const int blocks = (a.T + kRowWarps - 1) / kRowWarps;
        parts = blocks < parts ? blocks : parts;
        e = op_launch(norm_grad_kernel<T, N, NW, LAYER, true>, dim3(parts), dim3(kRowWarps * 32), 0, s, false, 1, a);
    } else if (nvec <= 512 * NW) {
        e = op_launch(norm_grad_kernel<T, N, NW, LAYER, false>, dim3(parts), dim3(round32((nvec + NW - 1) / NW)), 0, s, false,
                      1, a);
    } else {
        e = op_launch(norm_grad_wide_kernel<T, LAYER>, dim3(a.T), dim3(1024), 0, s, false, 1, a);
        if (e != cudaSuccess || (!a.dgain && !a.dbias)) return e;
        const int groups = (a.T + 7) / 8;
        parts = groups < parts ? groups : parts;
        parts = parts < 64 ? parts : 64;
        e = op_launch(norm_grad_columns_kernel<T, LAYER>, dim3((a.d + 31) / 32, parts), dim3(32, 8), 0, s, false, 1, a);
    }
    if (e != cudaSuccess || (!a.dgain && !a.dbias)) return e;
    return op_launch(norm_reduce_kernel, dim3((a.d + 31) / 32, a.dbias ? 2 : 1), dim3(32, 8), 0, s, true, 1,
                     static_cast<const float *>(a.part), parts, a.d, a.dgain, a.dbias);
}

template <class T, int N>
cudaError_t norm_by_kind(int kind, bool grad, const NormArgs &a, cudaStream_t s)
{
    if (kind == MOE_NORM_LAYER) return grad ? launch_norm_grad<T, N, true>(a, s) : launch_norm<T, N, true>(a, s);
    return grad ? launch_norm_grad<T, N, false>(a, s) : launch_norm<T, N, false>(a, s);
}

template <class T>
cudaError_t norm_by_width(int kind, bool grad, const NormArgs &a, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    if (a.d % W == 0) return norm_by_kind<T, W>(kind, grad, a, s);
    if (a.d % 2 == 0) return norm_by_kind<T, 2>(kind, grad, a, s);
    return norm_by_kind<T, 1>(kind, grad, a, s);
}

int norm_dispatch(int kind, int dtype, bool grad, const NormArgs &a, cudaStream_t s)
{
    const cudaError_t e = dtype == MOE_F32   ? norm_by_width<float>(kind, grad, a, s)
                          : dtype == MOE_F16 ? norm_by_width<__half>(kind, grad, a, s)
                                             : norm_by_width<__nv_bfloat16>(kind, grad, a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

bool norm_sizes_ok(int T, int d) { return T >= 0 && T <= MOE_MAX_TOKENS && d >= 1 && d <= 65536; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_norm_forward(int kind, int dtype, int T, int d, const void *x, const void *gain,
                                        const void *bias, float eps, void *y, float *stats, void *stream)
{
    if ((kind != MOE_NORM_RMS && kind != MOE_NORM_LAYER) || !dtype_known(dtype) || !norm_sizes_ok(T, d)) return MOE_EINVAL;
    if (!(eps >= 0.f) || (bias && kind != MOE_NORM_LAYER)) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!op_ptr(x) || !op_ptr(y) || !op_aligned16(gain) || !op_aligned16(bias) || !op_aligned16(stats)) return MOE_EINVAL;
    const size_t row = static_cast<size_t>(d) * dtype_size(dtype), all = T * row, sb = static_cast<size_t>(T) * 8;
    if (op_overlap(x, all, y, all) || op_overlap(gain, row, y, all) || op_overlap(bias, row, y, all) ||
        op_overlap(stats, sb, y, all) || op_overlap(stats, sb, x, all) || op_overlap(stats, sb, gain, row) ||
        op_overlap(stats, sb, bias, row))
        return MOE_EINVAL;
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    NormArgs a{T, d, x, gain, bias, eps, y, stats};
    return norm_dispatch(kind, dtype, false, a, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API long long moe_norm_workspace(int T, int d)
{
    if (!norm_sizes_ok(T, d)) return MOE_EINVAL;
    return static_cast<long long>(parts_for(T, d)) * 2 * d * 4;
}

extern "C" MOE_API int moe_norm_backward(int kind, int dtype, int T, int d, const void *x, const void *gain,
                                         const float *stats, const void *dy, void *dx, float *dgain, float *dbias,
                                         void *workspace, void *stream)
{
    if ((kind != MOE_NORM_RMS && kind != MOE_NORM_LAYER) || !dtype_known(dtype) || !norm_sizes_ok(T, d)) return MOE_EINVAL;
    if (dbias && kind != MOE_NORM_LAYER) return MOE_EINVAL;
    if (!op_aligned16(dgain) || !op_aligned16(dbias) || !op_aligned16(gain)) return MOE_EINVAL;
    const size_t row = static_cast<size_t>(d) * dtype_size(dtype), all = T * row, sb = static_cast<size_t>(T) * 8;
    const size_t gb = static_cast<size_t>(d) * 4, wb = static_cast<size_t>(parts_for(T, d)) * 2 * d * 4;
    if (op_overlap(dgain, gb, dbias, gb)) return MOE_EINVAL;
    if (T > 0) {
        if (!op_ptr(x) || !op_ptr(stats) || !op_ptr(dy) || !op_ptr(dx) || !op_ptr(workspace)) return MOE_EINVAL;
        const struct {
            const void *p;
            size_t n;
        } in[] = {{x, all}, {gain, row}, {stats, sb}, {dy, all}}, out[] = {{dx, all}, {dgain, gb}, {dbias, gb}, {workspace, wb}};
        for (int i = 0; i < 4; ++i) {
            for (const auto &b : in)
                if (op_overlap(out[i].p, out[i].n, b.p, b.n)) return MOE_EINVAL;
            for (int j = 0; j < i; ++j)
                if (op_overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MOE_EINVAL;
        }
    }
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no rows: the sums are 0
        if (dgain && cudaMemsetAsync(dgain, 0, gb, s) != cudaSuccess) return MOE_ECUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, gb, s) != cudaSuccess) return MOE_ECUDA;
        return MOE_OK;
    }
    NormArgs a{T, d, x, gain, nullptr, 0.f, nullptr, const_cast<float *>(stats), dy, dx, static_cast<float *>(workspace),
               dgain, dbias};
    return norm_dispatch(kind, dtype, true, a, s);
}
