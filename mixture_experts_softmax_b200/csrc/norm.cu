// norm.cu -- RMSNorm and LayerNorm of rows, and their gradients with the reductions of the gain's
// and the bias's gradient.
//
//   y  = (x - m) r g + b        m = mean(x) (0 for RMSNorm), r = 1 / sqrt(mean((x - m)^2) + eps)
//   dx = r (h - mean(h) - xh mean(h xh)),   h = dy g,  xh = (x - m) r   (no mean(h) for RMSNorm)
//   dg = sum over rows of dy xh,   db = sum over rows of dy
//
// Both directions are bound by memory traffic (forward: x in, y out; backward: x and dy in, dx out);
// a row is read once and held until its result is written: in registers, or in a ring of shared memory
// that asynchronous copies fill some rows ahead.  The variance is taken around the mean, not as a
// difference of squares, and the walk that takes it also corrects the mean.  The backward pass runs a fixed number of blocks that walk over the rows
// and keep the columns' sums of dg and db in registers; each block leaves one row of partial sums
// and a second, short kernel adds those in block order, so results do not depend on scheduling.
//
// Rows whose width is no multiple of 16 bytes still move in 16-byte vectors: rows r, r + P, r + 2 P ...
// (P = 16 bytes over their common divisor with the row) begin at the same place within a vector,
// so a block that takes rows of one such class has its columns at fixed places.
// Rows too wide for a block's registers are read again from the caches instead, with the columns' sums in shared memory
// or, wider still, taken by a kernel of their own.
//
// Measured on a B200: LayerNorm of 16,383 x 2560 fp32 53 to 57 us (91 to 98% of the copy bandwidth), of 8192 x 1537 fp16 22.5 us
// (34%), RMSNorm of the same 18.4; RMSNorm gradient of 8192 x 6144 bf16 66 us (71%: about 60 us for the rows, at 48% of all issue
// slots, and the reduction), LayerNorm gradient of 5003 x 1537 fp16 30 us (24%: each block waits for one row's sums after
// the other, some 2700 cycles a row).
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

// two row sums at once (the first for LayerNorm only), at one barrier
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

// The walk around a pivot near the mean (the rounded sum over the rounded 1 / d) leaves t = sum(x - pivot) and q = sum((x - pivot)^2);
// with m = t / d the mean is pivot + m and the variance q / d - m^2.  m is some roundings of the pivot, so nothing cancels,
// and a row of equal values gets its value as mean and results of 0 at any width.  The second sum costs up to 8%: 38.0 to
// 39.4 us at 8192 x 6144 bf16, 22.6 to 24.5 at 4097 x 2051 fp32, 52.7 to 52.8 at 16,383 x 2560 fp32.
__device__ __forceinline__ float corrected(float2 tq, float inv, float &mean)
{
    const float m = tq.x * inv, v = tq.y * inv, var = fmaf(-m, m, v);
    mean += m;
    if (v == __int_as_float(0x7f800000)) return v;   // squares beyond fp32, of m too perhaps; below that m^2 <= v
    return var < 0.f ? 0.f : var;                    // nan stays
}

template <class T>
__device__ __forceinline__ void st_words(T *p, const uint32_t (&w)[4])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// where the vectors of a row are: column c of a row is element c + shift of the vectors that hold it
template <class T>
struct Place {
    static constexpr int W = 16 / sizeof(T);
    int d, shift, nv;           // nv: vectors that hold a row
    // the first vector may begin with the row before's end, the last may end behind this row
    __device__ __forceinline__ bool inner(int v) const { return v * W >= shift && (v + 1) * W <= shift + d; }
    __device__ __forceinline__ bool has(int v, int e) const { return v * W + e >= shift && v * W + e < shift + d; }
    __device__ __forceinline__ int bytes(int v) const
    {
        const int n = (shift + d - v * W) * static_cast<int>(sizeof(T));
        return n < 16 ? n : 16;
    }
    // the bits of vector v that are this row's
    __device__ __forceinline__ uint4 keep(int v) const
    {
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m[j] = W == 4 ? (has(v, j) ? 0xffffffffu : 0u)
                          : (has(v, 2 * j) ? 0xffffu : 0u) | (has(v, 2 * j + 1) ? 0xffff0000u : 0u);
        return make_uint4(m[0], m[1], m[2], m[3]);
    }
    // vector v of a row whose first vector is at p; elements outside the row are 0 (and not read)
    __device__ __forceinline__ uint4 load(const T *p, int v) const
    {
        if (inner(v)) return __ldg(reinterpret_cast<const uint4 *>(p + v * W));
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (W == 4) {
                w[j] = has(v, j) ? __float_as_uint(p[v * W + j]) : 0u;
            } else {
                const uint16_t *h = reinterpret_cast<const uint16_t *>(p + v * W) + 2 * j;
                w[j] = (has(v, 2 * j) ? h[0] : 0u) | (has(v, 2 * j + 1) ? static_cast<uint32_t>(h[1]) << 16 : 0u);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the elements of vector v, at p, that are this row's
    __device__ __forceinline__ void store_part(T *p, int v, const uint32_t (&w)[4]) const
    {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if (!has(v, e)) continue;
            if constexpr (W == 4) p[e] = __uint_as_float(w[e]);
            else reinterpret_cast<uint16_t *>(p)[e] = static_cast<uint16_t>(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
        }
    }
};

__device__ __forceinline__ uint4 bits_and(uint4 a, uint4 k) { return make_uint4(a.x & k.x, a.y & k.y, a.z & k.z, a.w & k.w); }

// sum of a pair's halves
__device__ __forceinline__ float both(F2 a)
{
    const float2 f = unpack(a);
    return f.x + f.y;
}

// rows of whole vectors, held in registers
template <class T, int NV, bool LAYER, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 1024) norm_kernel(NormArgs a)
{
    op_begin();
    constexpr int W = 16 / sizeof(T);
    __shared__ float buf[32];
    __shared__ float2 buf2[32];
    const int nt = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x, nv = a.d / W;
    const int row = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.T) return;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.d) + tid;
    uint4 u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i * nt + tid < nv) u[i] = __ldg(x + i * nt);
    const float inv = 1.f / static_cast<float>(a.d);
    float mean = 0.f;
    if constexpr (LAYER) {
        F2 s = f2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * nt + tid < nv) {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) s = add2(s, pair_of<T>(u[i], e));
            }
        mean = row_sum<WARP>(both(s), buf) * inv;
    }
    F2 nm = f2(-mean, -mean), t = f2(0.f, 0.f), q = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i * nt + tid < nv) {
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                F2 c = pair_of<T>(u[i], e);
                if constexpr (LAYER) {
                    c = add2(c, nm);
                    t = add2(t, c);
                }
                q = fma2(c, c, q);
            }
        }
    const float2 tq = row_sums<LAYER, WARP>(both(t), both(q), buf2);
    const float var = LAYER ? corrected(tq, inv, mean) : tq.y * inv, r = 1.f / sqrtf(var + a.eps);
    nm = f2(-mean, -mean);
    if (tid == 0 && a.stats) *reinterpret_cast<float2 *>(a.stats + 2 * static_cast<size_t>(row)) = make_float2(mean, r);
    const F2 rr = f2(r, r);
    T *y = static_cast<T *>(a.y) + static_cast<size_t>(row) * a.d;
    const uint4 *gain = static_cast<const uint4 *>(a.gain), *bias = static_cast<const uint4 *>(a.bias);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * nt + tid;
        if (v >= nv) continue;
        uint4 g, b;
        if (gain) g = __ldg(gain + v);
        if (LAYER && bias) b = __ldg(bias + v);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            F2 h = pair_of<T>(u[i], e);
            if constexpr (LAYER) h = add2(h, nm);
            h = mul2(h, rr);
            if (LAYER && bias) h = gain ? fma2(h, pair_of<T>(g, e), pair_of<T>(b, e)) : add2(h, pair_of<T>(b, e));
            else if (gain) h = mul2(h, pair_of<T>(g, e));
            set_pair<T>(o, e, h);
        }
        st_words(y + v * W, o);
    }
}

// rows too wide for the kernels above: three walks, the second and third from the caches
template <class T, bool LAYER>
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormArgs a)
{
    op_begin();
    constexpr int W = 16 / sizeof(T);
    __shared__ float buf[32];
    __shared__ float2 buf2[32];
    const size_t first = static_cast<size_t>(blockIdx.x) * a.d;
    Place<T> at{a.d, static_cast<int>(first % W), 0};
    at.nv = (at.shift + a.d + W - 1) / W;
    const T *x = static_cast<const T *>(a.x) + first - at.shift;
    T *y = static_cast<T *>(a.y) + first - at.shift;
    const T *gain = static_cast<const T *>(a.gain), *bias = static_cast<const T *>(a.bias);
    const float inv = 1.f / static_cast<float>(a.d);
    float mean = 0.f;
    if constexpr (LAYER) {
        F2 s = f2(0.f, 0.f);
        for (int v = threadIdx.x; v < at.nv; v += blockDim.x) {
            const uint4 u = at.load(x, v);
#pragma unroll
            for (int e = 0; e < W / 2; ++e) s = add2(s, pair_of<T>(u, e));
        }
        mean = row_sum<false>(both(s), buf) * inv;
    }
    F2 t = f2(0.f, 0.f), q = f2(0.f, 0.f);
    for (int v = threadIdx.x; v < at.nv; v += blockDim.x) {
        const uint4 u = at.load(x, v);
        const bool in = at.inner(v);
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            F2 c = pair_of<T>(u, e);
            if constexpr (LAYER) {
                c = add2(c, f2(in || at.has(v, 2 * e) ? -mean : 0.f, in || at.has(v, 2 * e + 1) ? -mean : 0.f));
                t = add2(t, c);
            }
            q = fma2(c, c, q);
        }
    }
    const float2 tq = row_sums<LAYER, false>(both(t), both(q), buf2);
    const float var = LAYER ? corrected(tq, inv, mean) : tq.y * inv, r = 1.f / sqrtf(var + a.eps);
    if (threadIdx.x == 0 && a.stats)
        *reinterpret_cast<float2 *>(a.stats + 2 * static_cast<size_t>(blockIdx.x)) = make_float2(mean, r);
    for (int v = threadIdx.x; v < at.nv; v += blockDim.x) {
        const uint4 u = at.load(x, v);
        const int c0 = v * W - at.shift;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            const int c = min(max(c0 + 2 * e, 0), a.d - 1), c1 = min(max(c0 + 2 * e + 1, 0), a.d - 1);
            F2 h = mul2(add2(pair_of<T>(u, e), f2(-mean, -mean)), f2(r, r));
            if (gain) h = mul2(h, f2(to_f32(__ldg(gain + c)), to_f32(__ldg(gain + c1))));
            if (LAYER && bias) h = add2(h, f2(to_f32(__ldg(bias + c)), to_f32(__ldg(bias + c1))));
            set_pair<T>(o, e, h);
        }
        if (at.inner(v)) st_words(y + v * W, o);
        else at.store_part(y + v * W, v, o);
    }
}

// ---- rows through a ring of shared memory ---------------------------------------------------

__device__ __forceinline__ void row_copy16(uint32_t dst, const void *src, int bytes)
{
    // bytes (1 .. 16) are read, the rest of the 16 is filled with 0
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void row_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void row_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 row_lds(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
constexpr int kRowStages = 3, kGradStages = 2;   // rows of a ring, forward and backward
constexpr int kGradThreads = 384;                // two blocks an SM leave each thread 85 registers

// The rows of one block (or warp): row, row + step, ... of one class, n of them.
template <class T, bool WARP>
struct Rows {
    static constexpr int W = 16 / sizeof(T);
    Place<T> at;
    int nt, tid;                // threads of a row
    int row, step, n;
    __device__ __forceinline__ Rows(int T_, int d, int P)
    {
        nt = WARP ? 32 : blockDim.x;
        tid = WARP ? threadIdx.x & 31 : threadIdx.x;
        const int cls = blockIdx.x % P, per = WARP ? kRowWarps : 1;
        at.d = d;
        at.shift = static_cast<int>(static_cast<long>(cls) * d % W);
        at.nv = (at.shift + d + W - 1) / W;
        row = cls + P * static_cast<int>((blockIdx.x / P) * per + (WARP ? threadIdx.x >> 5 : 0));
        step = static_cast<int>(gridDim.x / P) * per * P;
        n = row < T_ ? (T_ - 1 - row) / step + 1 : 0;
    }
    // this thread's first vector of the first row
    template <class V> __device__ __forceinline__ V *start(V *p) const
    {
        return p + (static_cast<long>(row) * at.d - at.shift + tid * W);
    }
    // one value per column (gain, bias) at the columns' places, fill where there is none
    __device__ __forceinline__ void columns(char *dst, const void *src, float fill) const
    {
        T *out = reinterpret_cast<T *>(dst);
        const int n = at.nv * W, step = blockDim.x;
        for (int i0 = threadIdx.x; i0 < n; i0 += 8 * step) {
            T v[8];   // in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = i0 + k * step - at.shift;
                v[k] = src && c >= 0 && c < at.d ? __ldg(static_cast<const T *>(src) + c) : from_f32<T>(fill);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + k * step < n) out[i0 + k * step] = v[k];
        }
    }
};

// the forward pass for rows that are no multiple of 16 bytes
template <class T, int NV, bool LAYER, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 512) norm_shift_kernel(NormArgs a, int P)
{
    op_begin();
    constexpr int W = 16 / sizeof(T);
    extern __shared__ __align__(16) char row_smem[];
    __shared__ float buf[2][32];
    __shared__ float2 buf2[2][32];
    const Rows<T, WARP> rows(a.T, a.d, P);
    const Place<T> &at = rows.at;
    const int nt = rows.nt, tid = rows.tid, plane = nt * NV * 16;
    rows.columns(row_smem, a.gain, 1.f);
    if (LAYER) rows.columns(row_smem + plane, a.bias, 0.f);
    const uint32_t gains = smem_u32(row_smem) + tid * 16, biases = gains + plane;
    const uint32_t ring = gains + (LAYER ? 2 : 1) * plane + (WARP ? (threadIdx.x >> 5) * (kRowStages * plane) : 0);
    __syncthreads();
    const T *src = rows.start(static_cast<const T *>(a.x));
    T *dst = rows.start(static_cast<T *>(a.y));
    const long stride = static_cast<long>(rows.step) * a.d;
    int bytes[NV];              // 0: no such vector
    bool whole[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * nt + tid;
        bytes[i] = v < at.nv ? at.bytes(v) : 0;
        whole[i] = at.inner(v);
    }
    int left = rows.n, put = 0;
    auto issue = [&]() {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (bytes[i]) row_copy16(ring + put * plane + i * nt * 16, src + i * nt * W, bytes[i]);
        }
        row_commit();
        --left;
        src += stride;
        put = put + 1 == kRowStages ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < kRowStages - 1; ++i) issue();
    const float inv = 1.f / static_cast<float>(a.d);
    float2 *stats = reinterpret_cast<float2 *>(a.stats) + rows.row;
    int get = 0, parity = 0;
    for (int j = 0; j < rows.n; ++j) {
        issue();
        row_wait<kRowStages - 1>();
        const uint32_t st = ring + get * plane;
        get = get + 1 == kRowStages ? 0 : get + 1;
        uint4 u[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            u[i] = bytes[i] ? row_lds(st + i * nt * 16) : make_uint4(0, 0, 0, 0);
            if (bytes[i] && !whole[i]) u[i] = bits_and(u[i], at.keep(i * nt + tid));
        }
        float mean = 0.f;
        if constexpr (LAYER) {
            F2 s = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < W / 2; ++e) s = add2(s, pair_of<T>(u[i], e));
            mean = row_sum<WARP>(both(s), buf[parity]) * inv;
        }
        F2 nm = f2(-mean, -mean), t = f2(0.f, 0.f), q = f2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!bytes[i]) continue;
            const int v = i * nt + tid;
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                F2 c = pair_of<T>(u[i], e);
                if constexpr (LAYER) {
                    c = add2(c, whole[i] ? nm : f2(at.has(v, 2 * e) ? -mean : 0.f, at.has(v, 2 * e + 1) ? -mean : 0.f));
                    t = add2(t, c);
                }
                q = fma2(c, c, q);
            }
        }
        const float2 tq = row_sums<LAYER, WARP>(both(t), both(q), buf2[parity]);
        const float var = LAYER ? corrected(tq, inv, mean) : tq.y * inv, r = 1.f / sqrtf(var + a.eps);
        nm = f2(-mean, -mean);
        parity ^= 1;
        if (tid == 0 && a.stats) *stats = make_float2(mean, r);
        stats += rows.step;
        const F2 rr = f2(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!bytes[i]) continue;
            const uint4 g = row_lds(gains + i * nt * 16);
            uint4 b;
            if constexpr (LAYER) b = row_lds(biases + i * nt * 16);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const F2 x = pair_of<T>(u[i], e);
                if constexpr (LAYER) set_pair<T>(o, e, fma2(mul2(add2(x, nm), rr), pair_of<T>(g, e), pair_of<T>(b, e)));
                else set_pair<T>(o, e, mul2(mul2(x, rr), pair_of<T>(g, e)));
            }
            T *p = dst + i * nt * W;
            if (whole[i]) st_words(p, o);
            else at.store_part(p, i * nt + tid, o);
        }
        dst += stride;
    }
}

// ---- backward ------------------------------------------------------------------------

__device__ __forceinline__ float half_of(F2 a, int e) { return e & 1 ? unpack(a).y : unpack(a).x; }

// With h = dy g:  dx = r h - r mean(h) - xh (r mean(h xh)).  SHIFT: rows that are no multiple of 16 bytes.
// The arithmetic (about 18 instructions an element, half of them conversions) runs close to the
// memory traffic, so what a thread needs again after the row's sums it keeps as fp32 pairs where the
// registers allow it.
template <class T, int NV, bool LAYER, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : NV > 2 ? 512 : kGradThreads, WARP ? 5 : NV > 2 ? 1 : 2)
    norm_grad_kernel(NormArgs a, int P)
{
    constexpr int W = 16 / sizeof(T);
    constexpr bool kHold = NV * W <= 8 || (NV * W <= 16 && !LAYER);
    extern __shared__ __align__(16) char row_smem[];
    __shared__ float2 buf[2][32];
    op_begin();
    const Rows<T, WARP> rows(a.T, a.d, P);
    const Place<T> &at = rows.at;
    const int nt = rows.nt, tid = rows.tid, plane = nt * NV * 16;
    // the gain: shifted rows take it from shared memory, others through the L1 cache, which leaves the rings more room
    const uint32_t gains = smem_u32(row_smem) + tid * 16;
    const uint4 *gain16 = static_cast<const uint4 *>(a.gain) + tid;
    if (SHIFT) {
        rows.columns(row_smem, a.gain, 1.f);
        __syncthreads();
    }
    auto gain_of = [&](int i) {
        if (SHIFT) return row_lds(gains + i * nt * 16);
        if (a.gain) return __ldg(gain16 + i * nt);
        const uint32_t one = W == 4 ? __float_as_uint(1.f) : pack2<T>(1.f, 1.f);
        return make_uint4(one, one, one, one);
    };
    const uint32_t ring = gains + (SHIFT ? plane : 0) + (WARP ? (threadIdx.x >> 5) * (kGradStages * 2 * plane) : 0);
    const T *xs = rows.start(static_cast<const T *>(a.x)), *ds = rows.start(static_cast<const T *>(a.dy));
    T *dst = rows.start(static_cast<T *>(a.dx));
    const long stride = static_cast<long>(rows.step) * a.d;
    int bytes[NV];              // 0: no such vector
    bool whole[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * nt + tid;
        bytes[i] = v < at.nv ? (SHIFT ? at.bytes(v) : 16) : 0;
        whole[i] = !SHIFT || at.inner(v);
    }
    const float2 *stats = reinterpret_cast<const float2 *>(a.stats) + rows.row;
    int left = rows.n, put = 0;
    // the next row's copies, and its statistics
    auto issue = [&]() {
        float2 st = make_float2(0.f, 0.f);
        if (left > 0) {
            st = __ldg(stats);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!bytes[i]) continue;
                const uint32_t to = ring + put * (2 * plane) + i * nt * 16;
                row_copy16(to, xs + i * nt * W, SHIFT ? bytes[i] : 16);
                row_copy16(to + plane, ds + i * nt * W, SHIFT ? bytes[i] : 16);
            }
        }
        row_commit();
        --left;
        stats += rows.step;
        xs += stride;
        ds += stride;
        put = put + 1 == kGradStages ? 0 : put + 1;
        return st;
    };
    static_assert(kGradStages == 2, "one row's statistics are on their way");
    float2 coming = issue();
    const float inv = 1.f / static_cast<float>(a.d);
    F2 dg[NV][W / 2], db[LAYER ? NV : 1][W / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            dg[i][e] = f2(0.f, 0.f);
            if constexpr (LAYER) db[i][e] = f2(0.f, 0.f);
        }
    int get = 0, parity = 0;
    for (int j = 0; j < rows.n; ++j) {
        const float2 now = coming;
        coming = issue();
        row_wait<kGradStages - 1>();
        const uint32_t st = ring + get * (2 * plane);
        get = get + 1 == kGradStages ? 0 : get + 1;
        // kept from the sums to the results: xh and h, or the row as it came
        F2 xh[NV][W / 2], h[NV][W / 2];
        uint4 xr[NV], dr[NV];
        const F2 nm = f2(-now.x, -now.x), rr = f2(now.y, now.y);
        F2 t0 = f2(0.f, 0.f), t1 = f2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!bytes[i]) continue;
            uint4 xu = row_lds(st + i * nt * 16), du = row_lds(st + plane + i * nt * 16);
            if (!whole[i]) {   // values of the neighbouring rows: 0
                const uint4 k = at.keep(i * nt + tid);
                xu = bits_and(xu, k);
                du = bits_and(du, k);
            }
            const uint4 gu = gain_of(i);
            if constexpr (!kHold) {
                xr[i] = xu;
                dr[i] = du;
            }
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const F2 dy = pair_of<T>(du, e), hv = mul2(dy, pair_of<T>(gu, e));
                F2 c = pair_of<T>(xu, e);
                if constexpr (LAYER) {
                    c = add2(c, nm);
                    t0 = add2(t0, hv);
                    db[i][e] = add2(db[i][e], dy);
                }
                const F2 xv = mul2(c, rr);
                t1 = fma2(hv, xv, t1);
                dg[i][e] = fma2(dy, xv, dg[i][e]);
                if constexpr (kHold) {
                    h[i][e] = hv;
                    xh[i][e] = xv;
                }
            }
        }
        const float2 s = row_sums<LAYER, WARP>(both(t0), both(t1), buf[parity]);
        parity ^= 1;
        const float m0 = -now.y * (s.x * inv), m1 = -now.y * (s.y * inv);
        const F2 k0 = f2(m0, m0), k1 = f2(m1, m1);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!bytes[i]) continue;
            uint4 gu;
            if constexpr (!kHold) gu = gain_of(i);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                F2 xv, hv;
                if constexpr (kHold) {
                    xv = xh[i][e];
                    hv = h[i][e];
                } else {
                    hv = mul2(pair_of<T>(dr[i], e), pair_of<T>(gu, e));
                    xv = pair_of<T>(xr[i], e);
                    if constexpr (LAYER) xv = add2(xv, nm);
                    xv = mul2(xv, rr);
                }
                set_pair<T>(o, e, fma2(xv, k1, LAYER ? fma2(hv, rr, k0) : mul2(hv, rr)));
            }
            T *p = dst + i * nt * W;
            if (whole[i]) st_words(p, o);
            else at.store_part(p, i * nt + tid, o);
        }
        dst += stride;
    }
    // the block's sums, one row of [2, d]; a warp per row: the warps' sums joined in order first
    float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
    if constexpr (WARP) {
        row_wait<0>();
        __syncthreads();
        float *sum = reinterpret_cast<float *>(row_smem);   // the rows' space is free now
        constexpr int kSum = 32 * NV * W;
        for (int w = 0; w < kRowWarps; ++w) {
            if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int c = (i * 32 + tid) * W + e;
                        sum[c] = w ? sum[c] + half_of(dg[i][e / 2], e) : half_of(dg[i][e / 2], e);
                        if constexpr (LAYER)
                            sum[kSum + c] = w ? sum[kSum + c] + half_of(db[i][e / 2], e) : half_of(db[i][e / 2], e);
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
            part[c] = sum[c + at.shift];
            if constexpr (LAYER) part[a.d + c] = sum[kSum + c + at.shift];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * nt + tid;
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (at.has(v, e)) {
                    part[v * W + e - at.shift] = half_of(dg[i][e / 2], e);
                    if constexpr (LAYER) part[a.d + v * W + e - at.shift] = half_of(db[i][e / 2], e);
                }
        }
    }
}

// Rows wider than that: the second walk reads them from the caches, and the columns' sums (SUMS) are in
// shared memory, each column its thread's own.
template <class T, bool LAYER, bool SUMS>
__global__ void __launch_bounds__(1024) norm_grad_wide_kernel(NormArgs a, int P)
{
    constexpr int W = 16 / sizeof(T);
    extern __shared__ __align__(16) char row_smem[];
    __shared__ float2 buf[2][32];
    op_begin();
    const Rows<T, false> rows(a.T, a.d, P);
    const Place<T> &at = rows.at;
    float *dg = reinterpret_cast<float *>(row_smem), *db = dg + at.nv * W;
    if (SUMS)
        for (int i = threadIdx.x; i < at.nv * W * (LAYER ? 2 : 1); i += blockDim.x) dg[i] = 0.f;
    __syncthreads();
    const T *gain = static_cast<const T *>(a.gain);
    const bool gains16 = gain && at.shift == 0;
    auto gain_of = [&](int v, uint4 u, int e) {   // pair e of vector v's gains (u: loaded whole)
        if (gains16 && at.inner(v)) return pair_of<T>(u, e);
        const int c = v * W + 2 * e - at.shift;
        return gain ? f2(to_f32(__ldg(gain + min(max(c, 0), a.d - 1))), to_f32(__ldg(gain + min(max(c + 1, 0), a.d - 1))))
                    : f2(1.f, 1.f);
    };
    const float inv = 1.f / static_cast<float>(a.d);
    int parity = 0;
    for (int j = 0; j < rows.n; ++j) {
        const int row = rows.row + j * rows.step;
        const long first = static_cast<long>(row) * a.d - at.shift;
        const T *x = static_cast<const T *>(a.x) + first, *dy = static_cast<const T *>(a.dy) + first;
        T *dx = static_cast<T *>(a.dx) + first;
        const float mean = LAYER ? a.stats[2 * static_cast<size_t>(row)] : 0.f, r = a.stats[2 * static_cast<size_t>(row) + 1];
        const F2 nm = f2(-mean, -mean), rr = f2(r, r);
        F2 t0 = f2(0.f, 0.f), t1 = f2(0.f, 0.f);
#pragma unroll 2
        for (int v = threadIdx.x; v < at.nv; v += blockDim.x) {
            const uint4 xu = at.load(x, v), du = at.load(dy, v);
            const uint4 gu = gains16 && at.inner(v) ? __ldg(reinterpret_cast<const uint4 *>(gain + v * W)) : make_uint4(0, 0, 0, 0);
            F2 *sg = reinterpret_cast<F2 *>(dg + v * W), *sb = reinterpret_cast<F2 *>(db + v * W);
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                // outside the row both are 0: dy is 0 in every term
                const F2 dv = pair_of<T>(du, e), h = mul2(dv, gain_of(v, gu, e));
                F2 c = pair_of<T>(xu, e);
                if constexpr (LAYER) {
                    c = add2(c, nm);
                    t0 = add2(t0, h);
                }
                const F2 xh = mul2(c, rr);
                t1 = fma2(h, xh, t1);
                if constexpr (SUMS) {
                    sg[e] = fma2(dv, xh, sg[e]);
                    if constexpr (LAYER) sb[e] = add2(sb[e], dv);
                }
            }
        }
        const float2 s = row_sums<LAYER, false>(both(t0), both(t1), buf[parity]);
        parity ^= 1;
        const float m0 = -r * (s.x * inv), m1 = -r * (s.y * inv);
        const F2 k0 = f2(m0, m0), k1 = f2(m1, m1);
#pragma unroll 2
        for (int v = threadIdx.x; v < at.nv; v += blockDim.x) {
            const uint4 xu = at.load(x, v), du = at.load(dy, v);
            const uint4 gu = gains16 && at.inner(v) ? __ldg(reinterpret_cast<const uint4 *>(gain + v * W)) : make_uint4(0, 0, 0, 0);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const F2 h = mul2(pair_of<T>(du, e), gain_of(v, gu, e));
                F2 c = pair_of<T>(xu, e);
                if constexpr (LAYER) c = add2(c, nm);
                set_pair<T>(o, e, fma2(mul2(c, rr), k1, LAYER ? fma2(h, rr, k0) : mul2(h, rr)));
            }
            if (at.inner(v)) st_words(dx + v * W, o);
            else at.store_part(dx + v * W, v, o);
        }
    }
    if (!SUMS) return;
    __syncthreads();
    float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        part[c] = dg[c + at.shift];
        if (LAYER) part[a.d + c] = db[c + at.shift];
    }
}

// partial column sums of rows whose sums do not fit shared memory: a block takes 32 columns of every gridDim.y-th group of 8 rows
template <class T, bool LAYER>
__global__ void __launch_bounds__(256) norm_grad_columns_kernel(NormArgs a)
{
    __shared__ float red[2][8][32];
    op_begin();
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

// dgain / dbias = the sum of the blocks' partial rows, in block order within each of 32 strands
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *part, int parts, int d, float *dgain, float *dbias)
{
    __shared__ float red[32][33];
    op_begin();
    float *out = blockIdx.y ? dbias : dgain;
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (!out) return;   // the whole block
    float s = 0.f;
    if (c < d) {
        const float *p = part + static_cast<size_t>(blockIdx.y) * d + c;
        for (int i0 = threadIdx.y; i0 < parts; i0 += 32 * 8) {
            float v[8];   // in flight together
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i0 + 32 * k < parts ? __ldcg(p + static_cast<size_t>(i0 + 32 * k) * 2 * d) : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    // warp y joins the strands of column y
    const float t = warp_sum(red[threadIdx.x][threadIdx.y]);
    const int col = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < d) out[col] = t;
}

// ---- host -------------------------------------------------------------------------------

// most rows of partial sums a backward call keeps, the blocks of its launch: a multiple of 8, the most classes of
// rows.  Narrow rows leave room for 8 blocks an SM, as long as each has some ten rows to walk over.
int most_parts(int T, int d)
{
    if (d > 4096) return d <= 8192 ? 2 * kSms : d <= 32768 ? 152 : 64;
    const int an_sm = T / (10 * kSms);
    return (an_sm > 8 ? 8 : an_sm < 2 ? 2 : an_sm) * kSms / 8 * 8;
}

int parts_for(int T, int d)
{
    const int most = most_parts(T, d), rows = (T + 7) / 8 * 8;
    return rows < most ? rows : most;
}

int round32(int v) { return (v + 31) / 32 * 32; }

// classes of rows that begin at the same place within 16 bytes
int classes_of(int d, int W)
{
    int P = 1;
    while (static_cast<long>(P) * d % W) P *= 2;
    return P;
}

constexpr int kRowSmem = 225 * 1024;   // shared memory a ring may take

// A launch of one of the ring kernels: planes of shared memory for the columns and for the ring of a row, and
// blocks that fill the SMs by shared memory and registers, a multiple of P.
struct RingPlan {
    int block, grid;
    size_t smem;
    bool ok, early;
};

RingPlan ring_plan(int T, int nv, int NV, bool warp, int P, int columns, int planes, int most, int regs)
{
    RingPlan r;
    r.block = warp ? kRowWarps * 32 : round32((nv + NV - 1) / NV);
    const int nt = warp ? 32 : r.block;
    const size_t plane = static_cast<size_t>(nt) * NV * 16;
    r.smem = plane * columns + plane * planes * (warp ? kRowWarps : 1);
    r.ok = r.block <= 512 && r.smem <= static_cast<size_t>(kRowSmem);
    int occ = static_cast<int>(220 * 1024 / (r.smem + 1024));
    const int by_regs = 65536 / (regs * r.block);
    occ = occ < by_regs ? occ : by_regs;
    const int per = warp ? kRowWarps : 1, work = (T + per - 1) / per;
    int grid = kSms * (occ > 1 ? occ : 1);
    grid = grid < work ? grid : work;
    grid = grid < most ? grid : most;
    r.grid = (grid + P - 1) / P * P;
    // Several blocks an SM, but fewer than fit, would spread unevenly beside a predecessor's last blocks.  Gradients, us, with
    // the early start against without: 5003 x 1537 fp16 35.8 and 30.8, 1500 x 2560 bf16 29.2 and 24.3, 2000 x 1537 fp16 23.2 and
    // 21.0 (but 4000 x 1024 bf16 18.7 and 19.7); where the rule starts early: 8192 x 6144 bf16 66.3 and 68.2, 500 x 6144 19.7 and
    // 20.9, forward of 8192 x 1537 fp16 22.5 and 25.0.
    r.early = r.grid <= kSms || grid >= kSms * occ;
    return r;
}

inline cudaError_t launch_ring(void (*kernel)(NormArgs, int), const RingPlan &r, const NormArgs &a, int P, cudaStream_t s)
{
    if (r.smem > 40 * 1024) {   // near the 48 KB that need no leave, static arrays included
        // always the most that any width takes: the limit is the kernel's, shared by all calls, and one that set its own
        // would take the larger limit of another thread's call away before that call's launch
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
    }
    return op_launch_when(r.early, kernel, dim3(r.grid), dim3(r.block), r.smem, s, 1, a, P);
}

template <class T, bool LAYER>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const int P = classes_of(a.d, W);
    if (P == 1) {
        const int nvec = a.d / W;
        if (nvec <= 32 * 4)
            return op_launch(norm_kernel<T, 4, LAYER, true>, dim3((a.T + kRowWarps - 1) / kRowWarps), dim3(kRowWarps * 32), 0,
                             s, 1, a);
        if (nvec <= 1024 * 4)
            return op_launch(norm_kernel<T, 4, LAYER, false>, dim3(a.T), dim3(round32((nvec + 3) / 4)), 0, s, 1, a);
        if (nvec <= 1024 * 8)
            return op_launch(norm_kernel<T, 8, LAYER, false>, dim3(a.T), dim3(round32((nvec + 7) / 8)), 0, s, 1, a);
    } else {
        const int nv = (a.d + 2 * (W - 1)) / W;   // at the largest shift
        const bool warp = nv <= 32 * 2;
        const RingPlan r = ring_plan(a.T, nv, 2, warp, P, LAYER ? 2 : 1, kRowStages, 1 << 20, 64);
        if (r.ok)
            return launch_ring(warp ? norm_shift_kernel<T, 2, LAYER, true> : norm_shift_kernel<T, 2, LAYER, false>, r, a, P, s);
    }
    return op_launch(norm_wide_kernel<T, LAYER>, dim3(a.T), dim3(1024), 0, s, 1, a);
}

template <class T, bool LAYER, bool SHIFT>
cudaError_t launch_norm_grad_ring(const RingPlan &r, bool warp, int NV, const NormArgs &a, int P, cudaStream_t s)
{
    return launch_ring(warp     ? norm_grad_kernel<T, 2, LAYER, true, SHIFT>
                       : NV > 2 ? norm_grad_kernel<T, 4, LAYER, false, SHIFT>
                                : norm_grad_kernel<T, 2, LAYER, false, SHIFT>,
                       r, a, P, s);
}

template <class T, bool LAYER>
cudaError_t launch_norm_grad(const NormArgs &a, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const int P = classes_of(a.d, W), nv = (a.d + (P > 1 ? 2 : 1) * (W - 1)) / W;
    const bool warp = nv <= 32 * 2, sums = a.dgain || a.dbias;
    const int NV = nv <= 2 * kGradThreads ? 2 : 4;
    RingPlan r = ring_plan(a.T, nv, NV, warp, P, P > 1, 2 * kGradStages, most_parts(a.T, a.d), warp ? 96 : NV > 2 ? 128 : 80);
    cudaError_t e;
    if (r.ok) {
        e = P == 1 ? launch_norm_grad_ring<T, LAYER, false>(r, warp, NV, a, P, s)
                   : launch_norm_grad_ring<T, LAYER, true>(r, warp, NV, a, P, s);
    } else {
        // one block an SM: the sums take its shared memory
        r.block = 1024;
        r.smem = static_cast<size_t>(nv) * W * 4 * (LAYER ? 2 : 1);
        const bool fits = sums && r.smem <= static_cast<size_t>(kRowSmem);
        const int most = parts_for(a.T, a.d);
        r.grid = a.T < kSms ? a.T : kSms;
        if (fits && r.grid > most) r.grid = most;
        r.grid = (r.grid + P - 1) / P * P;
        if (!fits) r.smem = 0;
        e = launch_ring(fits ? norm_grad_wide_kernel<T, LAYER, true> : norm_grad_wide_kernel<T, LAYER, false>, r, a, P, s);
        if (e == cudaSuccess && sums && !fits) {
            const int groups = (a.T + 7) / 8;
            r.grid = groups < most ? groups : most;
            r.grid = r.grid < 64 ? r.grid : 64;
            e = op_launch(norm_grad_columns_kernel<T, LAYER>, dim3((a.d + 31) / 32, r.grid), dim3(32, 8), 0, s, 1, a);
        }
    }
    if (e != cudaSuccess || !sums) return e;
    return op_launch(norm_reduce_kernel, dim3((a.d + 31) / 32, a.dbias ? 2 : 1), dim3(32, 32), 0, s, 1,
                     static_cast<const float *>(a.part), r.grid, a.d, a.dgain, a.dbias);
}

template <class T>
cudaError_t norm_by_kind(int kind, bool grad, const NormArgs &a, cudaStream_t s)
{
    if (kind == MOE_NORM_LAYER) return grad ? launch_norm_grad<T, true>(a, s) : launch_norm<T, true>(a, s);
    return grad ? launch_norm_grad<T, false>(a, s) : launch_norm<T, false>(a, s);
}

int norm_dispatch(int kind, int dtype, bool grad, const NormArgs &a, cudaStream_t s)
{
    const cudaError_t e = dtype == MOE_F32   ? norm_by_kind<float>(kind, grad, a, s)
                          : dtype == MOE_F16 ? norm_by_kind<__half>(kind, grad, a, s)
                                             : norm_by_kind<__nv_bfloat16>(kind, grad, a, s);
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
    if (op_overlap(dgain, gb, dbias, gb) || op_overlap(dgain, gb, gain, row) || op_overlap(dbias, gb, gain, row)) return MOE_EINVAL;
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
        const int done = dgain ? op_status(cudaMemsetAsync(dgain, 0, gb, s)) : MOE_OK;
        return done == MOE_OK && dbias ? op_status(cudaMemsetAsync(dbias, 0, gb, s)) : done;
    }
    NormArgs a{T, d, x, gain, nullptr, 0.f, nullptr, const_cast<float *>(stats), dy, dx, static_cast<float *>(workspace),
               dgain, dbias};
    return norm_dispatch(kind, dtype, true, a, s);
}
