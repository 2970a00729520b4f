// rows.cu -- token rows sorted by expert and back, with the gates applied, and the gradients.
//
//   sort      a stable counting sort of the T * k routes by expert: offsets[e] = routes of experts
//             below e, slot[r] = offsets[e_r] + #{routes r' < r of the same expert}, perm its inverse,
//             rows[slot[t,j]] = x[t]
//   unsort    out[t] = sum_j gate[t,j] * rows[slot[t,j]]   (gate 1: the gradient of the sort)
//   gradient  drows[slot[t,j]] = gate[t,j] * dout[t],  dgate[t,j] = <dout[t], rows[slot[t,j]]>
//
// All are bound by memory traffic: each row is read once and written once, with 16-byte accesses
// where the row width allows them, and every sum has a fixed order.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kMaxSortExperts = 256;
constexpr int kMaxPicks = 16;

// ---- the order -------------------------------------------------------------------
//
// The routes are cut into one contiguous segment per warp.  Every warp counts its segment's routes
// per expert, a scan over warps (and blocks) turns the counts into each warp's first row of every
// expert, and a second walk over the segment places its routes: lanes with the same expert find
// one another with a match, so a route's rank is the number of earlier lanes of its group.

struct SortArgs {
    int T, k, E, n;             // n = T * k
    const int *idx;             // [T, k]; outside [0, E): a dropped route
    int *offsets;               // [E + 1]
    int *perm;                  // [n]
    int *slot;                  // [n]
};

__device__ __forceinline__ int expert_of(const SortArgs &a, int r)
{
    const int e = r < a.n ? __ldg(a.idx + r) : -1;
    return e >= 0 && e < a.E ? e : -1;
}

// counts of the segment [begin, end) into cnt[E] (this warp's own)
__device__ __forceinline__ void count_segment(const SortArgs &a, int begin, int end, int *cnt)
{
    const int lane = threadIdx.x & 31;
    for (int r0 = begin; r0 < end; r0 += 32) {
        const int e = expert_of(a, r0 + lane);
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(peers) - 1) cnt[e] += __popc(peers);
        __syncwarp();
    }
}

// place(r, row): row of every route of the segment (-1: dropped); next[e] = the warp's next row of e
template <class F>
__device__ __forceinline__ void place_segment(const SortArgs &a, int begin, int end, int *next, F &&place)
{
    const int lane = threadIdx.x & 31;
    for (int r0 = begin; r0 < end; r0 += 32) {
        const int r = r0 + lane, e = expert_of(a, r);
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        const int row = e >= 0 ? next[e] + __popc(peers & ((1u << lane) - 1)) : -1;
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) next[e] += __popc(peers);
        __syncwarp();
        if (r < a.n) place(r, row);
    }
}

// warp 0: exclusive scan of tot[E] into base[E + 1]
__device__ __forceinline__ void scan_experts(const int *tot, int *base, int E)
{
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane, v = e < E ? tot[e] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (e < E) base[e] = carry + s - v;
        carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) base[E] = carry;
}

// per-warp counts -> each warp's first row within the block; tot[e] = the block's count
template <int NW>
__device__ __forceinline__ void scan_warps(int *cnt, int *tot, int E)
{
    for (int e = threadIdx.x; e < E; e += NW * 32) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = s;
            s += c;
        }
        tot[e] = s;
    }
}

// The order of any number of routes, by one cluster of 1 to 8 blocks of 32 warps: at 16,384 routes
// a warp walks two steps; at the largest, 4 M routes, the rows to be moved outweigh it by far.
constexpr int kPlanWarps = 32;

__global__ void __launch_bounds__(kPlanWarps * 32) sort_plan_kernel(SortArgs a)
{
    __shared__ int cnt[kPlanWarps * kMaxSortExperts];
    __shared__ int tot[kMaxSortExperts], all[kMaxSortExperts], base[kMaxSortExperts + 1];
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank(), warp = threadIdx.x >> 5;
    griddep_launch_dependents();   // the copy of the rows waits for this kernel's end where it has to

    const int per = ((a.n + C * kPlanWarps - 1) / (C * kPlanWarps) + 31) / 32 * 32;
    // long: the last warps' segments may begin behind the end of the range of an int
    const long b0 = static_cast<long>(rank * kPlanWarps + warp) * per;
    const int begin = static_cast<int>(b0 < a.n ? b0 : a.n);
    const int end = static_cast<int>(b0 + per < a.n ? b0 + per : a.n);
    for (int i = threadIdx.x; i < kPlanWarps * a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    count_segment(a, begin, end, cnt + warp * a.E);
    __syncthreads();
    scan_warps<kPlanWarps>(cnt, tot, a.E);
    cl.sync();
    // the cluster's counts, and those of the blocks before this one
    int before = 0;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {   // E <= blockDim.x: one turn
        int sum = 0;
        for (int c = 0; c < C; ++c) {
            const int v = cl.map_shared_rank(tot, c)[e];
            before += c < rank ? v : 0;
            sum += v;
        }
        all[e] = sum;
    }
    cl.sync();   // no block reads another's counts, or ends, after this
    if (warp == 0) scan_experts(all, base, a.E);
    __syncthreads();
    if (threadIdx.x < a.E) {
        const int first = base[threadIdx.x] + before;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) cnt[w * a.E + threadIdx.x] += first;
    }
    if (rank == 0)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = base[e];
    __syncthreads();
    place_segment(a, begin, end, cnt + warp * a.E, [&](int r, int row) {
        a.slot[r] = row;
        if (row >= 0) a.perm[row] = r;
    });
    for (int r = base[a.E] + rank * static_cast<int>(blockDim.x) + threadIdx.x; r < a.n; r += C * blockDim.x)
        a.perm[r] = -1;   // behind the last row
}

// ---- the rows --------------------------------------------------------------------
//
// A unit of 2^lg lanes copies kUnroll vectors a lane of one token's row to each of its rows, all
// loads first.  Rows are moved as bytes: V is the widest vector that divides the row.

constexpr int kUnroll = 4;

// i / per for i < total: a 32-bit division where the range allows it
__device__ __forceinline__ int row_of(long i, int per, long total)
{
    return total <= 0x7fffffffL ? static_cast<int>(i) / per : static_cast<int>(i / per);
}

struct CopyArgs {
    const void *x;
    void *rows;
    int vpr;                    // vectors per row
    int upr;                    // units per row
    int lg;
    long units;                 // T * upr
};

template <class V, class S>
__device__ __forceinline__ void copy_unit(const CopyArgs &c, int k, int n, long unit, S &&slot_of, bool wait)
{
    const int lanes = 1 << c.lg, lane = threadIdx.x & (lanes - 1);
    const bool on = unit < c.units;
    const int t = on ? row_of(unit, c.upr, c.units) : 0;
    const int v0 = on ? static_cast<int>(unit - static_cast<long>(t) * c.upr) * lanes * kUnroll + lane : c.vpr;
    const V *src = static_cast<const V *>(c.x) + static_cast<size_t>(t) * c.vpr;
    V v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (v0 + u * lanes < c.vpr) v[u] = __ldg(src + v0 + u * lanes);
    if (wait) griddep_wait();   // x was there before the call; the slots are the previous kernel's
    if (!on) return;
    for (int j = 0; j < k; ++j) {
        const int row = slot_of(t * k + j);
        if (row < 0 || row >= n) continue;
        V *dst = static_cast<V *>(c.rows) + static_cast<size_t>(row) * c.vpr;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (v0 + u * lanes < c.vpr) dst[v0 + u * lanes] = v[u];
    }
}

template <class V>
__global__ void __launch_bounds__(256) sort_copy_kernel(CopyArgs c, const int *slot, int k, int n)
{
    const long unit = (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> c.lg;
    // plain loads: the slots are written while this kernel may already run
    copy_unit<V>(c, k, n, unit, [&](int r) { return *reinterpret_cast<const volatile int *>(slot + r); }, true);
}

// A small batch in one launch: every block finds the whole order by itself (it is a few steps of
// eight warps) and copies its share of the rows; block 0 writes the order out.
constexpr int kSmallWarps = 8;
constexpr int kSmallRoutes = 1024;

template <class V>
__global__ void __launch_bounds__(kSmallWarps * 32) sort_small_kernel(SortArgs a, CopyArgs c)
{
    __shared__ int cnt[kSmallWarps * kMaxSortExperts];
    __shared__ int tot[kMaxSortExperts], base[kMaxSortExperts + 1];
    __shared__ int slots[kSmallRoutes];
    const int warp = threadIdx.x >> 5;
    const int per = ((a.n + kSmallWarps - 1) / kSmallWarps + 31) / 32 * 32;
    const int begin = min(warp * per, a.n), end = min(begin + per, a.n);
    for (int i = threadIdx.x; i < kSmallWarps * a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    count_segment(a, begin, end, cnt + warp * a.E);
    __syncthreads();
    scan_warps<kSmallWarps>(cnt, tot, a.E);
    __syncthreads();
    if (warp == 0) scan_experts(tot, base, a.E);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
#pragma unroll
        for (int w = 0; w < kSmallWarps; ++w) cnt[w * a.E + e] += base[e];
    }
    __syncthreads();
    const bool first = blockIdx.x == 0;
    place_segment(a, begin, end, cnt + warp * a.E, [&](int r, int row) {
        slots[r] = row;
        if (first) {
            a.slot[r] = row;
            if (row >= 0) a.perm[row] = r;
        }
    });
    if (first) {
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = base[e];
        for (int r = base[a.E] + threadIdx.x; r < a.n; r += blockDim.x) a.perm[r] = -1;
    }
    __syncthreads();
    if (!c.x) return;
    const long unit = (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> c.lg;
    copy_unit<V>(c, a.k, a.n, unit, [&](int r) { return slots[r]; }, false);
}

// lanes of a unit and units of a row for rows of vpr vectors: short rows share a warp
void unit_shape(int vpr, int *lg, int *upr)
{
    *lg = vpr <= 8 * kUnroll ? 3 : vpr <= 16 * kUnroll ? 4 : 5;
    *upr = (vpr + (kUnroll << *lg) - 1) / (kUnroll << *lg);
}

template <class V>
cudaError_t launch_sort(const SortArgs &a, const void *x, void *rows, size_t row_bytes, cudaStream_t s)
{
    CopyArgs c{x, rows, static_cast<int>(row_bytes / sizeof(V)), 0, 0, 0};
    unit_shape(c.vpr, &c.lg, &c.upr);
    c.units = static_cast<long>(a.T) * c.upr;
    const unsigned grid = static_cast<unsigned>(((c.units << c.lg) + 255) / 256);
    if (a.n <= kSmallRoutes)
        return op_launch(sort_small_kernel<V>, dim3(x ? grid : 1), dim3(kSmallWarps * 32), 0, s, false, 1, a, c);
    // one block for up to 4 steps a warp, then as many as the cluster takes
    const int cluster = a.n <= 4096 ? 1 : a.n <= 8192 ? 2 : a.n <= 16384 ? 4 : 8;
    cudaError_t e = op_launch(sort_plan_kernel, dim3(cluster), dim3(kPlanWarps * 32), 0, s, false, cluster, a);
    if (e != cudaSuccess || !x) return e;
    return op_launch(sort_copy_kernel<V>, dim3(grid), dim3(256), 0, s, true, 1, c, static_cast<const int *>(a.slot), a.k,
                     a.n);
}

// ---- back, with the gates applied ---------------------------------------------------
//
// One thread forms N consecutive elements of out[t]: fp32 products summed in pick order, one
// rounding at the end.  A dropped route adds nothing, whatever its gate holds.

constexpr int kGroup = 4;   // picks handled together

struct UnsortArgs {
    int T, k, d;
    const void *rows;
    const int *slot;
    const float *gate;          // [T, k] or nullptr: 1
    void *out;
};

template <class R, class O, int N>
__global__ void __launch_bounds__(256) unsort_kernel(UnsortArgs a, int vpr, long items)
{
    const int n = a.T * a.k;
    const long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= items) return;
    const int t = row_of(i, vpr, items), c = static_cast<int>(i - static_cast<long>(t) * vpr) * N;
    const R *rows = static_cast<const R *>(a.rows) + c;
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kGroup) {
        // the loads of a group of picks are in flight together
        int row[kGroup];
        float g[kGroup];
        Raw<R, N> v[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            row[j] = j0 + j < a.k ? __ldg(a.slot + t * a.k + j0 + j) : -1;
            g[j] = a.gate && j0 + j < a.k ? __ldg(a.gate + t * a.k + j0 + j) : 1.f;
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (row[j] >= 0 && row[j] < n) v[j].load(rows + static_cast<size_t>(row[j]) * a.d);
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (row[j] >= 0 && row[j] < n) {
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] = fmaf(g[j], v[j].get(e), acc[e]);
            }
    }
    Raw<O, N> o;
    o.set([&](int e) { return acc[e]; });
    o.store(static_cast<O *>(a.out) + static_cast<size_t>(t) * a.d + c);
}

// ---- the gradient of the way back -----------------------------------------------------
//
// NT threads take a token.  For a group of G picks a thread has kSteps vectors of dout[t] and of every
// pick's row in flight together (more picks read dout[t] again, from the caches); it writes the
// picks' gradient rows and adds up the products for the gates' gradients in fp32, joined over
// the threads in a fixed tree.

struct UnsortGradArgs {
    int T, k, d;
    const void *dout, *rows;
    const int *slot;
    const float *gate;          // nullptr: 1
    void *drows;
    float *dgate;               // nullptr: not wanted
};

template <class R, class O, int N, int G, int NT>
__global__ void __launch_bounds__(256) unsort_grad_kernel(UnsortGradArgs a)
{
    constexpr int kTokens = 256 / NT, kWarps = NT / 32;
    // vectors of a row in flight: about 192 bytes a thread
    constexpr int kBytes = N * static_cast<int>(sizeof(O) + G * sizeof(R));
    constexpr int kSteps = kBytes >= 96 ? 2 : kBytes >= 48 ? 3 : kBytes >= 20 ? 4 : 8;
    __shared__ float red[2][kTokens * kWarps][G];
    const int n = a.T * a.k, lane = threadIdx.x % NT, sub = threadIdx.x / NT;
    const int t = blockIdx.x * kTokens + sub;
    if (NT == 32 && t >= a.T) return;   // NT == 256: the grid is T blocks
    const O *dout = static_cast<const O *>(a.dout) + static_cast<size_t>(t) * a.d;
    int parity = 0;
    for (int j0 = 0; j0 < a.k; j0 += G) {
        bool on[G];
        const R *src[G];
        R *dst[G];
        float g[G], dot[G];
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const int row = j0 + j < a.k ? __ldg(a.slot + t * a.k + j0 + j) : -1;
            on[j] = row >= 0 && row < n;
            const size_t at = on[j] ? static_cast<size_t>(row) * a.d : 0;
            src[j] = static_cast<const R *>(a.rows) + at;
            dst[j] = static_cast<R *>(a.drows) + at;
            g[j] = on[j] && a.gate ? __ldg(a.gate + t * a.k + j0 + j) : 1.f;
            dot[j] = 0.f;
        }
        for (int c0 = lane * N; c0 < a.d; c0 += NT * N * kSteps) {
            Raw<O, N> dv[kSteps];
            Raw<R, N> rv[kSteps][G];
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int c = c0 + u * NT * N;
                if (c >= a.d) continue;
                dv[u].load(dout + c);
                if (a.dgate) {
#pragma unroll
                    for (int j = 0; j < G; ++j)
                        if (on[j]) rv[u][j].load(src[j] + c);
                }
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int c = c0 + u * NT * N;
                if (c >= a.d) continue;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (!on[j]) continue;
                    Raw<R, N> o;
                    o.set([&](int e) { return g[j] * dv[u].get(e); });
                    o.store(dst[j] + c);
                    if (a.dgate) {
#pragma unroll
                        for (int e = 0; e < N; ++e) dot[j] = fmaf(dv[u].get(e), rv[u][j].get(e), dot[j]);
                    }
                }
            }
        }
        if (!a.dgate) continue;
#pragma unroll
        for (int j = 0; j < G; ++j) dot[j] = warp_sum(dot[j]);
        if constexpr (NT == 32) {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (lane == j && j0 + j < a.k) a.dgate[t * a.k + j0 + j] = dot[j];
        } else {
            // two buffers by turns: one barrier a group
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int j = 0; j < G; ++j) red[parity][threadIdx.x >> 5][j] = dot[j];
            }
            __syncthreads();
            if (lane < G && j0 + lane < a.k) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += red[parity][w][lane];
                a.dgate[t * a.k + j0 + lane] = s;   // 0 for a dropped route
            }
            parity ^= 1;
        }
    }
}

template <class R, class O, int N>
cudaError_t launch_unsort(const UnsortArgs &a, cudaStream_t s)
{
    const int vpr = a.d / N;
    const long items = static_cast<long>(a.T) * vpr;
    return op_launch(unsort_kernel<R, O, N>, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, s, false, 1,
                     a, vpr, items);
}

template <class R, class O, int N>
cudaError_t launch_unsort_grad(const UnsortGradArgs &a, cudaStream_t s)
{
    const dim3 grid(a.d / N <= 128 ? (a.T + 7) / 8 : a.T);   // a warp covers 128 vectors in a few steps
    if (a.k <= 2)
        return op_launch(a.d / N <= 128 ? unsort_grad_kernel<R, O, N, 2, 32> : unsort_grad_kernel<R, O, N, 2, 256>, grid,
                         dim3(256), 0, s, false, 1, a);
    return op_launch(a.d / N <= 128 ? unsort_grad_kernel<R, O, N, 4, 32> : unsort_grad_kernel<R, O, N, 4, 256>, grid,
                     dim3(256), 0, s, false, 1, a);
}

// the vector width by the row width: 16 bytes of the wider type's neighbour where d allows
template <class R, class O>
cudaError_t unsort_by_width(const UnsortArgs &a, cudaStream_t s)
{
    constexpr int W = sizeof(O) == 4 ? 4 : 8;
    if (a.d % W == 0) return launch_unsort<R, O, W>(a, s);
    if (a.d % 2 == 0) return launch_unsort<R, O, 2>(a, s);
    return launch_unsort<R, O, 1>(a, s);
}

template <class R, class O>
cudaError_t unsort_grad_by_width(const UnsortGradArgs &a, cudaStream_t s)
{
    constexpr int W = sizeof(O) == 4 ? 4 : 8;
    if (a.d % W == 0) return launch_unsort_grad<R, O, W>(a, s);
    if (a.d % 2 == 0) return launch_unsort_grad<R, O, 2>(a, s);
    return launch_unsort_grad<R, O, 1>(a, s);
}

// call f(R{}, O{}) for the pair of types, or MOE_EUNSUPPORTED
template <class F>
int by_types(int rows_dtype, int dtype, F &&f)
{
    if (dtype == MOE_F32) return rows_dtype == MOE_F32 ? f(float(), float()) : MOE_EUNSUPPORTED;
    if (dtype == MOE_BF16)
        return rows_dtype == MOE_BF16 ? f(__nv_bfloat16(), __nv_bfloat16())
               : rows_dtype == MOE_F32 ? f(float(), __nv_bfloat16()) : MOE_EUNSUPPORTED;
    return rows_dtype == MOE_F16 ? f(__half(), __half()) : rows_dtype == MOE_F32 ? f(float(), __half()) : MOE_EUNSUPPORTED;
}

bool sizes_ok(int T, int k, int d) { return T >= 0 && T <= MOE_MAX_TOKENS && k >= 1 && k <= kMaxPicks && d >= 1 && d <= 65536; }

int status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ECUDA; }

}  // namespace

int op_device()
{
    // major version per device, looked up once: 0 unknown
    static volatile int major[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();
        return MOE_ENODEV;
    }
    int m = dev < 64 ? major[dev] : 0;
    if (!m) {
        if (cudaDeviceGetAttribute(&m, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
            cudaGetLastError();
            return MOE_ENODEV;
        }
        if (dev < 64) major[dev] = m;
    }
    return m == 10 ? MOE_OK : MOE_ENODEV;   // built for sm_100a only
}

}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_sort_rows(int dtype, int T, int k, int E, int d, const void *x, const int32_t *idx,
                                     int32_t *offsets, int32_t *perm, int32_t *slot, void *rows, void *stream)
{
    if (!dtype_known(dtype) || !sizes_ok(T, k, d) || E < 1) return MOE_EINVAL;
    if (E > kMaxSortExperts) return MOE_EUNSUPPORTED;
    if (!op_ptr(offsets)) return MOE_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t n = static_cast<size_t>(T) * k, row = static_cast<size_t>(d) * dtype_size(dtype);
    if (T > 0) {
        if (!op_ptr(idx) || !op_ptr(perm) || !op_ptr(slot)) return MOE_EINVAL;
        if (!x != !rows) return MOE_EINVAL;   // both, or the order alone
        if (x && (!op_ptr(x) || !op_ptr(rows) || op_overlap(x, T * row, rows, n * row))) return MOE_EINVAL;
        // the order is read from idx by every block while others write it
        const size_t nb = n * 4, eb = (static_cast<size_t>(E) + 1) * 4;
        if (op_overlap(idx, nb, perm, nb) || op_overlap(idx, nb, slot, nb) || op_overlap(perm, nb, slot, nb) ||
            op_overlap(idx, nb, offsets, eb) || op_overlap(perm, nb, offsets, eb) || op_overlap(slot, nb, offsets, eb))
            return MOE_EINVAL;
    }
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    if (T == 0) return status(cudaMemsetAsync(offsets, 0, (static_cast<size_t>(E) + 1) * 4, s));
    const SortArgs a{T, k, E, static_cast<int>(n), idx, offsets, perm, slot};
    if (row % 16 == 0) return status(launch_sort<uint4>(a, x, rows, row, s));
    if (row % 8 == 0) return status(launch_sort<uint2>(a, x, rows, row, s));
    if (row % 4 == 0) return status(launch_sort<uint32_t>(a, x, rows, row, s));
    return status(launch_sort<uint16_t>(a, x, rows, row, s));
}

extern "C" MOE_API int moe_unsort_rows(int rows_dtype, int dtype, int T, int k, int d, const void *rows,
                                       const int32_t *slot, const float *gate, void *out, void *stream)
{
    if (!dtype_known(dtype) || !dtype_known(rows_dtype) || !sizes_ok(T, k, d)) return MOE_EINVAL;
    if (rows_dtype != dtype && rows_dtype != MOE_F32) return MOE_EUNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!op_ptr(rows) || !op_ptr(slot) || !op_ptr(out) || (gate && !op_aligned16(gate))) return MOE_EINVAL;
    const size_t n = static_cast<size_t>(T) * k, ob = static_cast<size_t>(T) * d * dtype_size(dtype);
    if (op_overlap(rows, n * d * dtype_size(rows_dtype), out, ob) || op_overlap(slot, n * 4, out, ob) ||
        op_overlap(gate, n * 4, out, ob))
        return MOE_EINVAL;
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    const UnsortArgs a{T, k, d, rows, slot, gate, out};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_types(rows_dtype, dtype, [&](auto r, auto o) { return status(unsort_by_width<decltype(r), decltype(o)>(a, s)); });
}

extern "C" MOE_API int moe_unsort_rows_backward(int rows_dtype, int dtype, int T, int k, int d, const void *dout,
                                                const void *rows, const int32_t *slot, const float *gate, void *drows,
                                                float *dgate, void *stream)
{
    if (!dtype_known(dtype) || !dtype_known(rows_dtype) || !sizes_ok(T, k, d)) return MOE_EINVAL;
    if (rows_dtype != dtype && rows_dtype != MOE_F32) return MOE_EUNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!op_ptr(dout) || !op_ptr(slot) || !op_ptr(drows) || (gate && !op_aligned16(gate))) return MOE_EINVAL;
    if (dgate && (!op_aligned16(dgate) || !op_ptr(rows))) return MOE_EINVAL;
    const size_t n = static_cast<size_t>(T) * k, db = static_cast<size_t>(T) * d * dtype_size(dtype);
    const size_t rb = n * d * dtype_size(rows_dtype);
    if (op_overlap(drows, rb, dout, db) || op_overlap(drows, rb, slot, n * 4) || op_overlap(drows, rb, gate, n * 4) ||
        op_overlap(drows, rb, dgate, n * 4) || (dgate && op_overlap(drows, rb, rows, rb)))
        return MOE_EINVAL;
    if (dgate && (op_overlap(dgate, n * 4, gate, n * 4) || op_overlap(dgate, n * 4, slot, n * 4) ||
                  op_overlap(dgate, n * 4, dout, db) || op_overlap(dgate, n * 4, rows, rb)))
        return MOE_EINVAL;
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    const UnsortGradArgs a{T, k, d, dout, rows, slot, gate, drows, dgate};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_types(rows_dtype, dtype,
                    [&](auto r, auto o) { return status(unsort_grad_by_width<decltype(r), decltype(o)>(a, s)); });
}
