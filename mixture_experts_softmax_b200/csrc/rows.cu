// rows.cu -- token rows sorted by expert and back, with the gates applied, and the gradients.
//
//   sort      a stable counting sort of the T * k routes by expert: offsets[e] = routes of experts
//             below e, slot[r] = offsets[e_r] + #{routes r' < r of the same expert}, perm its inverse,
//             rows[slot[t,j]] = x[t]
//   unsort    out[t] = sum_j gate[t,j] * rows[slot[t,j]]   (gate 1: the gradient of the sort)
//   gradient  drows[slot[t,j]] = gate[t,j] * dout[t],  dgate[t,j] = <dout[t], rows[slot[t,j]]>
//
// All are bound by memory traffic: each row is read once and written once, with 16-byte accesses
// where the row width allows them, and every sum has a fixed order.  Measured on a B200 at 8192 tokens, 2
// picks, 6144 wide: sort bf16 53 us (88% of the copy bandwidth; about 6 us of it are the order, which only few SMs can
// find), way back of fp32 rows into bf16 75 us and its bf16 gradient 78 us (both at the copy bandwidth).  Rows that
// are no multiple of 16 bytes move in narrower pieces, and the number of accesses limits them: gradient of
// 1021 tokens, 6 picks, 2051 fp32 wide 22 us (59%).  Small batches are a launch: 8 tokens 7 us.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kMaxSortExperts = 256;
constexpr int kMaxPicks = 16;

// ---- the order -------------------------------------------------------------------
//
// The routes are cut into one contiguous segment per warp.  A warp walks over its segment, counts the
// routes per expert and notes each one's rank among those: lanes with the same expert find one
// another by votes, so the rank is the count so far plus the number of earlier lanes of the group.
// A scan over warps (and blocks) turns the counts into each warp's first row of every expert, and
// a second, cheap walk adds that to the ranks.

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

constexpr int kBatch = 4;   // steps whose loads are in flight together

// the lanes of the warp whose expert is this lane's (none for a dropped route): one vote for each bit of an expert's number
__device__ __forceinline__ unsigned peers_of(int e, int bits)
{
    unsigned m = __ballot_sync(0xffffffffu, e >= 0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        if (b >= bits) break;
        const bool one = e & (1 << b);
        const unsigned v = __ballot_sync(0xffffffffu, one);
        m &= one ? v : ~v;
    }
    return m;
}

// Counts of the segment [begin, end) into cnt[e * stride] (this warp's own), and rank[r] = earlier routes of the segment
// with the same expert (nothing for a dropped route).
__device__ __forceinline__ void count_segment(const SortArgs &a, int begin, int end, int *cnt, int stride, int *rank)
{
    const int lane = threadIdx.x & 31, bits = 32 - __clz(a.E - 1);
    for (int r0 = begin; r0 < end; r0 += 32 * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) e[b] = r0 + 32 * b < end ? expert_of(a, r0 + 32 * b + lane) : -1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (r0 + 32 * b >= end) break;
            const unsigned peers = peers_of(e[b], bits);
            const int lower = __popc(peers & ((1u << lane) - 1)), so_far = e[b] >= 0 ? cnt[e[b] * stride] : 0;
            if (e[b] >= 0) rank[r0 + 32 * b + lane] = so_far + lower;
            __syncwarp();
            if (e[b] >= 0 && lower == 0) cnt[e[b] * stride] = so_far + __popc(peers);
            __syncwarp();
        }
    }
}

// place(r, row): row of every route of the segment (-1: dropped) = first[e] (the block's) + base[e * stride] (the warp's
// among the block's) + rank
template <class F>
__device__ __forceinline__ void place_segment(const SortArgs &a, int begin, int end, const int *first, const int *base, int stride,
                                              const int *rank, F &&place)
{
    const int lane = threadIdx.x & 31;
    for (int r0 = begin; r0 < end; r0 += 32 * kBatch) {
        int e[kBatch], k[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            e[b] = r0 + 32 * b < end ? expert_of(a, r0 + 32 * b + lane) : -1;
            k[b] = e[b] >= 0 ? rank[r0 + 32 * b + lane] : 0;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + 32 * b + lane;
            if (r0 + 32 * b < end && r < a.n) place(r, e[b] >= 0 ? first[e[b]] + base[e[b] * stride] + k[b] : -1);
        }
    }
}

// inclusive sum over the warp's lanes
__device__ __forceinline__ int lane_scan(int v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// warp 0: exclusive scan of tot[E] into base[E + 1], 8 experts a lane (E <= 256)
__device__ __forceinline__ void scan_experts(const int *tot, int *base, int E)
{
    const int lane = threadIdx.x & 31;
    int v[8], s = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = lane * 8 + i < E ? tot[lane * 8 + i] : 0;
        s += v[i];
    }
    int at = lane_scan(s) - s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (lane * 8 + i < E) base[lane * 8 + i] = at;
        at += v[i];
    }
    if (lane == 31) base[E] = at;
}

// cnt[e * stride + w], the NW warps' counts -> each warp's first row of e within the block; tot[e] = the block's count.
// A warp takes an expert, its lanes the warps' counts.
template <int NW>
__device__ __forceinline__ void scan_warps(int *cnt, int stride, int *tot, int E)
{
    const int lane = threadIdx.x & 31;
    for (int e = threadIdx.x >> 5; e < E; e += NW) {
        const int c = lane < NW ? cnt[e * stride + lane] : 0, s = lane_scan(c);
        if (lane < NW) cnt[e * stride + lane] = s - c;
        if (lane == 31) tot[e] = s;
    }
}

// The order of any number of routes, by one cluster of 1 to 8 blocks of 32 warps: at 16,384 routes
// a warp walks two steps; at the largest, 4 M routes, the rows to be moved outweigh it by far.  What it
// takes is latency: two walks, two cluster barriers and the scans.
constexpr int kPlanWarps = 32, kPlanStride = kPlanWarps + 1;   // 1: an expert's counts begin at another bank than the next one's

// write_perm: else the copy kernel does it, where those scattered words spread over all SMs
__global__ void __launch_bounds__(kPlanWarps * 32) sort_plan_kernel(SortArgs a, int write_perm)
{
    __shared__ int cnt[kPlanStride * kMaxSortExperts];
    __shared__ int tot[kMaxSortExperts], all[kMaxSortExperts], first[kMaxSortExperts], base[kMaxSortExperts + 1];
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank(), warp = threadIdx.x >> 5;
    op_begin();

    const int per = ((a.n + C * kPlanWarps - 1) / (C * kPlanWarps) + 31) / 32 * 32;
    // n is 2^22 at most, and the last segment begins less than 8500 behind its end
    const int begin = min((rank * kPlanWarps + warp) * per, a.n), end = min(begin + per, a.n);
    for (int i = threadIdx.x; i < kPlanStride * a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    count_segment(a, begin, end, cnt + warp, kPlanStride, a.slot);   // ranks where the rows will stand
    __syncthreads();
    scan_warps<kPlanWarps>(cnt, kPlanStride, tot, a.E);
    cl.sync();
    // The cluster's counts of every expert, and those of the blocks before this one: a thread takes
    // an expert and one of eight blocks.
    for (int i = threadIdx.x; i < kMaxSortExperts * 8; i += blockDim.x) {
        const int e = i >> 3, c = i & 7, v = e < a.E && c < C ? cl.map_shared_rank(tot, c)[e] : 0;
        int sum = v, before = c < rank ? v : 0;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        if (c == 0 && e < a.E) {
            all[e] = sum;
            first[e] = before;
        }
    }
    cl.barrier_arrive();           // this block has read the others' counts
    __syncthreads();
    if (warp == 0) scan_experts(all, base, a.E);
    __syncthreads();
    if (threadIdx.x < a.E) first[threadIdx.x] += base[threadIdx.x];   // this block's first row of the expert
    if (rank == 0)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = base[e];
    __syncthreads();
    place_segment(a, begin, end, first, cnt + warp, kPlanStride, a.slot, [&](int r, int row) {
        a.slot[r] = row;
        if (write_perm && row >= 0) a.perm[row] = r;
    });
    for (int r = base[a.E] + rank * static_cast<int>(blockDim.x) + threadIdx.x; r < a.n; r += C * blockDim.x)
        a.perm[r] = -1;   // behind the last row
    cl.barrier_wait();             // no block ends while another reads its counts
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

// perm: nullptr, or where the first unit of a token notes its routes
template <class V, class S>
__device__ __forceinline__ void copy_unit(const CopyArgs &c, int k, int n, long unit, S &&slot_of, int *perm)
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
    if (!on) return;
    for (int j0 = 0; j0 < k; j0 += kUnroll) {
        int row[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) row[j] = j0 + j < k ? slot_of(t * k + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (row[j] < 0 || row[j] >= n) continue;
            if (perm && v0 == j) perm[row[j]] = t * k + j0 + j;   // a lane each
            V *dst = static_cast<V *>(c.rows) + static_cast<size_t>(row[j]) * c.vpr;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (v0 + u * lanes < c.vpr) dst[v0 + u * lanes] = v[u];
        }
    }
}

template <class V>
__global__ void __launch_bounds__(256) sort_copy_kernel(CopyArgs c, const int *slot, int k, int n, int *perm)
{
    op_begin();   // before x too: its writer ended before the order's launch began, but only a thread's own wait shows it x
    const long unit = (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> c.lg;
    copy_unit<V>(c, k, n, unit, [&](int r) { return __ldg(slot + r); }, perm);
}

// A small batch in one launch: every block finds the whole order by itself (it is a few steps of
// eight warps) and copies its share of the rows; block 0 writes the order out.
constexpr int kSmallWarps = 8, kSmallStride = kSmallWarps + 1;
constexpr int kSmallRoutes = 1024;

template <class V>
__global__ void __launch_bounds__(kSmallWarps * 32) sort_small_kernel(SortArgs a, CopyArgs c)
{
    op_begin();
    __shared__ int cnt[kSmallStride * kMaxSortExperts];
    __shared__ int tot[kMaxSortExperts], base[kMaxSortExperts + 1];
    __shared__ int slots[kSmallRoutes];
    const int warp = threadIdx.x >> 5;
    const int per = ((a.n + kSmallWarps - 1) / kSmallWarps + 31) / 32 * 32;
    const int begin = min(warp * per, a.n), end = min(begin + per, a.n);
    for (int i = threadIdx.x; i < kSmallStride * a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    count_segment(a, begin, end, cnt + warp, kSmallStride, slots);
    __syncthreads();
    scan_warps<kSmallWarps>(cnt, kSmallStride, tot, a.E);
    __syncthreads();
    if (warp == 0) scan_experts(tot, base, a.E);
    __syncthreads();
    const bool first = blockIdx.x == 0;
    place_segment(a, begin, end, base, cnt + warp, kSmallStride, slots, [&](int r, int row) {
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
    copy_unit<V>(c, a.k, a.n, unit, [&](int r) { return slots[r]; }, nullptr);
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
        return op_launch(sort_small_kernel<V>, dim3(x ? grid : 1), dim3(kSmallWarps * 32), 0, s, 1, a, c);
    // one step a warp as far as the cluster goes
    const int cluster = a.n <= 2048 ? 2 : a.n <= 4096 ? 4 : 8;
    cudaError_t e = op_launch(sort_plan_kernel, dim3(cluster), dim3(kPlanWarps * 32), 0, s, cluster, a, x ? 0 : 1);
    if (e != cudaSuccess || !x) return e;
    return op_launch(sort_copy_kernel<V>, dim3(grid), dim3(256), 0, s, 1, c, static_cast<const int *>(a.slot), a.k,
                     a.n, a.perm);
}

// ---- back, with the gates applied ---------------------------------------------------
//
// nt threads take a token; a thread forms kSteps vectors of out[t] at a time, with the picks' rows of a group of G in
// flight together: fp32 products summed in pick order, one rounding at the end.  A dropped route adds
// nothing, whatever its gate holds.

struct UnsortArgs {
    int T, k, d;
    const void *rows;
    const int *slot;
    const float *gate;          // [T, k] or nullptr: 1
    void *out;
};

// first elements of the rows of picks j0 .. j0 + G - 1 of token t (-1: a dropped route), and their gates
template <int G>
__device__ __forceinline__ void picks_of(const int *slot, const float *gate, int t, int k, int j0, int n, int d, long (&at)[G],
                                         float (&g)[G])
{
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const int row = j0 + j < k ? __ldg(slot + t * k + j0 + j) : -1;
        const bool on = row >= 0 && row < n;
        at[j] = on ? static_cast<long>(row) * d : -1;
        g[j] = on && gate ? __ldg(gate + t * k + j0 + j) : 1.f;
    }
}

// steps that keep about `bytes` a thread in flight
constexpr int steps_of(int step_bytes, int bytes) { return step_bytes * 8 <= bytes ? 8 : step_bytes * 4 <= bytes ? 4 : step_bytes * 3 <= bytes ? 3 : 2; }

template <class R, int N, int G> constexpr int unsort_steps() { return steps_of(N * G * static_cast<int>(sizeof(R)), 64); }

// NT: nt where it is fixed (the steps are then at constant distances), else 0
template <class R, class O, int N, int G, int NT>
__global__ void __launch_bounds__(256) unsort_kernel(UnsortArgs a, int threads)
{
    op_begin();
    const int nt = NT ? NT : threads;
    constexpr int kSteps = unsort_steps<R, N, G>();
    const int n = a.T * a.k, sub = static_cast<int>(threadIdx.x) / nt, lane = static_cast<int>(threadIdx.x) - sub * nt;
    const int t = blockIdx.x * (blockDim.x / nt) + sub;
    if (t >= a.T) return;
    O *out = static_cast<O *>(a.out) + static_cast<size_t>(t) * a.d;
    const R *rows = static_cast<const R *>(a.rows);
    long at[G];
    float g[G];
    if (a.k <= G) picks_of<G>(a.slot, a.gate, t, a.k, 0, n, a.d, at, g);
    for (int c0 = lane * N; c0 < a.d; c0 += nt * N * kSteps) {
        float acc[kSteps][N];
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int e = 0; e < N; ++e) acc[u][e] = 0.f;
        for (int j0 = 0; j0 < a.k; j0 += G) {
            if (a.k > G) picks_of<G>(a.slot, a.gate, t, a.k, j0, n, a.d, at, g);
            Raw<R, N> v[kSteps][G];
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (at[j] >= 0 && c0 + u * nt * N < a.d) v[u][j].load(rows + at[j] + c0 + u * nt * N);
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (at[j] >= 0 && c0 + u * nt * N < a.d) {
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[u][e] = fmaf(g[j], v[u][j].get(e), acc[u][e]);
                    }
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            if (c0 + u * nt * N >= a.d) continue;
            Raw<O, N> o;
            o.set([&](int e) { return acc[u][e]; });
            o.store(out + c0 + u * nt * N);
        }
    }
}

// ---- the gradient of the way back -----------------------------------------------------
//
// nt threads, whole warps, take a token.  For a group of G picks a thread has kSteps vectors of dout[t] and of every
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

template <class R, class O, int N, int G>
constexpr int unsort_grad_steps() { return steps_of(N * static_cast<int>(sizeof(O) + G * sizeof(R)), 96); }

template <class R, class O, int N, int G, int NT>
__global__ void __launch_bounds__(256) unsort_grad_kernel(UnsortGradArgs a, int threads)
{
    op_begin();
    const int nt = NT ? NT : threads;
    constexpr int kSteps = unsort_grad_steps<R, O, N, G>();
    __shared__ float red[2][8][G];
    const int n = a.T * a.k, sub = static_cast<int>(threadIdx.x) / nt, lane = static_cast<int>(threadIdx.x) - sub * nt;
    const int last = blockIdx.x * (blockDim.x / nt) + sub, t = min(last, a.T - 1), warps = nt / 32;
    const bool real = last < a.T;   // else: only at the barriers
    const O *dout = static_cast<const O *>(a.dout) + static_cast<size_t>(t) * a.d;
    const R *rows = static_cast<const R *>(a.rows);
    R *drows = static_cast<R *>(a.drows);
    int parity = 0;
    for (int j0 = 0; j0 < a.k; j0 += G) {
        long at[G];
        float g[G], dot[G];
        picks_of<G>(a.slot, a.gate, t, a.k, j0, real ? n : 0, a.d, at, g);
#pragma unroll
        for (int j = 0; j < G; ++j) dot[j] = 0.f;
        for (int c0 = real ? lane * N : a.d; c0 < a.d; c0 += nt * N * kSteps) {
            Raw<O, N> dv[kSteps];
            Raw<R, N> rv[kSteps][G];
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int c = c0 + u * nt * N;
                if (c >= a.d) continue;
                dv[u].load(dout + c);
                if (a.dgate) {
#pragma unroll
                    for (int j = 0; j < G; ++j)
                        if (at[j] >= 0) rv[u][j].load(rows + at[j] + c);
                }
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int c = c0 + u * nt * N;
                if (c >= a.d) continue;
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (at[j] < 0) continue;
                    Raw<R, N> o;
                    o.set([&](int e) { return g[j] * dv[u].get(e); });
                    o.store(drows + at[j] + c);
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
        if (nt == 32) {
#pragma unroll
            for (int j = 0; j < G; ++j)
                if (lane == j && real && j0 + j < a.k) a.dgate[t * a.k + j0 + j] = dot[j];   // 0 for a dropped route
        } else {
            // two buffers by turns: one barrier a group
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int j = 0; j < G; ++j) red[parity][threadIdx.x >> 5][j] = dot[j];
            }
            __syncthreads();
            if (lane < G && real && j0 + lane < a.k) {
                float s = 0.f;
                for (int w = 0; w < warps; ++w) s += red[parity][sub * warps + w][lane];
                a.dgate[t * a.k + j0 + lane] = s;
            }
            parity ^= 1;
        }
    }
}

// Threads of a token for rows of `vecs` vectors, `steps` at a time.  16-byte vectors: as few threads as fill the row
// in as many rounds as 256 would take (a multiple of `unit`), which leaves none idle.  Narrower ones:
// 256 threads (or a warp for short rows), since their loads are what there is too few of in flight.
// A block holds as many tokens as make up 256 threads.
struct TokenShape {
    int nt, block, grid;
};

TokenShape token_shape(int T, int vecs, int steps, int unit, bool narrow)
{
    const int rounds = (vecs + 256 * steps - 1) / (256 * steps), per = (vecs + rounds * steps - 1) / (rounds * steps);
    TokenShape s;
    s.nt = narrow ? (vecs <= 128 ? 32 : 256) : (per + unit - 1) / unit * unit;
    const int tokens = 256 / s.nt;
    s.block = tokens * s.nt;
    s.grid = (T + tokens - 1) / tokens;
    return s;
}

template <class R, class O, int N, int G>
cudaError_t launch_unsort_group(const UnsortArgs &a, cudaStream_t s)
{
    const TokenShape sh = token_shape(a.T, a.d / N, unsort_steps<R, N, G>(), 8, N <= 2);
    void (*kernel)(UnsortArgs, int);
    if constexpr (N > 2) kernel = unsort_kernel<R, O, N, G, 0>;
    else kernel = sh.nt == 32 ? unsort_kernel<R, O, N, G, 32> : unsort_kernel<R, O, N, G, 256>;
    return op_launch(kernel, dim3(sh.grid), dim3(sh.block), 0, s, 1, a, sh.nt);
}

template <class R, class O, int N>
cudaError_t launch_unsort(const UnsortArgs &a, cudaStream_t s)
{
    return a.k <= 2 ? launch_unsort_group<R, O, N, 2>(a, s) : launch_unsort_group<R, O, N, 4>(a, s);
}

template <class R, class O, int N, int G>
cudaError_t launch_unsort_grad_group(const UnsortGradArgs &a, cudaStream_t s)
{
    const TokenShape sh = token_shape(a.T, a.d / N, unsort_grad_steps<R, O, N, G>(), 32, N <= 2);
    void (*kernel)(UnsortGradArgs, int);
    if constexpr (N > 2) kernel = unsort_grad_kernel<R, O, N, G, 0>;
    else kernel = sh.nt == 32 ? unsort_grad_kernel<R, O, N, G, 32> : unsort_grad_kernel<R, O, N, G, 256>;
    return op_launch(kernel, dim3(sh.grid), dim3(sh.block), 0, s, 1, a, sh.nt);
}

template <class R, class O, int N>
cudaError_t launch_unsort_grad(const UnsortGradArgs &a, cudaStream_t s)
{
    return a.k <= 2 ? launch_unsort_grad_group<R, O, N, 2>(a, s) : launch_unsort_grad_group<R, O, N, 4>(a, s);
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
        if (x && (!op_ptr(x) || !op_ptr(rows))) return MOE_EINVAL;
        // blocks read idx, x and the slots while others write the order and the rows
        const struct {
            const void *p;
            size_t n;
        } in[] = {{x, T * row}, {idx, n * 4}},
          out[] = {{offsets, (static_cast<size_t>(E) + 1) * 4}, {perm, n * 4}, {slot, n * 4}, {rows, n * row}};
        for (int i = 0; i < 4; ++i) {
            for (const auto &b : in)
                if (op_overlap(out[i].p, out[i].n, b.p, b.n)) return MOE_EINVAL;
            for (int j = 0; j < i; ++j)
                if (op_overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MOE_EINVAL;
        }
    }
    const int rc = op_device();
    if (rc != MOE_OK) return rc;
    if (T == 0) return op_status(cudaMemsetAsync(offsets, 0, (static_cast<size_t>(E) + 1) * 4, s));
    const SortArgs a{T, k, E, static_cast<int>(n), idx, offsets, perm, slot};
    if (row % 16 == 0) return op_status(launch_sort<uint4>(a, x, rows, row, s));
    if (row % 8 == 0) return op_status(launch_sort<uint2>(a, x, rows, row, s));
    if (row % 4 == 0) return op_status(launch_sort<uint32_t>(a, x, rows, row, s));
    return op_status(launch_sort<uint16_t>(a, x, rows, row, s));
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
    return by_types(rows_dtype, dtype, [&](auto r, auto o) { return op_status(unsort_by_width<decltype(r), decltype(o)>(a, s)); });
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
                    [&](auto r, auto o) { return op_status(unsort_grad_by_width<decltype(r), decltype(o)>(a, s)); });
}
