// w4.cu -- few rows times 4-bit expert weights with group scales:
//
//   y[r, n] = sum_k x[r, k] * q[e, k, n] * s[e, k / G, n]      for the rows r of expert e
//   gated:    gelu(x W) * (x Wv), the up-projection of the MoE section's step 3
//
// With few rows the weights' bytes bound it: each is read once, by asynchronous 16-byte copies into
// a ring of stages that every lane keeps for itself, so that the copies of the next stages run while one is
// multiplied.  The products run on mma.sync m16n8k16 with 16 features as rows and 8 token rows as
// columns: a weight enters as an exact 16-bit float, the fp32 sum over one group is
// multiplied by the group's scale and added up in fp32.  (The tcgen05 path wants both operands
// staged as 16-bit tiles; for 8 columns that staging alone moves four times the weights' bytes through shared memory.)
//
// Measured on a B200: gated up-projection of 16 rows over 8 experts of 6144 x 32768 (1.66 GB) 267 us at full clock, 96% of the
// copy bandwidth, and 306 to 331 us once the power limit holds the clock near 1.57 GHz (the integer pipe is the busiest then);
// down-projection of one row each over 2 experts of 32768 x 6144 48 us, 69%: its 48 tiles, cut 5 times, fill the
// SMs' places once, unevenly.  More rows cost more multiplies and x traffic: one expert of 6144 x 32768, gated, takes 40, 45, 69
// and 123 us for 1, 8, 16 and 32 rows, up to 7 and 10 us more for the last two where the power limit holds the clock.
//
// Packed layout (moe_w4_pack).  Features in blocks of 32, inputs in units of 128 (padded: value 0,
// scale 0).  A unit of a block is 2 KB, in the order of the lanes' multiply operands: input chunk of
// 64 (2) x feature tile of 16 (2) x lane (32) x step of 16 inputs (4 words).  Lane 4 g + c of the step
// holds the inputs 4 c .. 4 c + 3 of features g and g + 8: nibble i and i + 4 of its word are operand
// register i's first and second element, stored as value + 8.  The scales follow all weights:
// per block and group 32 bf16, in the order 4 g + i for feature g + 8 i.
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kBlockF = 32;            // features of a block: one warp's
constexpr int kUnitK = 128;            // inputs of a unit: one stage
constexpr int kUnitBytes = kBlockF * kUnitK / 2;
constexpr int kStages = 3;
constexpr int kWarps = 8;
constexpr int kMaxRows = 1024;
constexpr int kMaxWExperts = 1024;
constexpr int kXUnits = 16;            // units of one 8-row slab of staged x; fewer with more slabs
constexpr int kRedStride = 36;         // floats per row of a warp's partial sums: no bank conflicts
constexpr int kTail = 256;             // bytes behind the scales: the packing's range flag

struct W4Shape {
    int E, K, N, G;
    int blocks, units, per_unit;       // feature blocks, input units, groups of a unit
    size_t scales;                     // byte offset of the scales
    size_t bytes;
};

W4Shape shape_of(int E, int K, int N, int G)
{
    W4Shape s{E, K, N, G, (N + kBlockF - 1) / kBlockF, (K + kUnitK - 1) / kUnitK, kUnitK / G, 0, 0};
    const size_t u = static_cast<size_t>(E) * s.blocks * s.units;
    s.scales = u * kUnitBytes;
    s.bytes = s.scales + u * s.per_unit * kBlockF * 2 + kTail;
    return s;
}

// ---- packing -----------------------------------------------------------------------

// one thread a 32-bit word: lanes of a warp cover the 32 features of 8 inputs
__global__ void __launch_bounds__(256) w4_pack_kernel(W4Shape s, const int8_t *q, uint32_t *out, int *flag)
{
    op_begin();
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    const size_t total = static_cast<size_t>(s.E) * s.blocks * s.units * (kUnitBytes / 4);
    if (i >= total) return;
    // reading order: feature tile and row (16), then the two low bits of the input position
    const int g = i & 7, tile = (i >> 3) & 1, c = (i >> 4) & 3, step = (i >> 6) & 3, chunk = (i >> 8) & 1;
    const size_t unit = i >> 9;
    const int u = static_cast<int>(unit % s.units);
    const size_t eb = unit / s.units;
    const int b = static_cast<int>(eb % s.blocks), e = static_cast<int>(eb / s.blocks);
    const int k0 = u * kUnitK + chunk * 64 + step * 16 + c * 4, n0 = b * kBlockF + tile * 16 + g;
    const int8_t *p = q + static_cast<size_t>(e) * s.K * s.N;
    uint32_t w = 0;
    bool bad = false;
#pragma unroll
    for (int r = 0; r < 4; ++r)          // operand register: feature + 8 for odd ones, inputs + 2 for the upper two
#pragma unroll
        for (int h = 0; h < 2; ++h) {    // its low and high half
            const int n = n0 + (r & 1) * 8, k = k0 + (r >> 1) * 2 + h;
            const int v = n < s.N && k < s.K ? p[static_cast<size_t>(k) * s.N + n] : 0;
            bad |= v < -8 || v > 7;
            w |= static_cast<uint32_t>((v + 8) & 15) << (4 * r + 16 * h);
        }
    if (bad) *flag = 1;
    out[unit * (kUnitBytes / 4) + ((chunk * 2 + tile) * 32 + g * 4 + c) * 4 + step] = w;
}

__global__ void __launch_bounds__(256) w4_pack_scales_kernel(W4Shape s, const __nv_bfloat16 *in, __nv_bfloat16 *out)
{
    op_begin();
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    const size_t total = static_cast<size_t>(s.E) * s.blocks * s.units * s.per_unit * kBlockF;
    if (i >= total) return;
    const int f = i & 31;                // feature; written to place 4 g + i of feature g + 8 i
    const size_t group = i >> 5;
    const int groups = (s.K + s.G - 1) / s.G, padded = s.units * s.per_unit;
    const int gr = static_cast<int>(group % padded);
    const size_t eb = group / padded;
    const int n = static_cast<int>(eb % s.blocks) * kBlockF + f;
    const int e = static_cast<int>(eb / s.blocks);
    const bool real = n < s.N && gr < groups;
    out[group * kBlockF + (f & 7) * 4 + (f >> 3)] =
        real ? in[(static_cast<size_t>(e) * groups + gr) * s.N + n] : __float2bfloat16_rn(0.f);
}

// ---- the product ---------------------------------------------------------------------

struct W4Args {
    int E, K, N, R;
    int blocks, units;
    size_t scales;
    const void *x;              // [R, K]
    const int *offsets;         // [E + 1] or nullptr: one expert, all rows
    const uint8_t *w, *wv;
    void *y;                    // [R, N]
    int out_f32;
    int splits;                 // blocks of a cluster, each with its share of the units
    int kparts;                 // warps of a block that share a feature block's units
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

template <class T2>
__device__ __forceinline__ uint32_t bits_of(const T2 &v)
{
    uint32_t w;
    memcpy(&w, &v, 4);
    return w;
}
template <class T2>
__device__ __forceinline__ T2 as16(uint32_t w)
{
    T2 v;
    memcpy(&v, &w, 4);
    return v;
}

// The four operand pairs of a word of 4-bit values u = value + 8.  The integer and FMA pipes limit this kernel, not
// the tensor cores, so the fast form is a mask per pair: an integer v below 256 in the low byte of a half is the
// 16-bit float v * kTiny, on both sides of the smallest normal number of bf16 (2^-133) and among
// the subnormal ones of fp16 (2^-24).  Odd pairs, the features g + 8, hold 16 u.  The products' sums are
// then those of u, and -8 times the sum of the group's inputs, with which the accumulators start, makes them
// those of u - 8; the scale's factor takes the powers of two back.  bf16 inputs are staged at 2^100 times their
// value, which keeps the products in the normal range.  A phase whose inputs do not allow that (bf16 from 2^27 up,
// inf, nan) takes the exact form: an FMA per pair makes u - 8 of it, as an ordinary number.
// What the fast form costs: sums at the size of 8 times the inputs' sum, about twice the rounding of the plain products (fp32 results of
// one token down: 7.0e-7 of the largest, plain fp32 products 4.8e-7), and all columns of a pass share one phase's choice.
// What the exact form everywhere costs, us: 16 rows over 8 experts of 6144 x 32768, gated, 298 against 270; one token over 2
// experts of 32768 x 6144, fp16, 65 against 48; the decode step's 16 rows there 182 against 161.
template <class T> struct Deq;
template <> struct Deq<__nv_bfloat16> {
    static constexpr float kFast[2] = {0x1p33f, 0x1p29f};      // 2^133 / 2^100, and / 16
    static constexpr float kExact = 128.f;                     // operands are (u - 8) / 128
    static constexpr float kStart = -0x1p-30f;                 // -8 * 2^-133 * 2^100
    static constexpr uint32_t kLimit = 0x4d00;                 // 2^27, as bits
    static __device__ __forceinline__ uint32_t stage(uint32_t w)
    {
        return pack2<__nv_bfloat16>(__uint_as_float(w << 16) * 0x1p100f, __uint_as_float(w & 0xffff0000u) * 0x1p100f);
    }
    static __device__ __forceinline__ float sum2(uint32_t w) { return __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t exact(uint32_t v, int odd)
    {
        const float f = odd ? 0x1p122f : 0x1p126f;
        return bits_of(__hfma2(as16<__nv_bfloat162>(v), __floats2bfloat162_rn(f, f), __floats2bfloat162_rn(-0.0625f, -0.0625f)));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Deq<__half> {
    static constexpr float kFast[2] = {0x1p24f, 0x1p20f};
    static constexpr float kExact = 1.f;
    static constexpr float kStart = -0x1p-21f;                 // -8 * 2^-24
    static constexpr uint32_t kLimit = 0x7c00;                 // inf
    static __device__ __forceinline__ uint32_t stage(uint32_t w) { return w; }
    static __device__ __forceinline__ float sum2(uint32_t w)
    {
        const float2 f = __half22float2(as16<__half2>(w));
        return f.x + f.y;
    }
    // OR-ed into 1024, whose last place is 1: 1024 + u, 1024 + 16 u
    static __device__ __forceinline__ uint32_t exact(uint32_t v, int odd)
    {
        const float f = odd ? 0.0625f : 1.f, o = odd ? -72.f : -1032.f;
        return bits_of(__hfma2(as16<__half2>(v | 0x64006400u), __floats2half2_rn(f, f), __floats2half2_rn(o, o)));
    }
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// x rows [row0, row0 + rows) at inputs [k0, k0 + nk), PU units at most, on their way into shared memory in the order in
// which a lane takes its operands: within 64 inputs, input 16 j + 4 c + i at place 16 c + 4 j + i.  Inputs behind K
// are 0 (the weights there are too, but 0 times what the memory holds need not be).  The loads are all in flight
// together, before the barrier that frees the place.
template <class T, int G, int NB, int PU>
struct StageX {
    static constexpr int kPer = PU * kUnitK / 8, kPieces = 8 * NB * kPer / (kWarps * 32);   // 16-byte pieces: a row's, a thread's
    uint4 v[kPieces];
    __device__ __forceinline__ void load(const W4Args &a, int row0, int rows, int k0, int nk)
    {
        const uint16_t *x = static_cast<const uint16_t *>(a.x) + static_cast<size_t>(row0) * a.K;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = threadIdx.x + i * (kWarps * 32), r = p / kPer, kk = p % kPer * 8, k = k0 + kk;
            v[i] = make_uint4(0, 0, 0, 0);
            if (r >= rows || kk >= nk || k >= a.K) continue;
            const uint16_t *src = x + static_cast<size_t>(r) * a.K + k;
            if ((a.K & 7) == 0) {
                v[i] = __ldg(reinterpret_cast<const uint4 *>(src));
            } else {
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = k + e < a.K ? __ldg(src + e) : 0u;
                v[i] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
            }
        }
    }
    // an input that the fast form cannot take
    __device__ __forceinline__ bool beyond() const
    {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) most = __vmaxu2(most, w[j] & 0x7fff7fffu);
        }
        return (most & 0xffffu) >= Deq<T>::kLimit || (most >> 16) >= Deq<T>::kLimit;
    }
    // The inputs, and (fast) what the accumulators of each group and row start with: the pieces of a group are
    // those of G / 8 neighbouring lanes.  Rows behind the last one stay as they are: a product's column is its row's own.
    __device__ __forceinline__ void store(char *xs, int stride, float *starts, int rows, bool fast) const
    {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = threadIdx.x + i * (kWarps * 32), r = p / kPer, kk = p % kPer * 8;
            if (r >= rows) continue;                          // whole warps: a row has at least 64 pieces
            const int j = (kk >> 4) & 3, c = (kk >> 2) & 3;   // c is 0 or 2
            char *dst = xs + r * stride + (kk >> 6) * 128 + c * 32 + j * 8;
            uint4 u = v[i];
            if (fast) {
                float sum = Deq<T>::sum2(u.x) + Deq<T>::sum2(u.y) + (Deq<T>::sum2(u.z) + Deq<T>::sum2(u.w));
#pragma unroll
                for (int o = 1; o < G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (kk % G == 0) starts[kk / G * (8 * NB) + r] = sum * Deq<T>::kStart;
                u = make_uint4(Deq<T>::stage(u.x), Deq<T>::stage(u.y), Deq<T>::stage(u.z), Deq<T>::stage(u.w));
            }
            *reinterpret_cast<uint2 *>(dst) = make_uint2(u.x, u.y);
            *reinterpret_cast<uint2 *>(dst + 32) = make_uint2(u.z, u.w);
        }
    }
};

// One unit of a feature block: two chunks of 64 inputs, two feature tiles.  st: its stage, xu: the lane's inputs,
// start: the lane's pair of rows' starting values of the unit's first group.
template <class T, int G, int NB, bool FAST>
__device__ __forceinline__ void w4_unit(float (&acc)[2][NB][4], uint32_t st, uint32_t xu, int xrows, uint32_t start)
{
    const int lane = threadIdx.x & 31, g = lane >> 2;
    float part[2][NB][4];
    auto begin = [&](int group) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float v0 = 0.f, v1 = 0.f;
            if (FAST)
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v0), "=f"(v1) : "r"(start + (group * NB + nb) * 32));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                part[t][nb][0] = v0;
                part[t][nb][1] = v1;
                part[t][nb][2] = v0 * 16.f;
                part[t][nb][3] = v1 * 16.f;
            }
        }
    };
    // the group's sums times its scales: features g, g + 8, g + 16, g + 24
    auto flush = [&](int group) {
        uint32_t lo, hi;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(st + kUnitBytes + group * 64 + g * 8));
        const float f0 = FAST ? Deq<T>::kFast[0] : Deq<T>::kExact, f1 = FAST ? Deq<T>::kFast[1] : Deq<T>::kExact;
        const float s[4] = {__uint_as_float(lo << 16) * f0, __uint_as_float(lo & 0xffff0000u) * f1, __uint_as_float(hi << 16) * f0,
                            __uint_as_float(hi & 0xffff0000u) * f1};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][nb][i] = fmaf(s[2 * t + (i >> 1)], part[t][nb][i], acc[t][nb][i]);
    };
    begin(0);
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        uint4 w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) w[t] = lds128(st + (ch * 2 + t) * 512 + lane * 16);
#pragma unroll
        for (int half = 0; half < 2; ++half) {        // two steps of 16 inputs
            uint4 xv[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) xv[nb] = lds128(xu + nb * xrows + ch * 128 + half * 16);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t v = half ? (j ? w[t].w : w[t].z) : (j ? w[t].y : w[t].x), h = v >> 8;
                    uint32_t av[4] = {v & 0x000f000fu, v & 0x00f000f0u, h & 0x000f000fu, h & 0x00f000f0u};
                    if (!FAST) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) av[i] = Deq<T>::exact(av[i], i & 1);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        Deq<T>::mma(part[t][nb], av, j ? xv[nb].z : xv[nb].x, j ? xv[nb].w : xv[nb].y);
                }
            if (G == 32) {
                flush(ch * 2 + half);
                if (ch * 2 + half < 3) begin(ch * 2 + half + 1);
            }
        }
        if (G == 64) {
            flush(ch);
            if (ch == 0) begin(1);
        }
    }
    if (G == 128) flush(0);
}

__device__ __forceinline__ float gelu_of(float a)
{
    // 0.5 a (1 + tanh(z)) = a / (1 + exp(-2 z)),  z = sqrt(2 / pi) (a + 0.044715 a^3)
    const float k0 = 0.7978845608028654f, k1 = 0.044715f * 0.7978845608028654f;
    const float z = a * fmaf(k1, a * a, k0);
    return a / (1.f + expf(-2.f * z));
}

// One pass over the block's share of the weights for up to 8 NB rows.  own: a bit for each row that is the expert's to write.
template <class T, int G, bool GATED, int NB>
__device__ __forceinline__ void w4_pass(const W4Args &a, char *smem, int e, int row0, int rows, unsigned own)
{
    constexpr int kGroups = kUnitK / G;                       // of a unit
    constexpr int kStageBytes = kUnitBytes + kGroups * 64;
    constexpr int kPU = kXUnits / NB;                         // units of staged x
    constexpr int kXStride = kPU * kUnitK * 2 + 16;           // 16: neighbouring rows in different banks
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int fw = kWarps / a.kparts, kpart = warp / fw, slot = warp % fw;
    const int fwt = GATED ? fw / 2 : fw;                      // feature blocks of the block
    const int tile = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const int b = tile * fwt + slot % fwt;
    const bool on = b < a.blocks;
    const uint8_t *base = GATED && slot >= fwt ? a.wv : a.w;
    const size_t eb = static_cast<size_t>(e) * a.blocks + (on ? b : 0);
    const uint8_t *wsrc = base + eb * a.units * kUnitBytes + lane * 16;
    const uint8_t *ssrc = base + a.scales + eb * a.units * (kGroups * 64) + lane * 16;
    const int u0 = static_cast<int>(static_cast<long>(a.units) * split / a.splits);
    const int u1 = static_cast<int>(static_cast<long>(a.units) * (split + 1) / a.splits);

    char *xs = smem + kWarps * kStages * kStageBytes;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
    float *starts = reinterpret_cast<float *>(xs + 8 * NB * kXStride);
    const uint32_t xaddr = smem_u32(xs) + g * kXStride + c * 32, saddr = smem_u32(starts) + c * 8;

    float acc[2][NB][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][nb][i] = 0.f;

    int left = on && u0 + kpart < u1 ? (u1 - u0 - kpart + a.kparts - 1) / a.kparts : 0, put = 0;   // units to copy, the next one's stage
    const uint8_t *wnext = wsrc + static_cast<size_t>(u0 + kpart) * kUnitBytes;
    const uint8_t *snext = ssrc + static_cast<size_t>(u0 + kpart) * (kGroups * 64);
    const int wstep = a.kparts * kUnitBytes, sstep = a.kparts * (kGroups * 64);
    const uint32_t to = ring + lane * 16;
    auto issue = [&]() {
        if (left > 0) {
            const uint32_t dst = to + put * kStageBytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) cp16(dst + i * 512, wnext + i * 512);
            if (lane < 4 * kGroups) cp16(dst + kUnitBytes, snext);
        }
        cp_commit();
        --left;
        wnext += wstep;
        snext += sstep;
        put = put + 1 == kStages ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    int get = 0, u = u0 + kpart;                              // this warp's next unit
    for (int p = u0; p < u1; p += kPU) {
        const int pe = p + kPU < u1 ? p + kPU : u1;
        StageX<T, G, NB, kPU> sx;
        sx.load(a, row0, rows, p * kUnitK, (pe - p) * kUnitK);
        const bool fast = !__syncthreads_or(sx.beyond());     // and the last x is used up
        sx.store(xs, kXStride, starts, rows, fast);
        __syncthreads();
        for (; u < pe; u += a.kparts) {
            cp_wait<kStages - 2>();
            __syncwarp();                                     // the scales are other lanes' copies; the last stage is read
            issue();
            const uint32_t st = ring + get * kStageBytes;
            get = get + 1 == kStages ? 0 : get + 1;
            if (!on) continue;
            const uint32_t xu = xaddr + (u - p) * (kUnitK * 2), sa = saddr + (u - p) * (kGroups * 8 * NB * 4);
            if (fast) w4_unit<T, G, NB, true>(acc, st, xu, 8 * kXStride, sa);
            else w4_unit<T, G, NB, false>(acc, st, xu, 8 * kXStride, sa);
        }
    }

    // Join: every warp leaves its sums [row][feature] in the ring's place; the cluster's blocks share
    // the outputs and add the splits and warps in order.
    cp_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);
    constexpr int kWarpRed = NB * 8 * kRedStride;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[warp * kWarpRed + (nb * 8 + 2 * c + (i & 1)) * kRedStride + t * 16 + (i >> 1) * 8 + g] = acc[t][nb][i];
    cg::cluster_group cl = cg::this_cluster();
    if (a.splits > 1) cl.sync();
    else __syncthreads();
    const int width = fwt * kBlockF;
    for (int i = split * (kWarps * 32) + threadIdx.x; i < rows * width; i += a.splits * (kWarps * 32)) {
        const int n = i / width, f = i - n * width;           // width: a power of two times 32
        const int feature = tile * width + f;
        if (feature >= a.N || !(own >> n & 1)) continue;
        float v[2] = {0.f, 0.f};
        for (int s = 0; s < a.splits; ++s) {
            const float *src = a.splits > 1 ? cl.map_shared_rank(red, s) : red;
            for (int kp = 0; kp < a.kparts; ++kp)
#pragma unroll
                for (int q = 0; q < (GATED ? 2 : 1); ++q)
                    v[q] += src[(kp * fw + q * fwt + f / kBlockF) * kWarpRed + n * kRedStride + f % kBlockF];
        }
        const float y = GATED ? gelu_of(v[0]) * v[1] : v[0];
        const size_t at = static_cast<size_t>(row0 + n) * a.N + feature;
        if (a.out_f32) static_cast<float *>(a.y)[at] = y;
        else static_cast<T *>(a.y)[at] = from_f32<T>(y);
    }
    // no block overwrites its sums, or ends, while another reads them
    if (a.splits > 1) cl.sync();
    else __syncthreads();
}

// the n-th expert that has rows, and its rows; the whole warp asks together.  falls: the offsets go down somewhere so far
// (or in the same 32), which is the only way for an earlier range to hold one of these rows
__device__ __forceinline__ bool busy_expert(const W4Args &a, int n, int &e, int &r0, int &r1, bool &falls)
{
    falls = false;
    if (!a.offsets) {
        e = 0;
        r0 = 0;
        r1 = a.R;
        return n == 0;
    }
    const int lane = threadIdx.x & 31;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int mine = e0 + lane;
        int lo = 0, hi = 0;
        if (mine < a.E) {
            lo = max(__ldg(a.offsets + mine), 0);
            hi = __ldg(a.offsets + mine + 1);
        }
        falls |= __any_sync(0xffffffffu, hi < lo);
        hi = min(hi, a.R);
        unsigned m = __ballot_sync(0xffffffffu, lo < hi);
        const int here = __popc(m);
        if (n < here) {
            for (; n > 0; --n) m &= m - 1;
            const int at = __ffs(m) - 1;
            e = e0 + at;
            r0 = __shfl_sync(0xffffffffu, lo, at);
            r1 = __shfl_sync(0xffffffffu, hi, at);
            return true;
        }
        n -= here;
    }
    return false;
}

// the rows r0 .. r0 + 31 that no earlier expert's range holds, a bit each: a row in several ranges is the first one's,
// whichever block comes first
__device__ __forceinline__ unsigned rows_owned(const int *offsets, int e, int r0)
{
    const int r = r0 + (threadIdx.x & 31);
    bool mine = true;
    for (int i = 0; i < e; ++i) mine &= r < __ldg(offsets + i) || r >= __ldg(offsets + i + 1);
    return __ballot_sync(0xffffffffu, mine);
}

// MAXNB: the most slabs of 8 rows an expert can have (1, 2, or 4: any number); fewer leave the registers to the others.
template <class T, int G, bool GATED, int MAXNB>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_kernel(W4Args a)
{
    extern __shared__ __align__(16) char w4_smem[];
    op_begin();
    // All blocks of a cluster have the same expert: they leave, and pass, together.  The grid has a row of blocks for
    // every expert that can have work, not for every expert.
    for (int i = blockIdx.y;; i += gridDim.y) {
        int e, r0, r1;
        bool falls;
        if (!busy_expert(a, i, e, r0, r1, falls)) return;
        for (; r0 < r1; r0 += 32) {
            const int rows = min(r1 - r0, 32);
            const unsigned own = falls ? rows_owned(a.offsets, e, r0) : ~0u;
            if (MAXNB == 1 || rows <= 8) {
                w4_pass<T, G, GATED, 1>(a, w4_smem, e, r0, rows, own);
                continue;
            }
            if constexpr (MAXNB > 1) {
                if (MAXNB == 2 || rows <= 16) {
                    w4_pass<T, G, GATED, 2>(a, w4_smem, e, r0, rows, own);
                    continue;
                }
            }
            if constexpr (MAXNB > 2) w4_pass<T, G, GATED, 4>(a, w4_smem, e, r0, rows, own);
        }
    }
}

constexpr int smem_bytes(int G)
{
    // the ring, x with its rows' padding (most with four slabs of 8 rows), the starting values
    return kWarps * kStages * (kUnitBytes + kUnitK / G * 64) + 8 * (kXUnits * kUnitK * 2) + 4 * 8 * 16 +
           kXUnits * (kUnitK / G) * 8 * 4;
}

// How a call is cut: kparts warps share a feature block's inputs, `splits` blocks of a cluster the input range.
// The estimate counts microseconds as measured here with a ring of four stages (three now; it only ranks the cuts): a
// warp's step (one unit, eight warps a block) takes 0.53 in a block that has an SM to itself and 0.9 where two share one; a
// block's start and end 3, plus 0.17 for every row of every phase of staged x, plus 2 for a cluster.  slots: blocks that run
// together, fewer where clusters do not fill the groups of SMs, as measured on one B200.  It takes the rows to be spread over as
// many experts as can have some; where a batch goes to few of many, more splits would serve it better.  Examples (us): 2
// experts of 32768 x 6144, one row each, 5 splits (chosen) 48, 4 splits of two warps an input range 54, 2 of two 60, neither
// 123; 64 experts of 2048 x 1408, 2 kparts (chosen) 28.0, neither 30.1, 2 splits 34.0.
struct W4Cut {
    int splits, kparts;
};

W4Cut cut_of(int blocks, int units, int busy, int rows, bool gated)
{
    static const int slots[9] = {0, 296, 296, 279, 284, 280, 270, 259, 264};
    const int slabs = rows <= 8 ? 1 : rows <= 16 ? 2 : 4, phase = kXUnits / slabs;
    W4Cut best{1, 1};
    double least = 0;
    for (int kp = 1; kp <= (gated ? 4 : 8); kp *= 2) {
        const int fwt = kWarps / kp / (gated ? 2 : 1);
        const long tiles = static_cast<long>((blocks + fwt - 1) / fwt) * busy;
        for (int sp = 1; sp <= 8 && sp <= units; ++sp) {
            const long ctas = tiles * sp, full = ctas / slots[sp], rest = ctas - full * slots[sp];
            const int share = (units + sp - 1) / sp, walk = (share + kp - 1) / kp, phases = (share + phase - 1) / phase;
            const double ends = 3 + 0.17 * (rows < 32 ? rows : 32) * phases + (sp > 1 ? 2 : 0);
            double cost = full * (0.9 * walk + ends);
            if (rest) cost += (rest <= kSms && sp <= 2 ? 0.53 : 0.9) * walk + ends;
            if (least == 0 || cost < least) {
                least = cost;
                best = W4Cut{sp, kp};
            }
        }
    }
    return best;
}

template <class T, int G, bool GATED, int MAXNB>
cudaError_t launch_w4_rows(const W4Args &a, dim3 grid, cudaStream_t s)
{
    constexpr int smem = smem_bytes(G);
    static_assert(smem >= kWarps * 4 * 8 * kRedStride * 4, "the partial sums take the ring's place");
    const cudaError_t e =
        cudaFuncSetAttribute(w4_kernel<T, G, GATED, MAXNB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
    }
    return op_launch(w4_kernel<T, G, GATED, MAXNB>, grid, dim3(kWarps * 32), smem, s, a.splits, a);
}

template <class T, int G, bool GATED>
cudaError_t launch_w4(W4Args a, cudaStream_t s)
{
    // at most as many experts have work as there are rows
    const int busy = a.offsets && a.R < a.E ? a.R : a.E;
    const W4Cut cut = cut_of(a.blocks, a.units, busy, (a.R + busy - 1) / busy, GATED);
    a.splits = cut.splits;
    a.kparts = cut.kparts;
    const int fwt = kWarps / a.kparts / (GATED ? 2 : 1);
    const dim3 grid(static_cast<unsigned>((a.blocks + fwt - 1) / fwt * a.splits), busy);
    if (a.R <= 8) return launch_w4_rows<T, G, GATED, 1>(a, grid, s);
    return a.R <= 16 ? launch_w4_rows<T, G, GATED, 2>(a, grid, s) : launch_w4_rows<T, G, GATED, 4>(a, grid, s);
}

template <class T>
cudaError_t w4_by_group(int G, const W4Args &a, cudaStream_t s)
{
    if (a.wv) return G == 32 ? launch_w4<T, 32, true>(a, s) : G == 64 ? launch_w4<T, 64, true>(a, s) : launch_w4<T, 128, true>(a, s);
    return G == 32 ? launch_w4<T, 32, false>(a, s) : G == 64 ? launch_w4<T, 64, false>(a, s) : launch_w4<T, 128, false>(a, s);
}

int w4_sizes(int E, int K, int N, int G)
{
    if (E < 1 || K < 1 || N < 1 || K > 131072 || N > 131072) return MOE_EINVAL;
    if (E > kMaxWExperts || (G != 32 && G != 64 && G != 128)) return MOE_EUNSUPPORTED;
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API long long moe_w4_packed_bytes(int E, int K, int N, int group)
{
    const int rc = w4_sizes(E, K, N, group);
    return rc != MOE_OK ? rc : static_cast<long long>(shape_of(E, K, N, group).bytes);
}

extern "C" MOE_API int moe_w4_pack(int E, int K, int N, int group, const int8_t *q, const void *scales, void *packed,
                                   void *stream)
{
    int rc = w4_sizes(E, K, N, group);
    if (rc != MOE_OK) return rc;
    if (!op_ptr(q) || !op_ptr(scales) || !op_ptr(packed)) return MOE_EINVAL;
    const W4Shape sh = shape_of(E, K, N, group);
    if (op_overlap(q, static_cast<size_t>(E) * K * N, packed, sh.bytes) ||
        op_overlap(scales, static_cast<size_t>(E) * ((K + group - 1) / group) * N * 2, packed, sh.bytes))
        return MOE_EINVAL;
    if ((rc = op_device()) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *out = static_cast<uint8_t *>(packed);
    int *flag = reinterpret_cast<int *>(out + sh.bytes - kTail);
    const size_t words = sh.scales / 4, nscales = (sh.bytes - kTail - sh.scales) / 2;
    int bad = 0;
    if (cudaMemsetAsync(flag, 0, kTail, s) != cudaSuccess ||
        op_launch(w4_pack_kernel, dim3(static_cast<unsigned>((words + 255) / 256)), dim3(256), 0, s, 1, sh, q,
                  reinterpret_cast<uint32_t *>(out), flag) != cudaSuccess ||
        op_launch(w4_pack_scales_kernel, dim3(static_cast<unsigned>((nscales + 255) / 256)), dim3(256), 0, s, 1, sh,
                  static_cast<const __nv_bfloat16 *>(scales), reinterpret_cast<__nv_bfloat16 *>(out + sh.scales)) !=
            cudaSuccess ||
        cudaMemcpyAsync(&bad, flag, sizeof bad, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ECUDA;
    }
    return bad ? MOE_ERANGE : MOE_OK;
}

extern "C" MOE_API int moe_w4_matvec(int dtype, int out_dtype, int E, int K, int N, int group, int R, const void *x,
                                     const int32_t *offsets, const void *packed, const void *packed_v, void *y,
                                     void *stream)
{
    int rc = w4_sizes(E, K, N, group);
    if (rc != MOE_OK) return rc;
    if (!dtype_known(dtype) || !dtype_known(out_dtype) || R < 0) return MOE_EINVAL;
    if (dtype == MOE_F32 || (out_dtype != dtype && out_dtype != MOE_F32) || R > kMaxRows) return MOE_EUNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!op_ptr(x) || !op_ptr(packed) || !op_ptr(y) || !op_aligned16(offsets) || !op_aligned16(packed_v)) return MOE_EINVAL;
    if (!offsets && E != 1) return MOE_EINVAL;
    const W4Shape sh = shape_of(E, K, N, group);
    const size_t yb = static_cast<size_t>(R) * N * dtype_size(out_dtype);
    if (op_overlap(x, static_cast<size_t>(R) * K * 2, y, yb) || op_overlap(packed, sh.bytes, y, yb) ||
        op_overlap(packed_v, sh.bytes, y, yb) || op_overlap(offsets, (static_cast<size_t>(E) + 1) * 4, y, yb))
        return MOE_EINVAL;
    if ((rc = op_device()) != MOE_OK) return rc;
    const W4Args a{E, K, N, R, sh.blocks, sh.units, sh.scales, x, offsets, static_cast<const uint8_t *>(packed),
                   static_cast<const uint8_t *>(packed_v), y, out_dtype == MOE_F32, 1, 1};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return (dtype == MOE_BF16 ? w4_by_group<__nv_bfloat16>(group, a, s) : w4_by_group<__half>(group, a, s)) == cudaSuccess
               ? MOE_OK
               : MOE_ECUDA;
}
