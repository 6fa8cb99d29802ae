// twell_norm.cu -- the residual addition and RMS norm that stand before the FFN, forward and backward.
//
//   h = x + r,  s = 1 / sqrt(mean(h^2) + eps),  y = h s w
//   dx = s (g - xh mean(g xh)) + dh  with  xh = h s, g = dy w;   dw = sum over rows of dy xh
//
// Both passes are bounded by memory traffic where rows are wide: every element is read and written once, and a row
// stays in registers between its statistics and its output. A row is spread over `wpr` warps, CH chunks of 8 elements
// a thread. 16-bit rows are bounded as much by the instructions, so that the arithmetic is on pairs of fp32 numbers
// and a row's sum takes one exchange (30000 x 1024, fp32 stream, into e4m3: 56.1 us -> 49.8, what its bytes take). All
// sums are in fp32; y, the 8-bit codes and the gradients are rounded once, from the fp32 values (y from the unrounded
// h, so that it does not depend on the residual stream's type).
#include "twell_common.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxThreads = 1024;  // with one chunk a thread
constexpr int kNormLongThreads = 512;  // with more
constexpr int max_threads(int ch) { return ch == 1 ? kNormMaxThreads : kNormLongThreads; }
constexpr int kNormMinThreads = 128;  // rows of few columns share a block of this many threads

// How a row of d columns is spread over a block: at least `least` chunks of 8 elements a thread (`ch`), `wpr` warps a
// row, `rpb` rows a block. The backward pass takes one chunk a thread as far as a block goes: a row's values and its
// share of dw fill the registers (16384 rows of 2560: 103.8 us with one, 105.6 with two, 137.4 with four; 3000 rows of
// 8192 in bf16: 48.5 and 61.7). The forward pass: fwd_chunks.
struct NormShape {
    int ch, wpr, rpb;
    explicit NormShape(int d, int least = 1)
    {
        const int chunks = d / 8;
        ch = chunks <= kNormMaxThreads ? least : 4;
        wpr = (chunks + 32 * ch - 1) / (32 * ch);
        rpb = wpr * 32 >= kNormMinThreads ? 1 : kNormMinThreads / (wpr * 32);
    }
    int threads() const { return 32 * wpr * rpb; }
};
// A thread's row in its block and place in the row. Several rows a block: of one or two warps each (no division).
struct RowPlace {
    int sub, t;
    __device__ __forceinline__ RowPlace(int wpr, int rpb) : sub(0), t(static_cast<int>(threadIdx.x))
    {
        static_assert(kNormMinThreads == 128, "rows that share a block have one or two warps");
        if (rpb > 1) {
            sub = t >> (4 + wpr);
            t -= sub << (4 + wpr);
        }
    }
};

// How a thread takes part in the sums over its row: its warp's place in the row's slot of shared memory. Slots of up to
// 8 warps are read whole by every thread, so that they are filled up with zeros to 4 or 8.
struct RowSlot {
    int wpr, first, warp, fill;
    __device__ __forceinline__ RowSlot(int wpr, int sub, int t)
        : wpr(wpr), first(sub * 4), warp(sub * 4 + (t >> 5)), fill((t >> 5) == wpr - 1 && wpr <= 8 ? (8 - wpr) & 3 : 0)
    {
    }
};

// Sum (or maximum, of values >= 0) over a row; every thread of the block takes part.
template <bool MAX>
__device__ __forceinline__ float warp_reduce(float v)
{
    if constexpr (MAX) {
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, const RowSlot& k)
{
    v = warp_reduce<MAX>(v);
    if (k.wpr == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane <= k.fill) red[k.warp + lane] = lane == 0 ? v : 0.0f;
    __syncthreads();
    if (k.wpr <= 8) {
        const float4 a = *reinterpret_cast<const float4*>(red + k.first);
        v = MAX ? fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)) : (a.x + a.y) + (a.z + a.w);
        if (k.wpr > 4) {
            const float4 b = *reinterpret_cast<const float4*>(red + 4);
            const float u = MAX ? fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)) : (b.x + b.y) + (b.z + b.w);
            v = MAX ? fmaxf(v, u) : v + u;
        }
        return v;
    }
    return warp_reduce<MAX>(lane < k.wpr ? red[lane] : 0.0f);
}

// The sum over a row of which each thread holds CH chunks' sums, in the order of one chunk a thread, so that a row's
// result does not depend on how many rows are with it: the chunks' butterflies over the lanes share their shuffles (the
// halves of the lanes go on with one each), and the shared memory has a place for each chunk of each warp.
template <int CH>
__device__ __forceinline__ float row_sum(const float (&v)[CH], float* red, const RowSlot& k, int d)
{
    if constexpr (CH == 1) {
        return row_reduce<false>(v[0], red, k);
    } else {
        const int lane = threadIdx.x & 31, warps = (d + 255) / 256;  // warps of a row at one chunk a thread
        float s[CH / 2];
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
            const float keep = lane < 16 ? v[2 * i] : v[2 * i + 1], give = lane < 16 ? v[2 * i + 1] : v[2 * i];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
        }
        int chunk = lane >> 4;
        float u = s[0];
        if constexpr (CH == 4) {
            const bool low = (lane & 8) == 0;
            u = (low ? s[0] : s[1]) + __shfl_xor_sync(0xffffffffu, low ? s[1] : s[0], 8);
            chunk += low ? 0 : 2;
        } else {
            u += __shfl_xor_sync(0xffffffffu, u, 8);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        const int first = k.first * (CH / 2), mine = k.warp - k.first;
        if ((lane & (32 / CH - 1)) == 0) red[first + chunk * k.wpr + mine] = u;
        // an odd number of warps at two chunks leaves two places of the last four
        if (CH == 2 && (k.wpr & 1) && mine == 0 && (lane & 15) == 1) red[first + 2 * k.wpr + chunk] = 0.0f;
        __syncthreads();
        if (warps <= 8) {
            const float4 a = *reinterpret_cast<const float4*>(red + first);
            u = (a.x + a.y) + (a.z + a.w);
            if (warps > 4) {
                const float4 b = *reinterpret_cast<const float4*>(red + first + 4);
                u += (b.x + b.y) + (b.z + b.w);
            }
            return u;
        }
        u = lane < warps ? red[lane] : 0.0f;
        if (lane + 32 < warps) u += red[lane + 32];
        return warp_reduce<false>(u);
    }
}

// 8 elements as they lie in memory, to be unpacked later.
template <typename E>
struct Raw8 {
    uint4 v[sizeof(E) / 2];
    __device__ __forceinline__ void load(const E* p)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i)
            v[i] = *reinterpret_cast<const uint4*>(p + i * (16 / sizeof(E)));
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(F2 (&o)[4]) const
    {
        if constexpr (sizeof(E) == 2) {
            float f[8];
            unpack16(v[0], f, static_cast<__nv_bfloat16*>(nullptr));
            to_f2(f, o);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[2 * i] = F2::of(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                o[2 * i + 1] = F2::of(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        }
    }
};

struct NormFwdArgs {
    const void* x;
    const void* res;
    const void* w;
    void* h;
    void* y;
    uint8_t* y8;
    float* scale;
    float* rstd;
    int N, d, group, ng, wpr, rpb;
    float eps, inv_d;
};

// a.rpb rows a block.
template <typename T, typename R, int CH>
__global__ void __launch_bounds__(max_threads(CH)) add_rmsnorm_fwd_kernel(const NormFwdArgs a)
{
    __shared__ __align__(16) float red[2][kNormMaxD / 256];
    pdl_begin();
    const int per_row = 32 * a.wpr;
    const RowPlace at_row(a.wpr, a.rpb);
    const int t = at_row.t, sub = at_row.sub;
    const RowSlot slot(a.wpr, sub, t);
    const unsigned row = blockIdx.x * a.rpb + sub, d = a.d;
    const bool live = row < static_cast<unsigned>(a.N);
    const int chunks = live ? d / 8 : 0;
    const size_t base = static_cast<size_t>(row) * d + t * 8;
    const int step = per_row * 8;

    Raw8<T> x[CH];  // unpacked only when every load is under way
    Raw8<R> r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        x[i].clear();
        r[i].clear();
        if (t + i * per_row < chunks) {
            x[i].load(static_cast<const T*>(a.x) + base + i * step);
            if (a.res != nullptr) r[i].load(static_cast<const R*>(a.res) + base + i * step);
        }
    }
    F2 h[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        F2 u[4];
        x[i].get(h[i]);
        r[i].get(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[i][e] = h[i][e] + u[e];
    }
    float part[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        F2 ss2 = F2::of(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss2 = fma2(h[i][e], h[i][e], ss2);
        float odd;
        ss2.get(part[i], odd);
        part[i] += odd;
        if (a.h != nullptr && t + i * per_row < chunks) store8(static_cast<R*>(a.h) + base + i * step, h[i]);
    }
    const float ss = row_sum<CH>(part, red[0], slot, a.d);
    const float s = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    if (a.rstd != nullptr && t == 0 && t < chunks) a.rstd[row] = s;

    const F2 s2 = F2::of(s, s);
    float top[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        top[i] = 0.0f;
        if (t + i * per_row < chunks) {
            F2 w[4];
            load8(static_cast<const T*>(a.w) + t * 8 + i * step, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[i][e] = h[i][e] * s2 * w[e];
            if (a.y != nullptr) store8(static_cast<T*>(a.y) + base + i * step, h[i]);
            if (a.y8 != nullptr) {
                float v[8];
                from_f2(h[i], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) top[i] = fmaxf(top[i], fabsf(v[e]));
            }
        }
    }
    if (a.y8 == nullptr) return;
    if (a.group == a.d) {
#pragma unroll
        for (int i = 1; i < CH; ++i) top[0] = fmaxf(top[0], top[i]);
        top[0] = row_reduce<true>(top[0], red[1], slot);
#pragma unroll
        for (int i = 1; i < CH; ++i) top[i] = top[0];
    } else {  // groups of 128 columns: 16 lanes next to each other
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < CH; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = t + i * per_row;
        if (c >= chunks) continue;
        const Scale8 q = Scale8::of(top[i]);
        *reinterpret_cast<uint2*>(a.y8 + base + i * step) = q.pack8(h[i]);
        if (a.group == a.d ? c == 0 : (c & 15) == 0)
            a.scale[static_cast<size_t>(row) * static_cast<unsigned>(a.ng) + (c >> 4)] = q.scale();
    }
}

struct NormBwdArgs {
    const void* dy;
    const void* h;
    const void* w;
    const void* dh;
    const float* rstd;
    void* dx;
    float* part;  // [gridDim.x, d]
    int N, d, wpr, rpb;
    float inv_d;
};

// Rows blockIdx.x * rpb + ..., then every gridDim.x * rpb-th one; the rows' shares of dw are added in registers and
// a block leaves one partial row of dw, its rows' sums added in order. The weights wait in shared memory, read and
// written by their own thread alone: there are no registers for them beside a row's.
// With one chunk a thread an SM holds 1024 threads (64 registers each), with more 512.
constexpr int norm_threads_per_sm(int ch) { return ch == 1 ? 1024 : 512; }
template <typename T, typename R, typename G, int CH>
__global__ void __launch_bounds__(max_threads(CH), norm_threads_per_sm(CH) / max_threads(CH))
    add_rmsnorm_bwd_kernel(const NormBwdArgs a)
{
    __shared__ __align__(16) float red[2][kNormMaxThreads / 32];
    // A thread's 8 weights while the block goes over its rows, then its share of dw where a block has several rows.
    extern __shared__ float4 own[];  // [2][blockDim.x]
    pdl_begin();
    const int per_row = 32 * a.wpr;
    const RowPlace at_row(a.wpr, a.rpb);
    const int t = at_row.t, sub = at_row.sub;
    const RowSlot slot(a.wpr, sub, t);
    const int chunks = a.d / 8, step = per_row * 8;
    const F2 zero = F2::of(0.0f, 0.0f);
    F2 dw[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[i][e] = zero;
    }
    auto keep = [&](const F2 (&v)[4]) {
        float f[8];
        from_f2(v, f);
        own[threadIdx.x] = make_float4(f[0], f[1], f[2], f[3]);
        own[blockDim.x + threadIdx.x] = make_float4(f[4], f[5], f[6], f[7]);
    };
    auto kept = [&](F2 (&v)[4], int thread) {
        const float4 l = own[thread], h = own[blockDim.x + thread];
        v[0] = F2::of(l.x, l.y), v[1] = F2::of(l.z, l.w), v[2] = F2::of(h.x, h.y), v[3] = F2::of(h.z, h.w);
    };
    if (CH == 1) {
        F2 w[4] = {zero, zero, zero, zero};
        if (t < chunks) load8(static_cast<const T*>(a.w) + t * 8, w);
        keep(w);
    }
    // With 16-bit h and gradients the next row is requested before this one is reduced: too little would be in flight
    // otherwise (6000 x 5120: 72.5 -> 54.0 us, 16384 x 2048 without dh 45.2 -> 41.7). Wider rows would not fit the registers
    // (fp32 gradients of 31220 x 368: 25.8 us so, 31.0 with the next row).
    constexpr bool kAhead = CH == 1 && sizeof(R) == 2 && sizeof(G) == 2;
    const unsigned N = a.N, rows = gridDim.x * a.rpb;  // no sum of the two passes 32 bits
    Raw8<G> next_dy;
    Raw8<R> next_h;
    float next_s = 0.0f;
    next_dy.clear();  // zeros for the threads past the row's end, which request nothing
    next_h.clear();
    auto request = [&](unsigned row, size_t at) {
        if (row < N) {
            next_s = a.rstd[row];
            if (t < chunks) {
                next_dy.load(static_cast<const G*>(a.dy) + at);
                next_h.load(static_cast<const R*>(a.h) + at);
            }
        }
    };
    unsigned row = blockIdx.x * a.rpb + sub;
    size_t at = static_cast<size_t>(row) * a.d + t * 8;
    if constexpr (kAhead) request(row, at);
    int flip = 0;
    const size_t far = static_cast<size_t>(rows) * a.d;
    for (; row - sub < N; row += rows, at += far, flip ^= 1) {
        const bool live = row < N;
        const int mine = live ? chunks : 0;
        const float s = kAhead ? next_s : live ? a.rstd[row] : 0.0f;
        const F2 s2 = F2::of(s, s);
        Raw8<G> raw_dy[CH], dh[CH];  // unpacked only when every load is under way
        Raw8<R> raw_h[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (!kAhead) {
                raw_dy[i].clear();
                raw_h[i].clear();
            }
            if (t + i * per_row < mine) {
                if (!kAhead) {
                    raw_dy[i].load(static_cast<const G*>(a.dy) + at + i * step);
                    raw_h[i].load(static_cast<const R*>(a.h) + at + i * step);
                }
                if (CH == 1 && a.dh != nullptr) dh[i].load(static_cast<const G*>(a.dh) + at + i * step);
            }
        }
        F2 dy[CH][4], xh[CH][4];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if constexpr (kAhead) {
                next_dy.get(dy[i]);
                next_h.get(xh[i]);
            } else {
                raw_dy[i].get(dy[i]);
                raw_h[i].get(xh[i]);
            }
        }
        F2 p2 = zero;
        if (live) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                F2 w[4] = {zero, zero, zero, zero};
                if (CH == 1) kept(w, threadIdx.x);
                else if (t + i * per_row < mine) load8(static_cast<const T*>(a.w) + t * 8 + i * step, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xh[i][e] = xh[i][e] * s2;
                    dw[i][e] = fma2(dy[i][e], xh[i][e], dw[i][e]);
                    dy[i][e] = dy[i][e] * w[e];
                    p2 = fma2(dy[i][e], xh[i][e], p2);
                }
            }
        }
        if constexpr (kAhead) request(row + rows, at + far);
        float p, pb;
        p2.get(p, pb);
        p = row_reduce<false>(p + pb, red[flip], slot) * -a.inv_d;
        p2 = F2::of(p, p);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (t + i * per_row >= mine) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) dy[i][e] = fma2(xh[i][e], p2, dy[i][e]) * s2;
            if (a.dh != nullptr) {
                F2 o[4];
                if (CH > 1) dh[i].load(static_cast<const G*>(a.dh) + at + i * step);  // no registers for it before
                dh[i].get(o);
#pragma unroll
                for (int e = 0; e < 4; ++e) dy[i][e] = dy[i][e] + o[e];
            }
            store8(static_cast<G*>(a.dx) + at + i * step, dy[i]);
        }
    }
    if (CH == 1 && a.rpb > 1) {
        keep(dw[0]);
        __syncthreads();
        if (sub > 0) return;
        for (int s = 1; s < a.rpb; ++s) {
            F2 u[4];
            kept(u, s * per_row + t);
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[0][e] = dw[0][e] + u[e];
        }
    }
    float* part = a.part + static_cast<size_t>(blockIdx.x) * a.d + t * 8;
#pragma unroll
    for (int i = 0; i < CH; ++i)
        if (t + i * per_row < chunks) store8(part + i * step, dw[i]);
}

// dw[c] = sum over p of part[p][c]: 8 columns (a 32-byte sector) a block, 128 threads a column, each over every 128th
// partial row, their sums added by a fixed tree: the same dw from call to call.
constexpr int kDwCols = 8, kDwWays = 128;
__global__ void __launch_bounds__(kDwCols * kDwWays) add_rmsnorm_dw_kernel(const float* __restrict__ part, int P, int d,
                                                                           float* __restrict__ dw)
{
    __shared__ float sums[kDwWays][kDwCols + 1];
    pdl_begin();
    const int c = threadIdx.x % kDwCols, way = threadIdx.x / kDwCols;
    float v = 0.0f;
#pragma unroll 4
    for (int p = way; p < P; p += kDwWays) v += part[static_cast<size_t>(p) * d + blockIdx.x * kDwCols + c];
    sums[way][c] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31, col = threadIdx.x >> 5;
    if (col >= kDwCols) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kDwWays / 32; ++i) v += sums[32 * i + lane][col];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) dw[blockIdx.x * kDwCols + col] = v;
}

// Blocks of the backward pass: what an SM holds at once, on each SM, no more than rows. A block more than that
// would run alone at the end (2560 columns, 320 threads: 103.8 us with the 3 that fit, 124.5 with 4).
int bwd_blocks(int N, const NormShape& S, int sms)
{
    const int per_sm = std::max(1, norm_threads_per_sm(S.ch) / S.threads());
    const long long need = (static_cast<long long>(N) + S.rpb - 1) / S.rpb;
    return static_cast<int>(std::min<long long>(need, static_cast<long long>(sms) * per_sm));
}
// The workspace is sized for this many SMs, whatever the device, so that its size is the same with
// and without one; the launch uses the device's own number up to it.
constexpr int kNormMaxSms = 160;

// Chunks a thread of the forward pass. One while the rows do not fill the device's threads; then two, so that each
// thread has more under way and a row's sums take fewer warps (30000 x 1024 into e4m3 without a stream 32.5 -> 25.4 us,
// 2000 x 2048 in bf16 5.7 -> 5.5; with an fp32 stream within 3% either way), and four where a row of 16-bit elements is
// wide (8192 columns in bf16: 34.6 us with one, 33.5 with two, 29.4 with four; but 1024 columns 33.4 with two, 34.7 with
// four). A row of 256 columns or fewer is one warp's.
int fwd_chunks(int N, int d, twell_dtype res_dtype, int sms)
{
    if (d <= 256 || static_cast<long long>(N) * d <= 8ll * 2048 * sms) return 1;
    return res_dtype == TWELL_BF16 && d >= 4096 ? 4 : 2;
}

template <typename T, typename R>
twell_status run_norm_fwd(const NormFwdArgs& a, const NormShape& S, cudaStream_t s)
{
    auto kern = S.ch == 1   ? add_rmsnorm_fwd_kernel<T, R, 1>
                : S.ch == 2 ? add_rmsnorm_fwd_kernel<T, R, 2>
                            : add_rmsnorm_fwd_kernel<T, R, 4>;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>((static_cast<long long>(a.N) + S.rpb - 1) / S.rpb)),
                                  dim3(S.threads()), 0, s, a);
}

template <typename T, typename R, typename G>
twell_status run_norm_bwd(const NormBwdArgs& a, const NormShape& S, int blocks, float* dw, cudaStream_t s)
{
    auto kern = S.ch == 1 ? add_rmsnorm_bwd_kernel<T, R, G, 1> : add_rmsnorm_bwd_kernel<T, R, G, 4>;
    twell_status st = twell_host::launch_dep(kern, dim3(blocks), dim3(S.threads()), S.ch == 1 ? S.threads() * 32 : 0, s, a);
    if (st != TWELL_OK) return st;
    return twell_host::launch_dep(add_rmsnorm_dw_kernel, dim3(a.d / kDwCols), dim3(kDwCols * kDwWays), 0, s,
                                  static_cast<const float*>(a.part), blocks, a.d, dw);
}

}  // namespace
}  // namespace twell

size_t twell_host::norm_bwd_ws_bytes(int N, int d)
{
    if (N <= 0 || d % 8 != 0 || d > twell::kNormMaxD) return 0;
    const twell::NormShape S(d);
    return static_cast<size_t>(twell::bwd_blocks(N, S, twell::kNormMaxSms)) * d * 4;
}

using namespace twell_host;

static bool norm_types_ok(twell_dtype dtype, twell_dtype res_dtype)
{
    return (dtype == TWELL_BF16 && (res_dtype == TWELL_BF16 || res_dtype == TWELL_F32)) ||
           (dtype == TWELL_F32 && res_dtype == TWELL_F32);
}

extern "C" twell_status twell_add_rmsnorm_fwd(const void* x, const void* res, const void* w, int32_t N, int32_t d,
                                              float eps, twell_dtype dtype, twell_dtype res_dtype, void* h_out, void* y,
                                              void* y8, float* y8_scale, int32_t group, float* rstd, void* stream)
{
    if (N < 0 || d <= 0 || d % 8 != 0 || w == nullptr || !(eps >= 0.0f)) return TWELL_ERR_INVALID;
    if (y8 != nullptr && group != 0 && group != 128) return TWELL_ERR_UNSUPPORTED;
    if (!norm_types_ok(dtype, res_dtype) || d > twell::kNormMaxD) return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    if (x == nullptr || (y == nullptr && y8 == nullptr) || (y8 != nullptr && y8_scale == nullptr)) return TWELL_ERR_INVALID;
    if (!aligned16(x) || !aligned16(res) || !aligned16(w) || !aligned16(h_out) || !aligned16(y) || !aligned16(y8) ||
        !aligned16(y8_scale) || !aligned16(rstd))
        return TWELL_ERR_INVALID;
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    const twell::NormShape S(d, twell::fwd_chunks(N, d, res_dtype, dev.sm_count));
    const int g = group == 0 || d <= 128 ? d : group;
    const twell::NormFwdArgs a{x,    res, w, h_out, y,  static_cast<uint8_t*>(y8), y8_scale, rstd, N, d,
                               g, (d + g - 1) / g, S.wpr, S.rpb, eps, 1.0f / static_cast<float>(d)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == TWELL_F32) return twell::run_norm_fwd<float, float>(a, S, s);
    if (res_dtype == TWELL_F32) return twell::run_norm_fwd<__nv_bfloat16, float>(a, S, s);
    return twell::run_norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, S, s);
}

extern "C" twell_status twell_add_rmsnorm_bwd(const void* dy, const void* h, const void* w, const float* rstd,
                                              const void* dh, int32_t N, int32_t d, twell_dtype dtype,
                                              twell_dtype res_dtype, twell_dtype grad_dtype, void* dx, float* dw,
                                              void* ws, size_t ws_bytes, void* stream)
{
    if (N < 0 || d <= 0 || d % 8 != 0 || w == nullptr || dw == nullptr || !aligned16(dw)) return TWELL_ERR_INVALID;
    if (!norm_types_ok(dtype, res_dtype) || (grad_dtype != TWELL_BF16 && grad_dtype != TWELL_F32) ||
        d > twell::kNormMaxD)
        return TWELL_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0)
        return cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * 4, s) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
    if (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr) return TWELL_ERR_INVALID;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(w) || !aligned16(rstd) || !aligned16(dh) || !aligned16(dx))
        return TWELL_ERR_INVALID;
    if (ws == nullptr || !aligned16(ws) || ws_bytes < norm_bwd_ws_bytes(N, d)) return TWELL_ERR_WORKSPACE;
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    const twell::NormShape S(d);
    const int blocks = twell::bwd_blocks(N, S, std::min(dev.sm_count, twell::kNormMaxSms));
    const twell::NormBwdArgs a{dy, h, w, dh, rstd, dx, static_cast<float*>(ws), N, d, S.wpr, S.rpb,
                               1.0f / static_cast<float>(d)};
    using bf = __nv_bfloat16;
    const bool g32 = grad_dtype == TWELL_F32;
    if (dtype == TWELL_F32)
        return g32 ? twell::run_norm_bwd<float, float, float>(a, S, blocks, dw, s)
                   : twell::run_norm_bwd<float, float, bf>(a, S, blocks, dw, s);
    if (res_dtype == TWELL_F32)
        return g32 ? twell::run_norm_bwd<bf, float, float>(a, S, blocks, dw, s)
                   : twell::run_norm_bwd<bf, float, bf>(a, S, blocks, dw, s);
    return g32 ? twell::run_norm_bwd<bf, bf, float>(a, S, blocks, dw, s)
               : twell::run_norm_bwd<bf, bf, bf>(a, S, blocks, dw, s);
}
