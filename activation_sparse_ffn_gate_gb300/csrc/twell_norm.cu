// twell_norm.cu -- the residual addition and RMS norm that stand before the FFN, forward and backward.
//
//   h = x + r,  s = 1 / sqrt(mean(h^2) + eps),  y = h s w
//   dx = s (g - xh mean(g xh)) + dh  with  xh = h s, g = dy w;   dw = sum over rows of dy xh
//
// Both passes are bounded by memory traffic: every element is read and written once, and a row stays in
// registers between its statistics and its output. A row is spread over `wpr` warps, CH chunks of 8
// elements a thread. All sums are in fp32; y, the 8-bit codes and the gradients are rounded once, from the
// fp32 values (y from the unrounded h, so that it does not depend on the residual stream's type).
#include "twell_common.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxThreads = 1024;  // with one chunk a thread
constexpr int kNormLongThreads = 512;  // with more
constexpr int max_threads(int ch) { return ch == 1 ? kNormMaxThreads : kNormLongThreads; }
constexpr int kNormMinThreads = 128;  // rows of few columns share a block of this many threads

// How a row of d columns is spread over a block: `ch` chunks of 8 elements a thread, `wpr` warps a row, `rpb` rows
// a block. One chunk a thread as far as a block goes: more threads in flight hide more of the latency than
// longer threads save instructions (16384 rows of 2560, forward into e4m3: 72.7 us with one chunk, 75.0 with two,
// 91.0 with four; backward 103.8, 105.6, 137.4; 3000 rows of 8192 in bf16: 33.4 with one, 42.3 with two, backward
// 48.5 and 61.7).
struct NormShape {
    int ch, wpr, rpb;
    explicit NormShape(int d)
    {
        const int chunks = d / 8;
        ch = chunks <= kNormMaxThreads ? 1 : 4;
        wpr = (chunks + 32 * ch - 1) / (32 * ch);
        rpb = wpr * 32 >= kNormMinThreads ? 1 : kNormMinThreads / (wpr * 32);
    }
    int threads() const { return 32 * wpr * rpb; }
};

// Sum (or maximum, of values >= 0) over the `wpr` warps of a row; every thread of the block takes part.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, int wpr)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (wpr == 1) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp / wpr * wpr;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < wpr ? red[first + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

// 8 elements as they lie in memory, to be unpacked later.
template <typename E>
struct Raw8 {
    uint4 v[sizeof(E) / 2];
    __device__ __forceinline__ void load(const E* p)
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) v[i] = *reinterpret_cast<const uint4*>(p + i * (16 / sizeof(E)));
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&o)[8]) const
    {
        if constexpr (sizeof(E) == 2) {
            unpack16(v[0], o, static_cast<__nv_bfloat16*>(nullptr));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                o[4 * i] = __uint_as_float(v[i].x);
                o[4 * i + 1] = __uint_as_float(v[i].y);
                o[4 * i + 2] = __uint_as_float(v[i].z);
                o[4 * i + 3] = __uint_as_float(v[i].w);
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

// What follows the loads of one row: h = x + r is in `h`, its part of the weights comes from weight(i).
template <typename T, typename R, int CH, typename W>
__device__ __forceinline__ void finish_row(const NormFwdArgs& a, float (&h)[CH][8], long long row, int t, int chunks, size_t base,
                                           float (*red)[kNormMaxThreads / 32], const W& weight)
{
    const int per_row = 32 * a.wpr, step = per_row * 8;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
        if (a.h != nullptr && t + i * per_row < chunks) store8(static_cast<R*>(a.h) + base + i * step, h[i]);
    }
    ss = row_reduce<false>(ss, red[0], a.wpr);
    const float s = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    if (a.rstd != nullptr && t < chunks && t == 0) a.rstd[row] = s;

    float top[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        top[i] = 0.0f;
        if (t + i * per_row < chunks) {
            float w[8];
            weight(i, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = h[i][e] * s * w[e];
                top[i] = fmaxf(top[i], fabsf(h[i][e]));
            }
            if (a.y != nullptr) store8(static_cast<T*>(a.y) + base + i * step, h[i]);
        }
    }
    if (a.y8 == nullptr) return;
    if (a.group == a.d) {
#pragma unroll
        for (int i = 1; i < CH; ++i) top[0] = fmaxf(top[0], top[i]);
        top[0] = row_reduce<true>(top[0], red[1], a.wpr);
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
        const Scale8 q = Scale8::approx(top[i]);
        *reinterpret_cast<uint2*>(a.y8 + base + i * step) = q.pack8(h[i]);
        if (a.group == a.d ? c == 0 : (c & 15) == 0) a.scale[static_cast<size_t>(row) * a.ng + (c >> 4)] = q.scale;
    }
}

// a.rpb rows a block.
template <typename T, typename R, int CH>
__global__ void __launch_bounds__(max_threads(CH)) add_rmsnorm_fwd_kernel(const NormFwdArgs a)
{
    __shared__ float red[2][kNormMaxThreads / 32];
    pdl_begin();
    const int per_row = 32 * a.wpr;
    const int t = static_cast<int>(threadIdx.x) % per_row;
    const long long row = static_cast<long long>(blockIdx.x) * a.rpb + threadIdx.x / per_row;
    const bool live = row < a.N;
    const int chunks = live ? a.d / 8 : 0;
    const size_t base = static_cast<size_t>(live ? row : 0) * a.d + t * 8;
    const int step = per_row * 8;

    float h[CH][8], r[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = r[i][e] = 0.0f;
        if (t + i * per_row < chunks) {
            load8(static_cast<const T*>(a.x) + base + i * step, h[i]);
            if (a.res != nullptr) load8(static_cast<const R*>(a.res) + base + i * step, r[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += r[i][e];
    }
    finish_row<T, R, CH>(a, h, row, t, chunks, base, red,
                         [&](int i, float (&w)[8]) { load8(static_cast<const T*>(a.w) + t * 8 + i * step, w); });
}

// Rows blockIdx.x * rpb + ..., then every gridDim.x * rpb-th one; the next row is requested before this one is reduced,
// the weights stay in registers. One chunk a thread. For 16-bit rows, which put too little in flight one a block:
// 16384 x 2560 with a 16-bit stream 58.6 -> 53.9 us, 30000 x 1024 into e4m3 without one 37.7 -> 34.5. With an fp32
// stream it is not faster (2560 columns 72.9 -> 80.6).
constexpr int kFwdThreadsPerSm = 1024;
template <typename T, typename R>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_fwd_ahead_kernel(const NormFwdArgs a)
{
    __shared__ float red[2][2][kNormMaxThreads / 32];
    pdl_begin();
    const int per_row = 32 * a.wpr;
    const int t = static_cast<int>(threadIdx.x) % per_row, sub = static_cast<int>(threadIdx.x) / per_row;
    const int all = a.d / 8;
    const long long rows = static_cast<long long>(gridDim.x) * a.rpb;
    Raw8<T> next_x, weight;
    Raw8<R> next_r;
    auto request = [&](long long row) {
        next_x.clear();
        next_r.clear();
        if (row < a.N && t < all) {
            const size_t at = static_cast<size_t>(row) * a.d + t * 8;
            next_x.load(static_cast<const T*>(a.x) + at);
            if (a.res != nullptr) next_r.load(static_cast<const R*>(a.res) + at);
        }
    };
    request(static_cast<long long>(blockIdx.x) * a.rpb + sub);
    weight.clear();
    if (t < all) weight.load(static_cast<const T*>(a.w) + t * 8);
    int flip = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * a.rpb; r0 < a.N; r0 += rows, flip ^= 1) {
        const long long row = r0 + sub;
        const bool live = row < a.N;
        float h[1][8], r[8];
        next_x.get(h[0]);
        next_r.get(r);
        request(row + rows);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[0][e] += r[e];
        finish_row<T, R, 1>(a, h, row, t, live ? all : 0, static_cast<size_t>(live ? row : 0) * a.d + t * 8, red[flip],
                            [&](int, float (&w)[8]) { weight.get(w); });
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

// Rows blockIdx.x * rpb + ..., then every gridDim.x * rpb-th one; the weights stay in registers and
// the rows' shares of dw are added there too; a block leaves one partial row of dw, its rows' sums added in order.
// With one chunk a thread an SM holds 1024 threads (64 registers each), with more 512.
constexpr int norm_threads_per_sm(int ch) { return ch == 1 ? 1024 : 512; }
template <typename T, typename R, typename G, int CH>
__global__ void __launch_bounds__(max_threads(CH), norm_threads_per_sm(CH) / max_threads(CH)) add_rmsnorm_bwd_kernel(const NormBwdArgs a)
{
    __shared__ float red[2][kNormMaxThreads / 32];
    __shared__ float rows_dw[8 * kNormMinThreads];  // of a block with several rows
    pdl_begin();
    const int per_row = 32 * a.wpr;
    const int t = static_cast<int>(threadIdx.x) % per_row;
    const int sub = static_cast<int>(threadIdx.x) / per_row;
    const int chunks = a.d / 8, step = per_row * 8;
    constexpr int KW = CH <= 2 ? CH : 1;  // chunks whose weights stay in registers; else they are read again (L1)
    float dw[CH][8], w[KW][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = w[i % KW][e] = 0.0f;
        if (KW == CH && t + i * per_row < chunks) load8(static_cast<const T*>(a.w) + t * 8 + i * step, w[i % KW]);
    }
    const long long rows = static_cast<long long>(gridDim.x) * a.rpb;
    // With 16-bit h the next row is requested before this one is reduced: too little would be in flight otherwise
    // (16384 x 2048, 16-bit gradients: 52.9 -> 44.3 us). With fp32 h it would not fit the registers (1208 columns: 61 -> 75).
    constexpr bool kAhead = CH == 1 && sizeof(R) == 2;
    Raw8<G> next_dy;
    Raw8<R> next_h;
    float next_s = 0.0f;
    auto request = [&](long long row) {
        next_dy.clear();
        next_h.clear();
        next_s = 0.0f;
        if (row < a.N) {
            next_s = a.rstd[row];
            if (t < chunks) {
                next_dy.load(static_cast<const G*>(a.dy) + static_cast<size_t>(row) * a.d + t * 8);
                next_h.load(static_cast<const R*>(a.h) + static_cast<size_t>(row) * a.d + t * 8);
            }
        }
    };
    if constexpr (kAhead) request(static_cast<long long>(blockIdx.x) * a.rpb + sub);
    int flip = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * a.rpb; r0 < a.N; r0 += rows, flip ^= 1) {
        const bool live = r0 + sub < a.N;
        const int mine = live ? chunks : 0;
        const size_t base = static_cast<size_t>(live ? r0 + sub : 0) * a.d + t * 8;
        const float s = kAhead ? next_s : live ? a.rstd[r0 + sub] : 0.0f;
        float dy[CH][8], xh[CH][8], o[CH][8];
        float p = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[i][e] = xh[i][e] = o[i][e] = 0.0f;
            if (kAhead) {
                next_dy.get(dy[i]);
                next_h.get(xh[i]);
            }
            if (t + i * per_row < mine) {
                if (!kAhead) {
                    load8(static_cast<const G*>(a.dy) + base + i * step, dy[i]);
                    load8(static_cast<const R*>(a.h) + base + i * step, xh[i]);
                }
                if (a.dh != nullptr) load8(static_cast<const G*>(a.dh) + base + i * step, o[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (KW != CH && t + i * per_row < mine) load8(static_cast<const T*>(a.w) + t * 8 + i * step, w[i % KW]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[i][e] *= s;
                dw[i][e] = fmaf(dy[i][e], xh[i][e], dw[i][e]);
                dy[i][e] *= w[i % KW][e];
                p = fmaf(dy[i][e], xh[i][e], p);
            }
        }
        if constexpr (kAhead) request(r0 + rows + sub);
        p = row_reduce<false>(p, red[flip], a.wpr) * a.inv_d;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (t + i * per_row >= mine) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] = fmaf(s, fmaf(-xh[i][e], p, dy[i][e]), o[i][e]);
            store8(static_cast<G*>(a.dx) + base + i * step, o[i]);
        }
    }
    if (CH == 1 && a.rpb > 1) {
        store8(rows_dw + threadIdx.x * 8, dw[0]);
        __syncthreads();
        if (sub > 0) return;
        for (int s = 1; s < a.rpb; ++s) {
            float u[8];
            load8(rows_dw + (s * per_row + t) * 8, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[0][e] += u[e];
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

template <typename T, typename R>
twell_status run_norm_fwd(const NormFwdArgs& a, const NormShape& S, int sms, cudaStream_t s)
{
    const long long need = (static_cast<long long>(a.N) + S.rpb - 1) / S.rpb;
    if constexpr (sizeof(R) == 2) {
        if (S.ch == 1) {
            const long long blocks = std::min<long long>(need, static_cast<long long>(sms) * (kFwdThreadsPerSm / S.threads()));
            return twell_host::launch_dep(add_rmsnorm_fwd_ahead_kernel<T, R>, dim3(static_cast<unsigned>(blocks)), dim3(S.threads()), 0, s, a);
        }
    }
    auto kern = S.ch == 1 ? add_rmsnorm_fwd_kernel<T, R, 1> : add_rmsnorm_fwd_kernel<T, R, 4>;
    return twell_host::launch_dep(kern, dim3(static_cast<unsigned>(need)), dim3(S.threads()), 0, s, a);
}

template <typename T, typename R, typename G>
twell_status run_norm_bwd(const NormBwdArgs& a, const NormShape& S, int blocks, float* dw, cudaStream_t s)
{
    auto kern = S.ch == 1 ? add_rmsnorm_bwd_kernel<T, R, G, 1> : add_rmsnorm_bwd_kernel<T, R, G, 4>;
    twell_status st = twell_host::launch_dep(kern, dim3(blocks), dim3(S.threads()), 0, s, a);
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
    const twell::NormShape S(d);
    const int g = group == 0 || d <= 128 ? d : group;
    const twell::NormFwdArgs a{x,    res, w, h_out, y,  static_cast<uint8_t*>(y8), y8_scale, rstd, N, d,
                               g, (d + g - 1) / g, S.wpr, S.rpb, eps, 1.0f / static_cast<float>(d)};
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == TWELL_F32) return twell::run_norm_fwd<float, float>(a, S, dev.sm_count, s);
    if (res_dtype == TWELL_F32) return twell::run_norm_fwd<__nv_bfloat16, float>(a, S, dev.sm_count, s);
    return twell::run_norm_fwd<__nv_bfloat16, __nv_bfloat16>(a, S, dev.sm_count, s);
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
