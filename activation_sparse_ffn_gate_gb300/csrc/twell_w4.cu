// twell_w4.cu -- y = x W^T for at most 16 tokens with 4-bit weights: W[r][k] = s[r][k / group] (code - 8),
// and the quantiser that lays the weights out.
//
// The product is bounded by the weights' bytes, k / 2 a row, so they are stored the way the tensor
// cores' fragments want them: a tile of 16 rows by 128 columns is 1 KB, lane (g, c) of a warp (g < 8,
// c < 4) owning 32 consecutive bytes of it: for rows g and g + 8, the columns 32j + 8c .. + 7, j < 4. A
// word holds 8 columns of a row, column 2i in bits 4i .. 4i + 3 and column 2i + 1 in bits 16 + 4i ..., so
// one shift and mask gives the pair an mma.sync m16n8k16 register wants. The pair becomes bf16
// exactly (128 + code by a bit pattern, minus 136); rows are the product's 16-row side and tokens its
// 8 columns, a group's products are summed in fp32 by the tensor core and added to the total times
// the group's scale in fp32, so x and the codes enter exactly. Scales lie beside the tile in the same
// order ([g][half][128 / group]).
// A block takes one row tile, its warps every n-th column tile each; their sums are added in warp
// order in shared memory (no atomics: the same y from call to call).
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kW4MaxN = 16;
constexpr int kW4Warps = 8;

template <int GROUP>
struct W4Scales;  // the scales of one lane's two rows in a tile: [row half][128 / GROUP]
template <>
struct W4Scales<32> {
    uint4 v;
    __device__ __forceinline__ float get(int half, int grp) const
    {
        const uint32_t w = half ? (grp < 2 ? v.z : v.w) : (grp < 2 ? v.x : v.y);
        return __uint_as_float((grp & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <>
struct W4Scales<64> {
    uint2 v;
    __device__ __forceinline__ float get(int half, int grp) const
    {
        const uint32_t w = half ? v.y : v.x;
        return __uint_as_float((grp & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <>
struct W4Scales<128> {
    uint32_t v;
    __device__ __forceinline__ float get(int half, int) const
    {
        return __uint_as_float(half ? (v & 0xffff0000u) : (v << 16));
    }
};

// Codes of one pair of columns as bf16 values code - 8.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i)
{
    const uint32_t b = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), __floats2bfloat162_rn(136.0f, 136.0f));
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int GROUP, int NB>
__global__ void __launch_bounds__(32 * kW4Warps) w4_matvec_kernel(const __nv_bfloat16* __restrict__ x,
                                                                  const uint4* __restrict__ words,
                                                                  const W4Scales<GROUP>* __restrict__ scales, int N,
                                                                  int n, int k, int kt, __nv_bfloat16* __restrict__ y)
{
    constexpr int kGroups = 128 / GROUP, kPer = GROUP / 32;  // groups a tile, 32-column steps a group
    __shared__ float part[kW4Warps][16][8 * NB + 1];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    float acc[NB][4] = {};
    const size_t tile0 = static_cast<size_t>(blockIdx.x) * kt;
    for (int t = warp; t < kt; t += kW4Warps) {
        const uint4* wp = words + (tile0 + t) * 64 + 2 * lane;
        const uint4 w0 = ldg_stream16(wp), w1 = ldg_stream16(wp + 1);
        const W4Scales<GROUP> sc = scales[(tile0 + t) * 8 + g];
        uint4 xv[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 128 * t + 32 * j + 8 * c;
                xv[b][j] = make_uint4(0u, 0u, 0u, 0u);
                if (8 * b + g < N && col < k)
                    xv[b][j] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(8 * b + g) * k + col));
            }
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            float d[NB][4];
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                const int j = q * kPer + p;
                const uint32_t u = j == 0 ? w0.x : j == 1 ? w0.y : j == 2 ? w0.z : w0.w;
                const uint32_t v = j == 0 ? w1.x : j == 1 ? w1.y : j == 2 ? w1.z : w1.w;
                const uint32_t u0 = w4_pair(u, 0), u1 = w4_pair(u, 1), u2 = w4_pair(u, 2), u3 = w4_pair(u, 3);
                const uint32_t v0 = w4_pair(v, 0), v1 = w4_pair(v, 1), v2 = w4_pair(v, 2), v3 = w4_pair(v, 3);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (p == 0) mma_bf16_first(d[b], u0, v0, u1, v1, xv[b][j].x, xv[b][j].y);
                    else mma_bf16(d[b], u0, v0, u1, v1, xv[b][j].x, xv[b][j].y);
                    mma_bf16(d[b], u2, v2, u3, v3, xv[b][j].z, xv[b][j].w);
                }
            }
            const float s0 = sc.get(0, q), s1 = sc.get(1, q);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                acc[b][0] = fmaf(s0, d[b][0], acc[b][0]);
                acc[b][1] = fmaf(s0, d[b][1], acc[b][1]);
                acc[b][2] = fmaf(s1, d[b][2], acc[b][2]);
                acc[b][3] = fmaf(s1, d[b][3], acc[b][3]);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        part[warp][g][8 * b + 2 * c] = acc[b][0];
        part[warp][g][8 * b + 2 * c + 1] = acc[b][1];
        part[warp][g + 8][8 * b + 2 * c] = acc[b][2];
        part[warp][g + 8][8 * b + 2 * c + 1] = acc[b][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * N; i += blockDim.x) {
        const int r = i & 15, tok = i >> 4;
        const int row = blockIdx.x * 16 + r;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) v += part[w][r][tok];
        if (row < n) y[static_cast<size_t>(tok) * n + row] = __float2bfloat16_rn(v);
    }
}

// One tile of 16 rows by 128 columns a block, 8 columns a thread: s = bf16(max |w| over the group / 7),
// code = clamp(round(w / s), -8, 7) + 8; a group of zeros has s = 0 and codes 8.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const __nv_bfloat16* __restrict__ W, int n, int k, int kt,
                                                          int group, uint32_t* __restrict__ words,
                                                          __nv_bfloat16* __restrict__ scales, int32_t* status)
{
    __shared__ float tops[16][16];
    pdl_begin();
    const int r = threadIdx.x >> 4, w16 = threadIdx.x & 15, j = w16 >> 2, c = w16 & 3;
    const size_t tile = blockIdx.x;
    const int row = static_cast<int>(tile / kt) * 16 + r, col = static_cast<int>(tile % kt) * 128 + 8 * w16;
    float v[8] = {};
    if (row < n && col < k) load8(W + static_cast<size_t>(row) * k + col, v);
    float top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        top = fmaxf(top, fabsf(v[e]));
        bad |= !(fabsf(v[e]) <= 3.4e38f);
    }
    if (bad) report(status, TWELL_ERR_DEVICE_CHECK);
    tops[r][w16] = top;
    __syncthreads();
    const int per = group / 8;  // words a group
    top = 0.0f;
    for (int i = 0; i < per; ++i) top = fmaxf(top, tops[r][w16 / per * per + i]);
    const __nv_bfloat16 sb = __float2bfloat16_rn(top / 7.0f);
    const float s = __bfloat162float(sb);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = s > 0.0f ? fminf(fmaxf(rintf(v[e] / s), -8.0f), 7.0f) : 0.0f;
        word |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * (e >> 1) + 16 * (e & 1));
    }
    words[tile * 256 + ((r & 7) * 4 + c) * 8 + (r >> 3) * 4 + j] = word;
    if (w16 % per == 0) {
        const int ng = 128 / group;
        scales[tile * 16 * ng + ((r & 7) * 2 + (r >> 3)) * ng + w16 / per] = sb;
    }
}

template <int GROUP>
twell_status run_w4(const void* x, const void* words, const void* scales, int N, int n, int k, void* y, cudaStream_t s)
{
    auto kern = N <= 8 ? w4_matvec_kernel<GROUP, 1> : w4_matvec_kernel<GROUP, 2>;
    return twell_host::launch_dep(kern, dim3((n + 15) / 16), dim3(32 * kW4Warps), 0, s,
                                  static_cast<const __nv_bfloat16*>(x), static_cast<const uint4*>(words),
                                  static_cast<const W4Scales<GROUP>*>(scales), N, n, k, (k + 127) / 128,
                                  static_cast<__nv_bfloat16*>(y));
}

bool w4_shape_ok(int n, int k, int group) { return n > 0 && k > 0 && group > 0 && k % 32 == 0 && k % group == 0; }
bool w4_group_ok(int group) { return group == 32 || group == 64 || group == 128; }

}  // namespace
}  // namespace twell

using namespace twell_host;

extern "C" size_t twell_w4_words_bytes(int32_t n, int32_t k)
{
    if (n <= 0 || k <= 0) return 0;
    return (static_cast<size_t>(n) + 15) / 16 * ((static_cast<size_t>(k) + 127) / 128) * 1024;
}

extern "C" size_t twell_w4_scales_bytes(int32_t n, int32_t k, int32_t group)
{
    if (n <= 0 || k <= 0 || !twell::w4_group_ok(group)) return 0;
    return (static_cast<size_t>(n) + 15) / 16 * ((static_cast<size_t>(k) + 127) / 128) * 16 * (128 / group) * 2;
}

extern "C" twell_status twell_w4_quantize(const void* W, int32_t n, int32_t k, int32_t group, void* words, void* scales,
                                          int32_t* dev_status, void* stream)
{
    if (!twell::w4_shape_ok(n, k, group) || W == nullptr || words == nullptr || scales == nullptr ||
        dev_status == nullptr || !aligned16(W) || !aligned16(words) || !aligned16(scales))
        return TWELL_ERR_INVALID;
    if (!twell::w4_group_ok(group)) return TWELL_ERR_UNSUPPORTED;
    const long long tiles = ((n + 15ll) / 16) * ((k + 127ll) / 128);
    if (tiles > INT32_MAX) return TWELL_ERR_UNSUPPORTED;
    return launch_dep(twell::w4_quantize_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0,
                      static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(W), n, k, (k + 127) / 128, group,
                      static_cast<uint32_t*>(words), static_cast<__nv_bfloat16*>(scales), dev_status);
}

extern "C" twell_status twell_w4_matvec(const void* x, const void* words, const void* scales, int32_t N, int32_t n,
                                        int32_t k, int32_t group, void* y, void* stream)
{
    if (N < 0 || !twell::w4_shape_ok(n, k, group) || words == nullptr || scales == nullptr || !aligned16(words) ||
        !aligned16(scales))
        return TWELL_ERR_INVALID;
    if (N > twell::kW4MaxN || !twell::w4_group_ok(group)) return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    if (x == nullptr || y == nullptr || !aligned16(x) || !aligned16(y)) return TWELL_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (group == 32) return twell::run_w4<32>(x, words, scales, N, n, k, y, s);
    if (group == 64) return twell::run_w4<64>(x, words, scales, N, n, k, y, s);
    return twell::run_w4<128>(x, words, scales, N, n, k, y, s);
}
