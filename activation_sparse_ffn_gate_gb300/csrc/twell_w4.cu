// twell_w4.cu -- y = x W^T for at most 16 tokens with 4-bit weights: W[r][k] = s[r][k / group] (code - 8),
// and the quantiser that lays the weights out.
//
// The product is bounded by the weights' bytes, k / 2 a row, so they are stored the way the tensor
// cores' fragments want them: a tile of 16 rows by 128 columns is 1 KB, lane (g, c) of a warp (g < 8,
// c < 4) owning 32 consecutive bytes of it: for rows g and g + 8, the columns 32j + 8c .. + 7, j < 4. A
// word holds 8 columns of a row, column 2i in bits 4i .. 4i + 3 and column 2i + 1 in bits 16 + 4i ..., so
// one shift and mask gives the pair an mma.sync m16n8k16 register wants. The pair becomes bf16 exactly (or-ed into
// 128.0 it is 128 + code; minus 136); rows are the product's 16-row side and tokens its 8 columns, a group's
// products are summed in fp32 by the tensor core and added to the total times the group's scale in fp32, so x and
// the codes enter exactly. Scales lie beside the tile in the same order ([g][half][128 / group]).
// A block takes up to 4 row tiles and its warps every n-th column tile of them each: a fragment of x is loaded once
// for those row tiles, and a warp copies weights, scales and x into its own shared-memory ring a column tile
// ahead. The warps' sums are added in warp order in shared memory (no atomics: the same y from call to call).
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kW4MaxN = 16;
constexpr int kW4Warps = 8;   // most a block has
constexpr int kW4Slot = 1152; // bytes of a weight tile in the ring: its words, then its scales (at most 128 bytes)
constexpr int kW4Stages = 2;
constexpr int kW4Direct = 2;  // column tiles a warp may have to take them straight into registers
// Most row tiles a block, by the token columns (in eights).
constexpr int w4_tiles(int nb) { return nb == 1 ? 4 : 3; }
constexpr int w4_stage(int nb, int rt) { return rt * kW4Slot + nb * 2048; }  // 8 tokens by 128 columns of x: 2 KB
constexpr int w4_smem(int warps, int nb, int rt) { return warps * kW4Stages * w4_stage(nb, rt); }
// Warps a block: as many as let two blocks share an SM, whose 228 KB of shared memory hold both rings and the 1 KB that goes
// with each block. That is 8, but 7 with three row tiles and 9 to 16 tokens, where 8 left one block an SM and the
// grid, of two an SM, took two rounds (14336 x 4096, 16 tokens: 12.3 us with 8, 11.1 with 7; 24577 x 4096 26.5 and 22.9; 9745 x
// 8192 21.0 and 20.7; two row tiles and 8 warps: 13.3, 23.7, 23.0).
constexpr int kW4SmBytes = 228 * 1024, kW4BlockBytes = 1024;
constexpr int w4_warps(int nb, int rt)
{
    const int fit = (kW4SmBytes / 2 - kW4BlockBytes) / w4_smem(1, nb, rt);
    return fit < kW4Warps ? fit : kW4Warps;
}

template <int GROUP>
struct W4Scales;  // the scales of one lane's two rows in a tile: [row half][128 / GROUP]
template <>
struct W4Scales<32> {
    uint4 v;
    __device__ __forceinline__ void load(uint32_t at)
    {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    }
    __device__ __forceinline__ float get(int half, int grp) const
    {
        const uint32_t w = half ? (grp < 2 ? v.z : v.w) : (grp < 2 ? v.x : v.y);
        return __uint_as_float((grp & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <>
struct W4Scales<64> {
    uint2 v;
    __device__ __forceinline__ void load(uint32_t at)
    {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    }
    __device__ __forceinline__ float get(int half, int grp) const
    {
        const uint32_t w = half ? v.y : v.x;
        return __uint_as_float((grp & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <>
struct W4Scales<128> {
    uint32_t v;
    __device__ __forceinline__ void load(uint32_t at) { asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at)); }
    __device__ __forceinline__ float get(int half, int) const
    {
        return __uint_as_float(half ? (v & 0xffff0000u) : (v << 16));
    }
};

// A pair of columns of a word as bf16 values code - 8, exactly.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i)
{
    uint32_t b;  // (a & b) | c in one instruction
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(word >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
    uint32_t v;  // 1.0 b - 136.0
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(b), "r"(0x3f803f80u), "r"(0xc308c308u));
    return v;
}

__device__ __forceinline__ void w4_copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 w4_lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// One tile of weights against the tokens' fragments: group sums by the tensor core, added under their scales.
template <int GROUP, int NB>
__device__ __forceinline__ void w4_tile(const uint4& w0, const uint4& w1, const W4Scales<GROUP>& sc, const uint4 (&xv)[NB][4],
                                        float (&acc)[NB][4])
{
    constexpr int kGroups = 128 / GROUP, kPer = GROUP / 32;  // groups a tile, 32-column steps a group
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

// One row tile a block and at most kW4Direct column tiles a warp: everything is requested at once, into registers.
template <int GROUP, int NB>
__global__ void __launch_bounds__(32 * kW4Warps) w4_small_kernel(const __nv_bfloat16* __restrict__ x,
                                                                 const uint8_t* __restrict__ words,
                                                                 const uint8_t* __restrict__ scales, int N, int n, int k,
                                                                 int kt, __nv_bfloat16* __restrict__ y)
{
    constexpr int kGroups = 128 / GROUP, kScaleBytes = 32 * kGroups;
    __shared__ float part[kW4Warps][8 * NB][17];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, c = lane & 3;
    uint4 w0[kW4Direct], w1[kW4Direct], xv[kW4Direct][NB][4];
    W4Scales<GROUP> sc[kW4Direct];
#pragma unroll
    for (int i = 0; i < kW4Direct; ++i) {
        const int t = warp + i * warps;
        w0[i] = w1[i] = make_uint4(0u, 0u, 0u, 0u);
        sc[i] = {};
        if (t < kt) {
            const size_t tile = static_cast<size_t>(blockIdx.x) * kt + t;
            w0[i] = ldg_stream16(words + tile * 1024 + lane * 32);
            w1[i] = ldg_stream16(words + tile * 1024 + lane * 32 + 16);
            sc[i] = reinterpret_cast<const W4Scales<GROUP>*>(scales + tile * kScaleBytes)[g];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 128 * t + 32 * j + 8 * c;
                xv[i][b][j] = make_uint4(0u, 0u, 0u, 0u);
                if (8 * b + g < N && col < k)
                    xv[i][b][j] = __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(8 * b + g) * k + col));
            }
    }
    float acc[NB][4] = {};
#pragma unroll
    for (int i = 0; i < kW4Direct; ++i) w4_tile<GROUP, NB>(w0[i], w1[i], sc[i], xv[i], acc);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        part[warp][8 * b + 2 * c][g] = acc[b][0];
        part[warp][8 * b + 2 * c + 1][g] = acc[b][1];
        part[warp][8 * b + 2 * c][g + 8] = acc[b][2];
        part[warp][8 * b + 2 * c + 1][g + 8] = acc[b][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * N; i += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += part[w][i >> 4][i & 15];
        const int row = 16 * blockIdx.x + (i & 15);
        if (row < n) y[static_cast<size_t>(i >> 4) * n + row] = __float2bfloat16_rn(v);
    }
}

// Row tiles [nt * block / blocks, nt * (block + 1) / blocks), at most RT of them.
template <int GROUP, int NB, int RT>
__global__ void __launch_bounds__(32 * kW4Warps, 2) w4_matvec_kernel(const __nv_bfloat16* __restrict__ x,
                                                                     const uint8_t* __restrict__ words,
                                                                     const uint8_t* __restrict__ scales, int N, int n,
                                                                     int k, int nt, int kt, __nv_bfloat16* __restrict__ y)
{
    constexpr int kCols = 8 * NB;
    constexpr int kScaleBytes = 32 * (128 / GROUP);          // of a tile
    constexpr int kStage = w4_stage(NB, RT);                 // of a warp: the weight tiles, then x
    constexpr int kRing = kW4Stages * kStage;
    static_assert(RT * kCols * 17 * 4 <= kRing, "a warp leaves its sums in its ring");
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, c = lane & 3;
    const int r0 = static_cast<int>(static_cast<long long>(nt) * blockIdx.x / gridDim.x);
    const int tiles = static_cast<int>(static_cast<long long>(nt) * (blockIdx.x + 1) / gridDim.x) - r0;
    const uint32_t ring = smem_u32(smem) + warp * kRing;
    // this lane's pieces: of a weight tile 16 bytes at 16 lane and 512 behind, of x the chunk lane % 16 of rows
    // lane / 16, lane / 16 + 2, ... (chunks of odd rows swapped in fours, for the banks of the fragments' reads)
    const size_t first = static_cast<size_t>(r0) * kt + warp;
    const uint8_t* wsrc = words + first * 1024 + lane * 16;
    const uint8_t* ssrc = scales + first * kScaleBytes + lane * 16;
    size_t row_of[RT];  // row tile r, in tiles (a block with fewer repeats its last one: no branch between them)
#pragma unroll
    for (int r = 0; r < RT; ++r) row_of[r] = static_cast<size_t>(min(r, tiles - 1)) * kt;
    const int xrow = lane >> 4, xcol = (lane & 15) * 8;
    const __nv_bfloat16* xsrc = x + static_cast<size_t>(xrow) * k + 128 * warp + xcol;
    const size_t xstep = 2 * static_cast<size_t>(k);
    const uint32_t xdst = RT * kW4Slot + xrow * 256 + ((lane & 15) ^ (xrow << 2)) * 16;
    // rows of x past the last token are zeros in both stages; columns past the last one become so in their stage
    auto zero16 = [](uint32_t at) {
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
    };
#pragma unroll
    for (int i = 0; i < 4 * NB; ++i)
        if (2 * i + xrow >= N) {
#pragma unroll
            for (int s = 0; s < kW4Stages; ++s) zero16(ring + s * kStage + xdst + i * 512);
        }
    auto request = [&](int t, int stage) {
        if (t < kt) {
            const uint32_t st = ring + stage * kStage;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t dst = st + r * kW4Slot + lane * 16;
                const uint8_t* w = wsrc + row_of[r] * 1024;
                w4_copy16(dst, w);
                w4_copy16(dst + 512, w + 512);
                if (lane < kScaleBytes / 16) w4_copy16(dst + 1024, ssrc + row_of[r] * kScaleBytes);
            }
            if (128 * t + xcol < k) {
                const __nv_bfloat16* src = xsrc;
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i) {
                    if (2 * i + xrow < N) w4_copy16(st + xdst + i * 512, src);
                    src += xstep;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i)
                    if (2 * i + xrow < N) zero16(st + xdst + i * 512);
            }
            wsrc += warps * 1024;
            ssrc += warps * kScaleBytes;
            xsrc += warps * 128;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kW4Stages - 1; ++s) request(warp + s * warps, s);

    float acc[RT][NB][4] = {};
    int stage = 0;
    for (int t = warp; t < kt; t += warps) {
        __syncwarp();  // the stage to be overwritten has been read by all lanes
        request(t + (kW4Stages - 1) * warps, stage == 0 ? kW4Stages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kW4Stages - 1) : "memory");
        __syncwarp();  // all lanes' copies of this stage are visible
        const uint32_t st = ring + stage * kStage;
        uint4 xv[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xv[b][j] = w4_lds128(st + RT * kW4Slot + (8 * b + g) * 256 + ((4 * j + c) ^ ((g & 1) << 2)) * 16);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint32_t at = st + r * kW4Slot;
            const uint4 w0 = w4_lds128(at + lane * 32), w1 = w4_lds128(at + lane * 32 + 16);
            W4Scales<GROUP> sc;
            sc.load(at + 1024 + g * (kScaleBytes / 8));
            w4_tile<GROUP, NB>(w0, w1, sc, xv, acc[r]);
        }
        stage = stage + 1 == kW4Stages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // sums: [row tiles][token columns][17] of each warp, in its ring
    float* part = reinterpret_cast<float*>(smem + warp * kRing);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float* p = part + r * (kCols * 17);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            p[(8 * b + 2 * c) * 17 + g] = acc[r][b][0];
            p[(8 * b + 2 * c + 1) * 17 + g] = acc[r][b][1];
            p[(8 * b + 2 * c) * 17 + g + 8] = acc[r][b][2];
            p[(8 * b + 2 * c + 1) * 17 + g + 8] = acc[r][b][3];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * tiles * N; i += blockDim.x) {
        const int tok = i / (16 * tiles), row = i - tok * (16 * tiles);  // row of the block's tiles
        const float* p = reinterpret_cast<const float*>(smem) + (row >> 4) * (kCols * 17) + tok * 17 + (row & 15);
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += p[w * (kRing / 4)];
        if (16 * r0 + row < n) y[static_cast<size_t>(tok) * n + 16 * r0 + row] = __float2bfloat16_rn(v);
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

template <int GROUP, int NB, int RT>
twell_status launch_w4(const void* x, const void* words, const void* scales, int N, int n, int k, void* y, int blocks,
                       cudaStream_t s)
{
    const int nt = (n + 15) / 16, kt = (k + 127) / 128;
    // every warp takes the same number of column tiles where that is possible
    constexpr int kMost = w4_warps(NB, RT);
    static_assert(2 * (w4_smem(kMost, NB, RT) + kW4BlockBytes) <= kW4SmBytes, "run_w4's grid is two blocks an SM");
    const int each = (kt + kMost - 1) / kMost, warps = (kt + each - 1) / each;
    if (RT == 1 && each <= kW4Direct)
        return twell_host::launch_dep(w4_small_kernel<GROUP, NB>, dim3(blocks), dim3(32 * warps), 0, s,
                                      static_cast<const __nv_bfloat16*>(x), static_cast<const uint8_t*>(words),
                                      static_cast<const uint8_t*>(scales), N, n, k, kt, static_cast<__nv_bfloat16*>(y));
    const int smem = w4_smem(warps, NB, RT);
    auto kern = w4_matvec_kernel<GROUP, NB, RT>;
    static std::atomic<uint64_t> allowed{0};
    if (twell_host::allow_smem(kern, w4_smem(kMost, NB, RT), allowed) != TWELL_OK) return TWELL_ERR_CUDA;
    return twell_host::launch_dep(kern, dim3(blocks), dim3(32 * warps), smem, s, static_cast<const __nv_bfloat16*>(x),
                                  static_cast<const uint8_t*>(words), static_cast<const uint8_t*>(scales), N, n, k, nt,
                                  kt, static_cast<__nv_bfloat16*>(y));
}

template <int GROUP>
twell_status run_w4(const void* x, const void* words, const void* scales, int N, int n, int k, void* y, cudaStream_t s)
{
    twell_host::DevInfo dev;
    if (twell_host::dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    // two blocks an SM as long as their row tiles cover the rows, then whole rounds of them
    const int nt = (n + 15) / 16, slots = 2 * dev.sm_count, per = w4_tiles(N <= 8 ? 1 : 2);
    const int blocks = std::min(nt, slots * ((nt + per * slots - 1) / (per * slots)));  // no block without a tile
    const int most = (nt + blocks - 1) / blocks;
    if (N <= 8) {
        if (most == 1) return launch_w4<GROUP, 1, 1>(x, words, scales, N, n, k, y, blocks, s);
        if (most == 2) return launch_w4<GROUP, 1, 2>(x, words, scales, N, n, k, y, blocks, s);
        if (most == 3) return launch_w4<GROUP, 1, 3>(x, words, scales, N, n, k, y, blocks, s);
        return launch_w4<GROUP, 1, 4>(x, words, scales, N, n, k, y, blocks, s);
    }
    if (most == 1) return launch_w4<GROUP, 2, 1>(x, words, scales, N, n, k, y, blocks, s);
    if (most == 2) return launch_w4<GROUP, 2, 2>(x, words, scales, N, n, k, y, blocks, s);
    return launch_w4<GROUP, 2, 3>(x, words, scales, N, n, k, y, blocks, s);
}

bool w4_shape_ok(int n, int k, int group) { return n > 0 && k > 0 && group > 0 && k % 32 == 0 && k % group == 0; }
constexpr int kW4MaxDim = 1 << 24;
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
    if (!twell::w4_group_ok(group) || n > twell::kW4MaxDim || k > twell::kW4MaxDim) return TWELL_ERR_UNSUPPORTED;
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
    if (N > twell::kW4MaxN || !twell::w4_group_ok(group) || n > twell::kW4MaxDim || k > twell::kW4MaxDim)
        return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    if (x == nullptr || y == nullptr || !aligned16(x) || !aligned16(y)) return TWELL_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (group == 32) return twell::run_w4<32>(x, words, scales, N, n, k, y, s);
    if (group == 64) return twell::run_w4<64>(x, words, scales, N, n, k, y, s);
    return twell::run_w4<128>(x, words, scales, N, n, k, y, s);
}
