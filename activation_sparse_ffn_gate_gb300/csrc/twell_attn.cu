// twell_attn.cu -- attention of one new token per sequence over the paged key-value cache.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m),  t over the visible tokens
//
// What bounds it is the cache: every visible key and value is read once for all the query heads
// that share it, 2 x heads per key flops a byte, so the kernel is laid out to keep reads in flight.
//   - Split over the length. The work is the list of 16-token tiles of every (sequence, key head), in
//     that order, cut into equal contiguous ranges, one a warp of a grid of one block an SM: a batch
//     of ragged lengths and a single long sequence are balanced alike, and no range is empty of work
//     while another is long. A warp streams its tiles through its own shared-memory ring with
//     16-byte asynchronous copies (rows beyond the visible range are filled with zeros and never
//     read), across sequence boundaries, so that the ring stays full.
//   - The products are small matrix products with the tokens (for q . k) and the dimensions (for the
//     output) on the 16-row side of mma.sync m16n8k16 and the query heads on its 8 columns: a
//     group of up to 8 query heads costs what one does. tcgen05's 64 to 128 rows a tile would be
//     filled by 16 tokens a warp only after a block-wide exchange, and nothing here is bounded by
//     the products. The scores' fragment becomes the second product's operand by an 8x8 transpose
//     (movmatrix); with a bf16 cache the weights go in as hi + lo bf16 parts (~16 bits), with an
//     e4m3 cache as fp16 (11 bits).
//   - Running maximum m and sum l in fp32, per query head. For an e4m3 cache the value's scale s_t is
//     folded into the weight, w_t = p_t s_t, and m runs over score + log2 s_t, so that the fp16
//     weights stay in (0, 1] whatever the scales. The query is brought to [1, 2) by a power of two
//     before its fp16 rounding (exact for bf16 values down to 2^-14 of the largest).
//   - Joining. A (sequence, key head) that lies within one warp's range is finished there. Otherwise
//     each part leaves (m, l, unnormalised o) in fp32 in the workspace; a block whose whole range lies
//     in one (sequence, key head) first joins its warps' parts in shared memory, and a second kernel
//     joins what is left, in ascending order: the result does not depend on scheduling.
#include "twell_kv.cuh"
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kTileTokens = 16;
constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxSms = 160;    // the workspace is sized for this many blocks, whatever the device
constexpr int kAttnMaxWarps = 16;   // and this many warps a block
constexpr float kNegInf = -INFINITY;

// HD: head_dim; Q8: e4m3 cache; NT: query heads of one key head handled together, in eights.
template <int HD, bool Q8, int NT>
struct AttnCfg {
    static constexpr int kRow = HD * (Q8 ? 1 : 2);      // bytes of a token's key or value
    static constexpr int kChunks = kRow / 16;
    static constexpr int kSwizzle = kChunks % 8 == 0 ? 7 : (kChunks % 4 == 0 ? 3 : 1);
    static constexpr int kHalf = kTileTokens * kRow;    // bytes of a tile's keys (then its values)
    static constexpr int kStage = 2 * kHalf + (Q8 ? 2 * kTileTokens * 4 : 0);
    static constexpr int kWarps = HD == 256 ? (Q8 ? 8 : 4) : ((Q8 || HD == 64) && NT == 1 ? 16 : 8);
    static constexpr int kStages = std::min(8, 204800 / (kWarps * kStage));
    static constexpr int kMt = HD / 16;                 // 16-dimension tiles of the output
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kPartF = NT * kMt * 128;       // floats of a part's o, then NT * 16 of m and l
    static constexpr int kPart = kPartF + NT * 16;
    static constexpr int kJoin = kWarps * kPart * 4;    // the block's join, in the ring's place
    static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin);
};

struct AttnArgs {
    KvView c;
    const __nv_bfloat16* q;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* out;
    float* lse;
    int32_t* status;
    int64_t q_stride;      // elements between two sequences' queries
    int B, n_q, G, blocks; // blocks: groups of 8 NT query heads per key head
    int max_pages, window;
    float scale_log2;      // scale * log2(e)
    uint32_t* prefix;      // [B + 1] tiles before each sequence, of one key head
    int* desc;             // [workers] the (sequence, key head) that a worker's start is the first to split, or -1
    float* part;           // [2 * workers][kPart]
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The 8x8 transpose of a matrix of 16-bit elements held one row of four pairs per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t f16_pack(float lo, float hi) { return f16x2_rn(lo, hi); }

// The visible tokens of a sequence, [first, len), and its tiles, counted from the tile of `first`.
struct SeqSpan {
    int len, first, tile0, tiles;
    __device__ __forceinline__ SeqSpan(int raw_len, int cap, int window)
    {
        len = min(max(raw_len, 0), cap);
        first = window > 0 ? max(len - window, 0) : 0;
        tile0 = first / kTileTokens;
        tiles = len > 0 ? (len + kTileTokens - 1) / kTileTokens - tile0 : 0;
    }
};

// A place in the list of tiles: sequence b, key-head block hv (key head x block of query heads), tile.
struct Cursor {
    int b, hv, tile;
    SeqSpan s;
    __device__ __forceinline__ Cursor() : b(0), hv(0), tile(0), s(0, 0, 0) {}
    __device__ __forceinline__ void load(const AttnArgs& a)
    {
        s = SeqSpan(__ldg(a.lens + b), a.max_pages << a.c.page_shift, a.window);
    }
    // item < total: the place of the item-th tile
    __device__ __forceinline__ void seek(const AttnArgs& a, const uint32_t* prefix, int HV, long long item)
    {
        int lo = 0, hi = a.B;  // prefix[lo] * HV <= item < prefix[hi] * HV
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<long long>(prefix[mid]) * HV <= item) lo = mid;
            else hi = mid;
        }
        b = lo;
        const uint32_t n = prefix[b + 1] - prefix[b];
        const long long rem = item - static_cast<long long>(prefix[b]) * HV;
        hv = static_cast<int>(rem / n);
        tile = static_cast<int>(rem - static_cast<long long>(hv) * n);
        load(a);
    }
    __device__ __forceinline__ void next(const AttnArgs& a, int HV)
    {
        if (++tile < s.tiles) return;
        tile = 0;
        if (++hv < HV) return;
        hv = 0;
        do {
            if (++b >= a.B) return;
            load(a);
        } while (s.tiles == 0);
    }
};

// The list of `total` tiles cut into equal ranges: range w of W starts at total * w / W, formed from the
// quotient and the remainder of total / W so that each start costs a 32-bit division. Few tiles use
// fewer blocks, one tile a warp.
struct Ranges {
    long long quot;
    uint32_t rem, W;
    int blocks;
    __device__ __forceinline__ Ranges(long long total, int max_blocks, int warps)
    {
        const long long need = (total + warps - 1) / warps;
        blocks = static_cast<int>(need < 1 ? 1 : (need < max_blocks ? need : max_blocks));
        W = static_cast<uint32_t>(blocks * warps);
        quot = total / W;
        rem = static_cast<uint32_t>(total - quot * W);
    }
    __device__ __forceinline__ long long start(uint32_t w) const { return quot * w + rem * w / W; }
};

// Physical 16-byte chunk of a tile's row: spread so that the rows that are read together by the
// fragments of either product fall into different banks.
template <class C>
__device__ __forceinline__ int swizzled(int row, int chunk, bool q8)
{
    const int f = q8 ? (row & 6) ^ ((row & 1) << 2) : row;
    return chunk ^ (f & C::kSwizzle);
}

template <int HD, bool Q8, int NT>
struct AttnState {
    using C = AttnCfg<HD, Q8, NT>;
    static constexpr int kQ = Q8 ? (HD + 63) / 64 * 8 : HD / 16 * 2;  // query fragment registers per eight heads
    uint32_t q[NT][kQ];
    float qs[NT][2];     // factor of the raw scores of heads 2c, 2c + 1
    float m[NT][2], l[NT][2];
    float o[C::kMt][NT][4];

    __device__ __forceinline__ void reset()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = kNegInf;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < C::kMt; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
        }
    }

    __device__ __forceinline__ void load_q(const AttnArgs& a, int b, int hv, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
        const int kvh = hv / a.blocks, first = (hv % a.blocks) * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int j = first + n * 8 + g;
            const __nv_bfloat16* src = a.q + b * a.q_stride + static_cast<int64_t>(kvh * a.G + j) * HD;
            const bool live = j < a.G;
            if constexpr (!Q8) {
#pragma unroll
                for (int i = 0; i < HD / 16; ++i) {
                    q[n][2 * i] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * i + 2 * c)) : 0u;
                    q[n][2 * i + 1] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * i + 8 + 2 * c)) : 0u;
                }
                qs[n][0] = qs[n][1] = a.scale_log2;
            } else {
                uint32_t raw[kQ];
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < kQ / 8; ++i) {
                    const bool on = live && 4 * i + c < HD / 16;
                    const uint32_t* p = reinterpret_cast<const uint32_t*>(src + 64 * i + 16 * c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        raw[8 * i + e] = on ? __ldg(p + e) : 0u;
                        const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&raw[8 * i + e]));
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
                const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&raw[i]));
                    q[n][i] = f16x2_rn(f.x * down, f.y * down);
                }
                qs[n][0] = __shfl_sync(0xffffffffu, up, 8 * c) * a.scale_log2;
                qs[n][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4) * a.scale_log2;
            }
        }
    }

    // One tile: its keys at `st`, its values C::kHalf behind, its scales behind those; bit t of `vis` says
    // whether token t of the 16 is visible.
    __device__ __forceinline__ void tile(uint32_t st, uint32_t vis, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
        if constexpr (!Q8) {
            const int row = lane & 15, hi8 = lane >> 4;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
                uint32_t k[4];
                ldsm_x4(k, st + row * C::kRow + swizzled<C>(row, 2 * i + hi8, false) * 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(sc[n], k[0], k[1], k[2], k[3], q[n][2 * i], q[n][2 * i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kQ / 8; ++i) {
                uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0;
                if (HD % 64 == 0 || 4 * i + c < HD / 16) {
                    k0 = lds128(st + g * C::kRow + swizzled<C>(g, 4 * i + c, true) * 16);
                    k1 = lds128(st + (g + 8) * C::kRow + swizzled<C>(g + 8, 4 * i + c, true) * 16);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w0 = e == 0 ? k0.x : e == 1 ? k0.y : e == 2 ? k0.z : k0.w;
                    const uint32_t w1 = e == 0 ? k1.x : e == 1 ? k1.y : e == 2 ? k1.z : k1.w;
                    const uint32_t a0 = e4m3x2_f16x2(static_cast<uint16_t>(w0)), a1 = e4m3x2_f16x2(static_cast<uint16_t>(w1));
                    const uint32_t a2 = e4m3x2_f16x2(static_cast<uint16_t>(w0 >> 16)),
                                   a3 = e4m3x2_f16x2(static_cast<uint16_t>(w1 >> 16));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(sc[n], a0, a1, a2, a3, q[n][8 * i + 2 * e], q[n][8 * i + 2 * e + 1]);
                }
            }
        }

        // scores (base 2) of tokens g and g + 8 for heads 2c and 2c + 1; weights
        const bool on0 = (vis >> g) & 1u, on1 = (vis >> (g + 8)) & 1u;
        float ks0 = 1.0f, ks1 = 1.0f, vs0 = 1.0f, vs1 = 1.0f, lv0 = 0.0f, lv1 = 0.0f;
        if constexpr (Q8) {
            const uint32_t sp = st + 2 * C::kHalf;
            ks0 = __uint_as_float(lds32(sp + 4 * g));
            ks1 = __uint_as_float(lds32(sp + 4 * (g + 8)));
            vs0 = __uint_as_float(lds32(sp + 64 + 4 * g));
            vs1 = __uint_as_float(lds32(sp + 64 + 4 * (g + 8)));
            lv0 = __log2f(fmaxf(vs0, kAmaxMin));
            lv1 = __log2f(fmaxf(vs1, kAmaxMin));
        }
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x[4];
            x[0] = on0 ? fmaf(sc[n][0], qs[n][0] * ks0, lv0) : kNegInf;
            x[1] = on0 ? fmaf(sc[n][1], qs[n][1] * ks0, lv0) : kNegInf;
            x[2] = on1 ? fmaf(sc[n][2], qs[n][0] * ks1, lv1) : kNegInf;
            x[3] = on1 ? fmaf(sc[n][3], qs[n][1] * ks1, lv1) : kNegInf;
            float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, s));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, s));
            }
            if (__any_sync(0xffffffffu, t0 > m[n][0] || t1 > m[n][1])) {
                const float n0 = fmaxf(m[n][0], t0), n1 = fmaxf(m[n][1], t1);
                const float f0 = m[n][0] == kNegInf ? 0.0f : exp2_approx(m[n][0] - n0);
                const float f1 = m[n][1] == kNegInf ? 0.0f : exp2_approx(m[n][1] - n1);
                m[n][0] = n0;
                m[n][1] = n1;
                l[n][0] *= f0;
                l[n][1] *= f1;
#pragma unroll
                for (int i = 0; i < C::kMt; ++i) {
                    o[i][n][0] *= f0;
                    o[i][n][1] *= f1;
                    o[i][n][2] *= f0;
                    o[i][n][3] *= f1;
                }
            }
            const float b0 = m[n][0] == kNegInf ? 0.0f : m[n][0], b1 = m[n][1] == kNegInf ? 0.0f : m[n][1];
            float p[4];
            p[0] = exp2_approx(x[0] - lv0 - b0);
            p[1] = exp2_approx(x[1] - lv0 - b1);
            p[2] = exp2_approx(x[2] - lv1 - b0);
            p[3] = exp2_approx(x[3] - lv1 - b1);
            l[n][0] += p[0] + p[2];
            l[n][1] += p[1] + p[3];
            if constexpr (Q8) {
                ph[n][0] = transpose8(f16_pack(p[0] * vs0, p[1] * vs0));
                ph[n][1] = transpose8(f16_pack(p[2] * vs1, p[3] * vs1));
            } else {
                const uint32_t h0 = bf16x2_rn(p[0], p[1]), h1 = bf16x2_rn(p[2], p[3]);
                const float2 r0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
                const float2 r1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
                ph[n][0] = transpose8(h0);
                ph[n][1] = transpose8(h1);
                pl[n][0] = transpose8(bf16x2_rn(p[0] - r0.x, p[1] - r0.y));
                pl[n][1] = transpose8(bf16x2_rn(p[2] - r1.x, p[3] - r1.y));
            }
        }

        // o += v^T p: dimensions on the rows
        const uint32_t sv = st + C::kHalf;
        if constexpr (!Q8) {
            const int row = (lane & 7) + ((lane & 16) >> 1), odd = (lane >> 3) & 1;
#pragma unroll
            for (int i = 0; i < C::kMt; ++i) {
                uint32_t v[4];
                ldsm_x4_trans(v, sv + row * C::kRow + swizzled<C>(row, 2 * i + odd, false) * 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(o[i][n], v[0], v[1], v[2], v[3], ph[n][0], ph[n][1]);
                    mma_bf16(o[i][n], v[0], v[1], v[2], v[3], pl[n][0], pl[n][1]);
                }
            }
        } else {
            // lane (g, c): dimensions g HD / 8 ... of tokens 2c, 2c + 1, 2c + 8, 2c + 9
            constexpr int W = HD / 32;  // words of a token's dimensions
            constexpr int V = HD == 96 ? 1 : (W < 4 ? W : 4);  // words a load
#pragma unroll
            for (int w0 = 0; w0 < W; w0 += V) {
                uint32_t v[4][V];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * c + (r & 1) + (r >> 1) * 8;
                    const int byte = g * (HD / 8) + 4 * w0;
                    const uint32_t ad = sv + row * C::kRow + swizzled<C>(row, byte >> 4, true) * 16 + (byte & 15);
                    if constexpr (V == 4) {
                        const uint4 u = lds128(ad);
                        v[r][0] = u.x, v[r][1] = u.y, v[r][2] = u.z, v[r][3] = u.w;
                    } else if constexpr (V == 2) {
                        const uint2 u = lds64(ad);
                        v[r][0] = u.x, v[r][1] = u.y;
                    } else {
                        v[r][0] = lds32(ad);
                    }
                }
#pragma unroll
                for (int w = 0; w < V; ++w) {
                    const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
                    const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = h ? x1 : x0, y = h ? y1 : y0;
                        const uint32_t a0 = e4m3x2_f16x2(static_cast<uint16_t>(x)), a1 = e4m3x2_f16x2(static_cast<uint16_t>(x >> 16));
                        const uint32_t a2 = e4m3x2_f16x2(static_cast<uint16_t>(y)), a3 = e4m3x2_f16x2(static_cast<uint16_t>(y >> 16));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(o[2 * (w0 + w) + h][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                    }
                }
            }
        }
    }

    // l over the tokens of all lanes (m is the same in them already).
    __device__ __forceinline__ void close()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], s);
                l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], s);
            }
    }

    __device__ __forceinline__ void store_part(float* p, int lane) const
    {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < C::kMt; ++i)
                reinterpret_cast<float4*>(p)[(n * C::kMt + i) * 32 + lane] =
                    make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
            if (lane < 4) {
                p[C::kPartF + n * 16 + 2 * c] = m[n][0];
                p[C::kPartF + n * 16 + 2 * c + 1] = m[n][1];
                p[C::kPartF + n * 16 + 8 + 2 * c] = l[n][0];
                p[C::kPartF + n * 16 + 8 + 2 * c + 1] = l[n][1];
            }
        }
    }
};

// Final values of one fragment element group: dimension tile i, eight heads n, lane's four sums r with
// their heads' totals l; all 32 lanes of a warp call it for the same (n, i).
template <int HD, bool Q8, int NT>
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int hv, int n, int i, int lane, const float (&r)[4],
                                          float l0, float l1)
{
    const int g = lane >> 2, c = lane & 3;
    const int kvh = hv / a.blocks, first = (hv % a.blocks) * 8 * NT + n * 8;
    const float i0 = l0 > 0.0f || l0 != l0 ? 1.0f / l0 : 0.0f, i1 = l1 > 0.0f || l1 != l1 ? 1.0f / l1 : 0.0f;
    __nv_bfloat16* base = a.out + (static_cast<int64_t>(b) * a.n_q + kvh * a.G) * HD;
    if constexpr (!Q8) {  // rows g and g + 8 of the tile, heads 2c and 2c + 1
        const uint32_t x = transpose8(bf16x2_rn(r[0] * i0, r[1] * i1)), y = transpose8(bf16x2_rn(r[2] * i0, r[3] * i1));
        if (first + g < a.G) {
            uint32_t* p = reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(first + g) * HD + 16 * i + 2 * c);
            p[0] = x;
            p[4] = y;
        }
    } else {  // dimensions g HD / 8 + 2i and the next, heads 2c and 2c + 1
        const int d = g * (HD / 8) + 2 * i, j = first + 2 * c;
        if (j < a.G)
            *reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(j) * HD + d) = bf16x2_rn(r[0] * i0, r[2] * i0);
        if (j + 1 < a.G)
            *reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(j + 1) * HD + d) = bf16x2_rn(r[1] * i1, r[3] * i1);
    }
}

template <int NT>
__device__ __forceinline__ void store_lse(const AttnArgs& a, int b, int hv, int head, float m, float l)
{
    const int kvh = hv / a.blocks, j = (hv % a.blocks) * 8 * NT + head;
    if (a.lse != nullptr && j < a.G)
        a.lse[static_cast<int64_t>(b) * a.n_q + kvh * a.G + j] =
            l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

template <int HD, bool Q8, int NT>
__global__ void __launch_bounds__(AttnCfg<HD, Q8, NT>::kWarps * 32, 1) paged_attn_kernel(const AttnArgs a)
{
    using C = AttnCfg<HD, Q8, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t sums[32];
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + C::kSmem);  // [B + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_begin();

    // tiles before each sequence (of one key head): a scan over the lengths, by every block for itself
    const int cap = a.max_pages << a.c.page_shift;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, a.B);
    uint32_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = __ldg(a.lens + b);
        if ((raw < 0 || raw > cap) && blockIdx.x == 0) report(a.status, TWELL_ERR_DEVICE_CHECK);
        mine += SeqSpan(raw, cap, a.window).tiles;
    }
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += sums[w];
    run -= mine;
    for (int b = b0; b < b1; ++b) {
        prefix[b] = run;
        run += SeqSpan(__ldg(a.lens + b), cap, a.window).tiles;
        if (b == a.B - 1) prefix[a.B] = run;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= a.B; b += blockDim.x) a.prefix[b] = prefix[b];

    // sequences with nothing visible: zeros, lse = -inf
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (prefix[b + 1] != prefix[b]) continue;
        uint32_t* p = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(b) * a.n_q * HD);
        for (int i = threadIdx.x; i < a.n_q * HD / 2; i += blockDim.x) p[i] = 0u;
        if (a.lse != nullptr)
            for (int i = threadIdx.x; i < a.n_q; i += blockDim.x) a.lse[static_cast<int64_t>(b) * a.n_q + i] = kNegInf;
    }

    const int HV = a.c.heads * a.blocks;
    const long long total = static_cast<long long>(prefix[a.B]) * HV;
    const Ranges R(total, gridDim.x, C::kWarps);
    if (static_cast<int>(blockIdx.x) >= R.blocks) return;
    const int w = blockIdx.x * C::kWarps + warp;
    const long long start = R.start(w), end = R.start(w + 1);
    const long long c_start = R.start(blockIdx.x * C::kWarps), c_end = R.start((blockIdx.x + 1) * C::kWarps);

    // the block's range: within one (sequence, key head), or even all of it
    bool inside = false, whole = false;
    Cursor cur;  // where this warp's next tile to be used is
    if (start < total) cur.seek(a, prefix, HV, start);
    const long long seg0 = start - cur.tile;  // first tile of the (sequence, key head) at `start`
    if (c_end > c_start) {
        Cursor at;
        at.seek(a, prefix, HV, c_start);
        const long long s0 = c_start - at.tile, s1 = s0 + at.s.tiles;
        inside = c_end <= s1;
        whole = inside && s0 == c_start && s1 == c_end;
    }
    if (lane == 0) {
        int d = -1;
        if (w > 0 && start < total && start > seg0 && R.start(w - 1) <= seg0 && !whole)
            d = cur.b * HV + cur.hv;
        a.desc[w] = d;
    }

    const int n = static_cast<int>(end - start);
    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);
    Cursor ahead = cur;  // where the next tile to be requested is
    int page = 0;        // of token `lane` of that tile (lanes 0..15), -1 where nothing is read
    auto load_page = [&]() {
        page = -1;
        const int pos = (ahead.s.tile0 + ahead.tile) * kTileTokens + (lane & 15);
        if (pos >= ahead.s.first && pos < ahead.s.len) {
            page = __ldg(a.table + static_cast<int64_t>(ahead.b) * a.max_pages + (pos >> a.c.page_shift));
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.n_pages)) {
                report(a.status, TWELL_ERR_DEVICE_CHECK);
                page = -1;
            }
        }
    };
    // Requests a tile into a ring stage; returns its visible tokens (those of bad pages are left out) as bits.
    auto request = [&](int stage) -> uint32_t {
        const int pos = (ahead.s.tile0 + ahead.tile) * kTileTokens + (lane & 15);
        const int in_page = pos & ((1 << a.c.page_shift) - 1);
        const int head = ahead.hv / a.blocks;
        const uint32_t valid = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
        const int64_t off =
            page >= 0 ? (page * a.c.page_stride + head * a.c.head_stride + in_page * a.c.token_stride) * (Q8 ? 1 : 2) : 0;
        const uint32_t st = ring + stage * C::kStage;
        const uint8_t* kb = static_cast<const uint8_t*>(a.c.k);
        const uint8_t* vb = static_cast<const uint8_t*>(a.c.v);
#pragma unroll
        for (int i = 0; i < C::kHalf / 512; ++i) {
            const int id = i * 32 + lane, row = id / C::kChunks, ch = id % C::kChunks;
            const int64_t ro = __shfl_sync(0xffffffffu, off, row) + ch * 16;
            const bool on = (valid >> row) & 1u;
            const uint32_t dst = st + row * C::kRow + swizzled<C>(row, ch, Q8) * 16;
            cp_async16(dst, kb + ro, on);
            cp_async16(dst + C::kHalf, vb + ro, on);
        }
        if constexpr (Q8) {
            const int64_t so = page >= 0 ? page * a.c.scale_page + head * a.c.scale_head + in_page : 0;
            cp_async4(st + 2 * C::kHalf + 4 * lane, (lane < 16 ? a.c.k_scale : a.c.v_scale) + so, page >= 0);
        }
        return valid;
    };

    AttnState<HD, Q8, NT> S;
    int slot = 0;              // 0: the segment at the worker's start, 1: a later one
    uint32_t valid_ring = 0;   // lane i: the visible tokens of ring stage i's tile
    if (n > 0) load_page();
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
        if (s < n) {
            const uint32_t v = request(s);
            if (lane == s) valid_ring = v;
            ahead.next(a, HV);
            if (s + 1 < n) load_page();
        }
        cp_commit();
    }
    int stage = 0;
    for (int it = 0; it < n; ++it) {
        cp_wait<C::kStages - 2>();
        __syncwarp();
        const uint32_t vis = __shfl_sync(0xffffffffu, valid_ring, stage);
        {
            const int s = stage == 0 ? C::kStages - 1 : stage - 1;
            if (it + C::kStages - 1 < n) {
                const uint32_t v = request(s);
                if (lane == s) valid_ring = v;
                ahead.next(a, HV);
                if (it + C::kStages < n) load_page();
            }
            cp_commit();
        }
        if (it == 0 || cur.tile == 0) {
            S.load_q(a, cur.b, cur.hv, lane);
            S.reset();
        }
        S.tile(ring + stage * C::kStage, vis, lane);
        stage = stage + 1 == C::kStages ? 0 : stage + 1;

        const bool seg_end = cur.tile + 1 == cur.s.tiles;
        if (seg_end || it + 1 == n) {
            S.close();
            const bool complete = seg_end && it >= cur.tile;  // its first tile was this warp's too
            if (complete && !inside) {
#pragma unroll
                for (int e = 0; e < NT; ++e) {
#pragma unroll
                    for (int i = 0; i < C::kMt; ++i)
                        store_out<HD, Q8, NT>(a, cur.b, cur.hv, e, i, lane, S.o[i][e], S.l[e][0], S.l[e][1]);
                    if (lane < 4) {
                        store_lse<NT>(a, cur.b, cur.hv, e * 8 + 2 * lane, S.m[e][0], S.l[e][0]);
                        store_lse<NT>(a, cur.b, cur.hv, e * 8 + 2 * lane + 1, S.m[e][1], S.l[e][1]);
                    }
                }
            } else if (!inside) {
                S.store_part(a.part + (static_cast<int64_t>(w) * 2 + slot) * C::kPart, lane);
            }
        }
        if (seg_end) slot = 1;
        if (it + 1 < n) cur.next(a, HV);
    }
    cp_wait<0>();
    if (!inside) return;

    // every warp's range lies in one (sequence, key head): join the parts in shared memory
    __syncthreads();
    float* jp = reinterpret_cast<float*>(smem);
    if (n == 0) S.reset();
    S.store_part(jp + warp * C::kPart, lane);
    __syncthreads();
    Cursor at;
    at.seek(a, prefix, HV, c_start);
    float* dst = a.part + static_cast<int64_t>(blockIdx.x) * C::kWarps * 2 * C::kPart;
    for (int t = threadIdx.x; t < NT * C::kMt * 32; t += blockDim.x) {
        const int ni = t >> 5, e = ni / C::kMt, h = 2 * (lane & 3);  // (ni, lane): this thread's float4
        float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
        for (int p = 0; p < C::kWarps; ++p) {
            m0 = fmaxf(m0, jp[p * C::kPart + C::kPartF + e * 16 + h]);
            m1 = fmaxf(m1, jp[p * C::kPart + C::kPartF + e * 16 + h + 1]);
        }
        float r[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int p = 0; p < C::kWarps; ++p) {
            const float* pp = jp + p * C::kPart;
            const float pm0 = pp[C::kPartF + e * 16 + h], pm1 = pp[C::kPartF + e * 16 + h + 1];
            const float f0 = pm0 == kNegInf ? 0.0f : exp2_approx(pm0 - m0), f1 = pm1 == kNegInf ? 0.0f : exp2_approx(pm1 - m1);
            const float4 v = reinterpret_cast<const float4*>(pp)[t];
            r[0] = fmaf(v.x, f0, r[0]);
            r[1] = fmaf(v.y, f1, r[1]);
            r[2] = fmaf(v.z, f0, r[2]);
            r[3] = fmaf(v.w, f1, r[3]);
            l0 = fmaf(pp[C::kPartF + e * 16 + 8 + h], f0, l0);
            l1 = fmaf(pp[C::kPartF + e * 16 + 8 + h + 1], f1, l1);
        }
        if (whole) {
            store_out<HD, Q8, NT>(a, at.b, at.hv, e, ni % C::kMt, lane, r, l0, l1);
            if (ni % C::kMt == 0 && lane < 4) {
                store_lse<NT>(a, at.b, at.hv, e * 8 + h, m0, l0);
                store_lse<NT>(a, at.b, at.hv, e * 8 + h + 1, m1, l1);
            }
        } else {
            reinterpret_cast<float4*>(dst)[t] = make_float4(r[0], r[1], r[2], r[3]);
            if (ni % C::kMt == 0 && lane < 4) {
                dst[C::kPartF + e * 16 + h] = m0;
                dst[C::kPartF + e * 16 + h + 1] = m1;
                dst[C::kPartF + e * 16 + 8 + h] = l0;
                dst[C::kPartF + e * 16 + 8 + h + 1] = l1;
            }
        }
    }
}

// Joins the parts of the (sequence, key head)s that a worker of main block blockIdx.x was the first to
// split off: kGroups groups of threads, one float4 of the output a thread; a single split is shared
// by all groups (each takes every kGroups-th part), several are dealt out to them.
template <int HD, bool Q8, int NT>
struct JoinCfg {
    static constexpr int kElems = NT * (HD / 16) * 32;
    static constexpr int kGroups = 1024 / kElems;
    static constexpr int kThreads = kGroups * kElems;
};
template <int HD, bool Q8, int NT>
__global__ void __launch_bounds__(JoinCfg<HD, Q8, NT>::kThreads)
    paged_attn_join_kernel(const AttnArgs a, int main_blocks)
{
    using C = AttnCfg<HD, Q8, NT>;
    using J = JoinCfg<HD, Q8, NT>;
    constexpr int kElems = J::kElems, kGroups = J::kGroups;
    constexpr int kMaxParts = kAttnMaxSms + 2 * kAttnMaxWarps;
    __shared__ int s_desc[C::kWarps];
    __shared__ int s_list[kGroups][kMaxParts];  // parts in ascending order, -1 where there is none
    __shared__ float4 s_sum[J::kThreads];
    __shared__ float s_m[kGroups][NT * 8], s_l[kGroups][NT * 8];
    pdl_begin();
    const int HV = a.c.heads * a.blocks;
    const long long total = static_cast<long long>(a.prefix[a.B]) * HV;
    const Ranges R(total, main_blocks, C::kWarps);
    if (static_cast<int>(blockIdx.x) >= R.blocks) return;
    if (threadIdx.x < C::kWarps) s_desc[threadIdx.x] = a.desc[blockIdx.x * C::kWarps + threadIdx.x];
    __syncthreads();
    int owned = 0;
#pragma unroll
    for (int i = 0; i < C::kWarps; ++i) owned += s_desc[i] >= 0;
    const int grp = threadIdx.x / kElems, t = threadIdx.x % kElems;
    const int lane = threadIdx.x & 31;
    const int e = (t >> 5) / C::kMt, dim = (t >> 5) % C::kMt, h = 2 * (lane & 3);
    const bool shared_by_all = owned == 1;

    for (int k0 = 0; k0 < owned; k0 += shared_by_all ? 1 : kGroups) {
        // this group's split: the (k0 + grp)-th owned one (or the only one)
        const int want = shared_by_all ? 0 : k0 + grp;
        int wi = -1;
        for (int i = 0, s = 0; i < C::kWarps; ++i)
            if (s_desc[i] >= 0 && s++ == want) wi = i;
        const bool live = wi >= 0;
        int b = 0, hv = 0, count = 0;
        if (live) {
            b = s_desc[wi] / HV;
            hv = s_desc[wi] % HV;
            const uint32_t p0 = a.prefix[b], nt = a.prefix[b + 1] - p0;
            const long long I0 = static_cast<long long>(p0) * HV + static_cast<long long>(hv) * nt, I1 = I0 + nt;
            // candidates: the warps of the first block that holds some of [I0, I1), one for each block
            // between, the warps of the last; a block inside [I0, I1) has left one part, its first warp's
            const int blk0 = (static_cast<int>(blockIdx.x) * C::kWarps + wi - 1) / C::kWarps;
            const int blk1 = static_cast<int>((I1 * R.W + total - 1) / total - 1) / C::kWarps;
            const int mid = max(blk1 - blk0 - 1, 0);
            count = blk1 > blk0 ? 2 * C::kWarps + mid : C::kWarps;
            for (int i = t; i < count; i += kElems) {
                uint32_t w = blk0 * C::kWarps + i;
                bool one = false;
                if (i >= C::kWarps + mid) {
                    w = blk1 * C::kWarps + (i - C::kWarps - mid);
                } else if (i >= C::kWarps) {
                    w = (blk0 + 1 + i - C::kWarps) * C::kWarps;
                    one = true;
                }
                const uint32_t blk = w / C::kWarps * C::kWarps;
                const long long s = R.start(w), en = R.start(w + 1), cs = R.start(blk), ce = R.start(blk + C::kWarps);
                int entry = -1;
                if (one || (cs >= I0 && ce <= I1)) {
                    if (w == blk && ce > cs) entry = static_cast<int>(2 * w);
                } else if (en > s && s < I1 && en > I0) {
                    entry = static_cast<int>(2 * w + (s < I0 ? 1 : 0));
                }
                s_list[grp][i] = entry;
            }
        }
        __syncthreads();
        float m0 = kNegInf, m1 = kNegInf, l0 = 0.0f, l1 = 0.0f;
        float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int step = shared_by_all ? kGroups : 1;
#pragma unroll 4
        for (int p = shared_by_all ? grp : 0; p < count; p += step) {
            const int entry = s_list[grp][p];
            if (entry < 0) continue;
            const float* pp = a.part + static_cast<int64_t>(entry) * C::kPart;
            const float4 v = reinterpret_cast<const float4*>(pp)[t];
            const float2 pm = *reinterpret_cast<const float2*>(pp + C::kPartF + e * 16 + h);
            const float2 pl = *reinterpret_cast<const float2*>(pp + C::kPartF + e * 16 + 8 + h);
            const float n0 = fmaxf(m0, pm.x), n1 = fmaxf(m1, pm.y);
            const float f0 = m0 == kNegInf ? 0.0f : exp2_approx(m0 - n0), f1 = m1 == kNegInf ? 0.0f : exp2_approx(m1 - n1);
            const float g0 = pm.x == kNegInf ? 0.0f : exp2_approx(pm.x - n0),
                        g1 = pm.y == kNegInf ? 0.0f : exp2_approx(pm.y - n1);
            m0 = n0;
            m1 = n1;
            r[0] = r[0] * f0 + v.x * g0;
            r[1] = r[1] * f1 + v.y * g1;
            r[2] = r[2] * f0 + v.z * g0;
            r[3] = r[3] * f1 + v.w * g1;
            l0 = l0 * f0 + pl.x * g0;
            l1 = l1 * f1 + pl.y * g1;
        }
        if (shared_by_all) {  // the groups' sums, in group order
            s_sum[threadIdx.x] = make_float4(r[0], r[1], r[2], r[3]);
            if (dim == 0 && lane < 4) {
                s_m[grp][e * 8 + h] = m0;
                s_m[grp][e * 8 + h + 1] = m1;
                s_l[grp][e * 8 + h] = l0;
                s_l[grp][e * 8 + h + 1] = l1;
            }
            __syncthreads();
            m0 = m1 = kNegInf;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                m0 = fmaxf(m0, s_m[q][e * 8 + h]);
                m1 = fmaxf(m1, s_m[q][e * 8 + h + 1]);
            }
            r[0] = r[1] = r[2] = r[3] = l0 = l1 = 0.0f;
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const float q0 = s_m[q][e * 8 + h], q1 = s_m[q][e * 8 + h + 1];
                const float f0 = q0 == kNegInf ? 0.0f : exp2_approx(q0 - m0), f1 = q1 == kNegInf ? 0.0f : exp2_approx(q1 - m1);
                const float4 v = s_sum[q * kElems + t];
                r[0] = fmaf(v.x, f0, r[0]);
                r[1] = fmaf(v.y, f1, r[1]);
                r[2] = fmaf(v.z, f0, r[2]);
                r[3] = fmaf(v.w, f1, r[3]);
                l0 = fmaf(s_l[q][e * 8 + h], f0, l0);
                l1 = fmaf(s_l[q][e * 8 + h + 1], f1, l1);
            }
        }
        if (live && (!shared_by_all || grp == 0)) {
            store_out<HD, Q8, NT>(a, b, hv, e, dim, lane, r, l0, l1);
            if (dim == 0 && lane < 4) {
                store_lse<NT>(a, b, hv, e * 8 + h, m0, l0);
                store_lse<NT>(a, b, hv, e * 8 + h + 1, m1, l1);
            }
        }
        __syncthreads();
    }
}

template <int HD, bool Q8, int NT>
twell_status run_attn(const AttnArgs& a, int sms, cudaStream_t s)
{
    using C = AttnCfg<HD, Q8, NT>;
    static_assert(NT * C::kWarps <= kAttnMaxWarps, "the workspace holds kAttnMaxWarps warps' parts of eight heads");
    static_assert(C::kStages >= 2, "the ring overlaps copies with the products");
    auto kern = paged_attn_kernel<HD, Q8, NT>;
    const size_t smem = C::kSmem + (static_cast<size_t>(a.B) + 1) * 4;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return TWELL_ERR_CUDA;
    twell_status st = twell_host::launch_dep(kern, dim3(sms), dim3(C::kWarps * 32), smem, s, a);
    if (st != TWELL_OK) return st;
    return twell_host::launch_dep(paged_attn_join_kernel<HD, Q8, NT>, dim3(sms), dim3(JoinCfg<HD, Q8, NT>::kThreads), 0,
                                  s, a, sms);
}

template <int HD, bool Q8>
twell_status run_heads(AttnArgs& a, int sms, cudaStream_t s)
{
    // query heads of a key head are taken eight at a time, sixteen where there are more than eight and
    // the fragments of sixteen fit the registers
    constexpr int kMost = HD <= 128 ? 2 : 1;
    if (kMost == 2 && a.G > 8) {
        a.blocks = (a.G + 15) / 16;
        return run_attn<HD, Q8, kMost>(a, sms, s);
    }
    a.blocks = (a.G + 7) / 8;
    return run_attn<HD, Q8, 1>(a, sms, s);
}

struct AttnWs {
    size_t prefix = 0, desc = 0, part = 0, total = 0;
    AttnWs(int B, int hd)
    {
        auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
        const size_t workers = static_cast<size_t>(kAttnMaxSms) * kAttnMaxWarps;
        desc = up((static_cast<size_t>(B) + 1) * 4);
        part = desc + up(workers * 4);
        total = part + 2 * workers * (static_cast<size_t>(hd) * 8 + 16) * 4;
    }
};

}  // namespace
}  // namespace twell

size_t twell_host::paged_attn_ws_bytes(int B, int hd)
{
    return B > 0 && hd > 0 ? twell::AttnWs(B, hd).total : 0;
}

using namespace twell_host;

extern "C" twell_status twell_paged_attn_decode(const void* q, int64_t q_stride, const twell_kv_cache* cache,
                                                const int32_t* page_table, const int32_t* seq_lens, int32_t B,
                                                int32_t n_q_heads, int32_t max_pages, float scale, int32_t window,
                                                void* out, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                                void* stream)
{
    twell::AttnArgs a{};
    twell_status st = check_kv(cache, &a.c);
    if (st != TWELL_OK) return st;
    if (B < 0 || n_q_heads <= 0 || max_pages <= 0 || window < 0 || dev_status == nullptr || n_q_heads % a.c.heads != 0)
        return TWELL_ERR_INVALID;
    const int hd = a.c.hd;
    if (hd != 64 && hd != 96 && hd != 128 && hd != 256) return TWELL_ERR_UNSUPPORTED;
    const long long cap = static_cast<long long>(max_pages) << a.c.page_shift;
    if (B > twell::kAttnMaxSeqs || cap > INT32_MAX - 16 || B * (cap / twell::kTileTokens + 1) > INT32_MAX ||
        static_cast<long long>(B) * n_q_heads > INT32_MAX)
        return TWELL_ERR_UNSUPPORTED;
    if (B == 0) return TWELL_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr) return TWELL_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || q_stride % 8 != 0 ||
        (B > 1 && q_stride < static_cast<int64_t>(n_q_heads) * hd))
        return TWELL_ERR_INVALID;
    const twell::AttnWs L(B, hd);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < L.total) return TWELL_ERR_WORKSPACE;
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.table = page_table;
    a.lens = seq_lens;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.status = dev_status;
    a.q_stride = q_stride;
    a.B = B;
    a.n_q = n_q_heads;
    a.G = n_q_heads / a.c.heads;
    a.max_pages = max_pages;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.prefix = reinterpret_cast<uint32_t*>(base + L.prefix);
    a.desc = reinterpret_cast<int*>(base + L.desc);
    a.part = reinterpret_cast<float*>(base + L.part);
    const int sms = std::min(dev.sm_count, twell::kAttnMaxSms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.c.q8) {
        if (hd == 64) return twell::run_heads<64, true>(a, sms, s);
        if (hd == 96) return twell::run_heads<96, true>(a, sms, s);
        if (hd == 128) return twell::run_heads<128, true>(a, sms, s);
        return twell::run_heads<256, true>(a, sms, s);
    }
    if (hd == 64) return twell::run_heads<64, false>(a, sms, s);
    if (hd == 96) return twell::run_heads<96, false>(a, sms, s);
    if (hd == 128) return twell::run_heads<128, false>(a, sms, s);
    return twell::run_heads<256, false>(a, sms, s);
}
