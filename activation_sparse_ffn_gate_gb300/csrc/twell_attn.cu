// twell_attn.cu -- attention of one new token per sequence over the paged key-value cache.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t - m),  t over the visible tokens
//
// What bounds it is the cache: every visible key and value is read once for all the query heads
// that share it, 2 x heads per key flops a byte, so the kernel is laid out to keep reads in flight.
//   - Split over the length. The work is the list of 32-token tiles of every (sequence, key head), in
//     that order, cut into equal contiguous ranges, one a warp of a grid of one block an SM: a batch
//     of ragged lengths and a single long sequence are balanced alike, and no range is empty of work
//     while another is long. A warp streams its tiles, keys and values in turn, through its own
//     shared-memory ring with 16-byte asynchronous copies (rows beyond the visible range are filled
//     with zeros and never read), across sequence boundaries, so that the ring stays full.
//   - The products are small matrix products with the tokens (for q . k) and the dimensions (for the
//     output) on the 16-row side of mma.sync m16n8k16 and the query heads on its 8 columns: a
//     group of up to 8 query heads costs what one does. tcgen05's 64 to 128 rows a tile would be
//     filled by 16 tokens a warp only after a block-wide exchange, and nothing here is bounded by
//     the products. The scores' fragment becomes the second product's operand by an 8x8 transpose
//     (movmatrix); the weights go in as hi + lo parts, bf16 with a bf16 cache (~16 bits) and fp16 with an
//     e4m3 cache (22 bits, of the largest weight 2^-40).
//   - A batch of short sequences whose (sequence, key head)s about fill the SMs skips the list: one block each,
//     which needs no second kernel; a large batch of short ones is dealt out in whole (sequence, key head)s, equally
//     many a warp, and needs neither (the rules are in run_attn).
//   - Running maximum m and sum l in fp32, per query head. For an e4m3 cache the value's scale s_t is
//     folded into the weight, w_t = p_t s_t, and m runs over score + log2 s_t, so that the largest weight is
//     2^15 whatever the scales: the fp16 parts then hold weights down to 2^-40 of it (with a largest weight of 1
//     and one part, 131071 tokens of 2^-26 each, 0.2% of the sum, were lost). p_t is formed times 2^32, so that it
//     neither overflows nor vanishes as long as a sequence's scales lie within 2^90 of one another. The query is
//     brought to [1, 2) by a power of two before its fp16 rounding (exact for bf16 values down to 2^-14 of the largest).
//   - Joining. A (sequence, key head) that lies within one warp's range is finished there. The parts
//     (m, l, unnormalised o, fp32) of one that spans warps of a block are joined by the block, through
//     shared memory; one that spans blocks leaves a part a block in the workspace, and a second kernel
//     joins those. Parts are joined in ascending order: the result does not depend on scheduling.
#include "twell_kv.cuh"
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kTileTokens = 32;
constexpr int kMTiles = kTileTokens / 16;  // 16-token rows of a product
constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxSms = 160;   // the workspace is sized for this many blocks, whatever the device
constexpr int kAttnMaxWarps = 16;  // and this many warps a block
// When a block takes a whole (sequence, key head): see run_attn.
constexpr int kPairIdle = 2, kPairTiles = 8;
// When a warp takes whole ones: likewise.
constexpr int kWholeTiles = 8, kWholeExtra = 4;
constexpr float kNegInf = -INFINITY;
// An e4m3 cache's sums: l is held times 2^kLift, the weights and o times 2^kUp (see scores); scales under kScaleMin count
// as that in the running maximum.
constexpr float kLift = 32.0f, kUp = 15.0f;
constexpr float kWeight = 7.62939453125e-06f;        // 2^(kUp - kLift)
constexpr float kOut = 131072.0f;                    // 2^(kLift - kUp)
constexpr float kScaleMin = 2.8421709430404007e-14f;  // 2^-45

// HD: head_dim; Q8: e4m3 cache; NT: query heads of one key head handled together, in eights.
template <int HD, bool Q8, int NT>
struct AttnCfg {
    static constexpr int kRow = HD * (Q8 ? 1 : 2);      // bytes of a token's key or value
    static constexpr int kChunks = kRow / 16;
    static constexpr int kSwizzle = kChunks % 8 == 0 ? 7 : (kChunks % 4 == 0 ? 3 : 1);
    static constexpr int kHalf = kTileTokens * kRow;    // bytes of a tile's keys, or its values
    static constexpr int kSlot = kHalf + (Q8 ? 2 * kTileTokens * 4 : 0);  // with keys: both scales behind them
    // Enough warps to keep up with the copies, few enough for three slots each and for ranges that are many tiles
    // long: 64 sequences of up to 16384 tokens, e4m3, head_dim 128: 93.1 us with 12 warps, 93.8 with 8 (16 have too few
    // registers: 129.7); 8 of up to 32768, e4m3, head_dim 64: 35.3 with 16, 41.4 with 12, 41.5 with 8.
    static constexpr int kWarps = HD == 256 ? (Q8 ? 8 : 4) : NT == 2 || kHalf > 4096 ? 8 : kHalf > 2048 ? 12 : 16;
    static constexpr int kFit = 212000 / (kWarps * kSlot);
    static constexpr int kSlots = kFit >= 7 ? 7 : kFit >= 5 ? 5 : 3;  // odd: keys are requested while keys are used
    static_assert(kFit >= 3, "the ring overlaps copies with the products");
    static constexpr int kMt = HD / 16;                 // 16-dimension tiles of the output
    static constexpr int kF = kMt % 4 == 0 ? 4 : 3;     // of them joined and stored together
    static constexpr int kRing = kSlots * kSlot;        // bytes of a warp's ring
    static constexpr int kPartF = NT * kMt * 128;       // floats of a part's o, then NT * 16 of m and l
    static constexpr int kPart = kPartF + NT * 16;
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kPart * 4 <= kRing, "a warp leaves its last part in its ring");
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
    int pairs;             // 1: one block a (sequence, key head)
    int whole;             // 1: whole (sequence, key head)s, equally many a warp
    float scale_log2;      // scale * log2(e)
    int2* split;           // [blocks] the (sequence, key head) that a block's start is the first to split, or -1,
                           // and the last block that holds some of it
    float* block_part;     // [2 * blocks][kPart] 0: of a (sequence, key head) from an earlier block, 1: into a later
    float* head_part;      // [workers][kPart] a warp's part of a (sequence, key head) that ends inside its range
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
    // item < total: the place of the item-th tile; returns the first tile of its (sequence, key head)
    __device__ __forceinline__ long long seek(const AttnArgs& a, const uint32_t* prefix, int HV, long long item)
    {
        // its tile among those of one key head, were the heads of a sequence taken together
        const uint32_t at = (item >> 32) == 0 ? static_cast<uint32_t>(item) / HV : static_cast<uint32_t>(item / HV);
        int lo = 0, hi = a.B;  // prefix[lo] <= at < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= at) lo = mid;
            else hi = mid;
        }
        b = lo;
        const uint32_t n = prefix[b + 1] - prefix[b];
        const long long rem = item - static_cast<long long>(prefix[b]) * HV;
        hv = (rem >> 32) == 0 ? static_cast<int>(static_cast<uint32_t>(rem) / n) : static_cast<int>(rem / n);
        tile = static_cast<int>(rem - static_cast<long long>(hv) * n);
        load(a);
        return item - tile;
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

// The list of `total` tiles cut into W equal ranges, one a warp of as many blocks as that takes (fewer
// tiles than warps: one each). Range w starts at total * w / W, formed from the quotient and the
// remainder of total / W so that each start costs a 32-bit division.
struct Ranges {
    long long quot;
    uint32_t rem, W;
    int blocks;
    __device__ __forceinline__ Ranges() : quot(0), rem(0), W(1), blocks(1) {}
    __device__ __forceinline__ Ranges(long long total, int max_blocks, int warps)
    {
        const uint32_t most = static_cast<uint32_t>(max_blocks * warps);
        W = total >= most ? most : (total > 1 ? static_cast<uint32_t>(total) : 1u);
        blocks = static_cast<int>((W + warps - 1) / warps);
        quot = (total >> 32) == 0 ? static_cast<uint32_t>(total) / W : total / W;
        rem = static_cast<uint32_t>(total - quot * W);
    }
    __device__ __forceinline__ long long start(uint32_t w) const
    {
        w = min(w, W);
        return quot * w + rem * w / W;
    }
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

    // A query's fragments, as bf16: requested here, brought into their final form by finish_q.
    __device__ __forceinline__ static void load_q(uint32_t (&q)[NT][kQ], const AttnArgs& a, int b, int hv, int lane)
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
            } else {
#pragma unroll
                for (int i = 0; i < kQ / 8; ++i) {
                    const bool on = live && 4 * i + c < HD / 16;
                    const uint4* p = reinterpret_cast<const uint4*>(src + 64 * i + 16 * c);
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u), u = on ? __ldg(p) : zero, v = on ? __ldg(p + 1) : zero;
                    q[n][8 * i] = u.x, q[n][8 * i + 1] = u.y, q[n][8 * i + 2] = u.z, q[n][8 * i + 3] = u.w;
                    q[n][8 * i + 4] = v.x, q[n][8 * i + 5] = v.y, q[n][8 * i + 6] = v.z, q[n][8 * i + 7] = v.w;
                }
            }
        }
    }
    __device__ __forceinline__ void finish_q(const AttnArgs& a, int lane)
    {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            qs[n][0] = qs[n][1] = a.scale_log2;
            if constexpr (Q8) {
                // the largest magnitude, as bf16 bits, over the head's four lanes; its power of two taken out
                __nv_bfloat162 m2 = __float2bfloat162_rn(0.0f);
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const uint32_t u = q[n][i] & 0x7fff7fffu;
                    m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162*>(&u));
                }
                float top = fmaxf(__low2float(m2), __high2float(m2));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
                const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&q[n][i]));
                    q[n][i] = f16x2_rn(f.x * down, f.y * down);
                }
                qs[n][0] *= __shfl_sync(0xffffffffu, up, 8 * c);
                qs[n][1] *= __shfl_sync(0xffffffffu, up, 8 * c + 4);
            }
        }
    }

    // The weights of a tile's tokens from its keys at `st` (and both scales behind them), as fragments of the
    // second product; bit t of `vis` says whether token t is visible.
    uint32_t ph[kMTiles][NT][2], pl[kMTiles][NT][2];
    __device__ __forceinline__ void scores(uint32_t st, uint32_t vis, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
        float x[kMTiles][NT][4];
#pragma unroll
        for (int t = 0; t < kMTiles; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) x[t][n][0] = x[t][n][1] = x[t][n][2] = x[t][n][3] = 0.0f;
        if constexpr (!Q8) {
            const int row = lane & 15, hi8 = lane >> 4;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i)
#pragma unroll
                for (int t = 0; t < kMTiles; ++t) {
                    uint32_t k[4];
                    ldsm_x4(k, st + (16 * t + row) * C::kRow + swizzled<C>(row, 2 * i + hi8, false) * 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_bf16(x[t][n], k[0], k[1], k[2], k[3], q[n][2 * i], q[n][2 * i + 1]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < kQ / 8; ++i)
#pragma unroll
                for (int t = 0; t < kMTiles; ++t) {
                    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0;
                    if (HD % 64 == 0 || 4 * i + c < HD / 16) {
                        k0 = lds128(st + (16 * t + g) * C::kRow + swizzled<C>(g, 4 * i + c, true) * 16);
                        k1 = lds128(st + (16 * t + g + 8) * C::kRow + swizzled<C>(g, 4 * i + c, true) * 16);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w0 = e == 0 ? k0.x : e == 1 ? k0.y : e == 2 ? k0.z : k0.w;
                        const uint32_t w1 = e == 0 ? k1.x : e == 1 ? k1.y : e == 2 ? k1.z : k1.w;
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_f16(w0, a0, a2);
                        e4m3x4_f16(w1, a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(x[t][n], a0, a1, a2, a3, q[n][8 * i + 2 * e], q[n][8 * i + 2 * e + 1]);
                    }
                }
        }

        // scores (base 2) of tokens 16t + g and 16t + g + 8 for heads 2c and 2c + 1; with an e4m3 cache the values' scales
        // and their log2, which the maximum alone contains, rounded up, so that no weight is above 2^kUp however large the
        // scores are
        float vs[kMTiles][2], lv[kMTiles][2];
#pragma unroll
        for (int t = 0; t < kMTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tok = 16 * t + 8 * h + g;
                const bool on = (vis >> tok) & 1u;
                float ks = 1.0f;
                vs[t][h] = 1.0f;
                lv[t][h] = 0.0f;
                if constexpr (Q8) {
                    ks = __uint_as_float(lds32(st + C::kHalf + 4 * tok));
                    vs[t][h] = __uint_as_float(lds32(st + C::kHalf + 4 * kTileTokens + 4 * tok));
                    // of a value that is not finite: any, so that m and l, which do not depend on values, stay finite
                    lv[t][h] = __log2f(vs[t][h] < INFINITY ? fmaxf(vs[t][h], kScaleMin) : 1.0f);
                    vs[t][h] *= kWeight;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    x[t][n][2 * h] = on ? x[t][n][2 * h] * (qs[n][0] * ks) : kNegInf;
                    x[t][n][2 * h + 1] = on ? x[t][n][2 * h + 1] * (qs[n][1] * ks) : kNegInf;
                }
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float t0 = kNegInf, t1 = kNegInf;
#pragma unroll
            for (int t = 0; t < kMTiles; ++t) {
                if constexpr (Q8) {
                    t0 = fmaxf(t0, fmaxf(__fadd_ru(x[t][n][0], lv[t][0]), __fadd_ru(x[t][n][2], lv[t][1])));
                    t1 = fmaxf(t1, fmaxf(__fadd_ru(x[t][n][1], lv[t][0]), __fadd_ru(x[t][n][3], lv[t][1])));
                } else {
                    t0 = fmaxf(t0, fmaxf(x[t][n][0], x[t][n][2]));
                    t1 = fmaxf(t1, fmaxf(x[t][n][1], x[t][n][3]));
                }
            }
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
            auto weight = [](float x, float b) { return exp2_approx(Q8 ? x - b + kLift : x - b); };
#pragma unroll
            for (int t = 0; t < kMTiles; ++t) {
                float p[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    p[2 * h] = weight(x[t][n][2 * h], b0);
                    p[2 * h + 1] = weight(x[t][n][2 * h + 1], b1);
                }
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
                if constexpr (Q8) {
                    const float w0 = p[0] * vs[t][0], w1 = p[1] * vs[t][0], w2 = p[2] * vs[t][1], w3 = p[3] * vs[t][1];
                    const uint32_t h0 = f16x2_rn(w0, w1), h1 = f16x2_rn(w2, w3);
                    const float2 r0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                    const float2 r1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                    ph[t][n][0] = transpose8(h0);
                    ph[t][n][1] = transpose8(h1);
                    pl[t][n][0] = transpose8(f16x2_rn(w0 - r0.x, w1 - r0.y));
                    pl[t][n][1] = transpose8(f16x2_rn(w2 - r1.x, w3 - r1.y));
                } else {
                    const uint32_t h0 = bf16x2_rn(p[0], p[1]), h1 = bf16x2_rn(p[2], p[3]);
                    const float2 r0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h0));
                    const float2 r1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h1));
                    ph[t][n][0] = transpose8(h0);
                    ph[t][n][1] = transpose8(h1);
                    pl[t][n][0] = transpose8(bf16x2_rn(p[0] - r0.x, p[1] - r0.y));
                    pl[t][n][1] = transpose8(bf16x2_rn(p[2] - r1.x, p[3] - r1.y));
                }
            }
        }
    }

    // o += v^T p from the tile's values at `sv`: dimensions on the rows
    __device__ __forceinline__ void values(uint32_t sv, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
        if constexpr (!Q8) {
            const int row = (lane & 7) + ((lane & 16) >> 1), odd = (lane >> 3) & 1;
#pragma unroll
            for (int t = 0; t < kMTiles; ++t)
#pragma unroll
                for (int i = 0; i < C::kMt; ++i) {
                    uint32_t v[4];
                    ldsm_x4_trans(v, sv + (16 * t + row) * C::kRow + swizzled<C>(row, 2 * i + odd, false) * 16);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_bf16(o[i][n], v[0], v[1], v[2], v[3], ph[t][n][0], ph[t][n][1]);
                        mma_bf16(o[i][n], v[0], v[1], v[2], v[3], pl[t][n][0], pl[t][n][1]);
                    }
                }
        } else {
            // lane (g, c): dimensions g HD / 8 ... of tokens 16t + 2c, 2c + 1, 2c + 8, 2c + 9
            constexpr int W = HD / 32;  // words of a token's dimensions
            constexpr int V = HD == 96 ? 1 : (W < 4 ? W : 4);  // words a load
#pragma unroll
            for (int t = 0; t < kMTiles; ++t)
#pragma unroll
                for (int w0 = 0; w0 < W; w0 += V) {
                    uint32_t v[4][V];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 2 * c + (r & 1) + (r >> 1) * 8;
                        const int byte = g * (HD / 8) + 4 * w0;
                        const uint32_t ad =
                            sv + (16 * t + row) * C::kRow + swizzled<C>(row, byte >> 4, true) * 16 + (byte & 15);
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
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_f16(x, a0, a1);
                            e4m3x4_f16(y, a2, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                mma_f16(o[2 * (w0 + w) + h][n], a0, a1, a2, a3, ph[t][n][0], ph[t][n][1]);
                                mma_f16(o[2 * (w0 + w) + h][n], a0, a1, a2, a3, pl[t][n][0], pl[t][n][1]);
                            }
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

// Final values of F fragments next to each other: dimension tiles i .. i + F - 1, eight heads n, the lane's four sums
// each with their heads' totals l; all 32 lanes of a warp call it for the same (n, i). i is a multiple of F.
template <int HD, bool Q8, int NT, int F>
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int hv, int n, int i, int lane, const float (&r)[F][4],
                                          float l0, float l1)
{
    const int g = lane >> 2, c = lane & 3;
    const int kvh = hv / a.blocks, first = (hv % a.blocks) * 8 * NT + n * 8;
    constexpr float kOne = Q8 ? kOut : 1.0f;
    const float i0 = l0 > 0.0f || l0 != l0 ? kOne / l0 : 0.0f, i1 = l1 > 0.0f || l1 != l1 ? kOne / l1 : 0.0f;
    __nv_bfloat16* base = a.out + (static_cast<int64_t>(b) * a.n_q + kvh * a.G) * HD;
    if constexpr (!Q8) {  // rows g and g + 8 of a tile, heads 2c and 2c + 1
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const uint32_t x = transpose8(bf16x2_rn(r[f][0] * i0, r[f][1] * i1));
            const uint32_t y = transpose8(bf16x2_rn(r[f][2] * i0, r[f][3] * i1));
            if (first + g < a.G) {
                uint32_t* p = reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(first + g) * HD + 16 * (i + f) + 2 * c);
                p[0] = x;
                p[4] = y;
            }
        }
    } else {  // dimensions g HD / 8 + 2i and the 2F - 1 after it, heads 2c and 2c + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x[F];
#pragma unroll
            for (int f = 0; f < F; ++f)
                x[f] = h ? bf16x2_rn(r[f][1] * i1, r[f][3] * i1) : bf16x2_rn(r[f][0] * i0, r[f][2] * i0);
            const int head = first + 2 * c + h;
            if (head >= a.G) continue;
            uint32_t* p = reinterpret_cast<uint32_t*>(base + static_cast<int64_t>(head) * HD + g * (HD / 8) + 2 * i);
            if constexpr (F % 4 == 0) {
#pragma unroll
                for (int f = 0; f < F; f += 4) *reinterpret_cast<uint4*>(p + f) = make_uint4(x[f], x[f + 1], x[f + 2], x[f + 3]);
            } else {
#pragma unroll
                for (int f = 0; f < F; ++f) p[f] = x[f];
            }
        }
    }
}

template <bool Q8, int NT>
__device__ __forceinline__ void store_lse(const AttnArgs& a, int b, int hv, int head, float m, float l)
{
    const int kvh = hv / a.blocks, j = (hv % a.blocks) * 8 * NT + head;
    if (a.lse != nullptr && j < a.G)
        a.lse[static_cast<int64_t>(b) * a.n_q + kvh * a.G + j] =
            l == 0.0f ? kNegInf : (m + (log2f(l) - (Q8 ? kLift : 0.0f))) * 0.69314718055994531f;
}

// Parts joined for F float4 of o (fragments ni .. ni + F - 1 = eight heads x F dimension tiles, this lane) and the two
// heads they belong to: their maximum first, then the sums under it, so that no exponential waits for the one before.
template <class C, int F>
struct Joined {
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.0f, l1 = 0.0f;
    float r[F][4] = {};

    __device__ __forceinline__ Joined() {}
    // part(i), i < count: where part i is
    template <typename P>
    __device__ __forceinline__ Joined(int count, int ni, int lane, P part)
    {
        const int ml = C::kPartF + ni / C::kMt * 16 + 2 * (lane & 3);
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float2 pm = *reinterpret_cast<const float2*>(part(i) + ml);
            m0 = fmaxf(m0, pm.x);
            m1 = fmaxf(m1, pm.y);
        }
        const float b0 = m0 == kNegInf ? 0.0f : m0, b1 = m1 == kNegInf ? 0.0f : m1;
#pragma unroll 2
        for (int i = 0; i < count; ++i) {
            const float* p = part(i);
            const float2 pm = *reinterpret_cast<const float2*>(p + ml), pl = *reinterpret_cast<const float2*>(p + ml + 8);
            const float f0 = exp2_approx(pm.x - b0), f1 = exp2_approx(pm.y - b1);
            l0 = fmaf(pl.x, f0, l0);
            l1 = fmaf(pl.y, f1, l1);
#pragma unroll
            for (int f = 0; f < F; ++f) add(f, reinterpret_cast<const float4*>(p)[(ni + f) * 32 + lane], f0, f1);
        }
    }
    __device__ __forceinline__ void add(int f, const float4& v, float f0, float f1)
    {
        r[f][0] = fmaf(v.x, f0, r[f][0]);
        r[f][1] = fmaf(v.y, f1, r[f][1]);
        r[f][2] = fmaf(v.z, f0, r[f][2]);
        r[f][3] = fmaf(v.w, f1, r[f][3]);
    }
    __device__ __forceinline__ void store(float* part, int ni, int lane) const
    {
#pragma unroll
        for (int f = 0; f < F; ++f)
            reinterpret_cast<float4*>(part)[(ni + f) * 32 + lane] = make_float4(r[f][0], r[f][1], r[f][2], r[f][3]);
        if (ni % C::kMt == 0 && lane < 4) {
            float* ml = part + C::kPartF + ni / C::kMt * 16 + 2 * lane;
            *reinterpret_cast<float2*>(ml) = make_float2(m0, m1);
            *reinterpret_cast<float2*>(ml + 8) = make_float2(l0, l1);
        }
    }
};

template <int HD, bool Q8, int NT, int F>
__device__ __forceinline__ void store_joined(const AttnArgs& a, int bhv, int HV, int ni, int lane,
                                             const Joined<AttnCfg<HD, Q8, NT>, F>& J)
{
    constexpr int kMt = AttnCfg<HD, Q8, NT>::kMt;
    const int b = bhv / HV, hv = bhv % HV, e = ni / kMt;
    store_out<HD, Q8, NT, F>(a, b, hv, e, ni % kMt, lane, J.r, J.l0, J.l1);
    if (ni % kMt == 0 && lane < 4) {
        store_lse<Q8, NT>(a, b, hv, e * 8 + 2 * lane, J.m0, J.l0);
        store_lse<Q8, NT>(a, b, hv, e * 8 + 2 * lane + 1, J.m1, J.l1);
    }
}

// The results of a key-head block of a sequence with nothing visible: zeros, lse = -inf. By `threads` threads.
template <int HD, int NT>
__device__ __forceinline__ void empty_heads(const AttnArgs& a, int b, int hv, int thread, int threads)
{
    const int first = hv % a.blocks * 8 * NT, heads = min(8 * NT, a.G - first);
    const int64_t row = static_cast<int64_t>(b) * a.n_q + hv / a.blocks * a.G + first;
    uint32_t* p = reinterpret_cast<uint32_t*>(a.out + row * HD);
    for (int i = thread; i < heads * HD / 2; i += threads) p[i] = 0u;
    if (a.lse != nullptr && thread < heads) a.lse[row + thread] = kNegInf;
}

template <int HD, bool Q8, int NT>
__global__ void __launch_bounds__(AttnCfg<HD, Q8, NT>::kWarps * 32, 1) paged_attn_kernel(const AttnArgs a)
{
    using C = AttnCfg<HD, Q8, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t sums[32];
    // the (sequence, key head)s that span warps of this block: [0] the one that ends inside warp 0's range,
    // [1 + w] the one whose first part in this block is warp w's last; bhv -1: none
    __shared__ long long run_i0[C::kWarps + 1], run_i1[C::kWarps + 1];
    __shared__ int run_bhv[C::kWarps + 1];
    __shared__ long long warp_start[C::kWarps + 1];  // the warps' ranges
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + C::kSmem);  // [B + 1]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_begin();

    const int cap = a.max_pages << a.c.page_shift;
    const int HV = a.c.heads * a.blocks;
    long long whole_tiles = 0;  // tiles of the warp's whole (sequence, key head)s
    long long total = 0, seg0 = 0;  // tiles in the list; the first tile of the (sequence, key head) at this warp's start
    Cursor cur;                     // where this warp's next tile to be used is
    Ranges R;
    int w0 = 0;                     // the block's first range
    if (a.pairs) {
        // the list is the block's own (sequence, key head)
        cur.b = blockIdx.x / HV;
        cur.hv = blockIdx.x % HV;
        const int raw = __ldg(a.lens + cur.b);
        if ((raw < 0 || raw > cap) && threadIdx.x == 0) report(a.status, TWELL_ERR_DEVICE_CHECK);
        cur.s = SeqSpan(raw, cap, a.window);
        if (cur.s.tiles == 0) {
            empty_heads<HD, NT>(a, cur.b, cur.hv, threadIdx.x, blockDim.x);
            return;
        }
        total = cur.s.tiles;
        R = Ranges(total, 1, C::kWarps);
    } else if (a.whole) {
        // the warp's share of them, and the tiles in it
        const uint32_t P = static_cast<uint32_t>(a.B) * HV, W = gridDim.x * C::kWarps, v = blockIdx.x * C::kWarps + warp;
        const uint32_t p0 = static_cast<uint32_t>(static_cast<uint64_t>(P) * v / W);
        const uint32_t p1 = static_cast<uint32_t>(static_cast<uint64_t>(P) * (v + 1) / W);
        bool found = false;
        for (uint32_t p = p0; p < p1;) {
            const uint32_t b = p / HV, hv = p - b * HV, here = min(p1, (b + 1) * HV) - p;  // of one sequence
            const int raw = __ldg(a.lens + b);
            if ((raw < 0 || raw > cap) && lane == 0) report(a.status, TWELL_ERR_DEVICE_CHECK);
            const SeqSpan s(raw, cap, a.window);
            whole_tiles += static_cast<long long>(s.tiles) * here;
            if (s.tiles == 0) {
                for (uint32_t h = hv; h < hv + here; ++h) empty_heads<HD, NT>(a, b, h, lane, 32);
            } else if (!found) {
                found = true;
                cur.b = b;
                cur.hv = hv;
                cur.s = s;
            }
            p += here;
        }
    } else {
        // tiles before each sequence (of one key head): a scan over the lengths, by every block for itself, and
        // for up to kWarpSeqs sequences by every warp (all write the same values), which needs no barrier
        constexpr int kWarpSeqs = 128;
        if (a.B <= kWarpSeqs) {
            int raw[kWarpSeqs / 32];
#pragma unroll
            for (int i = 0; i < kWarpSeqs / 32; ++i) raw[i] = 32 * i + lane < a.B ? __ldg(a.lens + 32 * i + lane) : 0;
            uint32_t carry = 0;
#pragma unroll
            for (int i = 0; i < kWarpSeqs / 32; ++i) {
                if (32 * i >= a.B) break;
                if ((raw[i] < 0 || raw[i] > cap) && blockIdx.x == 0) report(a.status, TWELL_ERR_DEVICE_CHECK);
                const uint32_t mine = SeqSpan(raw[i], cap, a.window).tiles;
                uint32_t run = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t u = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += u;
                }
                if (32 * i + lane < a.B) prefix[32 * i + lane] = carry + run - mine;
                carry += __shfl_sync(0xffffffffu, run, 31);
            }
            if (lane == 0) prefix[a.B] = carry;
            __syncwarp();
        } else {
            const int per = (a.B + blockDim.x - 1) / blockDim.x;
            const int b0 = threadIdx.x * per, b1 = min(b0 + per, a.B);
            uint32_t mine = 0;
#pragma unroll 4
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
            for (int i = 0; i < warp; ++i) run += sums[i];
            run -= mine;
            for (int b = b0; b < b1; ++b) {
                prefix[b] = run;
                run += SeqSpan(__ldg(a.lens + b), cap, a.window).tiles;
                if (b == a.B - 1) prefix[a.B] = run;
            }
            __syncthreads();
        }
        // sequences with nothing visible: zeros, lse = -inf
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            if (prefix[b + 1] != prefix[b]) continue;
            uint32_t* p = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(b) * a.n_q * HD);
            for (int i = threadIdx.x; i < a.n_q * HD / 2; i += blockDim.x) p[i] = 0u;
            if (a.lse != nullptr)
                for (int i = threadIdx.x; i < a.n_q; i += blockDim.x) a.lse[static_cast<int64_t>(b) * a.n_q + i] = kNegInf;
        }
        total = static_cast<long long>(prefix[a.B]) * HV;
        R = Ranges(total, gridDim.x, C::kWarps);
        if (static_cast<int>(blockIdx.x) >= R.blocks) {
            if (threadIdx.x == 0) a.split[blockIdx.x] = make_int2(-1, 0);
            return;
        }
        w0 = blockIdx.x * C::kWarps;
    }
    const int w = w0 + warp;
    const long long start = a.whole ? 0 : R.start(w), end = a.whole ? whole_tiles : R.start(w + 1);
    if (a.pairs) cur.tile = static_cast<int>(start);
    else if (!a.whole && start < end) seg0 = cur.seek(a, prefix, HV, start);
    const int bhv0 = cur.b * HV + cur.hv;

    const int n = static_cast<int>(end - start);
    uint8_t* ring_ptr = smem + warp * C::kRing;
    const uint32_t ring = smem_u32(ring_ptr);
    Cursor ahead = cur;  // where the next tile to be requested is
    int page = 0;        // of token `lane` of that tile
    auto load_page = [&](const Cursor& at) -> int {
        const int pos = (at.s.tile0 + at.tile) * kTileTokens + lane;
        if (pos < at.s.first || pos >= at.s.len) return -1;
        return __ldg(a.table + static_cast<int64_t>(at.b) * a.max_pages + (pos >> a.c.page_shift));
    };
    // The tile whose keys and values are being requested: its visible tokens (those of bad pages are left out) as
    // bits and where its rows are. A tile that lies in one page is copied from one address: lane `lane` takes chunk
    // `lane`, `lane` + 32, ..., kStep bytes apart where a page's tokens are adjacent.
    constexpr int kElt = Q8 ? 1 : 2, kCopies = C::kHalf / 512;
    const bool packed = (1 << a.c.page_shift) >= kTileTokens && a.c.token_stride * kElt == C::kRow;
    uint32_t tile_vis = 0;
    int64_t tile_off = 0;  // bytes: of the tile, where it is copied from one address, else of token `lane`
    auto request = [&](const void* base, uint32_t dst) {
        const uint8_t* src = static_cast<const uint8_t*>(base);
        if (packed && tile_vis == 0xffffffffu) {
            src += tile_off + lane * 16;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int id = i * 32 + lane, row = id / C::kChunks, ch = id % C::kChunks;
                cp_async16(dst + row * C::kRow + swizzled<C>(row, ch, Q8) * 16, src + i * 512, true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int id = i * 32 + lane, row = id / C::kChunks, ch = id % C::kChunks;
                const int64_t ro = __shfl_sync(0xffffffffu, tile_off, row);
                cp_async16(dst + row * C::kRow + swizzled<C>(row, ch, Q8) * 16, src + ro + ch * 16, (tile_vis >> row) & 1u);
            }
        }
    };
    auto request_keys = [&](uint32_t dst) {  // of the tile at `ahead`, from `page`
        const int pos = (ahead.s.tile0 + ahead.tile) * kTileTokens + lane;
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.n_pages)) {
            if (pos >= ahead.s.first && pos < ahead.s.len) report(a.status, TWELL_ERR_DEVICE_CHECK);
            page = -1;
        }
        tile_vis = __ballot_sync(0xffffffffu, page >= 0);
        const int in_page = pos & ((1 << a.c.page_shift) - 1), head = ahead.hv / a.blocks;
        tile_off = page >= 0 ? (page * a.c.page_stride + head * a.c.head_stride + in_page * a.c.token_stride) * kElt : 0;
        if constexpr (Q8) {
            const int64_t so = page >= 0 ? page * a.c.scale_page + head * a.c.scale_head + in_page : 0;
            cp_async4(dst + C::kHalf + 4 * lane, a.c.k_scale + so, page >= 0);
            cp_async4(dst + C::kHalf + 4 * (kTileTokens + lane), a.c.v_scale + so, page >= 0);
        }
        if (packed && tile_vis == 0xffffffffu) tile_off = __shfl_sync(0xffffffffu, tile_off, 0);
        request(a.c.k, dst);
    };

    // Slots of the ring hold keys and values in turn; kSlots - 1 are requested ahead.
    constexpr int kAhead = (C::kSlots - 1) / 2;  // tiles
    AttnState<HD, Q8, NT> S;
    uint32_t vis_ring = 0;  // lane i: the visible tokens of the tile i (modulo 32) of the range
    if (n > 0) S.load_q(S.q, a, cur.b, cur.hv, lane);
    int pages[kAhead + 1];  // of the first tiles, requested together
    {
        Cursor at = cur;
#pragma unroll
        for (int s = 0; s <= kAhead; ++s) {
            pages[s] = s < n ? load_page(at) : -1;
            if (s + 1 < n) at.next(a, HV);
        }
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
        if (s < n) {
            page = pages[s];
            request_keys(ring + 2 * s * C::kSlot);
            if (lane == s) vis_ring = tile_vis;
        }
        cp_commit();
        if (s < n) {
            request(a.c.v, ring + (2 * s + 1) * C::kSlot);
            ahead.next(a, HV);
        }
        cp_commit();
    }
    page = pages[kAhead];
    S.reset();
    S.finish_q(a, lane);
    if (threadIdx.x <= C::kWarps) {
        run_bhv[threadIdx.x] = -1;
        warp_start[threadIdx.x] = R.start(w0 + threadIdx.x);
    }
    if (threadIdx.x == 0 && !a.pairs && !a.whole) {  // is this block's start the first to split its (sequence, key head)?
        int2 sp = make_int2(-1, 0);
        if (blockIdx.x > 0 && start > seg0 && R.start(w0 - C::kWarps) <= seg0) {
            const long long seg1 = seg0 + cur.s.tiles;  // the last tile is in the range of warp ceil(seg1 W / total) - 1
            sp = make_int2(bhv0, static_cast<int>((seg1 * R.W + total - 1) / total - 1) / C::kWarps);
        }
        a.split[blockIdx.x] = sp;
    }
    __syncthreads();  // run_bhv, warp_start

    Cursor next;
    uint32_t slot = 0, free_slot = C::kSlots - 1;  // to be used, to be requested into
    auto advance = [&]() {
        free_slot = slot;
        slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    };
    for (int it = 0; it < n; ++it) {
        cp_wait<C::kSlots - 2>();
        __syncwarp();  // all lanes' copies of this slot are visible, and the one before has been read by all
        const uint32_t vis = __shfl_sync(0xffffffffu, vis_ring, it & 31);
        const bool seg_end = cur.tile + 1 == cur.s.tiles;
        uint32_t next_q[NT][AttnState<HD, Q8, NT>::kQ];  // of the (sequence, key head) that the next tile begins
        if (seg_end && it + 1 < n) {
            next = cur;
            next.next(a, HV);
            S.load_q(next_q, a, next.b, next.hv, lane);
        }
        if (it + kAhead < n) {
            request_keys(ring + free_slot * C::kSlot);
            if (lane == ((it + kAhead) & 31)) vis_ring = tile_vis;
        }
        cp_commit();
        S.scores(ring + slot * C::kSlot, vis, lane);
        advance();
        cp_wait<C::kSlots - 2>();
        __syncwarp();
        if (it + kAhead < n) {
            request(a.c.v, ring + free_slot * C::kSlot);
            ahead.next(a, HV);
            if (it + kAhead + 1 < n) page = load_page(ahead);
        }
        cp_commit();
        S.values(ring + slot * C::kSlot, lane);
        advance();

        if (seg_end || it + 1 == n) {
            S.close();
            if (seg_end && it >= cur.tile) {  // its first tile was this warp's too
#pragma unroll
                for (int e = 0; e < NT; ++e) {
#pragma unroll
                    for (int i = 0; i < C::kMt; i += C::kF) {
                        float r[C::kF][4];
#pragma unroll
                        for (int f = 0; f < C::kF; ++f)
#pragma unroll
                            for (int k = 0; k < 4; ++k) r[f][k] = S.o[i + f][e][k];
                        store_out<HD, Q8, NT, C::kF>(a, cur.b, cur.hv, e, i, lane, r, S.l[e][0], S.l[e][1]);
                    }
                    if (lane < 4) {
                        store_lse<Q8, NT>(a, cur.b, cur.hv, e * 8 + 2 * lane, S.m[e][0], S.l[e][0]);
                        store_lse<Q8, NT>(a, cur.b, cur.hv, e * 8 + 2 * lane + 1, S.m[e][1], S.l[e][1]);
                    }
                }
            } else if (it + 1 < n) {  // ends inside the range, began before it
                S.store_part(a.head_part + static_cast<int64_t>(w) * C::kPart, lane);
                if (warp == 0 && lane == 0) {
                    run_i0[0] = seg0;
                    run_i1[0] = start + it + 1;
                    run_bhv[0] = bhv0;
                }
            } else {  // the last of the range
                cp_wait<0>();
                __syncwarp();
                S.store_part(reinterpret_cast<float*>(ring_ptr), lane);
                const long long i0 = end - 1 - cur.tile;
                if (lane == 0 && (i0 >= start || warp == 0)) {
                    run_i0[1 + warp] = i0;
                    run_i1[1 + warp] = i0 + cur.s.tiles;
                    run_bhv[1 + warp] = cur.b * HV + cur.hv;
                }
            }
            if (it + 1 < n) {
                cur = next;
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int i = 0; i < AttnState<HD, Q8, NT>::kQ; ++i) S.q[e][i] = next_q[e][i];
                S.reset();
                S.finish_q(a, lane);
            }
        } else {
            ++cur.tile;
        }
    }
    cp_wait<0>();
    __syncthreads();

    // join the parts of what spans warps: kF fragments of one of them a warp at a time
    constexpr int kF = C::kF, kItems = NT * C::kMt / kF;
    const uint32_t runs = __ballot_sync(0xffffffffu, lane <= C::kWarps && run_bhv[min(lane, C::kWarps)] >= 0);
    const int items = __popc(runs) * kItems;
    const long long c_start = warp_start[0], c_end = warp_start[C::kWarps];
    for (int it = warp; it < items; it += C::kWarps) {
        const int ni = it % kItems * kF;
        uint32_t rest = runs;  // the (it / kItems)-th run
        for (int i = it / kItems; i > 0; --i) rest &= rest - 1u;
        const int run = __ffs(rest) - 1;
        const long long i0 = run_i0[run], i1 = run_i1[run];
        const float* head = a.head_part + static_cast<int64_t>(w0) * C::kPart;
        // the run's warps: from run - 1 to the last whose range starts before i1; that one has left its part in
        // the workspace if its range goes on beyond i1
        const int first = max(run - 1, 0);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, lane == first || (lane < C::kWarps && lane > first && run != 0 &&
                                                                             warp_start[min(lane, C::kWarps)] < i1)));
        const bool last_head = run == 0 || (last != first && warp_start[last + 1] > i1);
        const Joined<C, kF> J(last - first + 1, ni, lane, [&](int i) {
            const int q = first + i;
            return q == last && last_head ? head + static_cast<int64_t>(q) * C::kPart
                                          : reinterpret_cast<const float*>(smem + q * C::kRing);
        });
        if (i0 >= c_start && i1 <= c_end) store_joined<HD, Q8, NT, kF>(a, run_bhv[run], HV, ni, lane, J);
        else J.store(a.block_part + (2 * static_cast<int64_t>(blockIdx.x) + (i0 < c_start ? 0 : 1)) * C::kPart, ni, lane);
    }
}

// Joins the parts of the (sequence, key head) that main block blockIdx.x's start is the first to split: the second part
// of the block before, the first ones of this and the following blocks. The parts' weights are formed once for the
// block; then kGroups groups of threads, one float4 of the output a thread, take every kGroups-th part.
template <int HD, bool Q8, int NT>
struct JoinCfg {
    static constexpr int kFrags = NT * (HD / 16);
    static constexpr int kGroups = std::max(1, 32 / kFrags);
    static constexpr int kThreads = kGroups * kFrags * 32;
    static constexpr int kBatch = 8;  // parts of a group requested before the weights are known
};
template <int HD, bool Q8, int NT>
__global__ void __launch_bounds__(JoinCfg<HD, Q8, NT>::kThreads, 1) paged_attn_join_kernel(const AttnArgs a)
{
    using C = AttnCfg<HD, Q8, NT>;
    using K = JoinCfg<HD, Q8, NT>;
    constexpr int kHeads = NT * 8;
    __shared__ float4 s_sum[K::kThreads];
    __shared__ float s_m[kAttnMaxSms + 1][kHeads], s_l[kAttnMaxSms + 1][kHeads];
    __shared__ float s_top[kHeads], s_tot[kHeads];
    pdl_begin();
    const int2 sp = a.split[blockIdx.x];
    if (sp.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp / K::kFrags, ni = warp % K::kFrags;
    const int count = sp.y - static_cast<int>(blockIdx.x) + 2;
    const float* first = a.block_part + (2 * static_cast<int64_t>(blockIdx.x) - 1) * C::kPart;
    auto part = [&](int p) { return first + (p == 0 ? 0 : 2 * static_cast<int64_t>(p) - 1) * C::kPart; };
    float4 v[K::kBatch];
#pragma unroll
    for (int i = 0; i < K::kBatch; ++i) {
        const int p = grp + i * K::kGroups;
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p < count) v[i] = reinterpret_cast<const float4*>(part(p))[ni * 32 + lane];
    }
    for (int i = threadIdx.x; i < count * kHeads; i += K::kThreads) {
        const int p = i / kHeads, h = i % kHeads;
        const float* ml = part(p) + C::kPartF + (h >> 3) * 16 + (h & 7);
        s_m[p][h] = ml[0];
        s_l[p][h] = ml[8];
    }
    __syncthreads();
    for (int h = warp; h < kHeads; h += K::kThreads / 32) {
        float top = kNegInf, tot = 0.0f;
        for (int p = lane; p < count; p += 32) top = fmaxf(top, s_m[p][h]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float b = top == kNegInf ? 0.0f : top;
        for (int p = lane; p < count; p += 32) {
            const float f = exp2_approx(s_m[p][h] - b);
            s_m[p][h] = f;
            tot = fmaf(s_l[p][h], f, tot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        if (lane == 0) {
            s_top[h] = top;
            s_tot[h] = tot;
        }
    }
    __syncthreads();
    Joined<C, 1> J;
    const int h = ni / C::kMt * 8 + 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < K::kBatch; ++i) {
        const int p = grp + i * K::kGroups;
        if (p < count) J.add(0, v[i], s_m[p][h], s_m[p][h + 1]);
    }
#pragma unroll 4
    for (int p = grp + K::kBatch * K::kGroups; p < count; p += K::kGroups)
        J.add(0, reinterpret_cast<const float4*>(part(p))[ni * 32 + lane], s_m[p][h], s_m[p][h + 1]);
    if (K::kGroups > 1) {  // the groups' sums, in group order
        s_sum[threadIdx.x] = make_float4(J.r[0][0], J.r[0][1], J.r[0][2], J.r[0][3]);
        __syncthreads();
        if (grp != 0) return;
#pragma unroll
        for (int q = 1; q < K::kGroups; ++q) J.add(0, s_sum[(q * K::kFrags + ni) * 32 + lane], 1.0f, 1.0f);
    }
    J.m0 = s_top[h];
    J.m1 = s_top[h + 1];
    J.l0 = s_tot[h];
    J.l1 = s_tot[h + 1];
    store_joined<HD, Q8, NT, 1>(a, sp.x, a.c.heads * a.blocks, ni, lane, J);
}

template <int HD, bool Q8, int NT>
twell_status run_attn(AttnArgs& a, int sms, cudaStream_t s)
{
    using C = AttnCfg<HD, Q8, NT>;
    static_assert(NT * C::kWarps <= kAttnMaxWarps, "the workspace holds kAttnMaxWarps warps' parts of eight heads");
    auto kern = paged_attn_kernel<HD, Q8, NT>;
    static std::atomic<uint64_t> allowed{0};
    if (twell_host::allow_smem(kern, C::kSmem + (kAttnMaxSeqs + 1) * 4, allowed) != TWELL_OK) return TWELL_ERR_CUDA;
    // One block for each (sequence, key head), without the list and its second kernel, where they fit the SMs and what the
    // page table's width lets be visible is few tiles a warp: at most kPairTiles, and at most kPairIdle times the share
    // of the SMs that would idle (38 sequences of up to 1000 / 2000 tokens, 4 key heads of 128: 12.3 / 18.0 us against 16.3 /
    // 20.2 through the list; but 8 of up to 2000 with 8 key heads, e4m3: 16.6 against 11.6).
    const long long cap = static_cast<long long>(a.max_pages) << a.c.page_shift;
    const long long seen = a.window > 0 ? std::min<long long>(cap, static_cast<long long>(a.window) + kTileTokens - 1) : cap;
    const long long pairs = static_cast<long long>(a.B) * a.c.heads * a.blocks;
    const long long each = (seen + static_cast<long long>(kTileTokens) * C::kWarps - 1) / (kTileTokens * C::kWarps);
    a.pairs = pairs <= sms && each <= kPairTiles && each * (sms - pairs) <= static_cast<long long>(kPairIdle) * sms;
    // More of them, of few tiles each: whole ones a warp, equally many, without the scan over the lengths, the search and
    // the second kernel; as long as the fullest warp has at most kWholeExtra tiles more than its share of the table's
    // width (125 sequences of 256 tokens, 8 key heads of 128: 32.1 -> 23.2 us; 40 of up to 53, 4 key heads of 256: 9.9 ->
    // 7.3; but 40 of up to 256 with 8 key heads, e4m3, 12.8 against 12.0 through the list).
    const long long warps = static_cast<long long>(sms) * C::kWarps, tiles = (seen + kTileTokens - 1) / kTileTokens;
    a.whole = !a.pairs && tiles <= kWholeTiles && (pairs + warps - 1) / warps * tiles <= pairs * tiles / warps + kWholeExtra;
    if (a.pairs)
        return twell_host::launch_dep(kern, dim3(static_cast<unsigned>(pairs)), dim3(C::kWarps * 32), C::kSmem, s, a);
    const size_t smem = C::kSmem + (static_cast<size_t>(a.B) + 1) * 4;
    twell_status st = twell_host::launch_dep(kern, dim3(sms), dim3(C::kWarps * 32), smem, s, a);
    if (st != TWELL_OK || a.whole) return st;
    return twell_host::launch_dep(paged_attn_join_kernel<HD, Q8, NT>, dim3(sms), dim3(JoinCfg<HD, Q8, NT>::kThreads), 0,
                                  s, a);
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
    size_t split = 0, block_part = 0, head_part = 0, total = 0;
    explicit AttnWs(int hd)
    {
        const size_t part = (static_cast<size_t>(hd) * 8 + 16) * 4;  // of eight heads
        block_part = kAttnMaxSms * sizeof(int2);
        head_part = block_part + 2 * kAttnMaxSms * 2 * part;
        total = head_part + static_cast<size_t>(kAttnMaxSms) * kAttnMaxWarps * part;
    }
};

}  // namespace
}  // namespace twell

size_t twell_host::paged_attn_ws_bytes(int B, int hd)
{
    return B > 0 && hd > 0 ? twell::AttnWs(hd).total : 0;
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
    if (B > twell::kAttnMaxSeqs || cap > INT32_MAX - twell::kTileTokens || B * (cap / twell::kTileTokens + 1) > INT32_MAX ||
        n_q_heads > 65535 || static_cast<long long>(B) * n_q_heads > INT32_MAX)
        return TWELL_ERR_UNSUPPORTED;
    if (B == 0) return TWELL_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr) return TWELL_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || q_stride % 8 != 0 ||
        (B > 1 && q_stride < static_cast<int64_t>(n_q_heads) * hd))
        return TWELL_ERR_INVALID;
    const twell::AttnWs L(hd);
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
    a.split = reinterpret_cast<int2*>(base + L.split);
    a.block_part = reinterpret_cast<float*>(base + L.block_part);
    a.head_part = reinterpret_cast<float*>(base + L.head_part);
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
