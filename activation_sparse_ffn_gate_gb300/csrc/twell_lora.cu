// twell_lora.cu -- low-rank adapters of many requests beside a shared projection: to each token's row y the product
// s B (A x) of its own adapter (or of none) is added, A [R, k] and B [n, R] of bf16.
//
// Tokens of one adapter go together, 16 MT of them a tile, so that its weights are read once a tile. A cluster of blocks does
// a tile: each block has a part of k for t = A x, the parts go to all blocks through distributed shared memory and are added
// there in one order, and each block then has a part of n for y + B t. So one launch does, t never reaches memory, and a
// single token's weights are spread over eight SMs. Both products are mma.sync with the tokens as rows; a warp's weights are
// its own, so that they go straight from memory into fragments. Which element of k (or of a rank) stands where in a fragment
// is free as long as both operands agree: a lane takes 16 adjacent bytes of a row, and 8 adjacent columns of y.
// t enters the second product as hi + lo bf16: 16 bits of it, for twice the products of a small rank.
#include "twell_mma.cuh"
#include "twell_ops.cuh"

namespace twell {
namespace {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 4096;
constexpr int kLoraMaxTokens = 1 << 20;
constexpr int kLoraMaxDim = 1 << 20;
constexpr int kLoraWarps = 8;
constexpr int kLoraThreads = 32 * kLoraWarps;
constexpr int kLoraCluster = 8;      // most blocks a tile
constexpr int kLoraSmallN = 512;     // up to here every cluster finds its tile from the ids itself
constexpr int kLoraSmallMT = 1;
constexpr int kLoraGroupThreads = 1024;

struct LoraArgs {
    const __nv_bfloat16 *a, *b, *x, *y;
    __nv_bfloat16* out;
    const float* scale;
    const int32_t *ranks, *ids;
    int32_t* status;
    int64_t ldx, ldy, ldo;
    int L, R, k, n, N;
    // of larger batches: the number of tiles, then a tile's adapter, first place in `order`, tokens
    const int32_t* n_tiles;
    const int4* tiles;
    const int32_t* order;
};

// Shared memory of a block: floats of the warps' sums (then the fragments of t), of the blocks' sums.
template <int MT, int RG, int RT>
struct LoraShape {
    static constexpr int kTok = 16 * MT;
    static constexpr int kWays = kLoraWarps / RG;     // warps that share a part of k
    static constexpr int kRanks = RG * RT * 8;
    static constexpr int kPitch = kRanks + 4;         // floats of a token's row
    static constexpr int kBlock = RT == 2 ? 16 : 32;  // ranks of which a lane takes a quarter at a time
    static constexpr int kFrags = kRanks / 16;
    static constexpr int kSum = kTok * kPitch;
    static constexpr int kFragFloats = MT * kFrags * 2 * 32 * 4;
    static constexpr int kWarpSums = kWays * kSum > kFragFloats ? kWays * kSum : kFragFloats;
    static constexpr size_t bytes(int cluster) { return sizeof(float) * (kWarpSums + static_cast<size_t>(cluster) * kSum); }
};

__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_blocks()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_cluster16(uint32_t at, const float4& v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// A token's adapter, L for none (-1, or one that does not exist, which is recorded).
__device__ __forceinline__ int lora_id(const LoraArgs& g, int id)
{
    if (id >= 0 && id < g.L) return id;
    if (id != -1) report(g.status, TWELL_ERR_DEVICE_CHECK);
    return g.L;
}

// Hi and lo parts of two numbers as bf16 pairs; what is not finite has no lo.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = bf16x2_rn(a, b);
    const float ha = __uint_as_float(hi << 16), hb = __uint_as_float(hi & 0xffff0000u);
    lo = bf16x2_rn(fabsf(ha) <= 3.4e38f ? a - ha : 0.0f, fabsf(hb) <= 3.4e38f ? b - hb : 0.0f);
}

// The tile of cluster `index` among those of at most kLoraSmallN tokens: tokens are taken in their order by one warp, each is
// given its number among those of its adapter, and every kTok-th of these begins a tile. All blocks of a cluster find the
// same. `count` has a place for each adapter.
template <int TOK>
__device__ __forceinline__ void lora_find(const LoraArgs& g, int index, int* count, uint16_t* number, int* tok, int& id, int& tokens)
{
    __shared__ int found[2];  // adapter, number of the tile's first token
    __shared__ int own[kLoraSmallN];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
    for (int i = tid; i < g.N; i += kLoraThreads) {
        own[i] = lora_id(g, g.ids[i]);
        count[own[i]] = 0;
    }
    if (tid == 0) found[0] = -1;
    if (tid < TOK) tok[tid] = -1;
    __syncthreads();
    if (tid < 32) {
        int tiles = 0;
        for (int i0 = 0; i0 < g.N; i0 += 32) {
            const int i = i0 + lane;
            const int mine = i < g.N ? own[i] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, mine);
            const int before = __popc(same & ((1u << lane) - 1));
            const int num = mine >= 0 ? count[mine] + before : 1;
            __syncwarp();
            if (mine >= 0) {
                number[i] = static_cast<uint16_t>(num);
                if (before == 0) count[mine] += __popc(same);
            }
            const unsigned first = __ballot_sync(0xffffffffu, num % TOK == 0);
            if ((first >> lane & 1) && tiles + __popc(first & ((1u << lane) - 1)) == index) {
                found[0] = mine;
                found[1] = num;
            }
            tiles += __popc(first);
            __syncwarp();
        }
    }
    __syncthreads();
    id = found[0];
    if (id < 0) return;
    tokens = min(count[id] - found[1], TOK);
    for (int i = tid; i < g.N; i += kLoraThreads)
        if (own[i] == id && static_cast<unsigned>(number[i] - found[1]) < static_cast<unsigned>(TOK)) tok[number[i] - found[1]] = i;
    __syncthreads();
}

template <int MT, int RG, int RT, bool SMALL>
__global__ void __launch_bounds__(kLoraThreads, MT == 4 ? 1 : 2) lora_kernel(const LoraArgs g)
{
    using S = LoraShape<MT, RG, RT>;
    extern __shared__ __align__(16) float lora_smem[];
    __shared__ int tok[S::kTok];
    pdl_begin();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5, gr = lane >> 2, c = lane & 3;
    const int blocks = static_cast<int>(cluster_blocks()), part = static_cast<int>(cluster_ctarank());
    const int index = static_cast<int>(blockIdx.x) / blocks;
    int id, tokens = 0;
    if constexpr (SMALL) {
        // the counts and numbers lie where the sums come later
        lora_find<S::kTok>(g, index, reinterpret_cast<int*>(lora_smem),
                           reinterpret_cast<uint16_t*>(reinterpret_cast<int*>(lora_smem) + g.L + 1), tok, id, tokens);
        if (id < 0) return;
    } else {
        if (index >= *g.n_tiles) return;
        const int4 t = g.tiles[index];
        id = t.x;
        tokens = t.z;
        if (tid < S::kTok) tok[tid] = tid < tokens ? g.order[t.y + tid] : -1;
        __syncthreads();
    }
    int rank = 0;
    if (id < g.L) {
        rank = g.ranks ? __ldg(g.ranks + id) : g.R;
        if (rank < 0 || rank > g.R) {
            report(g.status, TWELL_ERR_DEVICE_CHECK);
            rank = 0;
        }
    }
    const int nt_all = (g.n + 31) / 32, nt0 = static_cast<int>(static_cast<long long>(nt_all) * part / blocks),
              nt1 = static_cast<int>(static_cast<long long>(nt_all) * (part + 1) / blocks);
    if (rank == 0) {  // the same for all blocks of the cluster
        if (g.y == g.out) return;
        const int col0 = nt0 * 4, cols = min(nt1 * 4, g.n / 8) - col0;  // in chunks of 8
        for (int i = tid; i < tokens * cols; i += kLoraThreads) {
            const int t = tok[i / cols], col = (col0 + i % cols) * 8;
            *reinterpret_cast<uint4*>(g.out + t * g.ldo + col) = *reinterpret_cast<const uint4*>(g.y + t * g.ldy + col);
        }
        return;
    }
    if (blocks > 1) cluster_arrive();  // this block runs: the others may write to its shared memory

    // t = A x, this block's part of k: a warp has RT times 8 ranks and every kWays-th 64 columns
    const __nv_bfloat16* A = g.a + static_cast<int64_t>(id) * g.R * g.k;
    const int rg = warp % RG, way = warp / RG;
    float acc[MT][RT][4] = {};
    {
        const int kb_all = (g.k + 63) / 64, kb0 = static_cast<int>(static_cast<long long>(kb_all) * part / blocks),
                  kb1 = static_cast<int>(static_cast<long long>(kb_all) * (part + 1) / blocks);
        const __nv_bfloat16* xrow[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int t = tok[16 * m + 8 * s + gr];
                xrow[m][s] = t >= 0 ? g.x + t * g.ldx : nullptr;
            }
        const int row0 = rg * RT * 8 + gr;
        for (int kb = kb0 + way; kb < kb1 && rg * RT * 8 < rank; kb += S::kWays) {
            uint4 xv[2][MT][2], wv[2][RT];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = 64 * kb + 32 * h + 8 * c;
                const bool in = col < g.k;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    wv[h][r] = make_uint4(0u, 0u, 0u, 0u);
                    if (in && row0 + 8 * r < rank) wv[h][r] = ldg_stream16(A + static_cast<int64_t>(row0 + 8 * r) * g.k + col);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        xv[h][m][s] = make_uint4(0u, 0u, 0u, 0u);
                        if (in && xrow[m][s] != nullptr) xv[h][m][s] = __ldg(reinterpret_cast<const uint4*>(xrow[m][s] + col));
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint4 &u = xv[h][m][0], &v = xv[h][m][1], &w = wv[h][r];
                        mma_bf16(acc[m][r], u.x, v.x, u.y, v.y, w.x, w.y);
                        mma_bf16(acc[m][r], u.z, v.z, u.w, v.w, w.z, w.w);
                    }
        }
    }

    // y + B t, this block's part of n: a warp has every kLoraWarps-th 32 columns. The weights of its first ones are on their
    // way while t is put together.
    const __nv_bfloat16* B = g.b + static_cast<int64_t>(id) * g.n * g.R;
    constexpr int kKb = S::kRanks / S::kBlock, kPer = S::kBlock / 4, kWords = kPer / 2;
    uint32_t bw[kKb][4][kWords];
    auto load_b = [&](int nt) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = 32 * nt + 8 * (gr >> 1);
            const __nv_bfloat16* row = B + static_cast<int64_t>(col + 2 * u + (gr & 1)) * g.R;
#pragma unroll
            for (int kb = 0; kb < kKb; ++kb) {
                const int r0 = kb * S::kBlock + kPer * c;
#pragma unroll
                for (int w = 0; w < kWords; ++w) bw[kb][u][w] = 0u;
                if (col < g.n && r0 < rank) {
                    if constexpr (kWords == 4) {
                        const uint4 v = ldg_stream16(row + r0);
                        bw[kb][u][0] = v.x, bw[kb][u][1] = v.y, bw[kb][u][2] = v.z, bw[kb][u][3] = v.w;
                    } else {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + r0));
                        bw[kb][u][0] = v.x, bw[kb][u][1] = v.y;
                    }
                }
            }
        }
    };
    // what lies past the rank counts for nothing, whatever it is
    auto mask_b = [&] {
        if (rank % kPer == 0) return;
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const int left = rank - (kb * S::kBlock + kPer * c + 2 * w);
                const uint32_t keep = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
#pragma unroll
                for (int u = 0; u < 4; ++u) bw[kb][u][w] &= keep;
            }
    };
    if (nt0 + warp < nt1) load_b(nt0 + warp);

    float* sums = lora_smem;
    float* recv = lora_smem + S::kWarpSums;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float* p = sums + way * S::kSum + (16 * m + gr) * S::kPitch + 8 * (rg * RT + r) + 2 * c;
            *reinterpret_cast<float2*>(p) = make_float2(acc[m][r][0], acc[m][r][1]);
            *reinterpret_cast<float2*>(p + 8 * S::kPitch) = make_float2(acc[m][r][2], acc[m][r][3]);
        }
    __syncthreads();
    if (blocks > 1) cluster_wait();
    constexpr int kQuads = S::kRanks / 4;
    for (int i = tid; i < S::kTok * kQuads; i += kLoraThreads) {
        const int at = i / kQuads * S::kPitch + i % kQuads * 4;
        float4 v = *reinterpret_cast<const float4*>(sums + at);
#pragma unroll
        for (int w = 1; w < S::kWays; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(sums + w * S::kSum + at);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        float* to = recv + part * S::kSum + at;
        if (blocks == 1) {
            *reinterpret_cast<float4*>(to) = v;
        } else {
            for (int d = 0; d < blocks; ++d) st_cluster16(mapa_shared(smem_u32(to), d), v);
        }
    }
    if (blocks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // t, whole, under its scale, as the second product's fragments: [row tile][16 ranks][hi, lo][lane]
    uint4* frags = reinterpret_cast<uint4*>(sums);
    const float scale = __ldg(g.scale + id);
    for (int i = tid; i < MT * S::kFrags * 32; i += kLoraThreads) {
        const int l = i & 31, f = (i >> 5) % S::kFrags, m = (i >> 5) / S::kFrags;
        constexpr int kHalves = S::kBlock / 16;
        const int r0 = f / kHalves * S::kBlock + kPer * (l & 3) + 4 * (f % kHalves);
        const float* p = recv + (16 * m + (l >> 2)) * S::kPitch + r0;
        float4 v[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v[s] = *reinterpret_cast<const float4*>(p + s * 8 * S::kPitch);
            for (int d = 1; d < blocks; ++d) {
                const float4 u = *reinterpret_cast<const float4*>(p + d * S::kSum + s * 8 * S::kPitch);
                v[s].x += u.x, v[s].y += u.y, v[s].z += u.z, v[s].w += u.w;
            }
            // past the rank a row of zeros met x, which is NaN where x is infinite
            v[s].x = r0 < rank ? v[s].x * scale : 0.0f;
            v[s].y = r0 + 1 < rank ? v[s].y * scale : 0.0f;
            v[s].z = r0 + 2 < rank ? v[s].z * scale : 0.0f;
            v[s].w = r0 + 3 < rank ? v[s].w * scale : 0.0f;
        }
        uint4 hi, lo;
        split2(v[0].x, v[0].y, hi.x, lo.x);
        split2(v[1].x, v[1].y, hi.y, lo.y);
        split2(v[0].z, v[0].w, hi.z, lo.z);
        split2(v[1].z, v[1].w, hi.w, lo.w);
        frags[((m * S::kFrags + f) * 2 + 0) * 32 + l] = hi;
        frags[((m * S::kFrags + f) * 2 + 1) * 32 + l] = lo;
    }
    __syncthreads();

    int token[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) token[m][s] = tok[16 * m + 8 * s + gr];
    for (int nt = nt0 + warp; nt < nt1; nt += kLoraWarps) {
        const int col = 32 * nt + 8 * c;
        uint4 yv[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (col < g.n && token[m][s] >= 0) yv[m][s] = *reinterpret_cast<const uint4*>(g.y + token[m][s] * g.ldy + col);
        if (nt != nt0 + warp) load_b(nt);
        mask_b();
        float d[MT][4][4] = {};
#pragma unroll
        for (int f = 0; f < S::kFrags; ++f) {
            constexpr int kHalves = S::kBlock / 16;
            const int kb = f / kHalves, h = f % kHalves;
            if (kb * S::kBlock >= rank) break;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint4 a = frags[((m * S::kFrags + f) * 2 + p) * 32 + lane];
#pragma unroll
                    for (int u = 0; u < 4; ++u) mma_bf16(d[m][u], a.x, a.y, a.z, a.w, bw[kb][u][2 * h], bw[kb][u][2 * h + 1]);
                }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (col < g.n && token[m][s] >= 0) {
                    float v[8];
                    unpack16(yv[m][s], v, static_cast<__nv_bfloat16*>(nullptr));
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[2 * u] += d[m][u][2 * s];
                        v[2 * u + 1] += d[m][u][2 * s + 1];
                    }
                    store8(g.out + token[m][s] * g.ldo + col, v);
                }
    }
}

// The tiles of a larger batch: tokens counted by adapter, each adapter's given adjacent places in `order`, and a tile for each
// TOK of these. One block: the counts are in its shared memory, and 16384 ids are 64 KB. Which token of an adapter comes
// first is left to chance; a token's result does not depend on it.
template <int TOK>
__global__ void __launch_bounds__(kLoraGroupThreads) lora_group_kernel(const LoraArgs g, int32_t* n_tiles, int4* tiles, int32_t* order)
{
    extern __shared__ int count[];  // [L + 1] of tokens, then their first place
    __shared__ int warp_sum[2][32];
    pdl_begin();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= g.L; i += kLoraGroupThreads) count[i] = 0;
    __syncthreads();
    // every warp takes 32 tokens at a time; equal ids are counted by one lane
    const int rounds = (g.N + kLoraGroupThreads - 1) / kLoraGroupThreads;
    for (int r = 0; r < rounds; ++r) {
        const int i = r * kLoraGroupThreads + tid;
        const int id = i < g.N ? lora_id(g, g.ids[i]) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (id >= 0 && (same & ((1u << lane) - 1)) == 0) atomicAdd(count + id, __popc(same));
    }
    __syncthreads();
    const int per = (g.L + 1 + kLoraGroupThreads - 1) / kLoraGroupThreads, l0 = tid * per;
    int sum = 0, tsum = 0;
    for (int l = l0; l < min(l0 + per, g.L + 1); ++l) {
        sum += count[l];
        tsum += (count[l] + TOK - 1) / TOK;
    }
    int incl = sum, tincl = tsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, tincl, o);
        if (lane >= o) incl += u, tincl += v;
    }
    if (lane == 31) warp_sum[0][warp] = incl, warp_sum[1][warp] = tincl;
    __syncthreads();
    int w = warp_sum[0][lane], tw = warp_sum[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o), v = __shfl_up_sync(0xffffffffu, tw, o);
        if (lane >= o) w += u, tw += v;
    }
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0)), tbefore = __shfl_sync(0xffffffffu, tw, max(warp - 1, 0));
    int at = incl - sum + (warp ? before : 0), tile = tincl - tsum + (warp ? tbefore : 0);
    for (int l = l0; l < min(l0 + per, g.L + 1); ++l) {
        const int have = count[l];
        count[l] = at;
        for (int i = 0; i < have; i += TOK) tiles[tile++] = make_int4(l, at + i, min(TOK, have - i), 0);
        at += have;
    }
    if (tid == kLoraGroupThreads - 1) *n_tiles = tile;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
        const int i = r * kLoraGroupThreads + tid;
        const int v = i < g.N ? g.ids[i] : -1;
        const int id = i < g.N ? (v >= 0 && v < g.L ? v : g.L) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        const unsigned below = same & ((1u << lane) - 1);
        int first = 0;
        if (id >= 0 && below == 0) first = atomicAdd(count + id, __popc(same));
        first = __shfl_sync(0xffffffffu, first, __ffs(same) - 1);
        if (id >= 0) order[first + __popc(below)] = i;
    }
}

// A tile's blocks: as many as give each SM one.
int lora_blocks(long long tiles, int sms, int most)
{
    int b = 1;
    while (b < most && tiles * b < sms) b *= 2;
    return b;
}

template <typename K>
twell_status launch_lora(K kern, int clusters, int blocks, size_t smem, cudaStream_t s, const LoraArgs& g)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters) * static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, g) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

// Most blocks a tile whose sums fit an SM.
template <int MT, int RG, int RT>
constexpr int most_blocks()
{
    int b = kLoraCluster;
    while (b > 1 && LoraShape<MT, RG, RT>::bytes(b) > (MT == 4 ? 220u : 110u) * 1024u) b /= 2;
    return b;
}

template <int MT, int RG, int RT, bool SMALL>
twell_status run_lora(const LoraArgs& g, int clusters, int sms, cudaStream_t s)
{
    using S = LoraShape<MT, RG, RT>;
    constexpr int kMost = most_blocks<MT, RG, RT>();
    // the small batches' counts and numbers share the memory of the sums
    constexpr size_t kFind = SMALL ? sizeof(int) * (kLoraMaxAdapters + 1) + sizeof(uint16_t) * kLoraSmallN : 0;
    const int blocks = SMALL ? kMost : lora_blocks(g.N / S::kTok, sms, kMost);
    const size_t find = SMALL ? sizeof(int) * (g.L + 1) + sizeof(uint16_t) * kLoraSmallN : 0;
    auto kern = lora_kernel<MT, RG, RT, SMALL>;
    static std::atomic<uint64_t> allowed{0};
    if (twell_host::allow_smem(kern, std::max(S::bytes(kMost), kFind), allowed) != TWELL_OK) return TWELL_ERR_CUDA;
    return launch_lora(kern, clusters, blocks, std::max(S::bytes(blocks), find), s, g);
}

template <int MT, bool SMALL>
twell_status run_rank(const LoraArgs& g, int clusters, int sms, cudaStream_t s)
{
    if (g.R <= 16) return run_lora<MT, 1, 2, SMALL>(g, clusters, sms, s);
    if (g.R <= 32) return run_lora<MT, 1, 4, SMALL>(g, clusters, sms, s);
    if (g.R <= 64) return run_lora<MT, 2, 4, SMALL>(g, clusters, sms, s);
    return run_lora<MT, 4, 4, SMALL>(g, clusters, sms, s);
}

constexpr int kLoraMT = 4;
// Tiles of N tokens, at most.
long long lora_tiles(int N, int L, int tok) { return std::min<long long>(N, N / tok + std::min(N, L + 1)); }
// The workspace: the number of tiles, the tiles, the tokens' order.
size_t lora_order_at(int N) { return 16 + 16 * static_cast<size_t>(lora_tiles(N, kLoraMaxAdapters, 16 * kLoraMT)); }

}  // namespace
}  // namespace twell

using namespace twell_host;

size_t twell_host::lora_ws_bytes(int N)
{
    if (N <= twell::kLoraSmallN) return 0;
    return (twell::lora_order_at(N) + sizeof(int32_t) * static_cast<size_t>(N) + 15) / 16 * 16;
}

extern "C" twell_status twell_lora_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const twell_adapters* ad,
                                       const int32_t* ids, int32_t N, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                                       int32_t* dev_status, void* stream)
{
    if (ad == nullptr || N < 0 || ad->n_adapters <= 0 || ad->rank <= 0 || ad->k <= 0 || ad->n <= 0 || ad->rank % 8 != 0 ||
        ad->k % 8 != 0 || ad->n % 8 != 0)
        return TWELL_ERR_INVALID;
    if (ad->rank > twell::kLoraMaxRank || ad->n_adapters > twell::kLoraMaxAdapters || N > twell::kLoraMaxTokens ||
        ad->k > twell::kLoraMaxDim || ad->n > twell::kLoraMaxDim)
        return TWELL_ERR_UNSUPPORTED;
    if (N == 0) return TWELL_OK;
    const void* need[] = {y, x, ad->a, ad->b, ad->scale, ids, out, dev_status};
    for (const void* p : need)
        if (p == nullptr) return TWELL_ERR_INVALID;
    const void* rows[] = {y, x, ad->a, ad->b, out};
    for (const void* p : rows)
        if (!aligned16(p)) return TWELL_ERR_INVALID;
    const void* words[] = {ad->scale, ad->ranks, ids};
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) % sizeof(int32_t) != 0) return TWELL_ERR_INVALID;
    if (ldy % 8 != 0 || ldx % 8 != 0 || ldo % 8 != 0 || ldy < ad->n || ldx < ad->k || ldo < ad->n) return TWELL_ERR_INVALID;
    if ((y == out && ldy != ldo) || x == out) return TWELL_ERR_INVALID;
    const size_t need_ws = lora_ws_bytes(N);
    if (need_ws > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < need_ws)) return TWELL_ERR_WORKSPACE;
    using bf = __nv_bfloat16;
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    twell::LoraArgs g = {static_cast<const bf*>(ad->a), static_cast<const bf*>(ad->b), static_cast<const bf*>(x),
                         static_cast<const bf*>(y), static_cast<bf*>(out), ad->scale, ad->ranks, ids, dev_status,
                         ldx, ldy, ldo, ad->n_adapters, ad->rank, ad->k, ad->n, N, nullptr, nullptr, nullptr};
    if (N <= twell::kLoraSmallN)
        return twell::run_rank<twell::kLoraSmallMT, true>(
            g, static_cast<int>(twell::lora_tiles(N, g.L, 16 * twell::kLoraSmallMT)), dev.sm_count, s);
    constexpr int kTok = 16 * twell::kLoraMT;
    int32_t* n_tiles = static_cast<int32_t*>(ws);
    int4* tiles = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + 16);
    int32_t* order = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + twell::lora_order_at(N));
    const twell_status st = launch_dep(twell::lora_group_kernel<kTok>, dim3(1), dim3(twell::kLoraGroupThreads),
                                       sizeof(int) * (g.L + 1), s, g, n_tiles, tiles, order);
    if (st != TWELL_OK) return st;
    g.n_tiles = n_tiles;
    g.tiles = tiles;
    g.order = order;
    return twell::run_rank<twell::kLoraMT, false>(g, static_cast<int>(twell::lora_tiles(N, g.L, kTok)), dev.sm_count, s);
}
