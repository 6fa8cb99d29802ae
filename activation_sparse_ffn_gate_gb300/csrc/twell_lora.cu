// twell_lora.cu -- low-rank adapters of many requests beside a shared projection: to each token's row y the product
// s B (A x) of its own adapter (or of none) is added, A [R, k] and B [n, R] of bf16.
//
// Tokens of one adapter go together in tiles, so that its weights are read once a tile. Both products are mma.sync with the
// tokens as rows; a warp's weights, and its piece of x or y, are its own. Which element of k (or which rank) stands where in a
// fragment is free as long as both operands agree: a lane takes 16 adjacent bytes of a row, and 8 adjacent columns of y. They
// pass through slots of shared memory that belong to the lane, copied there a few pieces ahead, so that no barrier orders
// them. t = A x is summed in fp32 over warps and blocks in one order, and enters the second product as hi + lo bf16: 16 bits
// of it, for twice the products of a small rank.
// What costs a small batch is its chain of loads, what costs a large one its bytes; hence three ways:
// - Few tiles, each of which can have eight SMs: one kernel, a cluster of eight blocks a tile. Each has a part of k, the sums go
//   to all of them through distributed shared memory, and each then has a part of n, whose first pieces are on their way
//   meanwhile. One token, 2048 x 2048, rank 16: 3.5 us, of which the launch is 1.6; the rest is ids, x and A, the
//   exchange, y. One token of rank 64, 2048 x 4096: 5.0 us.
// - Up to 512 tokens else (1024 where the adapters are many): two kernels, whose blocks need not start together as a cluster's do.
//   The second one's blocks request their first copies as soon as they find room: beside two of the first's on an SM up to rank
//   16, where those end above it (at rank 32 the registers are short, at rank 64 the shared memory), and above rank 64 one takes
//   an SM for itself. 64 tokens with 64 adapters of ranks up to 64, 2048 x 4096: 10.1 us (16.1 in clusters; floor
//   3.0); 256 tokens with 64 adapters of rank 16, 2048 x 2048: 6.8 (9.6; floor 1.7).
// - Larger ones: the same two after a kernel that groups the tokens by adapter. 16384 tokens, 2048 x 4096, rank 16: 65 us, of
//   which grouping takes 6, the first product 15 (67 MB) and the second 44 (268 MB, 91% of the copy rate). Above rank 32 the
//   weights that each tile brings from L2 count: rank 64, 2048 x 2048: 61 us for 182 MB. Both products in one kernel, by a
//   block or a cluster a tile, were no faster: 84 us for those 16384 tokens, 22.6 against 23.7 for 3001 of rank 24; nor were rows
//   brought to L2 while the tokens are grouped (68, 24.2).
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
constexpr int kLoraClusterShift = 3, kLoraCluster = 1 << kLoraClusterShift;  // most blocks a tile
// Every block finds its tile from the ids itself up to so many tokens a thread, 32 adjacent ones of a warp at a time: always
// up to kLoraSmallN tokens, up to kLoraFindN where the adapters are many (lora_finds).
constexpr int kLoraFindPer = 2, kLoraFindMore = 4;
constexpr int kLoraSmallN = kLoraFindPer * kLoraThreads, kLoraFindN = kLoraFindMore * kLoraThreads;
// A larger batch's tiles have 32 tokens. With 16 their weights are read twice as often (9000 tokens, 1024 x 3000, rank 128: 99 us
// against 62; 16384 of rank 64, 2048 x 2048: 68 and 61; 3001 of rank 24: 25.2 and 23.3), which between 600 and 2400 tokens can be
// the quicker all the same (1000 of 8 adapters of rank 32: 11.7 and 14.2). With 64 they would be read half as often, but two
// blocks' rings no longer fit an SM.
constexpr int kLoraMT = 2;
// Most blocks of a tile that share its k where each leaves its own sums (325 tokens of few adapters of rank 64, 7312 x 704: 11.7 us,
// 12.5 with four; 256 of 64 adapters of rank 16, 2048 x 2048: 6.8 and 7.3), and of all tiles.
constexpr int kLoraParts = 8;
constexpr int kLoraSums = 1024;
constexpr int kLoraGroupThreads = 1024;
constexpr int kLoraPass = 16384;     // tokens of a larger batch that go together

struct LoraArgs {
    const __nv_bfloat16 *a, *b, *x, *y;
    __nv_bfloat16* out;
    const float* scale;
    const int32_t *ranks, *ids;
    int32_t* status;
    int64_t ldx, ldy, ldo;
    int L, R, k, n, N;
    uint64_t limit_ns;  // of a wait
    // of larger batches: the number of tiles; of each its adapter, first row in t, tokens and rank; and the tokens' numbers, with a
    // place for each token that a tile can have
    const int32_t* n_tiles;
    const int4* tiles;
    const int32_t* order;
};

// Shared memory of a block: of each warp a ring of copies (in which it also leaves its sums), the fragments of t, the blocks'
// sums. A ring's slots are the lane's own: 16 bytes a lane and vector, copied and read by the same lane.
// BOTH: the kernel does both products, else the first alone.
template <int MT, int RG, int RT, bool BOTH>
struct LoraShape {
    static constexpr int kTok = 16 * MT;
    static constexpr int kWays = kLoraWarps / RG;     // warps that share a part of k
    static constexpr int kWarpRanks = RT * 8;
    static constexpr int kRanks = RG * kWarpRanks;
    static constexpr int kPitch = kRanks + 4;         // floats of a token's row in the blocks' sums
    static constexpr int kBlock = RT == 2 ? 16 : 32;  // ranks of which a lane takes a quarter at a time
    static constexpr int kFrags = kRanks / 16;
    static constexpr int kSum = kTok * kPitch;
    static constexpr int kIn = (2 * MT + RT) * 512;                              // a stage of the first product: 32 columns
    static constexpr int kOut = 2 * MT * 512 + 4 * (kRanks / kBlock) * kBlock * 16;  // of the second: 32 columns of y and B's rows
    static constexpr int kWarpSums = kTok * kWarpRanks * 4;
    // room for three stages of the first product at least, and for kMinOut of the second beside the sums: a part of 512 columns
    // is two of them, on their way while t is put together
    static constexpr int kMinOut = RG == 4 ? 1 : 2;
    static constexpr int kRing = BOTH ? (3 * kIn > kWarpSums + kMinOut * kOut ? 3 * kIn : kWarpSums + kMinOut * kOut)
                                      : (MT == 1 && RG == 1 ? 6 : 12) * 1024;
    static constexpr int kInStages = kRing / kIn > 4 ? 4 : kRing / kIn;
    static constexpr int kOutStages = (kRing - kWarpSums) / kOut > 4 ? 4 : (kRing - kWarpSums) / kOut;
    static constexpr int kFragBytes = MT * kFrags * 2 * 512;
    static constexpr size_t bytes(int cluster)
    {
        if (BOTH) return kLoraWarps * kRing + kFragBytes + sizeof(float) * static_cast<size_t>(cluster) * kSum;
        return kLoraWarps * kRing + (cluster > 1 ? sizeof(float) * kTok * kRanks : 0);
    }
    // a warp's sum of (token, rank) in floats: quads of ranks are exchanged between rows, for the banks
    __device__ __forceinline__ static int at(int token, int rank)
    {
        return token * kWarpRanks + (((rank >> 2) ^ (token & (kWarpRanks / 4 - 1))) << 2) + (rank & 3);
    }
};

// Of the second product alone.
template <int MT, int RG, int RT>
struct LoraOutShape {
    using In = LoraShape<MT, RG, RT, false>;
    static constexpr int kRanks = In::kRanks, kBlock = In::kBlock, kFrags = In::kFrags, kStage = In::kOut;
    static constexpr int kRing = (MT == 1 ? (RG == 4 ? 18 : RG == 2 ? 10 : 6) : RT == 2 ? 9 : 12) * 1024;
    static constexpr int kStages = kRing / kStage;
    static constexpr size_t kBytes = kLoraWarps * kRing + In::kFragBytes;
};

// Copies of 16 or 8 bytes of which `bytes` are taken from memory and the rest is zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t at)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at));
    return r;
}

// The two halves of pdl_begin. A kernel that lets the next one start only after its own wait lets that one read, before it waits
// in turn, whatever was there before this kernel. lora_in_kernel and lora_out_kernel are the one such pair, and the exception to
// launch_dep's rule that a kernel begins with pdl_begin: lora_out_kernel reads ids, tiles, y and B before its wait, which is right
// only as long as lora_in_kernel waits first and lets it start then.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
// A store to another block's shared memory, counted on an mbarrier of that block's: whoever waits there for the bytes needs no fence
// from the sender (a cluster barrier behind plain stores was 1 us of a call).
__device__ __forceinline__ void st_counted16(uint32_t at, const float4& v, uint32_t bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(bar)
                 : "memory");
}

// The wait for the other blocks' stores. Whoever gives up records it and stays until they have come all the same (or for kLoraStayNs
// more), since they go on to write to this block's shared memory: from the cluster barrier on, which all have passed, they send
// without a wait of their own. Polls: try_wait may suspend a thread past any limit, and the sums are a microsecond away.
constexpr uint64_t kLoraStayNs = 2000000000ull;
__device__ __forceinline__ bool lora_wait(uint64_t* bar, int32_t* status, uint64_t limit_ns)
{
    bool in_time = true;
    for (const uint64_t t0 = globaltimer_ns();;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar))
            : "memory");
        if (ok) return in_time;
        const uint64_t spent = globaltimer_ns() - t0;
        if (spent <= limit_ns) continue;
        if (in_time) report(status, TWELL_ERR_TIMEOUT);
        in_time = false;
        if (spent - limit_ns > kLoraStayNs) return false;
    }
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

// Lo parts that split2 never gives (two NaNs): t was given up here.
constexpr uint32_t kLoraLost = 0xffffffffu;

// How many rows of adapter `id` count (0 for none, and where that number cannot be, which is recorded).
__device__ __forceinline__ int lora_rank(const LoraArgs& g, int id)
{
    if (id >= g.L) return 0;
    const int rank = g.ranks ? __ldg(g.ranks + id) : g.R;
    if (rank >= 0 && rank <= g.R) return rank;
    report(g.status, TWELL_ERR_DEVICE_CHECK);
    return 0;
}

// Blocks that share a tile, of `blocks` for `tiles` (the host knows only how many tiles there may be), as a power of two:
// divisions here and for the shares were 0.4 of 6.2 us before the first loads.
__device__ __forceinline__ int lora_sharers(int blocks, int tiles, int most)
{
    int s = 0;
    while (2 << s <= most && tiles << (s + 1) <= blocks) ++s;
    return s;
}
// Where block `part` of 2^shift has its share of n.
__device__ __forceinline__ int lora_share(int n, int part, int shift) { return n * part >> shift; }

// A tile of tokens of one adapter.
struct LoraTile {
    int id, rank;    // id -1: there is no such tile
    int first;       // its first row in t
    int tokens;
};

// Tile place(number of tiles) among those of at most PER kLoraThreads tokens: adapters in the order of their first tokens, each
// one's tokens in their own, TOK a tile; everyone who looks for a tile finds the same. Up to 32 tokens every warp does it by
// itself. More are counted by adapter in shared memory, with the least of each one's tokens (sums and minima: in any order the
// same), and the tiles before a token's are a scan over the tokens. Returns the tile's tokens, -1 past the last. `scratch`:
// kLoraFindBytes, free again afterwards.
constexpr size_t kLoraFindBytes = 2 * sizeof(int) * (kLoraMaxAdapters + 1);
template <int TOK, int PER, typename F>
__device__ __forceinline__ const int* lora_find(const LoraArgs& g, F place, void* scratch, LoraTile& tile)
{
    __shared__ int tok[kLoraWarps][TOK];
    __shared__ int found[3];  // adapter, number of the tile's first token, rank
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    tile.id = -1;
    tile.first = 0;
    if (g.N <= 32) {
        const int mine = lane < g.N ? lora_id(g, g.ids[lane]) : -1;
        const int rank = mine >= 0 ? lora_rank(g, mine) : 0;
        const unsigned same = __match_any_sync(0xffffffffu, mine), below = (1u << lane) - 1;
        const int num = __popc(same & below);
        const unsigned firsts = __ballot_sync(0xffffffffu, mine >= 0 && num % TOK == 0);
        const int index = place(__popc(firsts));
        const unsigned it = __ballot_sync(0xffffffffu, (firsts >> lane & 1) && __popc(firsts & below) == index);
        if (lane < TOK) tok[warp][lane] = -1;
        __syncwarp();
        if (it == 0) return nullptr;
        const int from = __ffs(it) - 1, base = __shfl_sync(0xffffffffu, num, from);
        tile.id = __shfl_sync(0xffffffffu, mine, from);
        tile.rank = __shfl_sync(0xffffffffu, rank, from);
        tile.tokens = min(__popc(__shfl_sync(0xffffffffu, same, from)) - base, TOK);
        if (mine == tile.id && num >= base && num < base + TOK) tok[warp][num - base] = lane;
        __syncwarp();
        return tok[warp];
    }
    static_assert(PER * kLoraWarps <= 32, "a warp adds up the totals");
    __shared__ int totals[2][32];              // tiles of each 32 tokens; tokens of the adapter
    int2* bins = static_cast<int2*>(scratch);  // [L + 1]: tokens of an adapter, the first of them
    int own[PER], rank[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) own[j] = j * kLoraThreads + tid < g.N ? __ldg(g.ids + j * kLoraThreads + tid) : 0;
    for (int i = tid; i <= g.L; i += kLoraThreads) bins[i] = make_int2(0, INT32_MAX);
    if (tid == 0) found[0] = -1;
    if (tid < TOK) tok[0][tid] = -1;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * kLoraThreads + tid;
        own[j] = i < g.N ? lora_id(g, own[j]) : -1;
        rank[j] = 0;
        if (j * kLoraThreads >= g.N) continue;
        rank[j] = own[j] >= 0 && own[j] < g.L && g.ranks ? __ldg(g.ranks + own[j]) : g.R;  // on its way while the tiles are counted
        if (i < g.N) {
            atomicAdd(&bins[own[j]].x, 1);
            atomicMin(&bins[own[j]].y, i);
        }
    }
    __syncthreads();
    int tiles[PER], before[PER];  // that begin with this token; before it in its 32
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = j * kLoraThreads + tid;
        tiles[j] = before[j] = 0;
        if (j * kLoraThreads >= g.N) continue;
        if (own[j] >= 0) {
            const int2 bin = bins[own[j]];
            if (bin.y == i) tiles[j] = (bin.x + TOK - 1) / TOK;
        }
        int incl = tiles[j];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        before[j] = incl - tiles[j];
        if (lane == 31) totals[0][j * kLoraWarps + warp] = incl;
    }
    __syncthreads();
    const int index = place(__reduce_add_sync(0xffffffffu, 32 * lane < g.N ? totals[0][lane] : 0));
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (j * kLoraThreads >= g.N) continue;
        const int at = before[j] + __reduce_add_sync(0xffffffffu, lane < j * kLoraWarps + warp ? totals[0][lane] : 0);
        if (index >= at && index < at + tiles[j]) {
            found[0] = own[j];
            found[1] = (index - at) * TOK;
            found[2] = own[j] == g.L ? 0 : rank[j];
        }
    }
    __syncthreads();
    tile.id = found[0];
    if (tile.id < 0) return nullptr;
    tile.tokens = min(bins[tile.id].x - found[1], TOK);
    tile.rank = found[2];
    if (tile.rank < 0 || tile.rank > g.R) {
        report(g.status, TWELL_ERR_DEVICE_CHECK);
        tile.rank = 0;
    }
    unsigned mine[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        mine[j] = __ballot_sync(0xffffffffu, own[j] == tile.id);
        if (lane == 0) totals[1][j * kLoraWarps + warp] = __popc(mine[j]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int num = __popc(mine[j] & ((1u << lane) - 1)) - found[1] +
                        __reduce_add_sync(0xffffffffu, lane < j * kLoraWarps + warp ? totals[1][lane] : 0);
        if (own[j] == tile.id && num >= 0 && num < TOK) tok[0][num] = j * kLoraThreads + tid;
    }
    __syncthreads();
    return tok[0];
}

// Tile place(number of tiles) of a batch, and the tokens of this lane's rows. `known`: of a larger batch, the tile whatever that
// number is, so that it is requested with it.
template <int MT, int FIND, typename F>
__device__ __forceinline__ bool lora_tile(const LoraArgs& g, F place, int known, uint8_t* smem, LoraTile& tile, int (&token)[MT][2])
{
    const int gr = (threadIdx.x & 31) >> 2;
    if constexpr (FIND != 0) {
        const int* tok = lora_find<16 * MT, FIND>(g, place, smem, tile);
        if (tile.id < 0) return false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) token[m][s] = tok[16 * m + 8 * s + gr];
        __syncthreads();  // the memory is free
    } else {
        // requested together: what lies past the last tile is some earlier call's
        const int n = *g.n_tiles, index = known >= 0 ? known : place(n);
        if (known < 0 && index >= n) return false;
        const int4 t = g.tiles[index];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) token[m][s] = g.order[index * 16 * MT + 16 * m + 8 * s + gr];
        if (index >= n) return false;
        tile = LoraTile{t.x, t.w, t.y, t.z};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (16 * m + 8 * s + gr >= tile.tokens) token[m][s] = -1;
    }
    return true;
}

// t = A x over one block's part of k: a warp has kWarpRanks ranks and every kWays-th 64 columns, 32 a stage. Leaves the warps'
// sums in their rings, which are free but for that; `between` runs once a warp's ring is (the copies of what comes next).
template <typename S, int MT, int RG, int RT, typename F>
__device__ __forceinline__ void lora_shrink(const LoraArgs& g, int id, int rank, int part, int shift, const int (&token)[MT][2],
                                            uint8_t* ring_at, F between)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, c = lane & 3;
    const uint32_t mine = smem_u32(ring_at) + lane * 16;
    const int rg = warp % RG, way = warp / RG;
    float acc[MT][RT][4] = {};
    {
        const int kb_all = (g.k + 63) / 64, kb0 = lora_share(kb_all, part, shift) + way, kb1 = lora_share(kb_all, part + 1, shift);
        const int row0 = rg * S::kWarpRanks + gr;
        // a warp whose ranks all lie past the adapter's has nothing to do
        const int stages = rg * S::kWarpRanks < rank && kb0 < kb1 ? (kb1 - kb0 + S::kWays - 1) / S::kWays * 2 : 0;
        // rows' addresses and how many bytes of a row's 16 there are: what a copy costs beside itself is one sum and one mask
        const char* A[RT];
        const char* X[MT][2];
        int a_bytes[RT], x_bytes[MT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const bool live = row0 + 8 * r < rank;
            A[r] = reinterpret_cast<const char*>(live ? g.a + (static_cast<int64_t>(id) * g.R + row0 + 8 * r) * g.k : g.a);
            a_bytes[r] = live ? 16 : 0;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool live = token[m][s] >= 0;
                X[m][s] = reinterpret_cast<const char*>(live ? g.x + token[m][s] * g.ldx : g.x);
                x_bytes[m][s] = live ? 16 : 0;
            }
        auto request = [&](int i, int slot) {
            if (i < stages) {
                const int col = 64 * (kb0 + (i >> 1) * S::kWays) + 32 * (i & 1) + 8 * c, in = col < g.k ? -1 : 0;
                const unsigned off = 2 * col & in;
                const uint32_t at = mine + slot * S::kIn;
#pragma unroll
                for (int r = 0; r < RT; ++r) copy16(at + r * 512, A[r] + off, a_bytes[r] & in);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int s = 0; s < 2; ++s) copy16(at + (RT + 2 * m + s) * 512, X[m][s] + off, x_bytes[m][s] & in);
            }
            copies_end();
        };
#pragma unroll
        for (int i = 0; i < S::kInStages; ++i) request(i, i);
        int slot = 0;
        for (int i = 0; i < stages; ++i) {
            copies_wait<S::kInStages - 1>();
            const uint32_t at = mine + slot * S::kIn;
            uint4 xv[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < 2; ++s) xv[m][s] = lds16(at + (RT + 2 * m + s) * 512);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint4 w = lds16(at + r * 512);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma_bf16(acc[m][r], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, w.x, w.y);
                    mma_bf16(acc[m][r], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, w.z, w.w);
                }
            }
            request(i + S::kInStages, slot);  // all of the slot has been read: the products have taken it
            slot = slot + 1 == S::kInStages ? 0 : slot + 1;
        }
    }
    copies_wait<0>();
    __syncwarp();  // the ring is free: what follows writes where other lanes' slots were
    between();
    float* sums = reinterpret_cast<float*>(ring_at);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            *reinterpret_cast<float2*>(sums + S::at(16 * m + gr, 8 * r + 2 * c)) = make_float2(acc[m][r][0], acc[m][r][1]);
            *reinterpret_cast<float2*>(sums + S::at(16 * m + 8 + gr, 8 * r + 2 * c)) = make_float2(acc[m][r][2], acc[m][r][3]);
        }
}

// The sum over the warps of four ranks of a token, from `smem`, the rings.
template <typename S, int RG>
__device__ __forceinline__ float4 lora_sum(const uint8_t* smem, int row, int quad)
{
    constexpr int kWarpQuads = S::kWarpRanks / 4;
    const float* from = reinterpret_cast<const float*>(smem + quad / kWarpQuads * S::kRing) + S::at(row, quad % kWarpQuads * 4);
    float4 v = *reinterpret_cast<const float4*>(from);
#pragma unroll
    for (int w = 1; w < S::kWays; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(from + w * RG * (S::kRing / 4));
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    return v;
}

// Four ranks of t under the scale, from r0 on: what lies past the rank is a row of zeros times x, NaN where x is infinite, and
// becomes 0. Hi parts in x and y, lo parts in z and w.
__device__ __forceinline__ uint4 lora_parts(const float4& v, int r0, int rank, float scale)
{
    uint4 o;
    split2(r0 < rank ? v.x * scale : 0.0f, r0 + 1 < rank ? v.y * scale : 0.0f, o.x, o.z);
    split2(r0 + 2 < rank ? v.z * scale : 0.0f, r0 + 3 < rank ? v.w * scale : 0.0f, o.y, o.w);
    return o;
}

// y + B t over 32-column pieces nt0, nt0 + 1, ... nt1 - 1 of a block, of which a warp takes every kLoraWarps-th, through STAGES
// slots of its own at `ring_at`.
template <int MT, int RG, int RT>
struct LoraOut {
    using S = LoraOutShape<MT, RG, RT>;
    static constexpr int kKb = S::kRanks / S::kBlock, kPer = S::kBlock / 4;  // ranks a lane takes at a time
    const LoraArgs& g;
    const char *B, *y[MT][2];  // of this lane: its first row of the adapter's, its tokens' rows
    char* out[MT][2];
    int y_bytes[MT][2], b_bytes[kKb];  // that there are of a copy's 16 or 8
    uint32_t mine;
    int rank, first, stages;
    __device__ __forceinline__ LoraOut(const LoraArgs& g, int id, int rank, int nt0, int nt1, const int (&token)[MT][2], const uint8_t* ring_at)
        : g(g), rank(rank)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, c = lane & 3;
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) b_bytes[kb] = 2 * min(max(rank - kb * S::kBlock - kPer * c, 0), kPer);
        B = reinterpret_cast<const char*>(g.b);
        if (b_bytes[0] > 0) B += ((static_cast<int64_t>(id) * g.n + 8 * (gr >> 1) + (gr & 1)) * g.R + kPer * c) * 2;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int t = max(token[m][s], 0);
                y[m][s] = reinterpret_cast<const char*>(g.y + t * g.ldy);
                out[m][s] = reinterpret_cast<char*>(g.out + t * g.ldo);
                y_bytes[m][s] = token[m][s] >= 0 ? 16 : 0;
            }
        mine = smem_u32(ring_at) + lane * 16;
        first = nt0 + 2 * warp;
        const int left = nt1 - first;  // a warp has pieces 0 and 1 of every 2 kLoraWarps
        stages = left > 0 ? (left - 1) / (2 * kLoraWarps) * 2 + min((left - 1) % (2 * kLoraWarps) + 1, 2) : 0;
    }
    __device__ __forceinline__ int column(int i) const { return 32 * (first + (i >> 1) * (2 * kLoraWarps) + (i & 1)); }
    __device__ __forceinline__ void request(int i, int slot) const
    {
        if (i < stages) {
            const int lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
            const int base = column(i), col = base + 8 * c, in = col < g.n ? -1 : 0, rows = base + 8 * (gr >> 1) < g.n ? -1 : 0;
            const unsigned off = 2 * col & in;
            const uint32_t at = mine + slot * S::kStage;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < 2; ++s) copy16(at + (2 * m + s) * 512, y[m][s] + off, y_bytes[m][s] & in);
            const char* from = B + static_cast<int64_t>(base & rows) * g.R * 2;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int kb = 0; kb < kKb; ++kb) {
                    // what lies past the rank becomes zeros, whatever it is
                    const uint32_t to = at + 2 * MT * 512 + (kb * 4 + u) * (kPer * 64);
                    if constexpr (kPer == 8) copy16(to, from + kb * (S::kBlock * 2), b_bytes[kb] & rows);
                    else copy8(to - lane * 8, from + kb * (S::kBlock * 2), b_bytes[kb] & rows);
                }
                from += 4 * g.R;
            }
        }
        copies_end();
    }
    // `frags`: t, [row tile][16 ranks][hi, lo][lane]
    template <int STAGES>
    __device__ __forceinline__ void run(const uint4* frags) const
    {
        const int lane = threadIdx.x & 31, c = lane & 3;
        int slot = 0;
        for (int i = 0; i < stages; ++i) {
            copies_wait<STAGES - 1>();
            const uint32_t at = mine + slot * S::kStage;
            const int col = column(i) + 8 * c;
            float d[MT][4][4] = {};
#pragma unroll
            for (int kb = 0; kb < kKb; ++kb) {
                if (kb * S::kBlock >= rank) break;
                uint4 bw[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t from = at + 2 * MT * 512 + (kb * 4 + u) * (kPer * 64);
                    if constexpr (kPer == 8) {
                        bw[u] = lds16(from);
                    } else {
                        const uint2 v = lds8(from - lane * 8);
                        bw[u] = make_uint4(v.x, v.y, 0u, 0u);
                    }
                }
#pragma unroll
                for (int h = 0; h < S::kBlock / 16; ++h)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const uint4 a = frags[((m * S::kFrags + kb * (S::kBlock / 16) + h) * 2 + p) * 32 + lane];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mma_bf16(d[m][u], a.x, a.y, a.z, a.w, h ? bw[u].z : bw[u].x, h ? bw[u].w : bw[u].y);
                        }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    uint4 y = lds16(at + (2 * m + s) * 512);
                    if (rank > 0) {
                        float v[8];
                        unpack16(y, v, static_cast<__nv_bfloat16*>(nullptr));
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            v[2 * u] += d[m][u][2 * s];
                            v[2 * u + 1] += d[m][u][2 * s + 1];
                        }
                        y = pack16(v, static_cast<__nv_bfloat16*>(nullptr));
                    }
                    if (col < g.n && y_bytes[m][s] > 0) *reinterpret_cast<uint4*>(out[m][s] + 2 * col) = y;
                }
            request(i + STAGES, slot);
            slot = slot + 1 == STAGES ? 0 : slot + 1;
        }
        copies_wait<0>();
    }
};

// A batch of few tiles, whole.
template <int MT, int RG, int RT>
__global__ void __launch_bounds__(kLoraThreads, 1) lora_kernel(const LoraArgs g)
{
    using S = LoraShape<MT, RG, RT, true>;
    extern __shared__ __align__(128) uint8_t lora_smem[];  // a warp's 512 bytes a vector begin on a 128-byte line
    pdl_begin();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5, gr = lane >> 2;
    constexpr int blocks = kLoraCluster, shift = kLoraClusterShift;
    const int part = static_cast<int>(cluster_ctarank());
    LoraTile tile;
    const int* tok = lora_find<S::kTok, kLoraFindPer>(g, [&](int) { return static_cast<int>(blockIdx.x) / blocks; }, lora_smem, tile);  // where the rings come later
    if (tile.id < 0) return;
    const int id = tile.id, rank = tile.rank;
    const int nt_all = (g.n + 31) / 32, nt0 = lora_share(nt_all, part, shift), nt1 = lora_share(nt_all, part + 1, shift);
    if (rank == 0) {  // the same for all blocks of the cluster
        if (g.y == g.out) return;
        const int col0 = nt0 * 4, cols = min(nt1 * 4, g.n / 8) - col0;  // in chunks of 8
        for (int i = tid; i < tile.tokens * cols; i += kLoraThreads) {
            const int t = tok[i / cols], col = (col0 + i % cols) * 8;
            *reinterpret_cast<uint4*>(g.out + t * g.ldo + col) = *reinterpret_cast<const uint4*>(g.y + t * g.ldy + col);
        }
        return;
    }
    constexpr int kQuads = S::kRanks / 4;
    __shared__ uint64_t bar;
    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&bar, static_cast<uint32_t>(blocks * tile.tokens * kQuads * 16));
    }
    cluster_arrive();  // this block runs and its barrier counts: the others may write to its shared memory

    int token[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < 2; ++s) token[m][s] = tok[16 * m + 8 * s + gr];
    uint8_t* const ring_at = lora_smem + warp * S::kRing;

    // the first pieces of the second product are on their way while t is put together
    const LoraOut<MT, RG, RT> out(g, id, rank, nt0, nt1, token, ring_at + S::kWarpSums);
    const float scale = __ldg(g.scale + id);
    lora_shrink<S, MT, RG, RT>(g, id, rank, part, shift, token, ring_at, [&] {
#pragma unroll
        for (int i = 0; i < S::kOutStages; ++i) out.request(i, i);
    });
    __syncthreads();
    cluster_wait();
    uint4* frags = reinterpret_cast<uint4*>(lora_smem + kLoraWarps * S::kRing);
    float* recv = reinterpret_cast<float*>(lora_smem + kLoraWarps * S::kRing + S::kFragBytes);
    for (int i = tid; i < tile.tokens * kQuads; i += kLoraThreads) {
        const int row = i / kQuads, quad = i % kQuads;
        const float4 v = lora_sum<S, RG>(lora_smem, row, quad);
        const uint32_t to = smem_u32(recv + part * S::kSum + row * S::kPitch + quad * 4);
#pragma unroll
        for (int d = 0; d < blocks; ++d) st_counted16(mapa_shared(to, d), v, mapa_shared(smem_u32(&bar), d));
    }
    const bool all = lora_wait(&bar, g.status, g.limit_ns);
    if (__syncthreads_or(!all)) {  // recorded
        copies_wait<0>();
        return;
    }
    // t, whole, under its scale, as the second product's fragments: [row tile][16 ranks][hi, lo][lane]
    for (int i = tid; i < MT * S::kFrags * 32; i += kLoraThreads) {
        const int l = i & 31, f = (i >> 5) % S::kFrags, m = (i >> 5) / S::kFrags;
        constexpr int kHalves = S::kBlock / 16;
        const int r0 = f / kHalves * S::kBlock + S::kBlock / 4 * (l & 3) + 4 * (f % kHalves);
        const float* p = recv + (16 * m + (l >> 2)) * S::kPitch + r0;
        uint4 t[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            // of a row without a token nothing was sent: what it holds stays in it
            float4 v = *reinterpret_cast<const float4*>(p + s * 8 * S::kPitch);
#pragma unroll
            for (int d = 1; d < blocks; ++d) {
                const float4 u = *reinterpret_cast<const float4*>(p + d * S::kSum + s * 8 * S::kPitch);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            t[s] = lora_parts(v, r0, rank, scale);
        }
        frags[((m * S::kFrags + f) * 2 + 0) * 32 + l] = make_uint4(t[0].x, t[1].x, t[0].y, t[1].y);
        frags[((m * S::kFrags + f) * 2 + 1) * 32 + l] = make_uint4(t[0].z, t[1].z, t[0].w, t[1].w);
    }
    __syncthreads();
    out.template run<S::kOutStages>(frags);
}

// t of a batch: a tile's rows of it, as lora_parts has them. A cluster of blocks shares a tile's k where tiles are few; each then
// adds up a share of the sums. With FIND each block of a tile leaves its own sums, [tile][part][token][rank], for the second
// product to add up: its blocks need not start together.
template <int MT, int RG, int RT, int FIND>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_in_kernel(const LoraArgs g, uint4* __restrict__ t_out)
{
    using S = LoraShape<MT, RG, RT, false>;
    extern __shared__ __align__(128) uint8_t lora_smem[];  // a warp's 512 bytes a vector begin on a 128-byte line
    pdl_wait();  // in this order: lora_out_kernel reads what the kernels before this one wrote without a wait for them
    pdl_next();
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5;
    int shift, blocks, index, part;  // of a cluster: the rank
    auto take = [&](int s) {
        shift = s, blocks = 1 << s, index = static_cast<int>(blockIdx.x) >> s, part = static_cast<int>(blockIdx.x) & (blocks - 1);
        return index;
    };
    if constexpr (FIND == 0) take(31 - __clz(static_cast<int>(cluster_blocks())));
    else index = -1;
    auto place = [&](int tiles) { return take(lora_sharers(static_cast<int>(gridDim.x), tiles, kLoraParts)); };
    int token[MT][2];
    LoraTile tile;
    if (!lora_tile<MT, FIND>(g, place, index, lora_smem, tile, token)) return;
    const int rank = tile.rank;
    if (rank == 0) return;
    constexpr int kQuads = S::kRanks / 4;
    const int quads = tile.tokens * kQuads;  // quad i is added up by block i % blocks
    __shared__ uint64_t bar;
    if (FIND == 0 && blocks > 1) {
        if (tid == 0) {
            mbar_init(&bar, 1);
            fence_mbar_init();
            mbar_arrive_expect_tx(&bar, static_cast<uint32_t>(blocks * ((quads + blocks - 1 - part) / blocks) * 16));
        }
        cluster_arrive();  // this block runs and its barrier counts
    }
    const float scale = __ldg(g.scale + tile.id);
    lora_shrink<S, MT, RG, RT>(g, tile.id, rank, part, shift, token, lora_smem + warp * S::kRing, [] {});
    __syncthreads();
    if constexpr (FIND != 0) {
        float4* to = reinterpret_cast<float4*>(t_out) + (static_cast<size_t>(index) * blocks + part) * (S::kTok * kQuads);
        for (int i = tid; i < quads; i += kLoraThreads) to[i] = lora_sum<S, RG>(lora_smem, i / kQuads, i % kQuads);
        return;
    }
    auto store = [&](int i, const float4& v) { t_out[static_cast<size_t>(tile.first) * kQuads + i] = lora_parts(v, i % kQuads * 4, rank, scale); };
    if (blocks == 1) {
        for (int i = tid; i < quads; i += kLoraThreads) store(i, lora_sum<S, RG>(lora_smem, i / kQuads, i % kQuads));
        return;
    }
    float4* recv = reinterpret_cast<float4*>(lora_smem + kLoraWarps * S::kRing);
    const int share = S::kTok * kQuads / blocks;
    cluster_wait();
    for (int i = tid; i < quads; i += kLoraThreads)
        st_counted16(mapa_shared(smem_u32(recv + part * share + i / blocks), i % blocks), lora_sum<S, RG>(lora_smem, i / kQuads, i % kQuads),
                     mapa_shared(smem_u32(&bar), i % blocks));
    const bool in_time = lora_wait(&bar, g.status, g.limit_ns);
    for (int i = part + tid * blocks; i < quads; i += kLoraThreads * blocks) {
        if (!in_time) {  // recorded; the second product leaves the tile's rows as they are
            t_out[static_cast<size_t>(tile.first) * kQuads + i].z = kLoraLost;
            continue;
        }
        float4 v = recv[i / blocks];
        for (int d = 1; d < blocks; ++d) {
            const float4 u = recv[d * share + i / blocks];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        store(i, v);
    }
}

// y + B t of a batch: a block has a tile's rows and a part of the columns, of which a warp takes every kLoraWarps-th 32. What it
// reads but t was there before the first product's kernel, which lets this one start after its own wait: the first pieces
// are on their way while that one runs. `most_parts`: of a tile's columns, by the number of tiles; 0: one of gridDim.x / most_tiles,
// whatever that number is. `in_blocks`: of the first product, with FIND.
template <int MT, int RG, int RT, int FIND>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_out_kernel(const LoraArgs g, const uint4* t_in, int most_tiles, int most_parts, int in_blocks)
{
    using S = LoraOutShape<MT, RG, RT>;
    extern __shared__ __align__(128) uint8_t lora_smem[];  // a warp's 512 bytes a vector begin on a 128-byte line
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5;
    int index = -1, in_parts = 1;
    unsigned parts = 1, part = 0;
    auto place = [&](int tiles) {
        if (FIND != 0) in_parts = 1 << lora_sharers(in_blocks, tiles, kLoraParts);
        if (most_parts == 0) return index;
        parts = max(1u, min(static_cast<unsigned>(most_parts), gridDim.x / max(tiles, 1)));
        part = blockIdx.x % parts;
        return index = static_cast<int>(blockIdx.x / parts);
    };
    if (most_parts == 0) {
        parts = gridDim.x / static_cast<unsigned>(most_tiles);
        part = blockIdx.x % parts;
        index = static_cast<int>(blockIdx.x / parts);
    }
    int token[MT][2];
    LoraTile tile;
    const bool is = lora_tile<MT, FIND>(g, place, index, lora_smem, tile, token);
    if (!is || (tile.rank == 0 && g.y == g.out)) {
        if (blockIdx.x == 0) pdl_wait();  // one block is enough for the grid not to be done before the one before it
        return;
    }
    const int rank = tile.rank;
    const unsigned nt_all = (g.n + 31) / 32;
    const int nt0 = static_cast<int>(nt_all * part / parts), nt1 = static_cast<int>(nt_all * (part + 1) / parts);
    const LoraOut<MT, RG, RT> out(g, tile.id, rank, nt0, nt1, token, lora_smem + warp * S::kRing);
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) out.request(i, i);
    const float scale = FIND != 0 && rank > 0 ? __ldg(g.scale + tile.id) : 0.0f;
    pdl_wait();
    pdl_next();
    bool lost = false;
    // t as the product's fragments
    uint4* frags = reinterpret_cast<uint4*>(lora_smem + kLoraWarps * S::kRing);
    constexpr int kQuads = S::kRanks / 4;
    if (rank > 0)
        for (int i = tid; i < MT * S::kFrags * 32; i += kLoraThreads) {
            const int l = i & 31, f = (i >> 5) % S::kFrags, m = (i >> 5) / S::kFrags;
            constexpr int kHalves = S::kBlock / 16, kPer = S::kBlock / 4;
            const int quad = (f / kHalves * S::kBlock + kPer * (l & 3)) / 4 + f % kHalves, row = 16 * m + (l >> 2);
            uint4 t[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                t[s] = make_uint4(0u, 0u, 0u, 0u);
                if (row + 8 * s >= tile.tokens) continue;
                if constexpr (FIND != 0) {
                    const float4* from = reinterpret_cast<const float4*>(t_in) + static_cast<size_t>(index) * in_parts * (16 * MT * kQuads) +
                                         (row + 8 * s) * kQuads + quad;
                    float4 u[kLoraParts];
#pragma unroll
                    for (int p = 0; p < kLoraParts; ++p)
                        if (p < in_parts) u[p] = __ldcg(from + p * (16 * MT * kQuads));
#pragma unroll
                    for (int p = 1; p < kLoraParts; ++p)
                        if (p < in_parts) u[0].x += u[p].x, u[0].y += u[p].y, u[0].z += u[p].z, u[0].w += u[p].w;
                    t[s] = lora_parts(u[0], 4 * quad, rank, scale);
                } else {
                    t[s] = __ldcg(t_in + static_cast<size_t>(tile.first + row + 8 * s) * kQuads + quad);
                    lost |= t[s].z == kLoraLost;
                }
            }
            frags[((m * S::kFrags + f) * 2 + 0) * 32 + l] = make_uint4(t[0].x, t[1].x, t[0].y, t[1].y);
            frags[((m * S::kFrags + f) * 2 + 1) * 32 + l] = make_uint4(t[0].z, t[1].z, t[0].w, t[1].w);
        }
    if constexpr (FIND == 0) {
        if (__syncthreads_or(lost)) {
            copies_wait<0>();
            return;
        }
    } else {
        __syncthreads();
    }
    out.template run<S::kStages>(frags);
}

// The tiles of a larger batch: tokens counted by adapter, a tile for each 16 kLoraMT of an adapter's, and
// their places in it in `order`. One block: the counts are in its shared memory, and a pass's ids are 64 KB, all requested before the
// first is counted. Which token of an adapter comes first is left to chance; a token's result does not depend on it.
__global__ void __launch_bounds__(kLoraGroupThreads) lora_group_kernel(const LoraArgs g, int32_t* n_tiles, int4* tiles, int32_t* order)
{
    constexpr int kTok = 16 * kLoraMT;                   // tokens a tile
    constexpr int kPer = kLoraPass / kLoraGroupThreads;  // tokens a thread
    extern __shared__ int count[];                       // [L + 1] of tokens, then their first place; [L + 1] of the first tiles
    __shared__ int warp_sum[2][32], s_tiles;
    pdl_begin();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int* first_tile = count + g.L + 1;
    int v[kPer];
#pragma unroll
    for (int r = 0; r < kPer; ++r) v[r] = r * kLoraGroupThreads + tid < g.N ? __ldg(g.ids + r * kLoraGroupThreads + tid) : INT32_MIN;
    for (int i = tid; i <= g.L; i += kLoraGroupThreads) count[i] = 0;
    __syncthreads();
    // a token's number among those of its adapter; a warp whose tokens have one adapter (most of a prompt's) counts them at once
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        if (r * kLoraGroupThreads >= g.N) break;
        const bool live = r * kLoraGroupThreads + tid < g.N;
        const int id = live ? lora_id(g, v[r]) : -1;
        const int first = __shfl_sync(0xffffffffu, id, 0);  // by all lanes, whatever they have
        const bool one = __all_sync(0xffffffffu, live && id == first);
        int num = 0;
        if (one) {
            if (lane == 0) num = atomicAdd(count + id, 32);
            num = __shfl_sync(0xffffffffu, num, 0) + lane;
        } else if (live) {
            num = atomicAdd(count + id, 1);
        }
        v[r] = live ? (id << 16) | num : -1;  // at most 4096 adapters and 2^15 tokens
    }
    __syncthreads();
    const int per = (g.L + kLoraGroupThreads) / kLoraGroupThreads, l0 = tid * per, l1 = min(l0 + per, g.L + 1);
    int sum = 0, tsum = 0;
    for (int l = l0; l < l1; ++l) {
        sum += count[l];
        tsum += (count[l] + kTok - 1) / kTok;
    }
    int incl = sum, tincl = tsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o), w = __shfl_up_sync(0xffffffffu, tincl, o);
        if (lane >= o) incl += u, tincl += w;
    }
    if (lane == 31) warp_sum[0][warp] = incl, warp_sum[1][warp] = tincl;
    __syncthreads();
    int w = warp_sum[0][lane], tw = warp_sum[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o), x = __shfl_up_sync(0xffffffffu, tw, o);
        if (lane >= o) w += u, tw += x;
    }
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0)), tbefore = __shfl_sync(0xffffffffu, tw, max(warp - 1, 0));
    int at = incl - sum + (warp ? before : 0), tile = tincl - tsum + (warp ? tbefore : 0);
    for (int l = l0; l < l1; ++l) {
        const int have = count[l];
        count[l] = at;
        first_tile[l] = tile;
        at += have;
        tile += (have + kTok - 1) / kTok;
    }
    if (tid == kLoraGroupThreads - 1) *n_tiles = s_tiles = tile;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        if (r * kLoraGroupThreads >= g.N) break;
        if (v[r] >= 0) {
            const int l = v[r] >> 16, num = v[r] & 0xffff;
            order[(first_tile[l] + num / kTok) * kTok + num % kTok] = r * kLoraGroupThreads + tid;
        }
    }
    for (int j = tid; j < s_tiles; j += kLoraGroupThreads) {
        int l = 0, len = g.L + 1;  // the last adapter whose tiles begin at j or before
        while (len > 1) {
            const int half = len >> 1;
            if (first_tile[l + half] <= j) l += half;
            len -= half;
        }
        const int from = count[l] + (j - first_tile[l]) * kTok;
        tiles[j] = make_int4(l, from, min(kTok, (l < g.L ? count[l + 1] : g.N) - from), lora_rank(g, l));
    }
}

// A tile's blocks in a cluster: as many as give each SM one (3001 tokens, 2560 x 2568: 23.3 us with two, 24.5 with one,
// 26.9 with four).
int lora_blocks(long long tiles, int sms)
{
    int b = 1;
    while (b < kLoraCluster && tiles * b < sms) b *= 2;
    return b;
}

template <typename... KArgs, typename... Args>
twell_status launch_lora(void (*kern)(KArgs...), int clusters, int blocks, size_t smem, cudaStream_t s, Args... args)
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
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

// Tiles of N tokens, at most.
long long lora_tiles(int N, int L, int tok) { return std::min<long long>(N, N / tok + std::min(N, L + 1)); }

constexpr int lora_ranks(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// Blocks of the first product where each leaves its own sums: as far as two an SM go (256 tokens with 64 adapters of rank 16, 2048 x
// 2048: 6.8 us, 8.3 with a second round of blocks; 300 of rank 64: 11.7 and 14.8).
int lora_in_blocks(int tiles, int sms) { return std::max(tiles, std::min(std::min(kLoraParts * tiles, 2 * sms), kLoraSums)); }

// Whether every block finds its tile itself. Beyond kLoraSmallN tokens its tiles of 16 can cost more weights than the grouping saves,
// unless the adapters are so many that tiles of 32 would be half empty (1000 tokens, 64 adapters of rank 16, 2048 x 2048: 10.4 us and
// 14.3 grouped; 1000 of 64 adapters of rank 64, 2048 x 4096: 21.2 and 28.5; 846 of 8 adapters of rank 128, 2048 x 2048: 21.5 and
// 19.7).
bool lora_finds(int N, int L) { return N <= kLoraSmallN || (N <= kLoraFindN && L >= N / 32); }

// What the workspace holds of a pass: the tiles and their tokens where they are grouped, and t; else the blocks' sums.
struct LoraWs {
    size_t tiles, order, t, total;
    LoraWs(int N, int R)
    {
        const int n = std::min(N, kLoraPass), tok = 16 * kLoraMT;
        const size_t most = static_cast<size_t>(lora_tiles(n, kLoraMaxAdapters, tok)), row = lora_ranks(R) * sizeof(float);
        tiles = 16;
        order = tiles + 16 * most;
        t = order + sizeof(int32_t) * tok * most;
        total = std::max(N > kLoraSmallN ? t + n * row : 0, N <= kLoraFindN ? 16 * kLoraSums * row : 0);
    }
};

// The two products of a batch whose tiles are found (by FIND, or in g).
template <int MT, int RG, int RT, int FIND>
twell_status run_products(const LoraArgs& g, uint4* t, int sms, cudaStream_t s)
{
    using S = LoraShape<MT, RG, RT, false>;
    using O = LoraOutShape<MT, RG, RT>;
    static_assert(!FIND || (kLoraFindBytes <= kLoraWarps * S::kRing && kLoraFindBytes <= kLoraWarps * O::kRing), "room to find a tile");
    const int most = static_cast<int>(lora_tiles(g.N, g.L, S::kTok));
    static_assert(2 * S::bytes(kLoraCluster) <= 226 * 1024, "two blocks an SM");
    auto in = lora_in_kernel<MT, RG, RT, FIND>;
    auto out = lora_out_kernel<MT, RG, RT, FIND>;
    static std::atomic<uint64_t> in_allowed{0}, out_allowed{0};
    if (twell_host::allow_smem(in, S::bytes(kLoraCluster), in_allowed) != TWELL_OK || twell_host::allow_smem(out, O::kBytes, out_allowed) != TWELL_OK)
        return TWELL_ERR_CUDA;
    // a block's part of the columns: two pieces a warp at least, and one round of two blocks an SM (tiles of 16 above rank 64 leave
    // room for one, 152 KB), or kOutRounds where the tiles alone are more
    constexpr int kOutRounds = 2;
    const long long places = 2ll * sms, most_parts = ((g.n + 31) / 32 + 2 * kLoraWarps - 1) / (2 * kLoraWarps);
    const int about = std::max(1, g.N / S::kTok);
    const bool one = most <= places;
    const long long out_blocks = one ? std::min(places, most * most_parts) : most * std::min((kOutRounds * places + about - 1) / about, most_parts);
    if (out_blocks > INT32_MAX) return TWELL_ERR_UNSUPPORTED;
    const dim3 out_grid(static_cast<unsigned>(out_blocks)), threads(kLoraThreads);
    const int by_tiles = one ? static_cast<int>(most_parts) : 0;
    if constexpr (FIND != 0) {
        const int in_blocks = lora_in_blocks(most, sms);
        const twell_status st = twell_host::launch_dep(in, dim3(static_cast<unsigned>(in_blocks)), threads, S::bytes(1), s, g, t);
        if (st != TWELL_OK) return st;
        return twell_host::launch_dep(out, out_grid, threads, O::kBytes, s, g, t, most, by_tiles, in_blocks);
    } else {
        const int blocks = lora_blocks(about, sms);
        const twell_status st = launch_lora(in, most, blocks, S::bytes(blocks), s, g, t);
        if (st != TWELL_OK) return st;
        return twell_host::launch_dep(out, out_grid, threads, O::kBytes, s, g, t, most, by_tiles, 0);
    }
}

// A batch whose blocks find their tiles: where the device holds all tiles' clusters at once, in one kernel; else in two, whose blocks need not
// start together.
template <int RG, int RT>
twell_status run_small(const LoraArgs& g, uint8_t* ws, int sms, cudaStream_t s)
{
    uint4* sums = reinterpret_cast<uint4*>(ws);
    if (g.N > kLoraSmallN) return run_products<1, RG, RT, kLoraFindMore>(g, sums, sms, s);
    using S = LoraShape<1, RG, RT, true>;
    static_assert(kLoraFindBytes <= kLoraWarps * S::kRing, "room to find a tile");
    static_assert(S::bytes(kLoraCluster) <= 224 * 1024, "a block's shared memory");
    const int tiles = static_cast<int>(lora_tiles(g.N, g.L, S::kTok));
    // (up to rank 32 two of its blocks share an SM: 30 tiles of rank 16, 2048 x 2048: 4.6 us and 5.0 in two kernels; 18 of rank 64, 2048
    // x 4096: 5.5 and 6.6; 30 of them: 10.0 and 7.0)
    if (tiles * kLoraCluster > (RG == 1 ? 2 : 1) * sms) return run_products<1, RG, RT, kLoraFindPer>(g, sums, sms, s);
    auto kern = lora_kernel<1, RG, RT>;
    static std::atomic<uint64_t> allowed{0};
    if (twell_host::allow_smem(kern, S::bytes(kLoraCluster), allowed) != TWELL_OK) return TWELL_ERR_CUDA;
    return launch_lora(kern, tiles, kLoraCluster, S::bytes(kLoraCluster), s, g);
}

template <int RG, int RT>
twell_status run_pass(LoraArgs g, uint8_t* ws, const LoraWs& at, int sms, cudaStream_t s)
{
    int32_t* n_tiles = reinterpret_cast<int32_t*>(ws);
    int4* tiles = reinterpret_cast<int4*>(ws + at.tiles);
    int32_t* order = reinterpret_cast<int32_t*>(ws + at.order);
    const twell_status st = twell_host::launch_dep(lora_group_kernel, dim3(1), dim3(kLoraGroupThreads), 2 * sizeof(int) * (g.L + 1), s, g,
                                                   n_tiles, tiles, order);
    if (st != TWELL_OK) return st;
    g.n_tiles = n_tiles;
    g.tiles = tiles;
    g.order = order;
    return run_products<kLoraMT, RG, RT, 0>(g, reinterpret_cast<uint4*>(ws + at.t), sms, s);
}

}  // namespace
}  // namespace twell

using namespace twell_host;

size_t twell_host::lora_ws_bytes(int N, int R)
{
    return N == 0 || R > twell::kLoraMaxRank ? 0 : twell::LoraWs(N, R).total;
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
    const size_t need_ws = lora_ws_bytes(N, ad->rank);
    if (need_ws > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < need_ws)) return TWELL_ERR_WORKSPACE;
    using bf = __nv_bfloat16;
    DevInfo dev;
    if (dev_info(&dev) != TWELL_OK) return TWELL_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    twell::LoraArgs g = {static_cast<const bf*>(ad->a), static_cast<const bf*>(ad->b), static_cast<const bf*>(x),
                         static_cast<const bf*>(y), static_cast<bf*>(out), ad->scale, ad->ranks, ids, dev_status,
                         ldx, ldy, ldo, ad->n_adapters, ad->rank, ad->k, ad->n, N, wait_limit_ns(), nullptr, nullptr, nullptr};
    uint8_t* w = static_cast<uint8_t*>(ws);
    if (twell::lora_finds(N, ad->n_adapters))
        return ad->rank <= 16   ? twell::run_small<1, 2>(g, w, dev.sm_count, s)
               : ad->rank <= 32 ? twell::run_small<1, 4>(g, w, dev.sm_count, s)
               : ad->rank <= 64 ? twell::run_small<2, 4>(g, w, dev.sm_count, s)
                                : twell::run_small<4, 4>(g, w, dev.sm_count, s);
    const twell::LoraWs at(N, ad->rank);
    for (int from = 0; from < N; from += twell::kLoraPass) {
        twell::LoraArgs p = g;
        p.N = N - from < twell::kLoraPass ? N - from : twell::kLoraPass;
        p.ids += from;
        p.x += from * ldx;
        p.y += from * ldy;
        p.out += from * ldo;
        const twell_status st = ad->rank <= 16   ? twell::run_pass<1, 2>(p, w, at, dev.sm_count, s)
                                : ad->rank <= 32 ? twell::run_pass<1, 4>(p, w, at, dev.sm_count, s)
                                : ad->rank <= 64 ? twell::run_pass<2, 4>(p, w, at, dev.sm_count, s)
                                                 : twell::run_pass<4, 4>(p, w, at, dev.sm_count, s);
        if (st != TWELL_OK) return st;
    }
    return TWELL_OK;
}
