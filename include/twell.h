/*
 * twell.h -- C ABI of the GB300 (sm_103a) activation-sparse gated FFN library (libtwell_gb300.so).
 *
 * The layer is  y = (ReLU(x Wg) * (x Wu)) Wd  with the gate activation kept in the tile-wise
 * ELL (TwELL) format. Passages that define each operation are cited by page title and section:
 *   [AIM] aimodeling.com news item "TwELL：Sakana AI与NVIDIA联合提出稀疏LLM推理加速20%，解决GPU批处理落地难题",
 *         summary paragraph n (¶n).
 *   [TG]  Telegram post "Sakana AI и NVIDIA представили TwELL ..." (ai_machinelearning_big_data),
 *         sections "Вот тут и решает TwELL", "Инференс", "Обучение".
 *   [PUL] pulsen.vercel.app "Sakana AI og NVIDIA introduserer TwELL ...", paragraph n.
 *   [TC]  Tencent Cloud "一文读懂 NVIDIA 与 Sakana AI 联手打造的稀疏 LLM 黑科技", sections 1-6.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Shapes: N tokens, d = d_model, f = d_ff, T = TwELL tile width, nt = ceil(f / T),
 *   K = hybrid per-row capacity.
 * - Weights are stored one row per hidden unit ("rows of Wu and Wd", [TG] "Инференс"):
 *   Wg_s = Wg^T, Wu_s = Wu^T and Wd_s = Wd are all [f, d] row-major. x, y, dy, dx are [N, d]
 *   row-major. So G = x Wg_s^T, U = x Wu_s^T, y = (ReLU(G) * U) Wd_s.
 * - Every pointer argument named as device memory must be device memory allocated by the
 *   caller; the library never allocates, never frees and keeps no pointer after a call returns.
 *   Struct arguments (twell_packed, twell_hybrid) are host structs that hold device pointers.
 * - Every call is asynchronous on `stream` (a cudaStream_t passed as void*; NULL = the legacy
 *   default stream). Outputs are valid once the stream reaches the call.
 * - Alignment: every device pointer must be 16-byte aligned; d must be a multiple of 8.
 * - Element type: TWELL_BF16 (bf16 storage, fp32 accumulation, tcgen05 tensor cores for the
 *   gate) or TWELL_F32 (fp32 storage and arithmetic on CUDA cores; small layers and tests).
 * - Errors: argument errors are detected on the host and returned before anything is launched
 *   (nothing is written). Conditions found on the device (a bounded wait that ran out, a
 *   failed device-side check, a full backup buffer) are written to *dev_status (one int32 in
 *   device memory, first error wins, never cleared by the library) as a twell_status code; read
 *   it with twell_read_status(). Launch failures return TWELL_ERR_CUDA.
 */
#ifndef TWELL_GB300_H
#define TWELL_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define TWELL_API __attribute__((visibility("default")))
#else
#define TWELL_API
#endif

typedef enum {
    TWELL_OK = 0,
    TWELL_ERR_INVALID = 1,     /* bad argument (null pointer, size, alignment, mismatch) */
    TWELL_ERR_UNSUPPORTED = 2, /* valid but not supported here (dtype, tile width, device) */
    TWELL_ERR_BACKUP_FULL = 3, /* hybrid: more overflow rows than backup_cap (device-reported) */
    TWELL_ERR_TIMEOUT = 4,     /* a bounded device-side wait ran out (device-reported) */
    TWELL_ERR_DEVICE_CHECK = 5,/* a device-side consistency check failed (device-reported) */
    TWELL_ERR_CUDA = 6,        /* a CUDA runtime call or kernel launch failed */
    TWELL_ERR_WORKSPACE = 7,   /* workspace missing or smaller than twell_workspace_bytes() */
    TWELL_ERR_POOL_EMPTY = 8   /* twell_kv_plan: fewer free pages than the step's tokens need (device-reported) */
} twell_status;

/* TWELL_E4M3 (8 bits, largest value 448) is an element type of the key-value cache only. */
typedef enum { TWELL_BF16 = 0, TWELL_F32 = 1, TWELL_E4M3 = 2 } twell_dtype;

typedef enum {
    TWELL_OP_GATE_PACK = 0,
    TWELL_OP_FFN_FUSED_FWD = 1,
    TWELL_OP_HYBRID_FWD = 2,
    TWELL_OP_HYBRID_BWD = 3,
    TWELL_OP_HYBRID_ROUTE = 4,
    TWELL_OP_FFN_UNION_FWD = 5,
    TWELL_OP_FFN_DECODE = 6,
    TWELL_OP_FFN_TILE_UNION_FWD = 7,
    TWELL_OP_FFN_GATE_UNION_FWD = 8,
    TWELL_OP_ADD_RMSNORM_BWD = 9, /* N rows of d columns; the other arguments are not used */
    TWELL_OP_PAGED_ATTN = 10,     /* N sequences, d = head_dim; the other arguments are not used */
    TWELL_OP_LORA_ADD = 11        /* N tokens, d = rank; the other arguments are not used */
} twell_op;

/* A TwELL matrix of gate activations a = ReLU(G), [n_rows, n_cols] ([TG] "Вот тут и решает TwELL";
 * [TC] §2). The columns are cut into nt = ceil(n_cols / tile) tiles of `tile` columns (the last
 * one partial when tile does not divide n_cols). For row r and tile t:
 *   cnt[r*nt + t]                 number of kept entries (g > 0) of that row in that tile;
 *   vals[(r*nt + t)*cap + k]      value of the k-th kept entry, k < cnt (element type `dtype`);
 *   idx [(r*nt + t)*cap + k]      its column inside the tile (0..tile-1), strictly ascending in k.
 * Slots k >= cnt are never written or read. cap must equal tile (lossless: a tile can never
 * overflow). tile is 64, 128 or 256. All three arrays are caller-owned device memory. */
typedef struct {
    int32_t n_rows;
    int32_t n_cols;
    int32_t tile;
    int32_t cap;
    twell_dtype dtype;
    void* vals;
    uint8_t* idx;
    uint16_t* cnt;
} twell_packed;

/* The hybrid training format ([TG] "Обучение"; [TC] §3): each row either fits in one
 * globally aligned sparse block of fixed capacity K or, when it has more than K nonzeros,
 * goes to a dense backup buffer. All pointers are caller-owned device memory.
 *   cnt[n_rows]          uint16: nonzeros of a light row (<= K), or 0xFFFF for a backup row;
 *   col[n_rows*K]        uint16: light rows' kept columns in ascending order (slots >= cnt: 0);
 *   a  [n_rows*K]        fp32: a = ReLU(g) at those columns (slots >= cnt: +0);
 *   u  [n_rows*K]        fp32: u = x Wu_s^T at those columns (filled by hybrid_fwd);
 *   backup_rows[backup_cap]  int32: backup row indices in ascending order;
 *   n_backup[1]          int32: number of overflow rows (may exceed backup_cap: then the call
 *                        reports TWELL_ERR_BACKUP_FULL, only backup_cap rows are stored and the
 *                        outputs of the other overflow rows are undefined);
 *   A_b[backup_cap*n_cols]   fp32: dense a rows of the backup rows;
 *   U_b[backup_cap*n_cols]   fp32: dense u rows of the backup rows (filled by hybrid_fwd);
 *   l1[1]                fp32: L1 term lambda * mean|h| (filled by hybrid_fwd);
 *   dev_status[1]        int32 device status word (see the conventions above).
 * Rows of a light row that are not written are never read; a row is in exactly one of the sparse
 * block and the backup. dtype must be TWELL_BF16 (the element type of x, weights, y, dy, dx). */
typedef struct {
    int32_t n_rows;
    int32_t n_cols;
    int32_t K;
    int32_t backup_cap;
    twell_dtype dtype;
    void* a;
    void* u;
    uint16_t* col;
    uint16_t* cnt;
    int32_t* backup_rows;
    int32_t* n_backup;
    void* A_b;
    void* U_b;
    float* l1;
    int32_t* dev_status;
} twell_hybrid;

/* ------------------------------------------------------------------------------------------
 * Sizes. Bytes of the three TwELL arrays for [n_rows, n_cols] with tile width `tile`
 * (cap = tile), and workspace bytes an operation needs (0 = none; then ws may be NULL).
 * Return 0 on invalid arguments.
 */
TWELL_API size_t twell_packed_vals_bytes(int32_t n_rows, int32_t n_cols, int32_t tile, twell_dtype dtype);
TWELL_API size_t twell_packed_idx_bytes(int32_t n_rows, int32_t n_cols, int32_t tile);
TWELL_API size_t twell_packed_cnt_bytes(int32_t n_rows, int32_t n_cols, int32_t tile);
TWELL_API size_t twell_workspace_bytes(twell_op op, int32_t N, int32_t d, int32_t f, int32_t tile, int32_t K,
                             int32_t backup_cap);

/* ------------------------------------------------------------------------------------------
 * Gate projection with the TwELL pack in its epilogue ([AIM] ¶3; [TG] "Вот тут и решает TwELL";
 * [PUL] ¶3; [TC] §2): G = x Wg_s^T accumulated in fp32, and in the same kernel, per token row
 * and column tile, a = ReLU(G) is packed as values + in-tile indices + count. A gate entry is
 * kept iff its fp32 accumulator is > 0. No dense G is written. x [N, d], Wg_s [f, d] (device,
 * element type `dtype`). `out` must describe an [N, f] TwELL matrix with out->tile = T; its
 * values are stored in out->dtype: TWELL_F32 keeps the fp32 accumulator exactly (allowed for
 * both input types), TWELL_BF16 rounds it to nearest even (bf16 inputs only).
 * ws/ws_bytes: workspace (twell_workspace_bytes(TWELL_OP_GATE_PACK, ...), currently 0).
 */
TWELL_API twell_status twell_gate_pack(const void* x, const void* Wg_s, int32_t N, int32_t d, int32_t f,
                             int32_t T, twell_dtype dtype, const twell_packed* out, void* ws,
                             size_t ws_bytes, int32_t* dev_status, void* stream);

/* Fused up+down projection over a TwELL matrix ([AIM] ¶3; [TG] "Инференс"; [PUL] ¶3; [TC] §2):
 * for every token row, walk only its packed nonzeros (column j, value a), gather row j of Wu_s
 * and of Wd_s, and accumulate y_r += a * (x_r . Wu_s[j]) * Wd_s[j] in fp32; y is stored in the
 * TwELL's dtype. The hidden activation h is never written to memory. Rows with no nonzeros get
 * y = 0. x [N, d], Wu_s / Wd_s [f, d], y [N, d] (device, element type `dtype`; the TwELL
 * values may be bf16 or fp32 independently, except that fp32 inputs need fp32 values).
 * d <= 8192 (bf16) / 4096 (fp32); f / tile <= 1024 tiles.
 * ws/ws_bytes: device workspace of at least twell_workspace_bytes(TWELL_OP_FFN_FUSED_FWD, N, d,
 * ...) bytes, 16-byte aligned, required when N > 0 (else TWELL_ERR_WORKSPACE). It holds the work
 * counter the kernel hands out rows from, a work plan (rows above 128 nonzeros are cut into items
 * of at most 128, walked by different warps, and their fp32 partial rows are added up in item
 * order by the last one to finish; the other rows are handed out longest class first) and those
 * partial rows: about 12 B per row plus N/8 (64 .. 4096) partial rows of 4*d bytes. The call
 * clears its header on `stream`, so two calls in flight at the same time must not share one
 * workspace. Its contents need not be initialised. y is the same bit for bit from call to call,
 * unless more rows want splitting than the N/8 item slots hold (those that find no room are
 * walked whole, and which ones those are depends on scheduling).
 * A corrupt TwELL (count above the tile width, in-tile index >= tile, column >= f) is reported
 * as TWELL_ERR_DEVICE_CHECK in *dev_status; such entries contribute nothing.
 */
TWELL_API twell_status twell_ffn_fused_fwd(const void* x, const void* Wu_s, const void* Wd_s,
                                 const twell_packed* a, int32_t N, int32_t d, int32_t f,
                                 twell_dtype dtype, void* y, void* ws, size_t ws_bytes,
                                 int32_t* dev_status, void* stream);

/* twell_ffn_fused_fwd with the down projection in fp16: Wd16_s is Wd_s converted once to fp16
 * (twell_convert_f16; the conversion is exact for every bf16 weight in [2^-17, 65504] in
 * magnitude, and loses no more than 2^-25 in absolute terms below that), and each h = a * u is
 * rounded once to fp16 (11 significant bits, against ~16 for the bf16 hi + lo pair of
 * twell_ffn_fused_fwd), which halves the tensor-core products of the down projection. Products
 * are accumulated in fp32, as there. bf16 x, Wu_s and y; TwELL values bf16 or fp32; d a multiple
 * of 256 in [512, 3072] (else TWELL_ERR_UNSUPPORTED). Workspace, determinism and error
 * reporting as twell_ffn_fused_fwd.
 */
TWELL_API twell_status twell_ffn_fused_fwd_f16down(const void* x, const void* Wu_s, const void* Wd16_s,
                                         const twell_packed* a, int32_t N, int32_t d, int32_t f,
                                         void* y, void* ws, size_t ws_bytes, int32_t* dev_status,
                                         void* stream);

/* n bf16 values at src to fp16 at dst (device pointers, no overlap), round to nearest even. A
 * finite value beyond the fp16 range is stored as infinity and reported as
 * TWELL_ERR_DEVICE_CHECK in *dev_status.
 */
TWELL_API twell_status twell_convert_f16(const void* src, void* dst, int64_t n, int32_t* dev_status,
                               void* stream);

/* dst [cols, rows] (fp16) = the transpose of src [rows, cols] (bf16, row-major) converted to fp16 with
 * the same rounding and overflow reporting as twell_convert_f16 (e.g. Wd_s [d_ff, d_model] ->
 * Wd16t_s [d_model, d_ff] for twell_ffn_union_fwd). rows <= 2,097,120 (else TWELL_ERR_UNSUPPORTED).
 * Device pointers; asynchronous on `stream`. */
TWELL_API twell_status twell_convert_f16_transposed(const void* src, void* dst, int32_t rows, int32_t cols,
                                                    int32_t* dev_status, void* stream);

/* The whole layer for a batch of at most 16 tokens (decoding) in two launches: the gate + pack of
 * twell_gate_pack (the same TwELL in *a_out, bit for bit) and, in the same kernel, the walk of each
 * column tile's kept entries by the CTAs that computed them ([AIM] ¶3; [TG] "Инференс"; [PUL] ¶3;
 * [TC] §2): the walk is separable by column tile, y_r = sum over tiles of sum over the tile's kept
 * j of a * (x_r . Wu_s[j]) * Wd_s[j]. Each CTA (half a column tile) forms u and h = a * u for its
 * units in fp32 (a as stored in the TwELL), adds h * Wd_s[j] in fp32 over its units in ascending
 * order and stores one fp32 partial row per token; a second kernel adds each token's partial rows
 * in a fixed order and stores y (bf16). y is the same bit for bit from call to call and does not
 * depend on scheduling; it agrees with twell_ffn_fused_fwd on the same TwELL to fp32 summation
 * order. bf16 x, Wg_s, Wu_s, Wd_s, y; 0 <= N <= 16, d_model a multiple of 64 up to 4096, tile 64,
 * 128 or 256 (else TWELL_ERR_UNSUPPORTED); a_out describes an [N, f] TwELL with tile T, values
 * bf16 or fp32. ws: twell_workspace_bytes(TWELL_OP_FFN_DECODE, N, d, f, T, 0, 0) bytes (a flag
 * and an fp32 partial row of d_model per (CTA, token): 2 * ceil(f / T) CTAs), 16-byte aligned,
 * required when N > 0; its contents need not be initialised, and two calls in flight at the same
 * time must not share it.
 */
TWELL_API twell_status twell_ffn_decode(const void* x, const void* Wg_s, const void* Wu_s, const void* Wd_s,
                              int32_t N, int32_t d, int32_t f, int32_t T, const twell_packed* a_out,
                              void* y, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/* The same y from the same TwELL for a layer too dense for the walk: with more than a few percent
 * of d_ff kept per token the union of the units a tile of 128 tokens keeps is nearly all of d_ff,
 * so the up and down projections are dense contractions over all of it, on the tensor cores ([TC]
 * §3: tensor cores for the heavy work). Steps: a is written into H [N, f_pad] (fp16, f_pad = f
 * rounded up to 64) at each row's kept columns, with a per-row keep mask; H = (x Wu_s^T) * a
 * (tcgen05 GEMM on SM pairs, the product formed in its epilogue where the mask is set, h stored in
 * place as fp16: 11 significant bits); y = H Wd16_s (tcgen05 GEMM on SM pairs over f_pad, fp16
 * operands, bf16 y). Wd16t_s is the transpose of Wd_s converted once to fp16 ([d, f]:
 * twell_convert_f16_transposed), so that the down GEMM reads both operands K-major. For N <= 512
 * the down product runs transposed (y^T = Wd16t_s H^T, rows of Wd16t_s on the MMA's M side, tokens in
 * tiles of up to 128, K split over a cluster of CTAs whose fp32 partials are added in a fixed order
 * in shared memory).
 * bf16 x, Wu_s, y; d and f multiples of 8; x [N, d], Wu_s [f, d], Wd16t_s [d, f], y [N, d], device,
 * 16-byte aligned. ws: twell_workspace_bytes(TWELL_OP_FFN_UNION_FWD, N, d, f, ...) bytes (H and the
 * masks, 2.125 * N * f_pad bytes), required when N > 0. A corrupt TwELL entry (count above the tile
 * width, column >= f) is reported as TWELL_ERR_DEVICE_CHECK in *dev_status and contributes nothing;
 * so is an a or h beyond the fp16 range.
 */
TWELL_API twell_status twell_ffn_union_fwd(const void* x, const void* Wu_s, const void* Wd16t_s,
                                 const twell_packed* a, int32_t N, int32_t d, int32_t f,
                                 twell_dtype dtype, void* y, void* ws, size_t ws_bytes,
                                 int32_t* dev_status, void* stream);

/* twell_gate_pack followed by twell_ffn_union_fwd, with the gate and the up projection in one
 * tensor-core GEMM: each tile of an SM pair computes g = x Wg_s^T and u = x Wu_s^T for the same 128
 * units (the pair's two CTAs load Wg_s and Wu_s rows respectively, x is shared), and its epilogue
 * packs ReLU(g) into *out -- the TwELL twell_gate_pack writes, bit for bit ([AIM] ¶3, [TC] §2:
 * the pack in the gate GEMM's epilogue) -- and stores h = a * u (a = the packed value; fp16, 11
 * significant bits; 0 where g <= 0) into the workspace; then y = H Wd16_s as in twell_ffn_union_fwd.
 * For N <= 128 both products run transposed, the weights on the MMA's M side and the tokens as its
 * N columns: each CTA stacks 64 units' Wg_s rows over their Wu_s rows, and two CTAs form one
 * 128-unit tile whose TwELL is the same, bit for bit; up to N = 512 the down product runs
 * transposed as in twell_ffn_union_fwd.
 * For layers whose density the walk no longer serves: the union of the units a tile of 128 tokens
 * keeps is then most of d_ff ([TC] §3: tensor cores for the heavy work).
 * bf16 x, Wg_s, Wu_s, y (dtype must be TWELL_BF16); d and f multiples of 8; T = 64 or 128 (else
 * TWELL_ERR_UNSUPPORTED); x [N, d], Wg_s / Wu_s [f, d], Wd16t_s [d, f] (twell_convert_f16_transposed
 * of Wd_s), y [N, d]; *out a TwELL of N rows, f columns, tile T, fp32 or bf16 values. Device
 * pointers, 16-byte aligned. ws: twell_workspace_bytes(TWELL_OP_FFN_GATE_UNION_FWD, N, d, f, ...)
 * bytes (H [N, f_pad] fp16, f_pad = f rounded up to 64), required when N > 0. An h beyond the fp16
 * range is recorded as TWELL_ERR_DEVICE_CHECK in *dev_status.
 */
TWELL_API twell_status twell_ffn_gate_union_fwd(const void* x, const void* Wg_s, const void* Wu_s,
                                      const void* Wd16t_s, int32_t N, int32_t d, int32_t f, int32_t T,
                                      twell_dtype dtype, const twell_packed* out, void* y, void* ws,
                                      size_t ws_bytes, int32_t* dev_status, void* stream);

/* y = (a * (x Wu_s^T)) Wd_s from the TwELL a, as tensor-core GEMMs over the units each tile of
 * 128 tokens keeps -- the tile's union U_m -- with the union's weight rows gathered ([TG] "Инференс":
 * the kernel gathers only the needed rows of Wu and Wd; [TC] §3: tensor cores take the heavy work).
 * Per tile m: H_m[r, p] = a[r, U_m[p]] * (x_r . Wu_s[U_m[p]]) over p < |U_m| (tcgen05, B = gathered
 * Wu_s rows, the product in the epilogue, h stored once as fp16), then y_m = H_m Wd16_s[U_m]
 * (tcgen05 over K = |U_m|, B = gathered rows of Wd16_s). Each weight row is read once per tile of
 * 128 tokens instead of once per token that keeps it. Wd16_s is Wd_s converted to fp16 once
 * (twell_convert_f16: the same values for weights of magnitude 2^-14 .. 65504; smaller ones move by
 * at most 2^-25); h carries 11 significant bits.
 * x [N, d] bf16, Wu_s [f, d] bf16, Wd16_s [f, d] fp16, y [N, d] bf16, all device, 32-byte aligned;
 * d a multiple of 64 (else TWELL_ERR_UNSUPPORTED); f <= 65535; a: any tile width, fp32 or bf16
 * values. ws: twell_workspace_bytes(TWELL_OP_FFN_TILE_UNION_FWD, N, d, f, ...) bytes, 32-byte
 * aligned, required when N > 0 (per tile: the union list and bitmap; H as fp16 [N, f rounded up to
 * 256]); its contents need not be initialised; two calls in flight at the same time must not share
 * it. A corrupt TwELL entry (count above the tile width, in-tile index >= T, column >= f) is
 * recorded as TWELL_ERR_DEVICE_CHECK and contributes nothing; so is an h beyond the fp16 range
 * (|h| >= 65520, stored as infinity).
 */
TWELL_API twell_status twell_ffn_tile_union_fwd(const void* x, const void* Wu_s, const void* Wd16_s,
                                                const twell_packed* a, int32_t N, int32_t d, int32_t f, void* y,
                                                void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/* Hybrid-format training forward ([TG] "Обучение"; [TC] §3), bf16 only (d_ff a multiple of
 * 64, d_model at most 4096, d_ff at most 65535): gate GEMM + TwELL pack,
 * routing of each row to the sparse block (nnz <= K) or to the dense backup (nnz > K, in
 * ascending row order), the up/down products (gathered rows of Wu_s / Wd_s for light rows,
 * dense tensor-core GEMMs for backup rows), y [N, d], and the L1 term
 * l1_coef * mean|h| over all N*f entries of h ([AIM] ¶4; [PUL] ¶4) into *ctx->l1.
 * ctx describes caller-owned buffers for N = ctx->n_rows, f = ctx->n_cols.
 * ws: at least twell_workspace_bytes(TWELL_OP_HYBRID_FWD, N, d, f, 0, K, backup_cap) bytes.
 */
TWELL_API twell_status twell_hybrid_fwd(const void* x, const void* Wg_s, const void* Wu_s, const void* Wd_s,
                              int32_t N, int32_t d, int32_t f, int32_t K, float l1_coef,
                              twell_dtype dtype, const twell_hybrid* ctx, void* y, void* ws,
                              size_t ws_bytes, void* stream);

/* Hybrid-format training backward ([TG] "Обучение": no product of two dense matrices for the
 * sparse rows), bf16 storage: given the context filled by twell_hybrid_fwd and dy [N, d],
 * computes the gradients of  <y, dy> + l1_coef * mean|h| :
 *   dh = dy_r . Wd_s[j] + l1_coef * sgn(h) / (N f),  du = dh * a,  dg = dh * u  (at kept entries)
 *   dx [N, d] (fp32)          = sum_j du * Wu_s[j] + dg * Wg_s[j]
 *   dWg_s, dWu_s, dWd_s [f, d] (fp32, overwritten) = sum_r dg x_r, du x_r, h dy_r.
 * Gradients are written in fp32: a bf16 copy of dx rounds its largest element by up to 2^-8 of
 * itself, more than the accuracy the layer is held to.
 * Backup rows take dh and dx from dense tensor-core GEMMs; the weight gradients of every kept
 * entry, light or backup, are summed per hidden unit in row order (deterministic). Same shape
 * limits as the forward.
 * ws: at least twell_workspace_bytes(TWELL_OP_HYBRID_BWD, N, d, f, 0, K, backup_cap) bytes; it
 * need not hold anything from the forward call (the context carries what the backward needs).
 */
TWELL_API twell_status twell_hybrid_bwd(const void* x, const void* Wg_s, const void* Wu_s, const void* Wd_s,
                              const twell_hybrid* ctx, const void* dy, int32_t N, int32_t d,
                              int32_t f, float l1_coef, float* dx, float* dWg_s, float* dWu_s,
                              float* dWd_s, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Dead-column compaction. The pages report that more than 30% of the gate's hidden units never
 * fire once training has settled ([PUL] ¶5). A unit that never fires adds nothing to y, so the
 * layer can run on the live units alone: count, per column, how often a calibration batch's TwELL
 * matrix keeps it (twell_column_activity), gather the rows of Wg_s, Wu_s and Wd_s of the columns
 * that fired (twell_gather_rows), and call twell_gate_pack / twell_ffn_fused_fwd with d_ff = the
 * number of live units. With the live columns kept in ascending order the compacted layer gives
 * the same y, bit for bit, on any batch whose active units are among them. The pages state the
 * observation, not this procedure.
 */

/* *total += the number of kept entries of `a` (the sum of its counts; device uint64, the caller
 * clears it): the batch's density is *total / (n_rows * n_cols), which is what a caller needs to
 * choose between twell_ffn_fused_fwd and twell_ffn_tile_union_fwd for the next batch. A count above
 * the tile width is reported as TWELL_ERR_DEVICE_CHECK and counts as 0. Asynchronous on `stream`. */
TWELL_API twell_status twell_count_nonzeros(const twell_packed* a, unsigned long long* total, int32_t* dev_status,
                                            void* stream);

/* col_counts[j] += the number of rows of `a` that keep column j (device int32 [a->n_cols]; the
 * call adds to what is there, the caller clears it). A bad entry (count above the tile width,
 * in-tile index >= tile, column >= n_cols) is reported as TWELL_ERR_DEVICE_CHECK in *dev_status
 * and skipped. */
TWELL_API twell_status twell_column_activity(const twell_packed* a, int32_t* col_counts, int32_t* dev_status,
                                   void* stream);

/* dst[i, :] = src[rows[i], :] for i < n (device; src [n_src, d], dst [n, d] row-major, element
 * type dtype, d * element size a multiple of 16 bytes, both 16-byte aligned; rows int32 [n]). A
 * row index outside [0, n_src) is reported as TWELL_ERR_DEVICE_CHECK and its output row is 0. */
TWELL_API twell_status twell_gather_rows(const void* src, int32_t n_src, const int32_t* rows, int32_t n,
                               int32_t d, twell_dtype dtype, void* dst, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------------------------
 * The operators of a decoder layer around the FFN. They take what stands before and beside it: the
 * residual addition with its RMS norm, the projections' products at decode batch sizes with 4-bit
 * weights, the paged key-value cache and the attention of one new token over it. The pages describe
 * the FFN only; these follow the conventions above (asynchronous, caller-owned memory, 16-byte
 * aligned pointers, host-checked arguments), and every launch is a programmatic dependent of the
 * one before it on its stream.
 */

/* h = x + res,  s = 1 / sqrt(mean(h^2) + eps),  y = h s w  for every row of x [N, d].
 * x, w [d] and y have type `dtype`, res and h_out `res_dtype`: (TWELL_BF16, TWELL_BF16),
 * (TWELL_BF16, TWELL_F32) or (TWELL_F32, TWELL_F32), else TWELL_ERR_UNSUPPORTED. res may be null
 * (then h = x); h_out (h rounded to res_dtype) and rstd [N] (s, fp32, for the backward call) are
 * written when not null. At least one of y and y8 must not be null. y8 [N, d] receives y in e4m3
 * with y8_scale [N, ng]: per group of `group` columns (0: one group a row, ng = 1; 128: ng =
 * ceil(d / 128); else TWELL_ERR_UNSUPPORTED), a = max(|y|, 2^-60), scale = a / 448, code = y * (448 / a)
 * rounded to nearest even; a code stands for code * scale. All sums are fp32; y and y8 are rounded
 * once, from the fp32 h. h_out may be res, and y may be x. d a multiple of 8 up to 16384.
 */
TWELL_API twell_status twell_add_rmsnorm_fwd(const void* x, const void* res, const void* w, int32_t N, int32_t d,
                                   float eps, twell_dtype dtype, twell_dtype res_dtype, void* h_out, void* y,
                                   void* y8, float* y8_scale, int32_t group, float* rstd, void* stream);

/* Gradients of <y, dy> + <h, dh> for the call above, from its h [N, d] (res_dtype; h_out, or x where
 * there was no res) and rstd [N]: dx [N, d] = s (g - xh mean(g xh)) + dh with xh = h s, g = dy w -- the
 * gradient of x and of res alike -- and dw [d] (fp32, overwritten) = sum over rows of dy xh. dy, dh
 * (null: zero) and dx have type grad_dtype, TWELL_BF16 or TWELL_F32 (the FFN's backward call gives an fp32
 * dx). dw is summed in a fixed order: the same from call to call. dx may be dy or dh. ws:
 * twell_workspace_bytes(TWELL_OP_ADD_RMSNORM_BWD, N, d, 1, 0, 0, 0) bytes.
 */
TWELL_API twell_status twell_add_rmsnorm_bwd(const void* dy, const void* h, const void* w, const float* rstd,
                                   const void* dh, int32_t N, int32_t d, twell_dtype dtype, twell_dtype res_dtype,
                                   twell_dtype grad_dtype, void* dx, float* dw, void* ws, size_t ws_bytes,
                                   void* stream);

/* A paged key-value cache (host struct; device memory owned by the caller). Key and value of token
 * slot s = page * page_size + offset and head h start at element
 *   page * page_stride + h * head_stride + offset * token_stride
 * of k and of v (head_dim contiguous elements). dtype is TWELL_BF16, or TWELL_E4M3 with the fp32 scales
 * k_scale, v_scale at page * scale_page_stride + h * scale_head_stride + offset: a code stands for
 * code * scale. page_size is a power of two up to 1024, head_dim a multiple of 16 up to 256,
 * n_pages * page_size < 2^31; strides in elements, k and v strides multiples of 16 bytes. Addresses are
 * formed in 64 bits. */
typedef struct {
    int32_t n_pages;
    int32_t page_size;
    int32_t n_kv_heads;
    int32_t head_dim;
    twell_dtype dtype;
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t page_stride;
    int64_t head_stride;
    int64_t token_stride;
    int64_t scale_page_stride;
    int64_t scale_head_stride;
} twell_kv_cache;

/* Writes n tokens' keys and values into the cache: k, v bf16, token i's heads at k + i * ldk (elements,
 * a multiple of 8, at least n_kv_heads * head_dim: slices of a fused projection are fine), to slot
 * slots[i] (device int32; -1: the token is skipped; any other slot outside the cache is reported as
 * TWELL_ERR_DEVICE_CHECK and skipped; where two tokens of a call have the same slot, what it then holds is not
 * defined: codes of one and a scale of the other among it). An e4m3 cache gets, per token and head, a = max(|values|, 2^-60), scale = a / 448 and the codes of
 * value * (448 / a), rounded to nearest even. */
TWELL_API twell_status twell_kv_append(const twell_kv_cache* cache, const void* k, const void* v, int64_t ldk,
                             int64_t ldv, const int32_t* slots, int32_t n, int32_t* dev_status, void* stream);

/* Reads n slots back: k_out, v_out bf16 [n, n_kv_heads, head_dim] (code * scale rounded once); rows of
 * slots -1 are zeros, and so are those of slots outside the cache, which are reported as
 * TWELL_ERR_DEVICE_CHECK. */
TWELL_API twell_status twell_kv_gather(const twell_kv_cache* cache, const int32_t* slots, int32_t n, void* k_out,
                             void* v_out, int32_t* dev_status, void* stream);

/* Attention of one new token per sequence over the cache. For sequence b < B and query head i (key head
 * i / (n_q_heads / n_kv_heads); n_q_heads a multiple of n_kv_heads): with len = seq_lens[b] and t over the
 * visible tokens [max(0, len - window), len) (window 0: all of them),
 *   out[b][i] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q[b][i] . k_t),  lse[b][i] = log sum_t p_t
 * (natural logarithm, fp32; lse may be null). Nothing visible: out = 0, lse = -inf. Token t of sequence
 * b is at offset t % page_size of page page_table[b * max_pages + t / page_size] (device int32; entries
 * past the last visible token are not read). q bf16, sequence b's heads at q + b * q_stride (elements, a
 * multiple of 8); out bf16 [B, n_q_heads, head_dim]. head_dim 64, 96, 128 or 256; B <= 4096, n_q_heads < 65536. A length
 * outside [0, max_pages * page_size] is clamped and reported as TWELL_ERR_DEVICE_CHECK; a page
 * outside the cache is reported and its tokens do not count. Sums, maxima and the join of split sequences
 * are fp32, in an order that the lengths, the batch, the table's width and the device's number of SMs fix: the same out
 * from call to call. Softmax weights meet the values in two 16-bit parts: 16 bits with a bf16 cache; with an e4m3 one 22
 * bits, down to 2^-40 of the sequence's largest weight times value scale, for value scales within 2^90 of one another. A
 * value that is not finite leaves lse alone. ws:
 * twell_workspace_bytes(TWELL_OP_PAGED_ATTN, B, head_dim, 1, 0, 0, 0) bytes; its contents need not be
 * initialised, and two calls in flight at the same time must not share it. */
TWELL_API twell_status twell_paged_attn_decode(const void* q, int64_t q_stride, const twell_kv_cache* cache,
                                     const int32_t* page_table, const int32_t* seq_lens, int32_t B,
                                     int32_t n_q_heads, int32_t max_pages, float scale, int32_t window, void* out,
                                     float* lse, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/* 4-bit weights W [n, k] with a bf16 scale per `group` columns (32, 64 or 128; k a multiple of 32 and of
 * group): W[r][c] = scale[r][c / group] * (code - 8), code 0..15. Layout, n rounded up to 16 and k to 128
 * (padding: codes 8, scales 0; n and k at most 2^24): words uint32 [ceil(n/16)][ceil(k/128)][8 g][4 c][2 half][4 j], a word
 * holding row 16 tile + 8 half + g, columns 128 tile + 32 j + 8 c + (0..7), column 2i of the 8 in bits
 * 4i..4i+3 and column 2i + 1 in bits 16+4i..19+4i; scales bf16 [ceil(n/16)][ceil(k/128)][8 g][2 half]
 * [128/group]. Sizes in bytes (0 on invalid arguments): */
TWELL_API size_t twell_w4_words_bytes(int32_t n, int32_t k);
TWELL_API size_t twell_w4_scales_bytes(int32_t n, int32_t k, int32_t group);

/* Quantises W [n, k] (bf16, row-major) into that layout: per group scale = bf16(max|w| / 7), code =
 * clamp(round(w / scale), -8, 7) + 8 (ties to even). A weight that is not finite is reported as
 * TWELL_ERR_DEVICE_CHECK. */
TWELL_API twell_status twell_w4_quantize(const void* W, int32_t n, int32_t k, int32_t group, void* words,
                               void* scales, int32_t* dev_status, void* stream);

/* y [N, n] = x W^T for x [N, k] (bf16), 0 <= N <= 16 (else TWELL_ERR_UNSUPPORTED), W as above: x and the
 * codes enter exactly, sums are fp32 in a fixed order, y is rounded once to bf16. A token's y is the same, bit for bit, in
 * any batch of up to 8 tokens, and in any of 9 to 16. */
TWELL_API twell_status twell_w4_matvec(const void* x, const void* words, const void* scales, int32_t N, int32_t n,
                             int32_t k, int32_t group, void* y, void* stream);

/* Rotary positions. A side (queries or keys) of B sequences of S tokens: element j of head h of token t of sequence b is
 * at in + b * in_batch + t * in_token + h * in_head + j and goes to out + b * out_batch + t * out_token + h * out_head + j.
 * in may be out, with the same strides (the call then works in place); else the two do not overlap. The heads of an output
 * lie apart, and so do the outputs of queries and keys; neither output lies over the other side's input (at its address it is
 * refused). Strides in elements; addresses need only the element type's alignment (16-byte vectors are used where the
 * addresses, strides and rot_dim allow them, 8-, 4- and 2-byte ones else). */
typedef struct {
    const void* in;
    void* out;
    int32_t n_heads;
    int64_t in_batch, in_token, in_head;
    int64_t out_batch, out_token, out_head;
} twell_rope_heads;

/* The first rot_dim values of each head (even, at most head_dim) are rot_dim / 2 pairs: (i, i + rot_dim / 2), or with
 * neighbours = 1 (2i, 2i + 1). Pair i of a token at position p is turned by t = 2 pi p turns[i] / 2^64:
 *   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t)
 * and the other values are copied. positions: device int32, of token t of sequence b at b * pos_batch + t (pos_batch 0: the
 * same for all sequences), any value. turns: device uint64 [rot_dim / 2], 2^64 times the turns a position, modulo 2^64: the
 * fraction of a turn is then off by 2^-33 and by the 2^-34 that the rounding of turns comes to, at most, at any position, and t,
 * whose rest after the nearest quarter is taken in fp32, by 2^-22. k may be null.
 * dtype TWELL_BF16 or TWELL_F32; products in fp32, rounded once. factor > 0; head_dim <= 1024 and B * S * head_dim < 2^31
 * (else TWELL_ERR_UNSUPPORTED). twell_rope_bwd takes gradients of the outputs to those of the inputs: the same with -t. */
TWELL_API twell_status twell_rope_fwd(const twell_rope_heads* q, const twell_rope_heads* k, const int32_t* positions,
                            int64_t pos_batch, const uint64_t* turns, float factor, int32_t B, int32_t S,
                            int32_t head_dim, int32_t rot_dim, int32_t neighbours, twell_dtype dtype, void* stream);
TWELL_API twell_status twell_rope_bwd(const twell_rope_heads* dq, const twell_rope_heads* dk, const int32_t* positions,
                            int64_t pos_batch, const uint64_t* turns, float factor, int32_t B, int32_t S,
                            int32_t head_dim, int32_t rot_dim, int32_t neighbours, twell_dtype dtype, void* stream);

/* The pages of a cache that no sequence has (host struct; device memory owned by the caller): ring int32 [n_pages], of which
 * the cells state[0], state[0] + 1, ... modulo n_pages hold the state[1] free pages; state[2] is 0 between calls and state[3]
 * 0. All pages free: ring 0, 1, 2, ..., state 0, n_pages, 0, 0. page_size as in twell_kv_cache. */
typedef struct {
    int32_t n_pages;
    int32_t page_size;
    int32_t* ring;
    int32_t* state;
} twell_page_pool;

/* The plan of a step of B requests (B <= 4096, else TWELL_ERR_UNSUPPORTED), on the device: request b has seq_lens[b] tokens
 * in the pages of row b of page_table [B, max_pages], and new_lens[b] new ones in this step (0: none; -1: it has ended). The
 * step's tokens are the requests' new ones, one request after the other: starts [B + 1] receives where each one's begin
 * (numbers past 2^31 - 1 as that). Token i of n_tokens receives its position in its sequence, its slot (for twell_kv_append)
 * and its owner: labels[b], or b without labels. Tokens past the last request's receive slot -1, position 0, owner -1.
 * New pages come from the ring's front, in the order of requests and positions, into the requests' rows; the pages of a
 * request that has ended go to its back, where later calls find them, its row stays as it is and its length becomes 0.
 * seq_lens_out [B] receives the lengths after the step and state_out [4] the pool's state; they may be seq_lens and
 * pool->state, and lie apart from everything else. A request gets nothing (length and row stay, its tokens receive slot -1 and position 0) if
 *  - the pages of the requests up to it that need any are more than the free ones: TWELL_ERR_POOL_EMPTY in *dev_status;
 *  - its length is negative, does not fit its row or exceeds 2^31 - 1024, its new tokens do not fit n_tokens, or new_lens[b] < -1:
 *    TWELL_ERR_DEVICE_CHECK.
 * More pages given back than are missing (none are taken back then), a state outside the ring (the ring then counts as empty: no
 * page is taken, and those of requests that have ended are put into its cells from 0 on, which are all that it has after
 * the step), and pages outside [0, n_pages) in a row or the ring (slot -1) are
 * TWELL_ERR_DEVICE_CHECK too. A page belongs to one request (one that two rows shared would be given back twice, which is noticed
 * only where the pages are then more than there are). Calls on one pool must follow one another. All integers: the same from call to call. */
TWELL_API twell_status twell_kv_plan(const twell_page_pool* pool, int32_t* page_table, int32_t max_pages,
                           const int32_t* seq_lens, const int32_t* new_lens, const int32_t* labels, int32_t B,
                           int32_t n_tokens, int32_t* slots, int32_t* positions, int32_t* owner, int32_t* starts,
                           int32_t* seq_lens_out, int32_t* state_out, int32_t* dev_status, void* stream);

/* Low-rank adapters of one projection (host struct of device pointers): a bf16 [n_adapters, rank, k], b bf16 [n_adapters, n,
 * rank], scale fp32 [n_adapters]; ranks int32 [n_adapters], or null: all `rank`. Of adapter i the first ranks[i] rows of a
 * and columns of b count; the others may hold anything. k, n and rank multiples of 8, rank <= 128, n_adapters <= 4096, k and
 * n <= 2^20. */
typedef struct {
    int32_t n_adapters;
    int32_t rank;
    int32_t k;
    int32_t n;
    const void* a;
    const void* b;
    const float* scale;
    const int32_t* ranks;
} twell_adapters;

/* out[i] = y[i] + scale[c] b[c] (a[c] x[i]) with c = ids[i], for N <= 2^20 tokens in any order; out[i] = y[i] where c = -1.
 * x [N, k], y and out [N, n] bf16, rows ldx, ldy and ldo elements apart (multiples of 8: slices of a fused projection are
 * fine). out may be y with the same stride (rows without an adapter are then not touched); else they do not overlap, and out
 * never overlaps x. Sums are fp32, in an order that the sizes, how many tokens each adapter has and the device's number of SMs
 * fix, and out is rounded once;
 * a[c] x[i] enters the second product with 16 bits or more. A row's result does not depend on the other tokens' rows or on
 * their order. An id outside [-1, n_adapters) or a rank outside [0, rank] is reported as
 * TWELL_ERR_DEVICE_CHECK and counts as -1. Blocks that share a token's sums wait for one another; should that wait run out,
 * TWELL_ERR_TIMEOUT is reported, and of those rows some columns, or all, stay as they were. ws: twell_workspace_bytes(TWELL_OP_LORA_ADD, N, rank, 1, 0, 0, 0) bytes; two calls
 * in flight at the same time must not share it. */
TWELL_API twell_status twell_lora_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const twell_adapters* ad,
                            const int32_t* ids, int32_t N, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                            int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------------------------
 * Test exports. They run the same device code as the calls above on a gate matrix the caller
 * provides, so packing and routing can be compared bit for bit with an independent reference.
 */

/* Dense [N, f] copy of a TwELL matrix (zeros outside the packed entries), in a->dtype. */
TWELL_API twell_status twell_unpack(const twell_packed* a, void* dense_out, int32_t* dev_status, void* stream);

/* TwELL pack of a given gate matrix G [N, f] (device, dtype): keep g > 0, values copied
 * unchanged. Uses the warp-ballot compaction of the gate epilogue. */
TWELL_API twell_status twell_pack_from_gate(const void* G, int32_t N, int32_t f, int32_t T, twell_dtype dtype,
                                  const twell_packed* out, int32_t* dev_status, void* stream);

/* Hybrid routing of a given gate matrix G [N, f] (device, bf16): the routing kernels of
 * twell_hybrid_fwd applied to pack(G) with tile width 128. Fills ctx->cnt, col, a,
 * backup_rows, n_backup, A_b (not u, U_b, l1). ws: twell_workspace_bytes(TWELL_OP_HYBRID_ROUTE). */
TWELL_API twell_status twell_hybrid_route_from_gate(const void* G, int32_t N, int32_t f, int32_t K,
                                          twell_dtype dtype, const twell_hybrid* ctx, void* ws,
                                          size_t ws_bytes, void* stream);

/* Dense fp32 G = x Wg_s^T [N, f] (row-major, ld = f) from the same tcgen05 mainloop as
 * twell_gate_pack, with a plain store epilogue (bf16 inputs only). */
TWELL_API twell_status twell_gate_gemm(const void* x, const void* Wg_s, int32_t N, int32_t d, int32_t f,
                             float* G_out, int32_t* dev_status, void* stream);

/* Hybrid routing of an already packed TwELL matrix `a` (fp32 values, tile 128, as written by
 * twell_gate_pack or twell_pack_from_gate) into ctx -- the same kernels and the same results as
 * the routing inside twell_hybrid_fwd / twell_hybrid_route_from_gate (ctx->cnt, col, a,
 * backup_rows, n_backup, A_b; not u, U_b, l1) -- without any workspace and without allocating.
 * The pages have no counterpart: this call exists for callers that cannot allocate device memory
 * or pass a workspace (code inside a framework whose caching allocator owns all device memory;
 * plug-in hosts whose interface carries only inputs and outputs; latency-critical loops where an
 * allocation would synchronise the device). ctx->u, ctx->U_b and ctx->l1 are not used and may be
 * null; cnt, n_backup, dev_status, and col and a (K > 0), backup_rows and A_b (backup_cap > 0)
 * are required.
 * Its only scratch, the overflow-row count of each 32-row block, is a fixed array of 32768 int32
 * inside the library: every GPU that loads the library keeps it (128 KB) until the process exits.
 * Limit: a->n_rows <= 1,048,576; larger inputs return TWELL_ERR_UNSUPPORTED before any launch.
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress), so make
 * that first call before any stream capture. All calls share the one array: two calls that
 * overlap on the GPU (different streams, no ordering between them) race and give wrong routes;
 * order them on one stream or with events. */
TWELL_API twell_status twell_hybrid_route_noalloc(const twell_packed* a, int32_t K,
                                                  const twell_hybrid* ctx, void* stream);

/* The bounded mbarrier wait that the library's kernels use (twell_lora_add has one of its own, under the same limit), on its own: one warp initialises an
 * mbarrier that expects one arrival and waits on it with a limit of limit_ms milliseconds. With
 * arrive != 0 the warp's lane 0 arrives first and the wait ends at once; with arrive == 0 nothing
 * ever arrives, the wait gives up after limit_ms, records TWELL_ERR_TIMEOUT in *dev_status and
 * the kernel returns, leaving the context usable. This is how failure detection is tested without
 * hanging or faulting a GPU: the limit of the real kernels' waits (TWELL_WAIT_LIMIT_MS, fractions
 * too, 2 s by default) takes the same path. limit_ms in [1, 10000], else TWELL_ERR_INVALID. */
TWELL_API twell_status twell_wait_probe(int32_t arrive, int32_t limit_ms, int32_t* dev_status, void* stream);

/* C[M, N] = A * B in fp32 from the tcgen05 GEMM used by the hybrid backup rows, bf16 operands:
 * A is [M, K] row-major (a_mn = 0) or [K, M] row-major (a_mn = 1); B is [N, K] row-major
 * (b_mn = 0) or [K, N] row-major (b_mn = 1); C is [M, N] row-major. N and the contiguous
 * extents must be multiples of 8. */
TWELL_API twell_status twell_gemm_test(const void* A, const void* B, int32_t M, int32_t N, int32_t K,
                                       int32_t a_mn, int32_t b_mn, float* C, int32_t* dev_status,
                                       void* stream);

/* ------------------------------------------------------------------------------------------
 * Status.
 */

/* Synchronises `stream`, then returns the code held in *dev_status (TWELL_OK if 0). */
TWELL_API twell_status twell_read_status(const int32_t* dev_status, void* stream);

/* Static text for a status code. */
TWELL_API const char* twell_status_string(twell_status s);

/* Number of SMs and the compute capability of the current device (for callers sizing work);
 * returns TWELL_ERR_CUDA without a device. */
TWELL_API twell_status twell_device_info(int32_t* sm_count, int32_t* cc_major, int32_t* cc_minor);

#ifdef __cplusplus
}
#endif

#endif /* TWELL_GB300_H */
