// Host-side declarations shared by the libftmoe translation units.
#pragma once

#include <cuda.h>
#include <nvtx3/nvToolsExt.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "ft_moe.h"

namespace ftmoe {

// Slots are grouped into blocks of this many rows for the warp-MMA (decode) path:
// one block is the N=8 side of an m16n8k16 MMA.
constexpr int kGemvBlock = 8;
// Align: slot counts up to this size are sorted by one CTA when its shared memory
// (32 E + 2 n + 2 E + 34 ints) fits; larger ones by three grid-wide passes over chunks of
// kAlignChunk slots.
constexpr int kAlignFusedMax = 8192;
constexpr int kAlignChunk = 2048;

// Everything one grouped warp-MMA launch needs. Rows of an expert matrix are the
// MMA M side (16 per warp tile); up to eight activation rows (slots of one block)
// are the N side; K is split across KSPLIT warps of the CTA.
struct GemvParams {
    const uint8_t *codes;    // [E][R][K/2]
    const uint8_t *scales;   // [E][R][K/group]
    const float *glob;       // [E][R]
    int64_t e_codes, e_scales, e_glob;  // per-expert strides (elements)
    int R, K, group;
    int up_off;              // gated: row offset of the up half (I_l)
    const uint16_t *act;     // bf16 rows of length K
    const int *n_pos_dev;    // routed: device count of padded positions
    int n_pos_static;        // shared: number of positions (tokens)
    const int *sorted_slot;  // routed: position -> slot (>= n_slots: padding)
    const int *block_expert; // routed: block -> expert
    int n_slots;             // routed: T*k; shared: T
    int top_k;               // routed: k (slot -> token); shared: 1
    int n_tiles;             // CTA tiles per block
    int num_experts;
    uint16_t *h_out;         // gated: bf16 [positions][h_ld]
    int h_ld;
    float *y_out;            // down: f32 [n_slots][R]
    const float *route_w;    // down, routed: [T*k]; nullptr = weight 1
    int *status;
    const float *sinv;       // fp8_block: scale_inv [E][R/128][K/128] (codes are then [E][R][K])
    int64_t e_sinv;          // fp8_block: per-expert stride of sinv (elements)
};

// Positions per block (the MMA N side) of the tensor-core prefill path.
constexpr int kTcBlock = 128;

// One grouped GEMM launch of the tensor-core path. Rows of expert e's matrix are
// e * R .. e * R + R - 1 of the bank; a unit is (block of kTcBlock positions, tile of
// 128 rows); gate_up units pair gate rows with the up rows up_off further down.
struct TcParams {
    const uint8_t *scales;   // [E][R][K/group]
    const float *glob;       // [E][R]
    int R, K, group, up_off, n_mtiles;
    const int *n_pos_dev;    // routed: device count of padded positions
    int n_pos_static;        // shared: number of tokens
    const int *sorted_slot;  // routed: position -> slot
    const int *block_expert; // routed: block -> expert
    int n_slots, top_k;
    int num_experts;         // routed: E (block_expert values index the banks); shared: 1
    uint16_t *h_out;         // gate_up: bf16 [positions][h_ld]
    int h_ld;
    float *y_out;            // down: fp32 [slots][y_ld]
    int y_ld;
    const float *route_w;    // down, routed: [T*k]
    const float *act_scale;  // per position: factor that undoes the B rows' f16 scaling (or null)
    int *status;
    int fp8;                 // fp8_block banks: codes [E][R][K] bytes, sinv below, no globals
    const float *sinv;       // fp8_block: scale_inv [E][R/128][K/128]
    int64_t e_sinv;          // fp8_block: per-expert stride of sinv (elements)
};
// One tensor-core grouped GEMM launch over up to two problems of the same stage, format
// and group (the routed experts, then the shared expert): units of problem 0, then of
// problem 1; K may differ between them.
struct TcLaunch {
    TcParams prob[2];
    int nprob;
    uint64_t wait_ns;   // limit of every barrier wait (0: the default, about two seconds)
    int skip_producer;  // fault injection: issue no copies, so the consumers' waits run out
    int scale_load_bytes;  // NVFP4 block scales read 16 (or 8, when some K/group is 8 mod 16) bytes at a time
};
// Fault injection armed by ft_moe_debug_inject_stall for the current ft_moe_forward call
// on this thread: the wait limit (0 = default) and whether the pipelined kernels skip
// their producer role.
void injected_stall(uint64_t *wait_ns, int *skip_producer);
// The operands of one problem: its bank's packed codes (rows_total rows) and the f16
// matrix its B operand comes from (act_rows rows of K).
struct TcOperands {
    const void *codes;
    int64_t rows_total;
    const void *act;
    int64_t act_rows;
};
bool tc_shape_ok(int K, int group, int rows_per_expert);
bool tc_shape_ok_fp8(int K, int rows_per_expert);
// nprob (1 or 2) problems in one launch; max_units bounds their total unit count.
cudaError_t launch_tc_gemm(const TcParams *probs, const TcOperands *ops, int nprob, bool gated, int max_units,
                           cudaStream_t s);
// B rows for the f16 tensor-core path: out[pos] = f16(src[row] * 2^-e), scale[pos] = 2^e,
// row = token of sorted_slot[pos] (or pos when sorted_slot is null; rows >= n_slots and
// padding slots give zero rows). pos < *n_pos_dev, or < n_pos_static when that is null.
cudaError_t launch_rows_to_f16(const uint16_t *src, int K, const int *sorted_slot, const int *n_pos_dev,
                               int n_pos_static, int n_slots, int top_k, int max_rows, uint16_t *out, float *scale,
                               cudaStream_t s, int *status);
// One W4A4 (native FP4) grouped GEMM problem: NVFP4 weight banks against NVFP4-quantized
// activation rows (codes, e4m3 scales per 16 elements, fp32 row scale per position).
struct W4Params {
    const uint8_t *w_scales;  // [E][R][K/group] e4m3
    const float *w_glob;      // [E][R]
    const uint8_t *a_scales;  // [positions][K/16] e4m3
    const float *a_glob;      // [positions]
    int R, K, group, up_off, n_mtiles;
    const int *n_pos_dev;     // routed: device count of padded positions
    int n_pos_static;         // shared: number of tokens
    const int *sorted_slot;   // routed: position -> slot
    const int *block_expert;  // routed: block -> expert
    int n_slots, top_k;
    int num_experts;          // routed: E; shared: 1
    float *h_out;             // gate_up: fp32 [positions][h_ld]
    int h_ld;
    float *y_out;             // down: fp32 [slots][y_ld]
    int y_ld;
    const float *route_w;     // down, routed: [T*k]
    int *status;
};
struct W4Launch {
    W4Params prob[2];
    int nprob;
    uint64_t wait_ns;
    int skip_producer;
};
struct W4Operands {
    const void *codes;        // the bank's packed weight codes
    int64_t rows_total;
    const void *act_codes;    // quantized activation codes, [act_rows][K/2]
    int64_t act_rows;
};
bool w4a4_shape_ok(int K, int rows_per_expert);
cudaError_t launch_w4a4_gemm(const W4Params *probs, const W4Operands *ops, int nprob, bool gated, int max_units,
                             cudaStream_t s);
// NVFP4 quantization of position rows (the token of sorted_slot[pos], or pos itself; bf16 or
// fp32 source rows of K elements, K a multiple of 16): codes [pos][K/2], e4m3 scales
// [pos][K/16], fp32 row scales [pos]; padding positions get zeros.
cudaError_t launch_quant_nvfp4(const void *src, bool f32_src, int K, const int *sorted_slot, const int *n_pos_dev,
                               int n_pos_static, int n_slots, int top_k, int max_rows, uint8_t *codes,
                               uint8_t *scales, float *glob, cudaStream_t s, int *status);

// 2D tiled tensor map (rows of `row_bytes` bytes, `inner` elements used per row) through
// the driver's cuTensorMapEncodeTiled; false when the driver refuses the shape. A box takes box_rows rows, row_step
// apart (at most 8, with box_rows * row_step <= 256).
bool make_tensor_map_2d(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t rows,
                        uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swz,
                        uint32_t row_step = 1);

// The same for a stack of `mats` matrices mat_bytes apart (a box takes box_mats of them; what it
// reaches beyond its matrix reads as zero). Lines come into L2 in pairs: a 128-byte wide box walks
// along the rows, and its next step reads the other half (64 decode rows over 256 experts: 152 us
// with single lines, 144 with pairs).
bool make_tensor_map_3d(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t rows,
                        uint64_t mats, uint64_t row_bytes, uint64_t mat_bytes, uint32_t box_inner, uint32_t box_rows,
                        CUtensorMapSwizzle swz, uint32_t box_mats = 1);

// A grouped bf16 product (group_gemm.cu). Forward uses x and w, dgrad dy and w, wgrad dy and x;
// `out` is y, dx or dw. Pointers, strides and sizes are the entry points', already checked.
enum { kGroupForward, kGroupDgrad, kGroupWgrad };
constexpr int kGroupMaxExperts = 1024;
struct GroupGemm {
    int form;
    const int *offs;             // [E + 1], or null (E = 1: all P rows)
    int E, P, N, K;
    const void *x, *w, *dy;
    int64_t ld_x, ld_dy, ld_out; // elements
    void *out;
    int out_f32, accumulate;
    int *status;
    int32_t *plan;               // not null: nothing is launched, the kernel's choice goes here
};
// What ft_moe_debug_group_plan reports.
inline void write_plan(int32_t *plan, int ctas, int tile, int split, bool counted)
{
    plan[0] = ctas;
    plan[1] = tile;
    plan[2] = split;
    plan[3] = counted;
}
cudaError_t launch_group_gemm(const GroupGemm &g, cudaStream_t s);
// A grouped e4m3 product with block scales (group_gemm_fp8.cu).
struct GroupGemm8 {
    const int *offs;
    int E, P, N, K;
    const void *x, *w;
    const float *xs, *ws;
    int64_t ld_x, ld_xs, ld_out;
    void *out;
    int out_f32;
    int *status;
    int32_t *plan;               // as in GroupGemm
};
cudaError_t launch_group_gemm_fp8(const GroupGemm8 &g, cudaStream_t s);
// A grouped MXFP4 product (group_gemm_mxfp4.cu).
struct GroupGemm4 {
    const int *offs;
    int E, P, N, K;
    const void *x, *w;           // packed e2m1 codes; ld_x in bytes
    const uint32_t *xs;          // [ceil(K / 128)][ld_xs] words of four scale bytes
    const uint8_t *ws;           // [E][ceil(N / 128)][ceil(K / 128)][512]
    int64_t ld_x, ld_xs, ld_out;
    void *out;
    int out_f32;
    int *status;
    int32_t *plan;               // as in GroupGemm
};
cudaError_t launch_group_gemm_mxfp4(const GroupGemm4 &g, cudaStream_t s);
// mxfp4_quant.cu. src: rows of K values (SwiGLU: of 2 K), strides in elements; codes: ld_codes in bytes.
struct Quant4Params {
    const void *src;
    int64_t ld_src;
    const float *w;              // SwiGLU: the rows' weights, or null
    int rows, K;
    uint8_t *codes;
    int64_t ld_codes;
    uint32_t *scales;            // words [ceil(K / 128)][ld_scales], or tiles
    int64_t ld_scales;
    int tile_rows;               // 0, or the rows of each weight matrix, whose scales go in tiles
};
cudaError_t launch_quantize_mxfp4(const Quant4Params &p, bool f32, cudaStream_t s);
cudaError_t launch_swiglu_quantize_mxfp4(const Quant4Params &p, cudaStream_t s);
cudaError_t launch_pack_mxfp4_scales(const uint8_t *src, int E, int N, int K, uint32_t *tiles, cudaStream_t s);
// expert_act.cu. Strides in elements; scales are [ceil(columns / 128)][ld_scales].
cudaError_t launch_quantize_fp8(const void *src, bool f32, int64_t ld, int rows, int K, uint8_t *codes, int64_t ld_codes,
                                float *scales, int64_t ld_scales, cudaStream_t s);
cudaError_t launch_swiglu(const void *gu, int64_t ld_gu, const float *w, int rows, int I, void *h, int64_t ld_h,
                          cudaStream_t s);
cudaError_t launch_swiglu_quantize_fp8(const void *gu, int64_t ld_gu, const float *w, int rows, int I, uint8_t *codes,
                                       int64_t ld_codes, float *scales, int64_t ld_scales, cudaStream_t s);
cudaError_t launch_swiglu_backward(const void *gu, int64_t ld_gu, const float *w, const void *dh, int64_t ld_dh, int rows,
                                   int I, void *dgu, int64_t ld_dgu, float *dw, cudaStream_t s);

// norm.cu. Strides in elements; scales are [ceil(H / 128)][ld_scales].
struct NormParams {
    const void *x, *residual, *w;  // residual may be null
    void *total, *y;               // total: with a residual only; y may be null
    int64_t ld_x, ld_residual, ld_total, ld_y;
    uint8_t *codes;                // may be null
    int64_t ld_codes;
    float *scales;
    int64_t ld_scales;
    float *rstd;                   // may be null
    float offset, eps;
    int rows, H;
    int total_f32, w_f32;
};
cudaError_t launch_rmsnorm(const NormParams &p, cudaStream_t s);
struct NormBackParams {
    const void *dy, *total, *w, *dtotal;  // dtotal may be null
    void *dx;
    int64_t ld_dy, ld_total, ld_dtotal, ld_dx;
    const float *rstd;
    float offset;
    int rows, H;
    int total_f32, w_f32;
    float *part;                          // [norm_parts][H], or null
};
constexpr int kMaxNormWidth = 16384;
// Rows of partial sums of the weight's gradient: a function of the sizes alone.
int norm_parts(int rows, int H);
cudaError_t launch_rmsnorm_backward(NormBackParams p, float *dw, int accumulate, void *workspace, cudaStream_t s);

// order.cu. Strides of x and out in bytes (dispatch), else in elements.
struct DispatchParams {
    const char *x;
    char *out;
    int64_t ld_x, ld_out;
    int row_bytes;
    int T, k, P;
    const int *slot, *count;                // count may be null
    const uint32_t *x_scale;                // [blocks][ld_xs]
    uint32_t *out_scale;
    int64_t ld_xs, ld_os;
    int blocks;                             // 0: no scales
    const float *w;
    float *row_w;                           // may be null
    int *pos;                               // may be null
    int small, clear, stream, team;         // set by the launch
};
cudaError_t launch_dispatch(DispatchParams p, cudaStream_t s);
struct CombineParams {
    const void *y, *add;                    // add may be null; of out's type
    void *out;
    int64_t ld_y, ld_add, ld_out;
    const int *pos;
    const float *w;                         // may be null: weights of 1
    const float *drow_w;
    float *dw;                              // may be null
    int T, k, P, H;
    int team;                               // set by the launch
};
cudaError_t launch_combine_rows(CombineParams p, bool y_f32, bool out_f32, cudaStream_t s);
struct CombineBackParams {
    const void *dout, *y;
    void *dy;
    int64_t ld_dout, ld_y, ld_dy;
    const int *pos;
    const float *w;                         // may be null
    float *dw;                              // may be null
    int T, k, P, H;
};
cudaError_t launch_combine_backward(const CombineBackParams &p, bool dout_f32, bool y_f32, cudaStream_t s);

// While one exists, the fault injection armed on this thread applies to the launches made; its
// end disarms it. (A call makes one when its arguments are checked: a refused call launches
// nothing and leaves the injection armed.)
struct StallScope {
    StallScope();
    ~StallScope();
    StallScope(const StallScope &) = delete;
    StallScope &operator=(const StallScope &) = delete;
};

int sm_count();

// Launch with programmatic stream serialization: the kernel may be scheduled before its
// predecessor in the stream finishes; it waits for it in pdl_wait() before touching
// memory (every kernel of the library starts with pdl_enter()).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}
// The same in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s,
                           const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
// Clusters of `cluster` CTAs (up to 8) of a kernel that can run at once: the grid of a persistent
// kernel. A die's SMs need not divide into whole clusters, and a cluster beyond this number would
// start only when another one ends: 152 SMs hold 76 pairs, but 36 clusters of four and 15 of eight.
// A static per kernel, always asked with the kernel's largest shared memory size; the answer is
// looked up once per device (threads that look it up together find the same).
struct ClusterLimit {
    std::atomic<int> found[64][9] = {};
    template <typename Kernel>
    int get(Kernel *kern, int cluster, int threads, size_t smem)
    {
        int dev = 0;
        if (cluster <= 1) return sm_count();
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || cluster > 8) return sm_count() / cluster;
        int n = found[dev][cluster].load(std::memory_order_relaxed);
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(cluster * sm_count());
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = cluster;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            const int all = sm_count() / cluster;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0 || n > all) n = all;
            found[dev][cluster].store(n, std::memory_order_relaxed);
        }
        return n;
    }
};
// launch_pdl inside a function returning cudaError_t: return the launch error, if any.
#define FT_LAUNCH(...)                                                                                         \
    do {                                                                                                       \
        const cudaError_t le_ = launch_pdl(__VA_ARGS__);                                                       \
        if (le_ != cudaSuccess) return le_;                                                                    \
    } while (0)
// An NVTX range named after the ABI call for the scope of the call (header-only NVTX 3:
// nothing is loaded unless a profiler is attached), so that profiles group each call's
// launches.
struct NvtxScope {
    explicit NvtxScope(const char *name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
    NvtxScope(const NvtxScope &) = delete;
    NvtxScope &operator=(const NvtxScope &) = delete;
};
#define FT_NVTX_RANGE(name) const NvtxScope ft_nvtx_scope_(name)

// Sets the thread-local error message (cleared for FT_OK) and returns `code`.
ft_status report_error(ft_status code, const char *message);
// Adds n to the calling thread's launch counter (ft_moe_launch_count).
void count_launches(int n);

cudaError_t launch_route(const float *logits, int T, int E, int k, int32_t *ids, float *w, cudaStream_t s);
// logits [T][E] (fp32) = x [T][H] . w [E][H]^T over bf16; H % 32 == 0.
cudaError_t launch_router_gemm(const uint16_t *x, const uint16_t *w, int T, int H, int E, float *logits,
                               cudaStream_t s);

// Align into caller buffers; `scratch` holds kAlignChunk-sized chunk counts and
// per-slot ranks (align_scratch_bytes). The zero_bytes at `zero` (a multiple of 4, the
// status word among them) are cleared first, in the align launch itself when it is a
// single CTA.
size_t align_scratch_bytes(int n_slots, int E);
cudaError_t launch_align(const int32_t *ids, int T, int k, int E, int B, int32_t *sorted_slot,
                         int32_t *block_expert, int32_t *expert_off, int32_t *n_padded, int *status,
                         void *scratch, cudaStream_t s, int *zero = nullptr, size_t zero_bytes = 0);

// K-split (1, 2, 4 or 8 warps per row tile) for a launch whose CTA-unit count at
// K-split 1 is max_blocks * units_per_block_ks1.
int gemv_ksplit(int max_blocks, int units_per_block_ks1, int K);
// p.n_tiles = CTA units per block: ceil(rows / (16 * 8 / ks)) with rows = I_l (gated) or H.
cudaError_t launch_gemv_gated(const GemvParams &p, int ks, int max_units, cudaStream_t s);
cudaError_t launch_gemv_down(const GemvParams &p, int ks, int max_units, cudaStream_t s);
// Lean register-fed GEMV (two 16-row tiles per warp): usable when K % 32 == 0 and
// (K / ks) % 128 == 0 and one expert's R x K codes take under 2 GB. p.n_tiles =
// ceil(rows / (pair_rows * 8 / ks)).
bool gemv_fast_ok(int K, int group, int ks, int R);

// One lean-GEMV launch over up to two problems (routed experts, shared expert); the
// down stage writes the slot-major y rows, and the combine runs as its own launch.
struct FastLaunch {
    GemvParams prob[2];
    int nprob;
    // Even split of the K steps over the CTAs (register-fed kernel, no in-CTA K split): a
    // unit shared by CTAs c and c + 1 leaves each piece's partial sums in
    // split_part[c][piece] and the second arrival on split_cnt[c] finishes it. Null: each
    // CTA takes whole units. split_cnt is zero at launch; at most kMaxSplitSlots CTAs.
    float *split_part;
    int *split_cnt;
};
constexpr int kMaxSplitSlots = 512;
constexpr size_t kSplitPartFloats = 2 * 256 * 8;  // two pieces x 256 threads x 8 partial sums
cudaError_t launch_gemv_fast(const FastLaunch &L, bool gated, int ks, int max_units, cudaStream_t s);

// The fused decode launch: the gate_up stage (gu, as for launch_gemv_fast with gated =
// true, its split buffers included), the down stage (dn) and the ordered combine in one
// persistent kernel. gu_done (one counter per block: the routed expert's blocks, then the
// shared expert's from shared_base) and done are zero at launch.
struct FusedLaunch {
    FastLaunch gu, dn;
    int *gu_done;
    int shared_base;
    int *done;
    const float *y, *y_sh;  // the down stage's outputs (dn.prob[0/1].y_out), combined in order
    void *out;
    int out_dtype, T, k, H;
    int *status;
    uint64_t wait_ns;       // limit of every cross-CTA wait (0: the default, about two seconds)
    int skip_publish;       // fault injection: gate_up publishes no finished units, so down's waits run out
};
// ks_gu in {1, 2, 4, 8}, ks_dn in {1, 2, 4}; max_units bounds the larger stage's unit count.
cudaError_t launch_gemv_fused(const FusedLaunch &F, int ks_gu, int ks_dn, int max_units, cudaStream_t s);

// fp8_block grouped GEMV (register-fed, any batch size): K a whole number of 128-element
// scale blocks per warp's share.
bool gemv_fp8_ok(int K, int ks);
cudaError_t launch_gemv_fp8(const FastLaunch &L, bool gated, int ks, int max_units, cudaStream_t s);

cudaError_t launch_combine(const float *y, const float *y_shared, int T, int k, int H, void *out, int out_dtype,
                           cudaStream_t s);

cudaError_t launch_pack_copy2d(const uint8_t *src, size_t src_pitch, uint8_t *dst, size_t dst_pitch,
                               size_t width, size_t height, cudaStream_t s);
cudaError_t launch_dequant(const uint8_t *codes, const uint8_t *scales, int rows, int K, int group,
                           uint16_t *out, cudaStream_t s);

}  // namespace ftmoe
