// Internal interface between the C-ABI entry points (sa_api.cu) and the
// kernel launchers (sa_perm.cu, sa_simt.cu, sa_tc.cu, sa_tc_ring.cu,
// sa_tc_chunk.cu).  Not installed.
#pragma once

#include <cuda.h>  // CUtensorMap (type only)
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "libsa.h"

namespace sa {

// Which attention a launch computes.
enum Path : int {
  kPathSA = 0,     // sliding window over the sigma-permuted rows
  kPathSWA = 1,    // trailing window over the original order
  kPathGated = 2,  // sigmoid-gated SA + SWA (SIMT kernel computes both in one pass)
};

// One attention problem, already validated on the host.
struct Problem {
  int B, n, Hq, Hkv, d, g;  // g = Hq / Hkv
  int window;               // SA window w (h = w / 2)
  int window_swa;           // SWA window
  int causal;               // SA causal rule
  float scale;              // softmax scale
  const void* q;
  const void* k;
  const void* v;
  const int32_t* perm;      // [B, n]; unused by SWA
  const float* gate_sa;     // [B, n, Hq] logits (gated only)
  const float* gate_swa;
  void* out;
  int32_t* err;             // device error word (never NULL here)
};

// Record a detail message for sa_last_error_message() and return `st`.
sa_status_t fail(sa_status_t st, const char* fmt, ...);

// Clear that message and return SA_OK.
sa_status_t succeed();

// Device error word owned by the library (used when the caller passes NULL).
int32_t* default_error_word();

// Bound, in SM cycles, on every pipeline wait of the tcgen05 kernels
// launched from now on (default ~2 s at the maximum clock; sa_set_wait_limit).
long long wait_limit_cycles();

// SIMT (CUDA-core) kernel: any window.  `path` selects SA, SWA or gated.
sa_status_t launch_simt(const Problem& pb, Path path, cudaStream_t stream);

// tcgen05 kernel.  `path` is kPathSA or kPathSWA.  gate != nullptr scales the
// output by sigmoid(gate logit); accumulate != 0 adds the previous contents
// of out (the gated merge's second pass).  Returns SA_ERR_UNSUPPORTED, with
// nothing launched, when the shape does not fit the kernel.
sa_status_t launch_tc(const Problem& pb, Path path, const float* gate, int accumulate,
                      cudaStream_t stream);

// True when launch_tc can run this problem / path.
bool tc_supported(const Problem& pb, Path path);

// tcgen05 kernel with a sliding K/V ring in shared memory (each CTA walks a
// contiguous run of tiles and fetches only the new rows of each window).
// Same contract as launch_tc; narrower spans only.
sa_status_t launch_ring(const Problem& pb, Path path, const float* gate, int accumulate,
                        cudaStream_t stream);
bool ring_supported(const Problem& pb, Path path);

// tcgen05 kernel streaming each tile's key span through shared memory in
// 128-key chunks with an online softmax: any window.  Same contract as
// launch_tc.
sa_status_t launch_chunk(const Problem& pb, Path path, const float* gate, int accumulate,
                         cudaStream_t stream);
bool chunk_supported(const Problem& pb, Path path);

// Tensor map of a row-major bf16 [rows, d] tensor for TMA copies of
// 64-column x box_rows boxes with the 128-byte swizzle (false if the driver
// entry point or the encoding fails).
bool encode_row_map(CUtensorMap* m, const void* base, uint64_t rows, int d, int box_rows);

// Tensor map of a bf16 tensor of 2 to 4 dimensions (innermost first; strides
// of the outer ones in bytes) for TMA copies of boxes with the 128-byte
// swizzle; elements outside are read as zeros.
bool encode_box_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims,
                    const uint64_t* strides, const uint32_t* box);

// Backward pass (sa_bwd.cu).  One path (SA or SWA) per call: the dQ kernel
// over query tiles (writes the rows' log2 normaliser and D, and the
// gate-logit gradient when a gate is given), then the dK/dV kernel over
// 128-key tiles.  out_mode: 0 bf16 store, 1 fp32 store, 2 fp32 add.
struct BwdArgs {
  const void* dout;    // bf16 [B, n, Hq, d]
  const float* gate;   // [B, n, Hq] logits or nullptr
  float* lse2;         // [B, n, Hq] workspace
  float* dsum;         // [B, n, Hq] workspace
  float* dgate;        // [B, n, Hq] or nullptr
  void* dq;            // [B, n, Hq, d]
  void* dk;            // [B, n, Hkv, d]
  void* dv;
  int out_mode;
};
bool bwd_supported(const Problem& pb, Path path);
sa_status_t launch_bwd(const Problem& pb, Path path, const BwdArgs& a, cudaStream_t stream);
// fp32 -> bf16 conversion of `count` values (a multiple of 4).
sa_status_t launch_to_bf16(const float* src, void* dst, size_t count, cudaStream_t stream);

// Receptive fields of stacked SA layers (sa_graph.cu).
size_t receptive_field_workspace_bytes(int n);
sa_status_t launch_receptive_field(const int32_t* perms, int layers, int n, int window, int causal,
                                   const int32_t* targets, int num_targets, int64_t* sizes,
                                   void* workspace, int32_t* err, cudaStream_t s);

// The gate projections and RoPE (sa_prologue.cu).
sa_status_t launch_gate_projection(const void* x, int tokens, int d_model, int hq, const void* w_sa,
                                   const void* w_swa, const float* b_sa, const float* b_swa,
                                   float* a_sa, float* a_swa, int32_t* err, cudaStream_t stream);
sa_status_t launch_rope(void* x, int batch, int n, int heads, int head_dim, double base,
                        cudaStream_t stream);

// The current device, and what the serving calls ask of it: its SM count (0
// unless it is an sm_103) and the library's error word there.  Looked up once
// per device; the runtime calls would take longer than a small launch.
struct DeviceInfo {
  int id, sms;
  int32_t* error_word;
};
bool device_info(DeviceInfo* info);

// Lets a kernel take `bytes` of dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem(uint32_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce != cudaSuccess) return ce;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  ce = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (ce == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return ce;
}

// Launches a kernel that may be set up while the kernel before it in the stream
// still runs (once each block of that one allows it or has ended), and orders
// itself: by begin_after or begin_alone, or by end_beside.  early = false: not before that one
// has ended.
template <class P>
cudaError_t launch_kernel(void (*kernel)(P), dim3 grid, unsigned threads, uint32_t smem, cudaStream_t stream,
                          const P& params, bool early = true) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, params);
}
#ifdef __CUDACC__
// The start of a kernel (all its threads): what came before it is done, and the
// next one may be set up.
__device__ __forceinline__ void begin_after() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// The same, but the next one is not set up before this one's blocks have ended:
// where nothing is gained by it (a plan of 1500 requests 10.5 us a call instead
// of 13.8, an append of 128 tokens 5.9 instead of 6.4).
__device__ __forceinline__ void begin_alone() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The end of a kernel that needs nothing of the one that it runs beside: its
// last block outlasts that one, so who waits for this kernel waits for both.
__device__ __forceinline__ void end_beside() {
  if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

// Attention over a paged cache, already validated on the host.
struct PagedProblem {
  int B, T, max_new, Hq, Hkv, d, g;
  int page, num_pages, max_pages;
  int window_swa;            // SWA window (swa and gated paths)
  int half;                  // SA half-width (sa and gated paths)
  int perm_rows, perm_len;
  float scale;
  long long q_stride, page_stride;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_lens;
  const void* q;
  const void* k;
  const void* v;
  const int32_t* perm;
  const int32_t* inv;
  const float* gate_sa;      // [T, Hq] logits (gated path)
  const float* gate_swa;
  void* out;
  int32_t* err;
  bool beside;               // the row or unit kernel runs beside the tile kernel
  int sa_limit;              // requests with more new tokens may go over sigma's order (paged_sa_tiled)
};

// Row kernel (sa_paged_rows.cu).  Requests with more than row_limit new
// tokens are skipped (swa path), or take their SWA term from swa_part, fp32
// [T, Hq, d], gate applied (gated path).  `part`: the workspace.
size_t paged_rows_workspace_bytes(const PagedProblem& pb, Path path, int row_limit, int sms);
sa_status_t launch_paged_rows(const PagedProblem& pb, Path path, int row_limit,
                              const float* swa_part, void* part, int sms, cudaStream_t stream);
// A unit of it: tokens, row groups of a kv head, rows; and its most keys.
void paged_unit_shape(const PagedProblem& pb, Path path, int row_limit, int* tb, int* rg, int* rows);
long long paged_unit_keys(const PagedProblem& pb, Path path, int tb);

// Unit kernel (sa_paged_unit.cu): the same for few units of few keys, a block
// each; no workspace.
bool paged_unit_fits(const PagedProblem& pb, Path path, int row_limit, int sms);
sa_status_t launch_paged_unit(const PagedProblem& pb, Path path, int row_limit,
                              const float* swa_part, int sms, cudaStream_t stream);

// Tile kernel (sa_paged_tiles.cu): the SWA path of requests with more than
// row_limit new tokens, into pb.out; with `gate` (logits [T, Hq]) as fp32
// gated rows into part_out [T, Hq, d] instead.
bool paged_tiles_supported(const PagedProblem& pb);
size_t paged_tiles_workspace_bytes(const PagedProblem& pb, bool sa, int sms);
sa_status_t launch_paged_tiles(const PagedProblem& pb, int row_limit, const float* gate,
                               float* part_out, void* workspace, int sms, cudaStream_t stream);
int paged_tile_tokens(const PagedProblem& pb);  // tokens of a tile

// The requests' tokens in sigma's order (sa_paged_order.cu), for those whose
// SA path the tile or member kernel takes (paged_sa_tiled).
struct SaOrder {
  uint2* list;     // [requests taken][cap] tokens in sigma's order: row of the
                   // caches at kv head 0 (0xffffffff: bad page), position
  int4* members;   // [T] new tokens in sigma's order, a request's from q_start on:
                   // first and last list entry of the window, row, position
  int32_t* chunks; // [T + B] key chunks before each of a request's tiles, from q_start + b on
  int4* info;      // [B] list number, members if the tile kernel takes the request, if the member kernel does
  int2* groups;    // [T / group + B] request and number of a group of its members (-1: none; not
                   // written where q_start is bad), a request's from q_start / group + b on
  int group;       // members of one (0: no groups)
  int cap;         // entries of one list
};
// Whether a request's SA path goes over its tokens in sigma's order: enough
// window keys in all, four times its length, to be worth listing them.  Measured
// (four requests, row kernel against order and what follows, us) at 2, 3, 4 and
// 5 times: 65 to 78, 88 to 58, 105 to 77, 144 to 73 (32 q heads on 8 kv heads, d =
// 128, length 16384, window 128), 44 to 170, 76 to 92, 84 to 98, 102 to 95 (window
// 512), 28 to 43, 46 to 40, 45 to 34, 51 to 34 (4096, 128); 90 to 75, 114 to 73, 151
// to 51, 176 to 56 (16 on 16, d = 64, 16384, 128).
__host__ __device__ inline bool paged_sa_tiled(int n, int len, int half, int row_limit) {
  return n > row_limit && (long long)n * (2LL * half + 1) >= 4LL * len;
}
inline bool paged_order_supported(const PagedProblem& pb) { return pb.B <= 1 << 27; }  // eight blocks each
// Which of the two kernels over that order takes the request: a tile of Bt
// members, perm_len / n places of sigma apart, against one member's window.
// Measured (three requests, member against tile kernel, us, at Bt perm_len over
// n (2 half + 1) of 32, 8, 7, 4 to 3.4, 2 and 0.5): 32 q heads on 8 kv heads,
// d = 128: - , 57 to 84, 86 to 100, - , 119 to 91, 518 to 210; 16 on 16, d = 64:
// 56 to 102, 71 to 106, - , - , 141 to 143, - ; 32 on 4, d = 64: - , - , - , 44 to
// 59, - , 279 to 167 (at 0.3).
__host__ __device__ inline bool paged_sa_members(int n, int Bt, int perm_len, int half) {
  return (long long)Bt * perm_len >= 3LL * n * (2LL * half + 1);
}
size_t paged_order_workspace_bytes(const PagedProblem& pb, int row_limit);
// beside: the kernel before it in the stream is the SWA tile kernel of the same
// call (or its join), beside which it may run.
sa_status_t launch_paged_order(const PagedProblem& pb, int row_limit, int tile_tokens, void* workspace,
                               int group, SaOrder* order, bool beside, cudaStream_t stream);
sa_status_t launch_paged_sa_tiles(const PagedProblem& pb, const SaOrder& order, const float* gate,
                                  const float* swa_part, void* workspace, int sms, cudaStream_t stream);

// Member kernel (sa_paged_members.cu): the same by warp-level matrix
// instructions, for members whose windows share little.
bool paged_members_supported(const PagedProblem& pb);
int paged_member_group(const PagedProblem& pb);      // members of a block
size_t paged_member_groups(const PagedProblem& pb);  // entries of SaOrder::groups
sa_status_t launch_paged_members(const PagedProblem& pb, const SaOrder& order, const float* gate,
                                 const float* swa_part, cudaStream_t stream);

// sigma^{-1} kernels.
sa_status_t launch_inverse_perm(const int32_t* perm, int32_t* inv, int batch, int n,
                                int32_t* err, cudaStream_t stream);

}  // namespace sa
