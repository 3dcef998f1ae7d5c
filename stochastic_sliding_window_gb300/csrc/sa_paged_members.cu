// Member kernel of the paged-cache attention: SA of requests that bring many new
// tokens whose windows share little, over the order that sa_paged_order.cu
// makes of a request's tokens.
//
// Mathematics.  In sigma's order a member's window (a new token's) is a run of
// list entries, and the members of a group follow each other in the list.  A
// warp takes a group, up to 16 query rows that share a kv head, and passes over
// the list from the first member's window to the last one's with an online
// softmax; a row attends to entry e where first <= e <= last of its window and
// the entry's token is not a later one.
//
// What bounds it: K and V rows from anywhere in the caches, 4 d bytes per entry
// for the group's members together.  Members s entries apart with windows of W
// entries cost a group of m members (m - 1) s + W entries; the tile kernel's
// groups of 256 rows share more, but compute 256 rows x all entries, of which
// each row uses W.  So the tile kernel (sa_paged_tiles.cu) takes the requests in
// which W is the larger part.  Warps work alone, a ring of cp.async stages each,
// as in the row kernel.  P is rounded to bf16 for the second product, as in the
// tile kernel; sums and O are fp32.
//
// Measured: three chunks of up to 501 tokens at 12000, 16 heads of d = 64, window
// 256, 45 to 49 us a call (79 by the tile kernel); two of up to 1024 at 16384, 32 q
// heads on 8 kv heads, d = 128, window 128, 49 us (70).  Blocks of 64 rows that
// share their stages read a third less, but their warps wait for each other at
// every stage: 96 us for the first.
#include "sa_paged_rows.cuh"

#include <cstring>

namespace sa {
namespace prow {

// A block is one warp, so that a finished one makes room at once: a gated chunk
// 85 us, with blocks of two and four warps 91 and 92.
constexpr int kMemberWarps = 1;
constexpr int kMemberThreads = 32 * kMemberWarps;
constexpr int kMemberRows = 16;
// Three stages where that leaves 16 warps an SM: 52 instead of 57 us for SA chunks
// with d = 64; with d = 128, where it leaves 8 instead of 12, 98 instead of 91.
template <int D>
constexpr int kMemberStages = D == 64 ? 3 : 2;
constexpr int kNoToken = 0x7fffffff;

struct MemberParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* q_start;
  const float* gate;      // [T, Hq] logits, or nullptr
  const float* swa_part;  // fp32 [T, Hq, D], added to the rows; nullptr: none
  __nv_bfloat16* out;
  SaOrder order;
  long long q_stride, groups;  // groups: of all kv heads
  int B, Hq, Hkv, g;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(kMemberThreads, D == 64 ? 16 : 12)
    sa_paged_members_kernel(const __grid_constant__ MemberParams P) {
  constexpr int kPitch = Pitch<D>;
  constexpr int kCpr = D / 8;
  constexpr int kStages = kMemberStages<D>;
  constexpr uint32_t kStageBytes = 2 * kKeys * kPitch;
  static_assert(16 * (D + 2) * 4 <= kStages * kStageBytes, "O in the ring");
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  begin_after();  // the order, and the SWA terms
  const long long id = (long long)blockIdx.x * kMemberWarps + warp;
  if (id >= P.groups) return;
  const int kvh = int(id % P.Hkv);
  const int2 group = P.order.groups[id / P.Hkv];
  if (unsigned(group.x) >= unsigned(P.B)) return;
  const int4 info = P.order.info[group.x];
  const int Mb = P.order.group;
  if (unsigned(group.y) >= unsigned(ceil_div(info.z, Mb))) return;
  const int nm = min(Mb, info.z - group.y * Mb), rows = nm * P.g;
  const int4* members = P.order.members + P.q_start[group.x] + group.y * Mb;
  const uint2* list = P.order.list + (long long)info.x * P.order.cap;
  const int4 mine = members[min(lane / P.g, nm - 1)];  // lanes 0-15: of row `lane`
  const int lo = __shfl_sync(0xffffffffu, mine.x, 0);
  const int entries = __shfl_sync(0xffffffffu, mine.y, rows - 1) + 1 - lo;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  const uint32_t sring = smem_u32(ring);
  const uint2 none = make_uint2(0xffffffffu, 0u);
  auto entry = [&](int i) {  // lanes 0-15: of tile i
    const int j = i * kKeys + lane;
    return lane < kKeys && j < entries ? list[lo + j] : none;
  };
  uint2 next = entry(0);
  // ---- Q, through the last stage
  constexpr uint32_t kOffQ = (kStages - 1) * kStageBytes;
  for (int i = lane; i < rows * kCpr; i += 32) {
    const int r = i / kCpr, c = i - r * kCpr, m = r / P.g;
    cp_async16(sring + kOffQ + r * kPitch + c * 16,
               P.q + (long long)members[m].z * P.q_stride + (kvh * P.g + r - m * P.g) * D + c * 8);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  const int tiles = ceil_div(entries, kKeys);
  int toks[kStages];  // lanes 0-15: the tokens of the tile in hand and of those loading
  auto issue = [&](int i) {  // tile i, whose entries are in `next`
    const uint32_t row = next.x == 0xffffffffu ? next.x : next.x + uint32_t(kvh);
    const int tok = next.x == 0xffffffffu ? kNoToken : int(next.y);
    next = entry(i + 1);
    load_tile<D>(P.k, P.v, sring + uint32_t(i % kStages) * kStageBytes, row);
    return tok;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    toks[i] = i < tiles ? issue(i) : 0;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  __syncwarp();  // Q
  Acc<D, 2> acc;
  acc.reset();
  acc.rows_of(sring + kOffQ, rows, 0, 1, true);
  int first[2][2];
  unsigned span[2][2];  // this lane's rows' windows, as entries from lo on
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = t * 8 + 2 * (lane & 3) + e;
      const int4 m = members[min(r / P.g, nm - 1)];
      first[t][e] = m.x - lo;
      span[t][e] = unsigned(m.y - m.x);
      acc.pos[t][e] = r < rows ? m.w : -1;
    }
  }
  __syncwarp();  // Q is read
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    toks[kStages - 1] = i + kStages - 1 < tiles ? issue(i + kStages - 1) : 0;
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t sk = sring + uint32_t(i % kStages) * kStageBytes;
    const int ta = __shfl_sync(0xffffffffu, toks[0], lane >> 2), tb = __shfl_sync(0xffffffffu, toks[0], (lane >> 2) + 8);
#pragma unroll
    for (int j = 0; j + 1 < kStages; ++j) toks[j] = toks[j + 1];
    const int ea = i * kKeys + (lane >> 2), eb = ea + 8;
    float s[2][4];
    acc.scores(sk, P.scale_log2, s);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (unsigned(ea - first[t][e]) > span[t][e] || ta > acc.pos[t][e]) s[t][e] = -INFINITY;
        if (unsigned(eb - first[t][e]) > span[t][e] || tb > acc.pos[t][e]) s[t][2 + e] = -INFINITY;
      }
    }
    acc.template absorb<false>(sk, s);
    __syncwarp();  // the stage is read
  }
  // ---- the rows, through the ring
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float* part = reinterpret_cast<float*>(ring);
  acc.sum_rows();
  acc.write(part, 16, rows);
  __syncwarp();
  // lanes 0-15: where row `lane` goes, and what it is multiplied by
  const int to = mine.z * P.Hq + kvh * P.g + lane % P.g;
  float mul = 0.f;
  if (lane < rows) {
    const float l = part[16 * D + 2 * lane + 1];
    mul = l == 0.f ? 0.f : 1.f / l;
    if (P.gate != nullptr) mul *= 1.f / (1.f + expf(-P.gate[to]));
  }
  constexpr int kBatch = 8;  // loads of several rows first (they do not pass the stores)
  for (int i0 = 0; i0 < rows * (D / 4); i0 += 32 * kBatch) {
    float4 y[kBatch];
    int row[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u + lane, r = i / (D / 4), c4 = i % (D / 4);
      row[u] = __shfl_sync(0xffffffffu, to, r & 15);
      if (r >= rows) row[u] = -1;
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (P.swa_part != nullptr && row[u] >= 0)
        y[u] = *reinterpret_cast<const float4*>(P.swa_part + size_t(row[u]) * D + c4 * 4);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u + lane, r = i / (D / 4), c4 = i % (D / 4);
      const float s = __shfl_sync(0xffffffffu, mul, r & 15);
      if (row[u] < 0) continue;
      const float4 o = *reinterpret_cast<const float4*>(part + r * D + c4 * 4);
      *reinterpret_cast<uint2*>(P.out + size_t(row[u]) * D + c4 * 4) =
          make_uint2(pack_bf16x2(fmaf(o.x, s, y[u].x), fmaf(o.y, s, y[u].y)),
                     pack_bf16x2(fmaf(o.z, s, y[u].z), fmaf(o.w, s, y[u].w)));
    }
  }
}

template <int D>
static cudaError_t launch_members(const MemberParams& P, unsigned grid, cudaStream_t stream) {
  const uint32_t smem = kMemberWarps * kMemberStages<D> * 2 * kKeys * Pitch<D>;
  const cudaError_t ce = allow_smem<sa_paged_members_kernel<D>>(smem);
  if (ce != cudaSuccess) return ce;
  return launch_kernel(sa_paged_members_kernel<D>, dim3(grid), kMemberThreads, smem, stream, P);
}

}  // namespace prow

int paged_member_group(const PagedProblem& pb) { return prow::kMemberRows / pb.g; }

size_t paged_member_groups(const PagedProblem& pb) {
  return pb.g > prow::kMemberRows ? 0 : size_t(pb.T) / paged_member_group(pb) + size_t(pb.B);
}

bool paged_members_supported(const PagedProblem& pb) {
  return pb.g <= prow::kMemberRows && double(paged_member_groups(pb)) * pb.Hkv < 2147483647.0;
}

sa_status_t launch_paged_members(const PagedProblem& pb, const SaOrder& order, const float* gate,
                                 const float* swa_part, cudaStream_t stream) {
  using namespace prow;
  MemberParams P;
  std::memset(&P, 0, sizeof(P));
  P.q = static_cast<const __nv_bfloat16*>(pb.q);
  P.k = static_cast<const __nv_bfloat16*>(pb.k);
  P.v = static_cast<const __nv_bfloat16*>(pb.v);
  P.q_start = pb.q_start;
  P.gate = gate;
  P.swa_part = swa_part;
  P.out = static_cast<__nv_bfloat16*>(pb.out);
  P.order = order;
  P.q_stride = pb.q_stride;
  P.groups = (long long)paged_member_groups(pb) * pb.Hkv;
  P.B = pb.B;
  P.Hq = pb.Hq;
  P.Hkv = pb.Hkv;
  P.g = pb.g;
  P.scale_log2 = pb.scale * 1.4426950408889634f;
  const unsigned grid = unsigned((P.groups + kMemberWarps - 1) / kMemberWarps);
  const cudaError_t ce = pb.d == 128 ? launch_members<128>(P, grid, stream) : launch_members<64>(P, grid, stream);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged member kernel launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
