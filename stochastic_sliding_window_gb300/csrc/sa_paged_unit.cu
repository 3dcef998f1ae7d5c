// Unit kernel of the paged-cache attention: few requests' few new tokens with
// windows of up to about a thousand keys (decoding steps of SA, SWA and gated
// layers).
//
// The same mathematics as the row kernel (sa_paged_rows.cu) for the same units
// of up to 16 query rows of a kv head, but a block of four warps per unit and
// nothing shared between blocks.  What bounds such a call is latency: a chain
// of dependent loads -- lengths, sigma^{-1}, sigma, block table, K and V -- and
// the launch.  So there is no scan over the requests, no second launch and no
// workspace: the grid names the unit; the block's threads resolve all keys at
// once, leave out those of later tokens (an SA window of a sequence at half
// its length holds half its keys), and put their rows' offsets in shared
// memory; its warps take every fourth tile of 16 keys, and their sums meet in
// shared memory at the end.  One token of one request, SWA window 128: 4.1 us on
// the GPU, 10.5 by the row and join kernels; SA, 64 requests at 32768 places: 12.5.
#include "sa_paged_rows.cuh"

#include <cstring>

namespace sa {
namespace prow {

constexpr int kUnitWarps = 4;
constexpr int kUnitThreads = 32 * kUnitWarps;
constexpr int kMostKeys = 1280;
constexpr int kRounds = kMostKeys / kUnitThreads + 1;  // window entries per thread

template <int D, int PATH, int NT>
__device__ __forceinline__ void unit(const Params& P) {
  constexpr int kPitch = Pitch<D>;
  constexpr int kCpr = D / 8;
  constexpr uint32_t kStageBytes = 2 * kKeys * kPitch;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_count[kRounds][kUnitWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // shared memory: Q rows, the keys' row numbers and tokens, the warps' stages
  const uint32_t off_list = uint32_t(P.R) * kPitch;
  const uint32_t off_tok = off_list + uint32_t(P.list_keys) * 4;
  const uint32_t off_ring = (off_tok + uint32_t(P.list_keys) * 4 + 127) / 128 * 128;
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + off_list);
  int* toks = reinterpret_cast<int*>(smem + off_tok);
  uint8_t* ring = smem + off_ring + uint32_t(warp) * uint32_t(P.stages) * kStageBytes;
  const uint32_t sring = smem_u32(ring);

  const int HR = P.Hkv * P.rg;
  const int hr = int(blockIdx.x % unsigned(HR));
  const int grp = int(blockIdx.x / unsigned(HR)) % P.gmax;
  const int b = int(blockIdx.x / unsigned(HR)) / P.gmax;
  const Request rq = load_request<PATH>(P, b, hr == 0 && grp == 0 && tid == 0);
  if (grp >= rq.groups) return;
  const int i0 = grp * P.tb, nt = min(P.tb, rq.n - i0);
  const int pos0 = rq.len - rq.n + i0;
  const int t0 = rq.q0 + i0;
  const int kvh = hr / P.rg;
  const int h0 = kvh * P.g + (hr - kvh * P.rg) * 16;
  const int rows = P.rg > 1 ? min(16, P.g - (hr - kvh * P.rg) * 16) : nt * P.g;
  const bool swa_here = PATH == kPathSWA || (PATH == kPathGated && rq.tsw > 0);

  for (int i = tid; i < rows * kCpr; i += kUnitThreads) {
    const int r = i / kCpr, c = i - r * kCpr;
    const int tk = P.rg > 1 ? 0 : r / P.g;
    cp_async16(smem_u32(smem) + r * kPitch + c * 16,
               P.q + (long long)(t0 + tk) * P.q_stride + (h0 + r - tk * P.g) * D + c * 8);
  }

  // ---- the keys
  const int32_t* table = P.table + (long long)b * P.max_pages;
  auto place = [&](int at, int tok, int page) {  // entry `at` of the list
    uint32_t row = 0xffffffffu;
    if (unsigned(page) < unsigned(P.num_pages)) {
      row = uint32_t(page) * uint32_t(P.page_rows) + uint32_t(page_in(P, tok)) * uint32_t(P.Hkv) + uint32_t(kvh);
    } else {
      atomicOr(P.err, SA_ERRBIT_RANGE);
      tok = 0x7fffffff;
    }
    list[at] = row;
    toks[at] = tok;
  };
  int sa_tiles = 0, sa_keys = 0;
  if (PATH != kPathSWA) {
    const int p = P.inv[(long long)b * P.perm_stride + pos0];
    int slo = 0, shi = 0;
    if (unsigned(p) < unsigned(P.perm_len)) {
      slo = max(0, p - P.half);
      shi = int(min((long long)P.perm_len, (long long)p + P.half + 1));
    } else if (tid == 0) {
      atomicOr(P.err, SA_ERRBIT_RANGE);
    }
    int tok[kRounds];
    unsigned mine[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int j = slo + k * kUnitThreads + tid;
      tok[k] = j < shi ? P.perm[(long long)b * P.perm_stride + j] : -1;
      if (j < shi && unsigned(tok[k]) >= unsigned(P.perm_len)) {
        atomicOr(P.err, SA_ERRBIT_RANGE);
        tok[k] = -1;
      }
      if (tok[k] > pos0) tok[k] = -1;  // a later token
    }
    int page[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      page[k] = tok[k] >= 0 ? table[page_col(P, tok[k])] : 0;
      mine[k] = __ballot_sync(0xffffffffu, tok[k] >= 0);
      if (lane == 0) s_count[k][warp] = __popc(mine[k]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      int at = sa_keys;
#pragma unroll
      for (int w = 0; w < kUnitWarps; ++w) {
        if (w < warp) at += s_count[k][w];
        sa_keys += s_count[k][w];
      }
      if (tok[k] >= 0) place(at + __popc(mine[k] & ((1u << lane) - 1u)), tok[k], page[k]);
    }
    sa_tiles = (sa_keys + kKeys - 1) / kKeys;
    if (tid < sa_tiles * kKeys - sa_keys) {
      list[sa_keys + tid] = 0xffffffffu;
      toks[sa_keys + tid] = 0x7fffffff;
    }
  }
  int tiles = sa_tiles;
  if (swa_here) {
    const int lo = max(0, pos0 - P.w + 1), keys = pos0 + nt - lo;
    const int base = sa_tiles * kKeys;
    tiles += (keys + kKeys - 1) / kKeys;
    for (int k = tid; k < (tiles - sa_tiles) * kKeys; k += kUnitThreads) {
      if (k < keys) {
        place(base + k, lo + k, table[page_col(P, lo + k)]);
      } else {
        list[base + k] = 0xffffffffu;
        toks[base + k] = 0x7fffffff;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // Q
  __syncthreads();

  // ---- this warp's tiles
  int issued = warp;  // next tile to load
  auto issue = [&](int stage) {
    if (issued < tiles) {
      load_tile<D>(P.k, P.v, sring + uint32_t(stage) * kStageBytes, list[issued * kKeys + (lane & 15)]);
      issued += kUnitWarps;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i + 1 < P.stages; ++i) issue(i);
  Acc<D, NT> acc;
  acc.reset();
  acc.rows_of(smem_u32(smem), rows, pos0, P.g, P.rg > 1);
  // gated: what the SA path left when the SWA path begins
  float stash[PATH == kPathGated ? D / 16 : 1][NT][4], sm[NT][2], sl[NT][2];
  bool swapped = PATH != kPathGated;
  auto swap = [&]() {
    swapped = true;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < (PATH == kPathGated ? D / 16 : 0); ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) stash[i][n][e] = acc.o[i][n][e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sm[n][e] = acc.m[n][e];
        sl[n][e] = acc.l[n][e];
      }
    }
    acc.reset();
  };
  int stage = 0, fill = P.stages - 1;
  for (int t = warp; t < tiles; t += kUnitWarps) {
    issue(fill);
    fill = fill + 1 == P.stages ? 0 : fill + 1;
    if (P.stages == 3)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    if (!swapped && t >= sa_tiles) swap();
    acc.tile(sring + uint32_t(stage) * kStageBytes, toks + t * kKeys, t >= sa_tiles ? unsigned(P.w) : 0x7fffffffu,
             false, P.scale_log2);
    __syncwarp();
    stage = stage + 1 == P.stages ? 0 : stage + 1;
  }
  if (!swapped) swap();

  // ---- the warps' parts, through their stages (gated: SA's behind SWA's)
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float* part = reinterpret_cast<float*>(ring);
  acc.sum_rows();
  acc.write(part, P.R, rows);
  if (PATH == kPathGated) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < (PATH == kPathGated ? D / 16 : 0); ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.o[i][n][e] = stash[i][n][e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc.m[n][e] = sm[n][e];
        acc.l[n][e] = sl[n][e];
      }
    }
    acc.sum_rows();
    acc.write(part + P.slot_floats, P.R, rows);
  }
  __syncthreads();
  const float* parts = reinterpret_cast<const float*>(smem + off_ring);
  const int warp_floats = P.stages * int(kStageBytes / 4);
  for (int i = tid; i < rows * (D / 4); i += kUnitThreads) {
    const int r = i / (D / 4), c4 = i - r * (D / 4);
    const int tk = P.rg > 1 ? 0 : r / P.g;
    const size_t row = size_t(t0 + tk) * P.Hq + h0 + r - tk * P.g;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int path = 0; path < (PATH == kPathGated ? 2 : 1); ++path) {
      const bool is_swa = PATH == kPathSWA || (PATH == kPathGated && path == 0);
      const float* pw = parts + path * P.slot_floats;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kUnitWarps; ++w) m = fmaxf(m, pw[w * warp_floats + P.R * D + 2 * r]);
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kUnitWarps; ++w) {
        const float* q = pw + w * warp_floats;
        const float pm = q[P.R * D + 2 * r];
        const float f = pm == -INFINITY ? 0.f : fast_exp2(pm - m);
        l = fmaf(f, q[P.R * D + 2 * r + 1], l);
        const float4 v = *reinterpret_cast<const float4*>(q + r * D + c4 * 4);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
      }
      float s = l == 0.f ? 0.f : 1.f / l;
      if (PATH == kPathGated) s *= 1.f / (1.f + expf(-(is_swa ? P.gate_swa : P.gate_sa)[row]));
      y.x = fmaf(a.x, s, y.x);
      y.y = fmaf(a.y, s, y.y);
      y.z = fmaf(a.z, s, y.z);
      y.w = fmaf(a.w, s, y.w);
    }
    if (PATH == kPathGated && !swa_here) {
      const float4 v = *reinterpret_cast<const float4*>(P.swa_part + row * D + c4 * 4);
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    *reinterpret_cast<uint2*>(P.out + row * D + c4 * 4) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
}

template <int D, int PATH, int NT>
__global__ void __launch_bounds__(kUnitThreads, 2) sa_paged_unit_kernel(const __grid_constant__ Params P) {
  if (P.beside) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else {
    begin_after();
  }
  unit<D, PATH, NT>(P);
  end_beside();
}

template <int D, int PATH, int NT>
static cudaError_t launch_rows_of(const Params& P, unsigned grid, uint32_t smem, cudaStream_t stream) {
  const cudaError_t ce = allow_smem<sa_paged_unit_kernel<D, PATH, NT>>(200u * 1024);
  if (ce != cudaSuccess) return ce;
  return launch_kernel(sa_paged_unit_kernel<D, PATH, NT>, dim3(grid), kUnitThreads, smem, stream, P);
}

template <int D, int PATH>
static cudaError_t launch_unit(const Params& P, unsigned grid, uint32_t smem, cudaStream_t stream) {
  return P.R <= 8 ? launch_rows_of<D, PATH, 1>(P, grid, smem, stream) : launch_rows_of<D, PATH, 2>(P, grid, smem, stream);
}

}  // namespace prow

// Units of up to 1280 keys (their list and stages fit two blocks to an SM).  Very
// many of very few keys are left to the row kernel, whose warps go from unit to
// unit without a block's latency for each; so are those of calls with tiles,
// where most units would be empty blocks (a gated chunk took 142 us instead of
// 114).  Measured (unit against row kernel, us; a token each, 32 q heads on 8 kv heads, d = 128): window 128, 8 requests
// 4.8 to 11.5, 128 18 to 20, 1000 126 to 113; window 512, 128 53 to 59, 1000 325
// to 367; window 1024, 8 14 to 17, 1000 598 to 687.
bool paged_unit_fits(const PagedProblem& pb, Path path, int row_limit, int sms) {
  int tb, rg, rows;
  paged_unit_shape(pb, path, row_limit, &tb, &rg, &rows);
  if (paged_unit_keys(pb, path, tb) > prow::kMostKeys) return false;
  const long long heads = (long long)pb.Hkv * rg;
  const long long units = (pb.T + tb - 1) / tb * heads;
  const long long most = path == kPathSWA ? min(pb.max_new, row_limit) : pb.max_new;
  const bool few = units < 32LL * sms || (paged_unit_keys(pb, path, tb) > 256 && pb.max_new <= row_limit);
  return few && (most + tb - 1) / tb * pb.B * heads <= 65536;
}

sa_status_t launch_paged_unit(const PagedProblem& pb, Path path, int row_limit, const float* swa_part,
                              int sms, cudaStream_t stream) {
  using namespace prow;
  Params P;
  fill_params(&P, pb, path, row_limit, swa_part);
  P.gmax = ((path == kPathSWA ? min(pb.max_new, row_limit) : pb.max_new) + P.tb - 1) / P.tb;
  P.slot_floats = (P.R * (pb.d + 2) + 3) / 4 * 4;
  P.list_keys = int(paged_unit_keys(pb, path, P.tb)) + 2 * kKeys;
  const uint32_t pitch = uint32_t(pb.d) * 2 + 16;
  auto bytes = [&](int stages) {
    return (uint32_t(P.R) * pitch + uint32_t(P.list_keys) * 8 + 127) / 128 * 128 +
           uint32_t(kUnitWarps * stages) * 2 * kKeys * pitch;
  };
  const unsigned grid = unsigned(P.gmax) * unsigned(pb.B) * unsigned(pb.Hkv * P.rg);
  // Three stages where two such blocks still fit an SM and are all that it gets:
  // 33 requests with a window of 512 11.7 us instead of 14.0, but 128 with a window
  // of 128 17.9 instead of 15.6, as a third block fits with two stages.
  P.stages = grid <= 2u * unsigned(sms) && bytes(3) <= kMaxSmem / 2 - 1024 ? 3 : 2;
  const uint32_t smem = bytes(P.stages);
  cudaError_t ce;
  if (pb.d == 128)
    ce = path == kPathSWA ? launch_unit<128, kPathSWA>(P, grid, smem, stream)
         : path == kPathSA ? launch_unit<128, kPathSA>(P, grid, smem, stream)
                           : launch_unit<128, kPathGated>(P, grid, smem, stream);
  else
    ce = path == kPathSWA ? launch_unit<64, kPathSWA>(P, grid, smem, stream)
         : path == kPathSA ? launch_unit<64, kPathSA>(P, grid, smem, stream)
                           : launch_unit<64, kPathGated>(P, grid, smem, stream);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged unit kernel launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
