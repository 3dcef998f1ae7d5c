// Serving over a paged K/V cache: the C-ABI entry points, the plan of a step
// (block tables, slots and positions from the requests' lengths) and the
// writer of new keys and values.  The attention itself is in
// sa_paged_rows.cu and sa_paged_unit.cu (few new tokens) and sa_paged_tiles.cu
// and sa_paged_members.cu (many).
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "sa_internal.h"

namespace sa {
namespace paged {

// ------------------------------------------------------------------ plan
//
// q_start = exclusive sum of n_b, and the pages request b takes are the
// exclusive sum S_b of need_b = ceil((c_b + n_b) / P) - ceil(c_b / P), so
// token i of request b (position p = c_b + i, table column p / P) lies in the
// page that column held before, or, past the owned columns, in
// free[num_free - 1 - (S_b + column - owned_b)].  Nothing is read back from
// what is written, so one launch does it: every block scans all lengths (a few
// KB from L2) and then places its own kTokens tokens by a binary search among
// the request starts in shared memory.  A page that is taken always begins
// with a new token, whose thread writes the table entry.
//
// Bound by latency: two passes over the lengths (check, then scan), a search
// and two dependent loads, then one 8-byte store per token.  A step of 64
// single tokens takes 4.0 us on the GPU, 1500 requests with 250 000 tokens 10.

constexpr int kPlanThreads = 512;
constexpr int kTokens = 1024;  // tokens per block

struct PlanParams {
  const int32_t* new_lens;
  const int32_t* cached;
  const int32_t* free_pages;
  const int32_t* num_free;
  int32_t* table;
  int32_t* q_start;
  int32_t* seq_lens;
  int32_t* slots;
  int32_t* positions;
  int32_t* counts;
  int32_t* err;
  int B, max_pages, free_capacity, page, num_pages, max_tokens;
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) sa_paged_plan_kernel(const __grid_constant__ PlanParams P) {
  __shared__ long long s_sum[2][kPlanThreads / 32];
  __shared__ int s_scan[2][kPlanThreads / 32];
  __shared__ int s_start[kPlanThreads + 1], s_take[kPlanThreads];
  __shared__ int s_cached[kPlanThreads], s_row[kPlanThreads];
  begin_alone();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = P.page;
  const int nfree = *P.num_free;
  // check: totals in 64 bits
  long long tokens = 0, pages = 0;
  int bad = nfree < 0 || nfree > P.free_capacity;
  for (int b = tid; b < P.B; b += kPlanThreads) {
    const int n = P.new_lens[b], c = P.cached[b];
    const long long len = (long long)n + c;
    if (n < 0 || c < 0 || len > (long long)P.max_pages * page || len > 2147483647LL) {
      bad = 1;
    } else {
      tokens += n;
      pages += (len + page - 1) / page - (c + (long long)page - 1) / page;
    }
  }
  bad = __syncthreads_or(bad);
  tokens = warp_sum(tokens);
  pages = warp_sum(pages);
  if (lane == 0) {
    s_sum[0][warp] = tokens;
    s_sum[1][warp] = pages;
  }
  __syncthreads();
  tokens = pages = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    tokens += s_sum[0][w];
    pages += s_sum[1][w];
  }
  if (bad || tokens > P.max_tokens || pages > nfree) {  // uniform over the grid
    if (blockIdx.x == 0) {
      for (int b = tid; b < P.B; b += kPlanThreads) P.seq_lens[b] = P.cached[b];
      for (int b = tid; b <= P.B; b += kPlanThreads) P.q_start[b] = 0;
      if (tid == 0) {
        P.counts[0] = 0;
        P.counts[1] = 0;
        P.counts[2] = nfree;
        atomicOr(P.err, SA_ERRBIT_RANGE);
      }
    }
    for (int t = blockIdx.x * kTokens + tid; t < min(P.max_tokens, int(blockIdx.x + 1) * kTokens); t += kPlanThreads) {
      P.slots[t] = -1;
      P.positions[t] = -1;
    }
    return;
  }
  const int t0 = blockIdx.x * kTokens, t1 = min(P.max_tokens, t0 + kTokens);
  int base = 0, pbase = 0;  // tokens and pages of the requests before this chunk
  for (int b0 = 0, chunk = 0; b0 < P.B; b0 += kPlanThreads, ++chunk) {
    const bool writer = chunk % int(gridDim.x) == int(blockIdx.x);
    const int b = b0 + tid;
    int n = 0, c = 0, take = 0;
    if (b < P.B) {
      n = P.new_lens[b];
      c = P.cached[b];
      take = int((unsigned(c) + unsigned(n) + unsigned(page) - 1u) / unsigned(page) -
                 (unsigned(c) + unsigned(page) - 1u) / unsigned(page));
    }
    int sn = n, st = take;  // inclusive scans
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, sn, o), d = __shfl_up_sync(0xffffffffu, st, o);
      if (lane >= o) {
        sn += a;
        st += d;
      }
    }
    __syncthreads();  // the previous chunk's searches are done
    if (lane == 31) {
      s_scan[0][warp] = sn;
      s_scan[1][warp] = st;
    }
    __syncthreads();
    int tn = 0, tt = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) {
        sn += s_scan[0][w];
        st += s_scan[1][w];
      }
      tn += s_scan[0][w];
      tt += s_scan[1][w];
    }
    s_start[tid + 1] = base + sn;
    if (tid == 0) s_start[0] = base;
    s_take[tid] = pbase + st - take;
    s_cached[tid] = c;
    s_row[tid] = b;
    if (writer && b < P.B) {
      P.q_start[b + 1] = base + sn;
      P.seq_lens[b] = c + n;
      if (b == 0) P.q_start[0] = 0;
    }
    __syncthreads();
    const int end = base + tn;
    for (int t = max(t0, base) + tid; t < min(t1, end); t += kPlanThreads) {
      int lo = 0, hi = kPlanThreads - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int cc = s_cached[lo], pos = cc + (t - s_start[lo]);
      const int col = int(unsigned(pos) / unsigned(page)), in = pos - col * page;
      const int owned = int((unsigned(cc) + unsigned(page) - 1u) / unsigned(page));
      int32_t* entry = P.table + (long long)s_row[lo] * P.max_pages + col;
      const int id = col < owned ? *entry : P.free_pages[nfree - 1 - (s_take[lo] + col - owned)];
      if (col >= owned && in == 0) *entry = id;
      const bool ok = unsigned(id) < unsigned(P.num_pages);
      if (!ok) atomicOr(P.err, SA_ERRBIT_RANGE);
      P.slots[t] = ok ? id * page + in : -1;
      P.positions[t] = pos;
    }
    base = end;
    pbase += tt;
  }
  for (int t = max(t0, base) + tid; t < t1; t += kPlanThreads) {
    P.slots[t] = -1;
    P.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    P.counts[0] = base;
    P.counts[1] = pbase;
    P.counts[2] = nfree - pbase;
  }
}

// ------------------------------------------------------------------ append
//
// A copy with a rotation on the way: each (token, head) row of q, k and v is
// read once and written once.  Bound by HBM.  A thread takes the same 8 pairs
// (x_k, x_{k + d/2}) of several heads of one token, two 16-byte loads and two
// 16-byte stores each: it finds the token's rows once, loads up to three heads
// before the block's angles are computed, and holds its cosines and sines in
// registers.  (With an item of any token and head at a time, found by
// divisions, its angles read from shared memory, a thread spent 290
// instructions per item and nine prompts of up to 4096 tokens took 163 us
// against 111; 105 at the copy rate.  Four heads at a time spill at the 64
// registers of 8 blocks of 128 threads to an SM: 130 us.  Streaming loads and
// stores took 110, but the attention that follows reads what is written here.)
// The angle of position p at frequency f_k = base^(-2k/d) / (2 pi) turns per
// token is p f_k mod 1: with f_k as a 64-bit fraction of a turn the product
// wraps by itself, exact to p 2^-64 of a turn, and its top 32 bits give the
// angle to 2^-32 of a turn -- no 64-bit floating point, any position.

constexpr int kAppendThreads = 128;
constexpr int kAppendPre = 3;       // heads per thread loaded at a time
constexpr int kMaxAngles = 1024;    // angle slots per block

struct AppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;
  const int32_t* slots;
  const int32_t* positions;
  __nv_bfloat16* kc;
  __nv_bfloat16* vc;
  __nv_bfloat16* qo;
  int32_t* err;
  long long ks, vs, qs, page_stride;
  int T, Hkv, Hq, d, page;
  int rows_end;  // num_pages * page_size
  int rope;
  int tpb;       // tokens per block
  int gpt;       // groups of threads per token (a group takes a head at a time)
  uint64_t freq[128];  // turns per token, as fractions of 2^64
};

struct AppendRow {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  int rot;
};

// Where head row `hh` of token t (its cache row at `slot`) comes from and goes.
__device__ __forceinline__ AppendRow append_row(const AppendParams& P, int t, int slot, int hh) {
  AppendRow r;
  if (hh >= 2 * P.Hkv) {
    const int h = hh - 2 * P.Hkv;
    r.src = P.q + (long long)t * P.qs + h * P.d;
    r.dst = P.qo + ((long long)t * P.Hq + h) * P.d;
    r.rot = 1;
    return r;
  }
  const int isv = hh >= P.Hkv, h = hh - (isv ? P.Hkv : 0);
  const int pg = int(unsigned(slot) / unsigned(P.page)), in = slot - pg * P.page;
  const long long at = (long long)pg * P.page_stride + ((long long)in * P.Hkv + h) * P.d;
  r.src = isv ? P.v + (long long)t * P.vs + h * P.d : P.k + (long long)t * P.ks + h * P.d;
  r.dst = (isv ? P.vc : P.kc) + at;
  r.rot = P.rope && !isv;
  return r;
}

// Slot of token t, or -1 where nothing is to be written.
__device__ __forceinline__ int append_slot(const AppendParams& P, int t) {
  const int slot = P.slots[t];
  if (slot == -1) return -1;
  if (unsigned(slot) >= unsigned(P.rows_end) || (P.rope && P.positions[t] < 0)) {
    atomicOr(P.err, SA_ERRBIT_RANGE);
    return -1;
  }
  return slot;
}

template <bool kVec>
__global__ void __launch_bounds__(kAppendThreads, 8) sa_paged_append_kernel(const __grid_constant__ AppendParams P) {
  __shared__ __align__(16) float2 s_cs[kMaxAngles];
  begin_alone();
  const int half = P.d / 2;
  const int t0 = blockIdx.x * P.tpb;
  const int ntok = min(P.tpb, P.T - t0);
  const int heads = 2 * P.Hkv + P.Hq;
  auto angles = [&]() {
    for (int a = threadIdx.x; a < ntok * half; a += kAppendThreads) {
      const int tk = a / half, k = a - tk * half;
      const uint64_t turns = P.freq[k] * uint64_t(uint32_t(P.positions[t0 + tk]));
      const float x = float(int32_t(uint32_t(turns >> 32))) * 0x1p-31f;  // half turns in [-1, 1]
      float s, c;
      sincospif(x, &s, &c);
      s_cs[a] = make_float2(c, s);
    }
    __syncthreads();
  };
  if constexpr (kVec) {
    const int per_head = half / 8;
    const int grp = int(threadIdx.x) / per_head, k = (int(threadIdx.x) - grp * per_head) * 8;
    const int tk = grp / P.gpt, h0 = grp - tk * P.gpt, t = t0 + tk;
    const bool on = tk < ntok;  // (groups beyond tpb gpt have no token)
    const __nv_bfloat16* const ksrc = P.k + (long long)t * P.ks + k;
    const __nv_bfloat16* const vsrc = P.v + (long long)t * P.vs + k;
    const __nv_bfloat16* const qsrc = P.q + (long long)t * P.qs + k;
    uint4 lo[kAppendPre], hi[kAppendPre];
    auto fetch = [&](int hh, int u) {
      if (!on || hh >= heads) return;
      const __nv_bfloat16* src = hh >= 2 * P.Hkv ? qsrc + (hh - 2 * P.Hkv) * P.d
                                 : hh >= P.Hkv ? vsrc + (hh - P.Hkv) * P.d
                                               : ksrc + hh * P.d;
      lo[u] = *reinterpret_cast<const uint4*>(src);
      hi[u] = *reinterpret_cast<const uint4*>(src + half);
    };
#pragma unroll
    for (int u = 0; u < kAppendPre; ++u) fetch(h0 + u * P.gpt, u);
    const int slot = on ? append_slot(P, t) : -1;
    const int pg = int(unsigned(slot) / unsigned(P.page)), in = slot - pg * P.page;
    const long long at = (long long)pg * P.page_stride + (long long)in * P.Hkv * P.d + k;
    __nv_bfloat16* const qdst = P.qo + (long long)t * P.Hq * P.d + k;
    float4 cs[4];  // cosine and sine of two pairs each
    if (P.rope) {
      angles();
      if (on) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = *reinterpret_cast<const float4*>(&s_cs[tk * half + k + 2 * e]);
      }
    }
    if (slot < 0) return;
    for (int h1 = h0; h1 < heads; h1 += kAppendPre * P.gpt) {
      if (h1 != h0) {
#pragma unroll
        for (int u = 0; u < kAppendPre; ++u) fetch(h1 + u * P.gpt, u);
      }
#pragma unroll
      for (int u = 0; u < kAppendPre; ++u) {
        const int hh = h1 + u * P.gpt;
        if (hh >= heads) break;
        const bool isv = hh >= P.Hkv && hh < 2 * P.Hkv;
        if (P.rope && !isv) {
          uint32_t* pl = reinterpret_cast<uint32_t*>(&lo[u]);
          uint32_t* ph = reinterpret_cast<uint32_t*>(&hi[u]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 bl = *reinterpret_cast<__nv_bfloat162*>(&pl[e]);
            __nv_bfloat162 bh = *reinterpret_cast<__nv_bfloat162*>(&ph[e]);
            const float2 l = __bfloat1622float2(bl), h = __bfloat1622float2(bh);
            const float4 a = cs[e];
            bl = __floats2bfloat162_rn(l.x * a.x - h.x * a.y, l.y * a.z - h.y * a.w);
            bh = __floats2bfloat162_rn(h.x * a.x + l.x * a.y, h.y * a.z + l.y * a.w);
            pl[e] = *reinterpret_cast<uint32_t*>(&bl);
            ph[e] = *reinterpret_cast<uint32_t*>(&bh);
          }
        }
        __nv_bfloat16* dst = hh >= 2 * P.Hkv ? qdst + (hh - 2 * P.Hkv) * P.d
                             : isv ? P.vc + at + (hh - P.Hkv) * P.d
                                   : P.kc + at + hh * P.d;
        *reinterpret_cast<uint4*>(dst) = lo[u];
        *reinterpret_cast<uint4*>(dst + half) = hi[u];
      }
    }
  } else {
    if (P.rope) angles();
    const int per_head = half, per_tok = heads * per_head, items = ntok * per_tok;
    for (int idx = threadIdx.x; idx < items; idx += kAppendThreads) {
      const int tk = idx / per_tok, rem = idx - tk * per_tok;
      const int hh = rem / per_head, k = rem - hh * per_head;
      const int slot = append_slot(P, t0 + tk);
      if (slot < 0) continue;
      const AppendRow r = append_row(P, t0 + tk, slot, hh);
      __nv_bfloat16 lo = r.src[k], hi = r.src[k + half];
      if (r.rot) {
        const float l = __bfloat162float(lo), h = __bfloat162float(hi);
        const float2 a = s_cs[tk * half + k];
        lo = __float2bfloat16_rn(l * a.x - h * a.y);
        hi = __float2bfloat16_rn(h * a.x + l * a.y);
      }
      r.dst[k] = lo;
      r.dst[k + half] = hi;
    }
  }
}

// ------------------------------------------------------------------ host

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

static sa_status_t check_sizes(const sa_paged_params_t* p, Path path) {
  if (p == nullptr) return fail(SA_ERR_INVALID_ARG, "params is NULL");
  if (p->batch < 1 || p->tokens < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1)
    return fail(SA_ERR_INVALID_ARG, "batch and head counts must be >= 1, tokens >= 0");
  if (p->num_q_heads % p->num_kv_heads != 0)
    return fail(SA_ERR_INVALID_ARG, "num_q_heads (%d) must be a multiple of num_kv_heads (%d)",
                p->num_q_heads, p->num_kv_heads);
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(SA_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", p->head_dim);
  if (p->page_size < 1 || p->num_pages < 1 || p->max_pages < 1)
    return fail(SA_ERR_INVALID_ARG, "page_size, num_pages and max_pages must be >= 1");
  if (double(p->num_pages) * p->page_size >= 2147483648.0)
    return fail(SA_ERR_UNSUPPORTED, "num_pages * page_size must be below 2^31");
  if (p->window < 1) return fail(SA_ERR_INVALID_ARG, "window must be >= 1");
  if (p->kernel < SA_PAGED_AUTO || p->kernel > SA_PAGED_TILES)
    return fail(SA_ERR_INVALID_ARG, "unknown kernel selector %d", p->kernel);
  const long long row = (long long)p->num_q_heads * p->head_dim;
  const long long page_elems = (long long)p->page_size * p->num_kv_heads * p->head_dim;
  if ((p->q_stride != 0 && p->q_stride < row) || p->q_stride % 8 != 0)
    return fail(SA_ERR_INVALID_ARG, "q_stride must be 0, or a multiple of 8 and at least %lld", row);
  if ((p->page_stride != 0 && p->page_stride < page_elems) || p->page_stride % p->head_dim != 0)
    return fail(SA_ERR_INVALID_ARG, "page_stride must be 0, or a multiple of head_dim and at least %lld",
                page_elems);
  const double stride = double(p->page_stride ? p->page_stride : page_elems);
  if (stride / p->head_dim * p->num_pages >= 4294967295.0)
    return fail(SA_ERR_UNSUPPORTED, "a cache of more than 2^32 rows of head_dim");
  if (double(p->tokens) * p->num_q_heads >= 2147483647.0)
    return fail(SA_ERR_UNSUPPORTED, "tokens * num_q_heads too large");
  if (path != kPathSWA) {
    if (p->perm_len < 1 || (p->perm_rows != 1 && p->perm_rows != p->batch))
      return fail(SA_ERR_INVALID_ARG, "perm_len must be >= 1, perm_rows 1 or batch");
    if (p->kernel == SA_PAGED_TILES)
      return fail(SA_ERR_UNSUPPORTED, "the tile kernel alone runs swa_paged_forward only");
  }
  return SA_OK;
}

static PagedProblem make_problem(const sa_paged_params_t* p, Path path) {
  PagedProblem pb;
  std::memset(&pb, 0, sizeof(pb));
  pb.B = p->batch;
  pb.T = p->tokens;
  pb.max_new = p->max_new > 0 && p->max_new < p->tokens ? p->max_new : p->tokens;
  pb.Hq = p->num_q_heads;
  pb.Hkv = p->num_kv_heads;
  pb.d = p->head_dim;
  pb.g = pb.Hq / pb.Hkv;
  pb.page = p->page_size;
  pb.num_pages = p->num_pages;
  pb.max_pages = p->max_pages;
  pb.window_swa = path == kPathGated && p->window_swa > 0 ? p->window_swa : p->window;
  pb.half = p->window / 2;
  pb.sa_limit = 0x7fffffff;
  pb.perm_rows = p->perm_rows;
  pb.perm_len = p->perm_len;
  pb.scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt(float(pb.d));
  pb.q_stride = p->q_stride ? p->q_stride : (long long)pb.Hq * pb.d;
  pb.page_stride = p->page_stride ? p->page_stride : (long long)pb.page * pb.Hkv * pb.d;
  pb.table = p->block_table;
  pb.q_start = p->q_start;
  pb.seq_lens = p->seq_lens;
  return pb;
}

// Which kernels a call runs.  A request with n new tokens has n g query rows
// per kv head.  The row kernel's warps take 16 rows over a run of keys, so that
// more rows read the keys again; the tile kernel's blocks take 256.  Measured for
// SWA (row against tile kernel, us; 32 q heads on 8 kv heads, d = 128): 16
// requests over 16384 keys each, 16 rows 138 to 130, 32 rows 196 to 125, 64 rows
// 275 to 118; 64 over 4096, 125 to 164, 179 to 143, 375 to 180; 16 with a window
// of 512, 12 to 16, 16 to 16, 29 to 16.
// A gated call with tiles runs two or three kernels after another: 48 rows of 16
// requests, SA window 128, SWA window 256, 51 against 53 (2 requests 12 against
// 28); SWA window 1024, 87 against 70.
constexpr int kSwaRows = 16, kGatedRows = 64, kWideGatedRows = 32, kWideWindow = 512;

struct Choice {
  bool tiles;     // SWA (or the gated pair's SWA term) of requests beyond row_limit by tiles
  bool order;     // SA of such requests over sigma's order, where paged_sa_tiled says so:
  bool sa_tiles;  //   some may go to the tile kernel,
  bool members;   //   some to the member kernel (paged_sa_members)
  bool rows, unit;
  int row_limit;  // new tokens per request that the row kernel still takes
};

static Choice choose(const PagedProblem& pb, Path path, int kernel, int sms) {
  Choice c{false, false, false, false, true, false, 0x7fffffff};
  if (kernel != SA_PAGED_ROWS && paged_tiles_supported(pb)) {
    if (kernel == SA_PAGED_TILES) return Choice{true, false, false, false, false, false, 0};
    const int most = path == kPathSWA                                        ? kSwaRows
                     : path == kPathGated && pb.window_swa > kWideWindow ? kWideGatedRows
                                                                             : kGatedRows;
    const int limit = pb.g >= most ? 1 : most / pb.g;
    if (pb.max_new > limit) {
      c.tiles = path != kPathSA;
      c.order = path != kPathSWA && paged_order_supported(pb);
      c.row_limit = limit;
    }
    if (c.order) {  // (requests of limit + 1 to max_new new tokens)
      const int bt = paged_tile_tokens(pb);
      c.members = paged_members_supported(pb) && paged_sa_members(limit + 1, bt, pb.perm_len, pb.half);
      c.sa_tiles = !c.members || !paged_sa_members(pb.max_new, bt, pb.perm_len, pb.half);
    }
  }
  // few units of few keys: the unit kernel instead of the row kernel
  if (paged_unit_fits(pb, path, c.row_limit, sms)) {
    c.unit = true;
    c.rows = false;
  }
  return c;
}

static size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct Workspace {
  size_t rows, tiles, order, swa_part;  // parts, in this order (both tile kernels use `tiles`)
  size_t total() const { return rows + tiles + order + swa_part; }
};

static Workspace workspace_parts(const PagedProblem& pb, Path path, const Choice& c, int sms) {
  Workspace w{0, 0, 0, 0};
  if (c.rows) w.rows = round256(paged_rows_workspace_bytes(pb, path, c.row_limit, sms));
  if (c.tiles) w.tiles = round256(paged_tiles_workspace_bytes(pb, false, sms));
  if (c.sa_tiles) {
    const size_t sa = round256(paged_tiles_workspace_bytes(pb, true, sms));
    w.tiles = w.tiles > sa ? w.tiles : sa;
  }
  if (c.order) {
    w.order = paged_order_workspace_bytes(pb, c.row_limit);
  }
  if (c.tiles && path == kPathGated) w.swa_part = round256(size_t(pb.T) * pb.Hq * pb.d * 4);
  return w;
}

static sa_status_t run(const sa_paged_params_t* prm, Path path, const void* q, const void* k,
                       const void* v, const int32_t* perm, const int32_t* inv,
                       const float* gate_sa, const float* gate_swa, void* out, void* ws,
                       size_t ws_bytes, cudaStream_t stream) {
  sa_status_t st = check_sizes(prm, path);
  if (st != SA_OK) return st;
  if (prm->tokens == 0) return succeed();  // nothing to compute: empty tensors have no address
  if (!q || !k || !v || !out || !prm->block_table || !prm->q_start || !prm->seq_lens)
    return fail(SA_ERR_INVALID_ARG, "q, caches, out, block_table, q_start and seq_lens must be non-NULL");
  if (path != kPathSWA && (!perm || !inv))
    return fail(SA_ERR_INVALID_ARG, "perm and inv_perm must be non-NULL");
  if (path == kPathGated && (!gate_sa || !gate_swa))
    return fail(SA_ERR_INVALID_ARG, "both gate logit arrays must be non-NULL");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return fail(SA_ERR_INVALID_ARG, "q, the caches and out must be 16-byte aligned");
  if (out == q || out == k || out == v) return fail(SA_ERR_INVALID_ARG, "out aliases an input");
  DeviceInfo dev;
  if (!device_info(&dev)) return fail(SA_ERR_CUDA, "cannot resolve the current device and its error word");
  const int sms = dev.sms;
  if (sms == 0) return fail(SA_ERR_UNSUPPORTED, "device is not sm_103");
  PagedProblem pb = make_problem(prm, path);
  const Choice ch = choose(pb, path, prm->kernel, sms);
  if (prm->kernel == SA_PAGED_TILES && !ch.tiles)
    return fail(SA_ERR_UNSUPPORTED, "the tile kernel takes at most 64 query heads per kv head");
  const Workspace parts = workspace_parts(pb, path, ch, sms);
  const size_t need = parts.total();
  if (need > 0 && (ws == nullptr || ws_bytes < need))
    return fail(SA_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (need > 0 && !aligned(ws, 256))
    return fail(SA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  pb.q = q;
  pb.k = k;
  pb.v = v;
  pb.perm = perm;
  pb.inv = inv;
  pb.gate_sa = gate_sa;
  pb.gate_swa = gate_swa;
  pb.out = out;
  pb.err = prm->err ? prm->err : dev.error_word;
  char* const w = static_cast<char*>(ws);
  float* const swa_part = parts.swa_part ? reinterpret_cast<float*>(w + parts.rows + parts.tiles + parts.order) : nullptr;
  if (ch.tiles) {
    st = launch_paged_tiles(pb, ch.row_limit, gate_swa, swa_part, w + parts.rows, sms, stream);
    if (st != SA_OK) return st;
  }
  if (ch.order) {
    pb.sa_limit = ch.row_limit;
    SaOrder order;
    st = launch_paged_order(pb, ch.row_limit, paged_tile_tokens(pb), w + parts.rows + parts.tiles,
                            ch.members ? paged_member_group(pb) : 0, &order, ch.tiles, stream);
    if (st == SA_OK && ch.members) st = launch_paged_members(pb, order, gate_sa, swa_part, stream);
    if (st == SA_OK && ch.sa_tiles) st = launch_paged_sa_tiles(pb, order, gate_sa, swa_part, w + parts.rows, sms, stream);
    if (st != SA_OK) return st;
  }
  pb.beside = (ch.tiles || ch.order) && path != kPathGated;  // (gated: it adds the SWA tiles' part)
  if (ch.unit) {
    st = launch_paged_unit(pb, path, ch.row_limit, swa_part, sms, stream);
    if (st != SA_OK) return st;
  }
  if (ch.rows) {
    st = launch_paged_rows(pb, path, ch.row_limit, swa_part, w, sms, stream);
    if (st != SA_OK) return st;
  }
  return succeed();
}

}  // namespace paged
}  // namespace sa

using namespace sa;

extern "C" sa_status_t swa_paged_forward(const sa_paged_params_t* params, const void* q,
                                         const void* k_cache, const void* v_cache, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream) {
  return paged::run(params, kPathSWA, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, out,
                    workspace, workspace_bytes, stream);
}

extern "C" sa_status_t sa_paged_forward(const sa_paged_params_t* params, const void* q,
                                        const void* k_cache, const void* v_cache,
                                        const int32_t* perm, const int32_t* inv_perm, void* out,
                                        void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
  return paged::run(params, kPathSA, q, k_cache, v_cache, perm, inv_perm, nullptr, nullptr, out,
                    workspace, workspace_bytes, stream);
}

extern "C" sa_status_t sa_swa_gated_paged_forward(
    const sa_paged_params_t* params, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* perm, const int32_t* inv_perm, const float* gate_sa_logits,
    const float* gate_swa_logits, void* out, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
  return paged::run(params, kPathGated, q, k_cache, v_cache, perm, inv_perm, gate_sa_logits,
                    gate_swa_logits, out, workspace, workspace_bytes, stream);
}

extern "C" size_t sa_paged_workspace_size(const sa_paged_params_t* params, int32_t path) {
  if (path < 0 || path > 2) return 0;
  const Path pt = path == 0 ? kPathSWA : path == 1 ? kPathSA : kPathGated;
  if (paged::check_sizes(params, pt) != SA_OK || params->tokens == 0) return 0;
  DeviceInfo dev;
  if (!device_info(&dev) || dev.sms == 0) return 0;
  const int sms = dev.sms;
  const PagedProblem pb = paged::make_problem(params, pt);
  return paged::workspace_parts(pb, pt, paged::choose(pb, pt, params->kernel, sms), sms).total();
}

extern "C" sa_status_t sa_paged_plan(const int32_t* new_lens, const int32_t* cached_lens,
                                     int32_t batch, int32_t* block_table, int32_t max_pages,
                                     const int32_t* free_pages, int32_t free_capacity,
                                     const int32_t* num_free, int32_t page_size, int32_t num_pages,
                                     int32_t max_tokens, int32_t* q_start, int32_t* seq_lens,
                                     int32_t* slots, int32_t* positions, int32_t* counts,
                                     int32_t* d_err, cudaStream_t stream) {
  if (batch < 1 || max_pages < 1 || page_size < 1 || num_pages < 1 || max_tokens < 0 || free_capacity < 0)
    return fail(SA_ERR_INVALID_ARG, "batch, max_pages, page_size and num_pages must be >= 1, "
                "max_tokens and free_capacity >= 0");
  if (!new_lens || !cached_lens || !block_table || !num_free || !q_start || !seq_lens || !counts ||
      (max_tokens > 0 && (!slots || !positions)) || (free_capacity > 0 && !free_pages))
    return fail(SA_ERR_INVALID_ARG, "NULL pointer");
  if (seq_lens == cached_lens || seq_lens == new_lens || q_start == new_lens ||
      q_start == cached_lens || counts == num_free)
    return fail(SA_ERR_INVALID_ARG, "an output aliases an input");
  if (double(num_pages) * page_size >= 2147483648.0)
    return fail(SA_ERR_UNSUPPORTED, "num_pages * page_size must be below 2^31");
  if (max_tokens > 2147483647 - paged::kTokens || page_size > (1 << 30))
    return fail(SA_ERR_UNSUPPORTED, "max_tokens or page_size too large");
  paged::PlanParams P;
  P.new_lens = new_lens;
  P.cached = cached_lens;
  P.free_pages = free_pages;
  P.num_free = num_free;
  P.table = block_table;
  P.q_start = q_start;
  P.seq_lens = seq_lens;
  P.slots = slots;
  P.positions = positions;
  P.counts = counts;
  DeviceInfo dev;
  if (!device_info(&dev)) return fail(SA_ERR_CUDA, "cannot resolve the current device and its error word");
  P.err = d_err ? d_err : dev.error_word;
  P.B = batch;
  P.max_pages = max_pages;
  P.free_capacity = free_capacity;
  P.page = page_size;
  P.num_pages = num_pages;
  P.max_tokens = max_tokens;
  const int grid = max_tokens > paged::kTokens ? (max_tokens + paged::kTokens - 1) / paged::kTokens : 1;
  const cudaError_t ce =
      launch_kernel(paged::sa_paged_plan_kernel, dim3(unsigned(grid)), paged::kPlanThreads, 0, stream, P);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "plan launch: %s", cudaGetErrorString(ce));
  return succeed();
}

extern "C" sa_status_t sa_paged_append(const sa_paged_append_params_t* p, const void* k,
                                       const void* v, const void* q, const int32_t* slots,
                                       const int32_t* positions, void* k_cache, void* v_cache,
                                       void* q_out, cudaStream_t stream) {
  using namespace paged;
  if (p == nullptr) return fail(SA_ERR_INVALID_ARG, "params is NULL");
  if (p->tokens < 0 || p->num_kv_heads < 1 || p->num_q_heads < 0 || p->page_size < 1 ||
      p->num_pages < 1 || p->head_dim < 2 || p->head_dim % 2 != 0 || p->head_dim > 256)
    return fail(SA_ERR_INVALID_ARG, "need tokens >= 0, num_kv_heads, page_size, num_pages >= 1 and "
                "an even head_dim <= 256");
  if (double(p->num_pages) * p->page_size >= 2147483648.0)
    return fail(SA_ERR_UNSUPPORTED, "num_pages * page_size must be below 2^31");
  const bool rope = p->rope_base != 0.0;
  if (rope && !(p->rope_base > 1.0)) return fail(SA_ERR_INVALID_ARG, "rope_base must be 0 or > 1");
  const bool with_q = q != nullptr || q_out != nullptr;
  if (with_q && !rope) return fail(SA_ERR_INVALID_ARG, "q is rotated only: it needs rope_base");
  const int d = p->head_dim, hq = with_q ? p->num_q_heads : 0, hkv = p->num_kv_heads;
  if (with_q && hq < 1) return fail(SA_ERR_INVALID_ARG, "num_q_heads must be >= 1 when q is given");
  if (2.0 * hkv + hq > 65536.0) return fail(SA_ERR_UNSUPPORTED, "too many heads");
  if (p->tokens == 0) return succeed();
  if (!k || !v || !slots || !k_cache || !v_cache || (rope && !positions) || (with_q && (!q || !q_out)))
    return fail(SA_ERR_INVALID_ARG, "NULL pointer");
  if (q_out != nullptr && (q_out == q || q_out == k || q_out == v))
    return fail(SA_ERR_INVALID_ARG, "q_out aliases an input");
  if (k_cache == v_cache || k_cache == k || v_cache == v)
    return fail(SA_ERR_INVALID_ARG, "a cache aliases an input or the other cache");
  AppendParams P;
  std::memset(&P, 0, sizeof(P));
  P.ks = p->k_stride ? p->k_stride : (long long)hkv * d;
  P.vs = p->v_stride ? p->v_stride : (long long)hkv * d;
  P.qs = p->q_stride ? p->q_stride : (long long)hq * d;
  P.page_stride = p->page_stride ? p->page_stride : (long long)p->page_size * hkv * d;
  if (P.ks < (long long)hkv * d || P.vs < (long long)hkv * d || P.qs < (long long)hq * d ||
      P.page_stride < (long long)p->page_size * hkv * d)
    return fail(SA_ERR_INVALID_ARG, "a stride is shorter than its row or page");
  P.k = static_cast<const __nv_bfloat16*>(k);
  P.v = static_cast<const __nv_bfloat16*>(v);
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.slots = slots;
  P.positions = positions;
  P.kc = static_cast<__nv_bfloat16*>(k_cache);
  P.vc = static_cast<__nv_bfloat16*>(v_cache);
  P.qo = static_cast<__nv_bfloat16*>(q_out);
  DeviceInfo dev;
  if (!device_info(&dev)) return fail(SA_ERR_CUDA, "cannot resolve the current device and its error word");
  P.err = p->err ? p->err : dev.error_word;
  P.T = p->tokens;
  P.Hkv = hkv;
  P.Hq = hq;
  P.d = d;
  P.page = p->page_size;
  P.rows_end = p->num_pages * p->page_size;
  P.rope = rope ? 1 : 0;
  const int half = d / 2;
  if (rope) {
    const double inv_two_pi = 0.15915494309189533576888376337251;
    for (int i = 0; i < half; ++i)
      P.freq[i] = uint64_t(std::ldexp(std::pow(p->rope_base, -2.0 * i / d) * inv_two_pi, 64));
  }
  const bool vec = d % 16 == 0 && aligned(k, 16) && aligned(v, 16) && aligned(k_cache, 16) &&
                   aligned(v_cache, 16) && (!with_q || (aligned(q, 16) && aligned(q_out, 16))) &&
                   P.ks % 8 == 0 && P.vs % 8 == 0 && P.qs % 8 == 0 && P.page_stride % 8 == 0;
  // tokens per block such that its groups of threads, gpt to a token, are in
  // work for up to kAppendPre heads each: with the fewest idle
  const int groups = kAppendThreads / (vec ? half / 8 : half > kAppendThreads ? kAppendThreads : half);
  const int heads = 2 * hkv + hq;
  int tpb = 1;
  double best = 0;
  for (int rounds = 1; rounds <= kAppendPre; ++rounds) {
    const int n = groups / ((heads + rounds - 1) / rounds);
    const double used = double(n) * heads / (double(groups) * rounds);
    if (n > 0 && used >= best) {
      best = used;
      tpb = n;
    }
  }
  if (tpb * half > kMaxAngles) tpb = kMaxAngles / half;
  // no fewer blocks than would fill the GPU
  const int even = p->tokens / 304;
  if (tpb > even) tpb = even;
  P.tpb = tpb < 1 ? 1 : tpb;
  P.gpt = groups / P.tpb;
  const unsigned grid = unsigned((p->tokens + P.tpb - 1) / P.tpb);
  const cudaError_t ce = launch_kernel(vec ? sa_paged_append_kernel<true> : sa_paged_append_kernel<false>, dim3(grid),
                                       kAppendThreads, 0, stream, P);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "append launch: %s", cudaGetErrorString(ce));
  return succeed();
}
