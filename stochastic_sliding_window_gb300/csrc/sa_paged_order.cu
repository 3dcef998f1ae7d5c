// A request's tokens in sigma's order, for the SA tiles of the paged-cache
// attention (sa_paged_tiles.cu).
//
// For each request that brings many new tokens, one block passes over its row
// of sigma and keeps, in order, the entries that name a token there is
// (sigma[q] < length): the list, with each token's row in the caches.  The new
// tokens among them are the members; a member at place q has the window
// |q' - q| <= h, the run of list entries between two binary searches over the
// places, each within h entries of its own.  Last, the tiles' key chunks are
// summed, which is what the tile kernel's schedule needs to know.
//
// Bound by latency and one SM's loads: perm_len * 4 bytes read, 12 bytes per
// token written, in rounds of 16384 entries whose order is found by ballots
// and one scan over the block's 32 warps.
#include "sa_internal.h"

#include <cstring>

namespace sa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 16;  // entries of sigma per thread and round
constexpr int kChunk = 128;

struct Params {
  const int32_t* perm;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_lens;
  int32_t* err;
  SaOrder order;
  long long perm_stride, page_rows;
  int T, max_new, max_pages, page, num_pages, perm_len, half, row_limit, Bt, Hkv, lists;
};

__device__ __forceinline__ int new_tokens(const Params& P, int b, int* len) {
  const int q0 = P.q_start[b], q1 = P.q_start[b + 1];
  *len = P.seq_lens[b];
  const int n = q1 - q0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= P.T && n <= P.max_new && n <= *len &&
                  (long long)*len <= (long long)P.max_pages * P.page && *len <= P.perm_len;
  return ok && paged_sa_tiled(n, *len, P.half, P.row_limit) ? n : 0;
}

__global__ void __launch_bounds__(kThreads) sa_paged_order_kernel(const __grid_constant__ Params P) {
  __shared__ int s_a[kWarps], s_b[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x;
  // list number: the requests before this one that are taken too
  int before = 0, len;
  for (int i = tid; i < b; i += kThreads) before += new_tokens(P, i, &len) > 0;
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) s_a[warp] = before;
  __syncthreads();
  before = __reduce_add_sync(0xffffffffu, s_a[lane]);
  int n = new_tokens(P, b, &len);
  if (before >= P.lists && n > 0) {  // only where requests claim the same rows
    if (tid == 0) atomicOr(P.err, SA_ERRBIT_RANGE);
    n = 0;
  }
  if (n == 0) {
    if (tid == 0) P.order.info[b] = make_int2(before, 0);
    return;
  }
  const int q0 = P.q_start[b], c = len - n;
  uint2* list = P.order.list + (long long)before * P.order.cap;
  int32_t* place = P.order.place + (long long)before * P.order.cap;
  int4* members = P.order.members + q0;
  const int32_t* sigma = P.perm + (long long)b * P.perm_stride;
  const int32_t* table = P.table + (long long)b * P.max_pages;
  const unsigned below = (1u << lane) - 1u;
  int entries = 0, found = 0;  // list entries and members so far
  for (int base = 0; base < P.perm_len; base += kThreads * kEach) {
    // a warp takes 32 kEach entries that follow each other
    const int from = base + warp * (32 * kEach) + lane;
    int tok[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int q = from + 32 * j;
      tok[j] = q < P.perm_len ? sigma[q] : -1;
      if (q < P.perm_len && unsigned(tok[j]) >= unsigned(P.perm_len)) {
        atomicOr(P.err, SA_ERRBIT_RANGE);
        tok[j] = -1;
      }
      if (tok[j] >= len) tok[j] = -1;
    }
    int pg[kEach];
    int count = 0, mine = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      pg[j] = tok[j] >= 0 ? table[unsigned(tok[j]) / unsigned(P.page)] : 0;
      count += __popc(__ballot_sync(0xffffffffu, tok[j] >= 0));
      mine += __popc(__ballot_sync(0xffffffffu, tok[j] >= c));
    }
    __syncthreads();  // the last round's sums are read
    if (lane == 0) {
      s_a[warp] = count;
      s_b[warp] = mine;
    }
    __syncthreads();
    const int ca = s_a[lane], cb = s_b[lane];
    int at = entries + __reduce_add_sync(0xffffffffu, lane < warp ? ca : 0);
    int am = found + __reduce_add_sync(0xffffffffu, lane < warp ? cb : 0);
    entries += __reduce_add_sync(0xffffffffu, ca);
    found += __reduce_add_sync(0xffffffffu, cb);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const unsigned have = __ballot_sync(0xffffffffu, tok[j] >= 0);
      const unsigned fresh = __ballot_sync(0xffffffffu, tok[j] >= c);
      if (tok[j] >= 0) {
        const int e = at + __popc(have & below);
        uint32_t row = 0xffffffffu;
        if (unsigned(pg[j]) < unsigned(P.num_pages))
          row = uint32_t(pg[j]) * uint32_t(P.page_rows) +
                uint32_t(unsigned(tok[j]) % unsigned(P.page)) * uint32_t(P.Hkv);
        else
          atomicOr(P.err, SA_ERRBIT_RANGE);
        list[e] = make_uint2(row, uint32_t(tok[j]));
        place[e] = from + 32 * j;
        const int m = am + __popc(fresh & below);
        if (tok[j] >= c && m < n) members[m] = make_int4(e, from + 32 * j, 0, tok[j]);
      }
      at += __popc(have);
      am += __popc(fresh);
    }
  }
  // sigma names each token once, else the rows of some are left as they were
  if (found != n && tid == 0) atomicOr(P.err, SA_ERRBIT_RANGE);
  found = min(found, n);
  __syncthreads();
  for (int m = tid; m < found; m += kThreads) {
    const int4 x = members[m];
    int lo = max(0, x.x - P.half), hi = x.x;  // first entry with place >= q - h
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (place[mid] >= x.y - P.half) hi = mid; else lo = mid + 1;
    }
    int lo2 = x.x, hi2 = int(min((long long)entries - 1, (long long)x.x + P.half));  // last with place <= q + h
    while (lo2 < hi2) {
      const int mid = (lo2 + hi2 + 1) >> 1;
      if ((long long)place[mid] <= (long long)x.y + P.half) lo2 = mid; else hi2 = mid - 1;
    }
    members[m] = make_int4(lo, lo2, q0 + x.w - c, x.w);
  }
  __syncthreads();
  // the tiles' chunks, summed
  int32_t* chunks = P.order.chunks + q0 + b;
  const int tiles = (found + P.Bt - 1) / P.Bt;
  int sum = 0;
  for (int g0 = 0; g0 < tiles; g0 += kThreads) {
    const int g = g0 + tid;
    int x = 0;
    if (g < tiles) {
      const int first = g * P.Bt, last = min(found, first + P.Bt) - 1;
      x = (members[last].y + 1 - members[first].x + kChunk - 1) / kChunk;
    }
    int in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += up;
    }
    __syncthreads();
    if (lane == 31) s_a[warp] = in;
    __syncthreads();
    const int wa = s_a[lane];
    const int off = sum + __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    sum += __reduce_add_sync(0xffffffffu, wa);
    if (g < tiles) chunks[g] = off + in - x;
  }
  if (tid == 0) {
    chunks[tiles] = sum;
    P.order.info[b] = make_int2(before, found);
  }
}

// The most requests that can be taken: each has more than row_limit tokens.
long long lists(const PagedProblem& pb, int row_limit) {
  return min((long long)pb.B, (long long)pb.T / (row_limit + 1LL));
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t paged_order_workspace_bytes(const PagedProblem& pb, int row_limit) {
  const size_t n = size_t(lists(pb, row_limit)) * size_t(pb.perm_len);
  return round256(n * 8) + round256(n * 4) + round256(size_t(pb.T) * 16) +
         round256((size_t(pb.T) + size_t(pb.B)) * 4) + round256(size_t(pb.B) * 8);
}

sa_status_t launch_paged_order(const PagedProblem& pb, int row_limit, int tile_tokens, void* workspace,
                               SaOrder* order, cudaStream_t stream) {
  const size_t n = size_t(lists(pb, row_limit)) * size_t(pb.perm_len);
  char* w = static_cast<char*>(workspace);
  order->list = reinterpret_cast<uint2*>(w);
  w += round256(n * 8);
  order->place = reinterpret_cast<int32_t*>(w);
  w += round256(n * 4);
  order->members = reinterpret_cast<int4*>(w);
  w += round256(size_t(pb.T) * 16);
  order->chunks = reinterpret_cast<int32_t*>(w);
  w += round256((size_t(pb.T) + size_t(pb.B)) * 4);
  order->info = reinterpret_cast<int2*>(w);
  order->cap = pb.perm_len;
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.perm = pb.perm;
  P.table = pb.table;
  P.q_start = pb.q_start;
  P.seq_lens = pb.seq_lens;
  P.err = pb.err;
  P.order = *order;
  P.perm_stride = pb.perm_rows == 1 ? 0 : pb.perm_len;
  P.page_rows = pb.page_stride / pb.d;
  P.T = pb.T;
  P.max_new = pb.max_new;
  P.max_pages = pb.max_pages;
  P.page = pb.page;
  P.num_pages = pb.num_pages;
  P.perm_len = pb.perm_len;
  P.half = pb.half;
  P.row_limit = row_limit;
  P.Bt = tile_tokens;
  P.Hkv = pb.Hkv;
  P.lists = int(lists(pb, row_limit));
  sa_paged_order_kernel<<<unsigned(pb.B), kThreads, 0, stream>>>(P);
  const cudaError_t ce = cudaGetLastError();
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged order launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
