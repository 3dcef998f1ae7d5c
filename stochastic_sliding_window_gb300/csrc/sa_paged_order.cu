// A request's tokens in sigma's order, for SA of many new tokens over a paged
// cache (sa_paged_members.cu, sa_paged_tiles.cu).
//
// For each request that brings many new tokens, a cluster of eight blocks
// passes over its row of sigma, an eighth each, and keeps, in order, the entries
// that name a token there is (sigma[q] < length): the list, with each token's
// row in the caches.  Beside it stand, for every 32 places of sigma, which of
// them are in the list and how many are before: rank(q), the list entries at
// places below q, is then one 8-byte load and a population count.  The new
// tokens in the list are the members; a member at place q has the window
// |q' - q| <= h, the list entries rank(q - h) to rank(q + h + 1) - 1.  Last, the
// tiles' key chunks are summed, which is what the tile kernel's schedule needs.
//
// Bound by latency, not by its 4 bytes per place read and 8 per token written:
// sigma, the block table and the ranks one after the other, two cluster
// barriers, and the launch.  A block holds up to 4096 places of its eighth in
// registers between the count and the writing; longer rows of sigma are read a
// second time.  Two requests of 1024 new tokens, 32768 places: 38 us of 180 for
// the gated call with one block per request, whose members were placed by
// binary searches; then the call took 140, with the order found beside the SWA
// tiles.
#include "sa_internal.h"

#include <cstring>

namespace sa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 4;     // places of sigma per thread and round
constexpr int kCluster = 8;  // blocks per request
constexpr int kChunk = 128;

struct Params {
  const int32_t* perm;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_lens;
  int32_t* err;
  SaOrder order;
  uint2* words;  // [lists][cap / 32] of each 32 places: which are in the list, entries before them
  int2* groups;  // SaOrder's
  int2* mark;    // [T] members in sigma's order, a request's from q_start on: place, position
  long long perm_stride, page_rows;
  int T, max_new, max_pages, page, num_pages, perm_len, half, row_limit, Bt, Hkv, lists, beside;
};

__device__ __forceinline__ int new_tokens(const Params& P, int b, int* len) {
  const int q0 = P.q_start[b], q1 = P.q_start[b + 1];
  *len = P.seq_lens[b];
  const int n = q1 - q0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= P.T && n <= P.max_new && n <= *len &&
                  (long long)*len <= (long long)P.max_pages * P.page && *len <= P.perm_len;
  return ok && paged_sa_tiled(n, *len, P.half, P.row_limit) ? n : 0;
}

__device__ __forceinline__ void cluster_sync() {  // also for what its blocks wrote to memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory of block `rank` of the cluster at the place of `p` here.
__device__ __forceinline__ int2 load_peer(const int2* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  int2 v;
  asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void order_request(const Params& P) {
  __shared__ int s_a[kWarps], s_b[kWarps];
  __shared__ int2 s_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
  int len;
  int n = new_tokens(P, b, &len);
  // list number: the requests before this one that are taken too
  int before = 0, other;
  for (int i = tid; i < b; i += kThreads) before += new_tokens(P, i, &other) > 0;
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) s_a[warp] = before;
  __syncthreads();
  before = __reduce_add_sync(0xffffffffu, s_a[lane]);
  if (before >= P.lists && n > 0) {  // only where requests claim the same rows
    if (tid == 0) atomicOr(P.err, SA_ERRBIT_RANGE);
    n = 0;
  }
  const bool by_members = P.order.group > 0 && paged_sa_members(n, P.Bt, P.perm_len, P.half);
  if (P.order.group > 0 && rank == 0) {
    const int q0 = P.q_start[b], q1 = P.q_start[b + 1];
    if (q0 >= 0 && q1 >= q0 && q1 <= P.T) {
      const int base = q0 / P.order.group + b, end = q1 / P.order.group + b;
      for (int s = base + tid; s <= end; s += kThreads)
        P.groups[s] = by_members && (long long)(s - base) * P.order.group < n ? make_int2(b, s - base) : make_int2(-1, 0);
    }
  }
  if (n == 0) {  // (so for every block of the cluster)
    if (tid == 0 && rank == 0) P.order.info[b] = make_int4(before, 0, 0, 0);
    return;
  }
  const int q0 = P.q_start[b], c = len - n;
  uint2* list = P.order.list + (long long)before * P.order.cap;
  uint2* words = P.words + (long long)before * ((P.order.cap + 31) / 32);
  int2* mark = P.mark + q0;
  const int32_t* sigma = P.perm + (long long)b * P.perm_stride;
  const int32_t* table = P.table + (long long)b * P.max_pages;
  const unsigned below = (1u << lane) - 1u;
  // this block's places, in rounds of kThreads kEach; a warp takes 32 kEach that follow each other
  const int share = ((P.perm_len - 1) / (kCluster * 32) + 1) * 32;
  const long long first = (long long)rank * share;
  const int begin = int(min(first, (long long)P.perm_len));
  const int end = int(min(first + share, (long long)P.perm_len));
  int tok[kEach], pg[kEach];
  auto load = [&](int base, bool report) {  // places `base` + .. of a round
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const long long q = (long long)base + warp * (32 * kEach) + 32 * j + lane;
      tok[j] = q < end ? sigma[q] : -1;
      if (q < end && unsigned(tok[j]) >= unsigned(P.perm_len)) {
        if (report) atomicOr(P.err, SA_ERRBIT_RANGE);
        tok[j] = -1;
      }
      if (tok[j] >= len) tok[j] = -1;
    }
  };
  auto pages = [&]() {
#pragma unroll
    for (int j = 0; j < kEach; ++j) pg[j] = tok[j] >= 0 ? table[unsigned(tok[j]) / unsigned(P.page)] : 0;
  };
  const bool once = end - begin <= kThreads * kEach;
  int count = 0, mine = 0;  // this warp's entries and members
  long long next = begin;
  do {
    load(int(next), true);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      count += __popc(__ballot_sync(0xffffffffu, tok[j] >= 0));
      mine += __popc(__ballot_sync(0xffffffffu, tok[j] >= c));
    }
    next += kThreads * kEach;
  } while (next < end);
  if (once) pages();
  __syncthreads();  // s_a has been read
  if (lane == 0) {
    s_a[warp] = count;
    s_b[warp] = mine;
  }
  __syncthreads();
  if (warp == 0) {
    const int x = __reduce_add_sync(0xffffffffu, s_a[lane]), y = __reduce_add_sync(0xffffffffu, s_b[lane]);
    if (lane == 0) s_total = make_int2(x, y);
  }
  cluster_sync();
  const int2 peer = lane < kCluster ? load_peer(&s_total, lane) : make_int2(0, 0);
  const int entries = __reduce_add_sync(0xffffffffu, peer.x);
  const int members = __reduce_add_sync(0xffffffffu, peer.y);
  int at0 = __reduce_add_sync(0xffffffffu, lane < rank ? peer.x : 0);
  int am0 = __reduce_add_sync(0xffffffffu, lane < rank ? peer.y : 0);
  next = begin;
  do {
    const int base = int(next);
    if (!once) {
      load(base, false);
      pages();
      count = mine = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        count += __popc(__ballot_sync(0xffffffffu, tok[j] >= 0));
        mine += __popc(__ballot_sync(0xffffffffu, tok[j] >= c));
      }
      __syncthreads();  // the last round's sums are read
      if (lane == 0) {
        s_a[warp] = count;
        s_b[warp] = mine;
      }
      __syncthreads();
    }
    const int ca = s_a[lane], cb = s_b[lane];
    int at = at0 + __reduce_add_sync(0xffffffffu, lane < warp ? ca : 0);
    int am = am0 + __reduce_add_sync(0xffffffffu, lane < warp ? cb : 0);
    at0 += __reduce_add_sync(0xffffffffu, ca);
    am0 += __reduce_add_sync(0xffffffffu, cb);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const long long q32 = (long long)base + warp * (32 * kEach) + 32 * j;
      const unsigned have = __ballot_sync(0xffffffffu, tok[j] >= 0);
      const unsigned fresh = __ballot_sync(0xffffffffu, tok[j] >= c);
      if (lane == 0 && q32 < end) words[q32 >> 5] = make_uint2(have, uint32_t(at));
      if (tok[j] >= 0) {
        uint32_t row = 0xffffffffu;
        if (unsigned(pg[j]) < unsigned(P.num_pages))
          row = uint32_t(pg[j]) * uint32_t(P.page_rows) +
                uint32_t(unsigned(tok[j]) % unsigned(P.page)) * uint32_t(P.Hkv);
        else
          atomicOr(P.err, SA_ERRBIT_RANGE);
        list[at + __popc(have & below)] = make_uint2(row, uint32_t(tok[j]));
        const int m = am + __popc(fresh & below);
        if (tok[j] >= c && m < n) mark[m] = make_int2(int(q32) + lane, tok[j]);
      }
      at += __popc(have);
      am += __popc(fresh);
    }
    next += kThreads * kEach;
  } while (next < end);
  // sigma names each token once, else the rows of some are left as they were
  if (members != n && tid == 0 && rank == 0) atomicOr(P.err, SA_ERRBIT_RANGE);
  const int found = min(members, n);
  cluster_sync();  // (also: nobody exits before its s_total is read)
  auto entries_below = [&](long long q) {
    if (q >= P.perm_len) return entries;
    const uint2 w = words[q >> 5];
    return int(w.y) + __popc(w.x & ((1u << (q & 31)) - 1u));
  };
  auto window_first = [&](int q) { return entries_below(max(0, q - P.half)); };
  auto window_last = [&](int q) { return entries_below((long long)q + P.half + 1) - 1; };
  for (int m = rank * kThreads + tid; m < found; m += kCluster * kThreads) {
    const int2 x = mark[m];
    P.order.members[q0 + m] = make_int4(window_first(x.x), window_last(x.x), q0 + x.y - c, x.y);
  }
  if (rank != kCluster - 1) return;
  // the tiles' chunks, summed
  int32_t* chunks = P.order.chunks + q0 + b;
  const int tiles = (found + P.Bt - 1) / P.Bt;
  int sum = 0;
  for (int g0 = 0; g0 < tiles; g0 += kThreads) {
    const int g = g0 + tid;
    int x = 0;
    if (g < tiles) {
      const int m0 = g * P.Bt, m1 = min(found, m0 + P.Bt) - 1;
      x = (window_last(mark[m1].x) - window_first(mark[m0].x) + kChunk) / kChunk;
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
    P.order.info[b] = make_int4(before, by_members ? 0 : found, by_members ? found : 0, 0);
  }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    sa_paged_order_kernel(const __grid_constant__ Params P) {
  if (P.beside) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else {
    begin_after();
  }
  order_request(P);
  end_beside();  // (the SWA tiles)
}

// The most requests that can be taken: each has more than row_limit tokens.
long long lists(const PagedProblem& pb, int row_limit) {
  return min((long long)pb.B, (long long)pb.T / (row_limit + 1LL));
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t word_bytes(const PagedProblem& pb, int row_limit) {
  return round256(size_t(lists(pb, row_limit)) * ((size_t(pb.perm_len) + 31) / 32) * 8);
}

}  // namespace

size_t paged_order_workspace_bytes(const PagedProblem& pb, int row_limit) {
  const size_t n = size_t(lists(pb, row_limit)) * size_t(pb.perm_len);
  return round256(n * 8) + word_bytes(pb, row_limit) + round256(size_t(pb.T) * 24) +
         round256((size_t(pb.T) + size_t(pb.B)) * 4) + round256(size_t(pb.B) * 16) +
         round256(paged_member_groups(pb) * 8);
}

sa_status_t launch_paged_order(const PagedProblem& pb, int row_limit, int tile_tokens, void* workspace,
                               int group, SaOrder* order, bool beside, cudaStream_t stream) {
  const size_t n = size_t(lists(pb, row_limit)) * size_t(pb.perm_len);
  char* w = static_cast<char*>(workspace);
  order->list = reinterpret_cast<uint2*>(w);
  w += round256(n * 8);
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.words = reinterpret_cast<uint2*>(w);
  w += word_bytes(pb, row_limit);
  order->members = reinterpret_cast<int4*>(w);
  P.mark = reinterpret_cast<int2*>(w + size_t(pb.T) * 16);
  w += round256(size_t(pb.T) * 24);
  order->chunks = reinterpret_cast<int32_t*>(w);
  w += round256((size_t(pb.T) + size_t(pb.B)) * 4);
  order->info = reinterpret_cast<int4*>(w);
  w += round256(size_t(pb.B) * 16);
  P.groups = reinterpret_cast<int2*>(w);
  order->groups = P.groups;
  order->group = group;
  order->cap = pb.perm_len;
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
  P.beside = beside;
  const cudaError_t ce =
      launch_kernel(sa_paged_order_kernel, dim3(unsigned(pb.B) * kCluster), kThreads, 0, stream, P);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged order launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
