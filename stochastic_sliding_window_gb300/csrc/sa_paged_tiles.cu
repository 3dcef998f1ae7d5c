// Tile kernel of the paged-cache attention for requests that bring many new
// tokens, on the 5th-generation tensor cores: SWA (any window, full causal
// among them), and SA over the order that sa_paged_order.cu makes of a
// request's tokens.
//
// Mathematics.  A tile is up to 256 query rows that share a kv head -- the g
// query heads of Bt = floor(256 / g) consecutive new tokens, row r = t g + j
// -- as two halves of M = 128.  Its keys, positions max(0, p_first - w + 1)
// to p_last, are cut into chunks of 128.  One pass with an online softmax:
//   S = Q K^T (TMEM),  P = 2^(scale log2(e) S - ref),  O += P V (TMEM),
// where ref is the row's running maximum, raised (and O and the sum rescaled)
// only when a chunk exceeds it by more than 2^8.  P is rounded to bf16, the
// operand type of the second product; sums and O are fp32.
//
// What bounds it: the tensor cores, 4 d multiply-adds per row and key.  A half's
// softmax must run beside the other half's MMAs, and a half's two MMAs of a
// chunk beside its own softmax; so a chunk's scores are taken in two parts of
// 64 keys, each with its own barriers, and P V of one part and Q K of the next
// chunk's part run while the other part is in its softmax.  Masks are applied
// only in the parts that a window's end crosses.
//
// Measured (2048 new tokens at the end of 32768, every key in the window, 32 q
// heads on 8 kv heads, d = 128: 1.06 PFLOP; 568 us at cuBLAS's burst rate):
//   one MMA warp, softmax over 128 columns at once         857-880 us (one producer)
//   64-key parts, two MMA warps, softmax loop unrolled         935 us
//   the same, the loop over the parts not unrolled         854-875 us, two producers and a shorter start 745-805
//   S of all 128 keys by one MMA of N = 128, P in parts        937 us
//   the halves taking turns, 16 softmax warps in pairs         882 us
// The unrolled softmax loop does not fit the instruction cache beside the
// other roles' code.  What is left between 770 and the tensor cores' time is
// the chain S -> softmax -> P V -> S of a part (1900 cycles, of which 640 are
// the MMAs of one half).
//
// SA.  In sigma's order -- the request's tokens listed by their place in sigma,
// those that do not exist yet left out -- every row's window is a run of
// consecutive entries, and the new tokens (members) that follow each other in
// the list share most of theirs.  So a tile is Bt members that follow each
// other, its keys the list from the first one's window to the last one's, and
// the rest is as for SWA, but for the causal rule among the new tokens
// themselves (older keys precede every row) and rows that TMA cannot box.
// (Members far apart share little: sa_paged_members.cu takes those requests.)
//
// Split.  One block per SM.  All chunks of all tiles, laid end to end
// (request, kv head, tile, chunk), are cut into equal runs, one per block, so
// ragged batches balance; each block finds its run by a scan over the
// requests' lengths.  Where tiles are long (32 chunks or more on average) a
// run may end inside a tile: both parts leave fp32 partials in the workspace
// and the join kernel merges them in order.  Else a tile belongs to the run
// it starts in.
// Measured with tiles cut from 8 chunks on instead: a mixed batch of 9 chunks a
// tile 56 us instead of 43, a gated chunk 115 instead of 114.
//
// Roles (12 warps, SA 14):
//   warps 0, 3  producers, of Q and K and of V: TMA.  A lane takes a page of the
//               chunk and loads its run of rows in two boxes of 128-byte rows,
//               the largest power of two in the run from its start and as many
//               rows up to its end, which may overlap.  (One warp for both, with
//               boxes of 64, 16, 4 and 1 rows, nine rounds of them for a ragged
//               run, took 5400 cycles a chunk where pages of 48 tokens end
//               anywhere: 78.5 us for the mixed batch against 58, and 857
//               against 815 for the long prompt.)
//               SA: warps 0, 3, 12 and 13, rows from anywhere by cp.async
//   warps 1, 2  the elected lane issues the MMAs of half 0, of half 1; warp 1
//               owns TMEM
//   warps 4-11  softmax and epilogue: warp 4 + 4 h + i takes rows 32 i .. of
//               half h, a row a thread, 64 columns at a time
// TMEM (512 columns): S of half h in [128 h, +128), each part's overwritten by
// its bf16 P in the first 32 of its 64 columns; O of half h in [256 + d h, +d).
// Order of the MMAs of a half: for each chunk c of a tile and part u, O += P V of
// part u of chunk c - 1, then S = Q K of part u of chunk c -- one thread, one
// tensor pipe, which runs MMAs in the order of their issue, so S may overwrite
// the P that the MMA before it reads.
// Every wait is bounded (SA_ERRBIT_TIMEOUT).
#include "sa_internal.h"
#include "sa_tc_common.cuh"

#include <cstring>

namespace sa {
namespace ptile {

using namespace tcc;

constexpr int kThreads = 384;
constexpr int kSaThreads = 448;     // SA: two more producers
constexpr int kMmaWarp = 1;
constexpr int kFirstSoftmaxWarp = 4;
constexpr int kRows = 2 * kBM;
constexpr int kKC = 128;            // keys per chunk: of one load
constexpr int kSub = 64;            // keys per part of a chunk: of one softmax step
constexpr float kRescaleLog2 = 8.f;
constexpr int kCutChunks = 32;      // tiles this long on average may be cut
constexpr int kBoxes = 7;           // boxes of up to 64 rows
constexpr uint32_t kMaxSmem = 232448;

struct Desc {  // per block: the tile that starts in its run and ends beyond it
  int valid, c1, t0, rows, kvh, pad;
};

struct Params {
  CUtensorMap tq;           // q [T, Hq, D] in boxes of a tile's rows
  CUtensorMap tk[kBoxes], tv[kBoxes]; // caches [pages, page, Hkv, D] in boxes of 2^i rows of a page
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_lens;
  const float* gate;      // [T, Hq] logits: fp32 gated rows into part_out
  __nv_bfloat16* out;
  float* part_out;        // [T, Hq, D], with gate
  float* part;            // partials [blocks][2][D/4][256] float4, then [blocks][2][256] (m, l)
  Desc* desc;             // nullptr: tiles are never cut
  int32_t* err;
  int B, T, max_new, row_limit, Hq, Hkv, g, Bt, page, num_pages, max_pages, w;
  uint32_t off_k, off_v, off_bad, off_seg, off_bar;
  float scale_log2;
  long long timeout_cycles;
  // SA: what sa_paged_order.cu made of sigma, and the rows that it numbers
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_stride;
  SaOrder order;
  const float* swa_part;  // fp32 [T, Hq, D], added to the rows; nullptr: none
};

// Barriers (8 bytes each).  A phase is one use; chunks and tiles are counted
// over the block's whole run.
template <int NS>
struct Bars {
  enum : uint32_t {
    kQfull = 0,           // Q rows of tile x landed
    kQfree = 1,           // both halves' last S MMA of tile x done
    kKfull = 2,           // [NS] K rows of chunk c landed
    kKfree = kKfull + NS, // [NS] both S MMAs of chunk c done
    kVfull = kKfree + NS, // [NS]
    kVfree = kVfull + NS, // [NS] both O MMAs of chunk c done
    kSfull = kVfree + NS, // [2 h + u] S of the half's part u of a chunk in TMEM
    kPfull = kSfull + 4,  // [2 h + u] its P written (4 warps)
    kPVdone = kPfull + 4, // [2 h + u] its O MMA done
    kOfree = kPVdone + 4, // [h] the half's O of tile x read out (4 warps)
    kSegFull = kOfree + 2, // [4] the entry of tile x written
    kSegFree = kSegFull + 4, // [4] and read by every softmax warp and the MMA warp
    kDrain = kSegFree + 4, // [h]
    kNum = kDrain + 2,
  };
};

__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// MMAs and commits of the warp's elected lane: every lane computes the
// operands, so that they are warp-uniform values.  kAdd: D is added to.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}
// A from TMEM (P), B from shared memory (V), D in TMEM (O).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The same 32 bytes where the address is known to be 16-byte aligned only.
__device__ __forceinline__ void st_global_2v4(void* p, const uint32_t (&r)[8]) {
  reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ void tma_box4(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ schedule

// sum_{i=0}^{n-1} floor((a i + b) / m), a, b >= 0: lattice points under a line,
// counted by Euclid's descent -- take out the integer parts of slope and
// offset, then exchange the axes.
// (a n + b fits 32 bits: 64-bit divisions take several times as long, and a
// block does nothing else until its run is found.)
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long s = 0;
  while (n > 0) {
    s += (long long)n * (n - 1) / 2 * (a / m) + (long long)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t t = a;
    a = m;
    m = t;
  }
  return s;
}

// a / b, both >= 0: in 32 bits where that is enough.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)(uint32_t(a) / uint32_t(b)) : a / b;
}

// SA: n counts the request's members (its new tokens in sigma's order) and its
// keys are entries of the list of its tokens in that order.
struct Request {
  int q0, n, len, b;
};
template <bool SA>
__device__ __forceinline__ Request load_request(const Params& P, int b, bool report) {
  Request r;
  r.b = b;
  r.q0 = P.q_start[b];
  const int q1 = P.q_start[b + 1];
  r.len = P.seq_lens[b];
  if (SA) {  // (checked where the order was made; 0 members where it was not)
    r.n = P.order.info[b].y;
    return r;
  }
  r.n = q1 - r.q0;
  const bool ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= P.T && r.n <= P.max_new && r.n <= r.len &&
                  (long long)r.len <= (long long)P.max_pages * P.page;
  if (!ok) {
    if (report && q1 != r.q0) atomicOr(P.err, SA_ERRBIT_RANGE);
    r.n = 0;
  }
  if (r.n <= P.row_limit) r.n = 0;
  return r;
}

// First key and the key after the last of tile `grp` of a request.
template <bool SA>
__device__ __forceinline__ int tile_lo(const Params& P, const Request& r, int grp) {
  if (SA) return P.order.members[r.q0 + grp * P.Bt].x;
  return max(0, r.len - r.n + grp * P.Bt - P.w + 1);
}
template <bool SA>
__device__ __forceinline__ int tile_hi(const Params& P, const Request& r, int grp) {
  if (SA) return P.order.members[r.q0 + min(r.n, (grp + 1) * P.Bt) - 1].y + 1;
  return r.len - r.n + min(r.n, (grp + 1) * P.Bt);
}
__device__ __forceinline__ int num_tiles(const Params& P, const Request& r) {
  return (r.n + P.Bt - 1) / P.Bt;
}
// Chunks of the request's first `k` tiles (of one kv head).
template <bool SA>
__device__ __forceinline__ long long chunks_before(const Params& P, const Request& r, int k);
template <bool SA>
__device__ __forceinline__ int tile_chunks(const Params& P, const Request& r, int grp) {
  if (SA) return int(chunks_before<SA>(P, r, grp + 1) - chunks_before<SA>(P, r, grp));
  return (tile_hi<SA>(P, r, grp) - tile_lo<SA>(P, r, grp) + kKC - 1) / kKC;
}
template <bool SA>
__device__ __forceinline__ long long chunks_before(const Params& P, const Request& r, int k) {
  if (SA) return P.order.chunks[r.q0 + r.b + k];
  const int nt = num_tiles(P, r);
  long long s = 0;
  if (k == nt && k > 0) {  // the last tile may be short
    --k;
    s = tile_chunks<SA>(P, r, k);
  }
  // tiles whose window reaches the first key: hi = c + (i + 1) Bt keys, at most
  // the request's length (a full tile ends there or before)
  const int c = r.len - r.n;
  const int reach = P.w - 1 - c;  // largest first-token offset with lo = 0
  const int ka = reach < 0 ? 0 : min(reach / P.Bt + 1, k);
  s += floor_sum(uint32_t(ka), kKC, uint32_t(P.Bt), uint32_t(c) + uint32_t(P.Bt + kKC - 1));
  s += (k - ka) * (((long long)P.Bt + P.w - 1 + kKC - 1) / kKC);
  return s;
}

// A block's run of chunks and where it starts; found once by warp 0.
struct Start {
  long long begin, end, tile_off;  // tile_off: chunks of the first tile before `begin`
  int b, kvh, grp, cut;
};

// One tile's part in the run.
struct Seg {
  Request r;
  int b, kvh, grp;
  int c0, c1, nch;  // chunks [c0, c1) of nch
  long long pos;    // run position of chunk c0
};

// What the other roles need of it, in shared memory (slot: tile number mod 4).
struct Shared {
  int t0, nt, pos0, lo;  // first token's row, tokens, first position, first key (SA:
                         // t0 is the first member's index, pos0 unused)
  int kvh, c0, c1, nch;
  int a[2], b[2];        // each half's chunks [a, b) of [c0, c1): those its rows have keys in
  int more;              // another tile part follows
  int join;              // last block that holds a part of a tile cut here
  int pad[2];
};

struct Cursor {
  long long pos, end;
  Request r;
  int b, kvh, grp, off, cut, nt;
  bool done;
};
template <bool SA>
__device__ __forceinline__ Cursor make_cursor(const Params& P, const Start& s) {
  Cursor c;
  c.pos = s.begin;
  c.end = s.end;
  c.b = s.b;
  c.kvh = s.kvh;
  c.grp = s.grp;
  c.off = int(s.tile_off);
  c.cut = s.cut;
  c.done = s.begin >= s.end;
  c.nt = 0;
  if (!c.done) {
    c.r = load_request<SA>(P, c.b, false);
    c.nt = num_tiles(P, c.r);
  }
  return c;
}
template <bool SA>
__device__ __forceinline__ void next_tile(const Params& P, Cursor& c) {
  c.off = 0;
  if (++c.grp < c.nt) return;
  c.grp = 0;
  if (++c.kvh < P.Hkv) return;
  c.kvh = 0;
  do {
    if (++c.b >= P.B) {
      c.done = true;
      return;
    }
    c.r = load_request<SA>(P, c.b, false);
  } while (c.r.n == 0);
  c.nt = num_tiles(P, c.r);
}
// Whether a tile part follows the one that next_seg returned last.
__device__ __forceinline__ bool more_segs(const Cursor& c) { return !c.done && c.pos < c.end; }
// The next tile part of the run; false at its end.
template <bool SA>
__device__ __forceinline__ bool next_seg(const Params& P, Cursor& c, Seg& s) {
  if (c.done) return false;
  if (!c.cut && c.off != 0) {  // the tile cut here is the previous block's
    c.pos += tile_chunks<SA>(P, c.r, c.grp) - c.off;
    next_tile<SA>(P, c);
    if (c.done) return false;
  }
  if (c.pos >= c.end) return false;
  s.r = c.r;
  s.b = c.b;
  s.kvh = c.kvh;
  s.grp = c.grp;
  s.nch = tile_chunks<SA>(P, c.r, c.grp);
  s.c0 = c.off;
  s.c1 = c.cut ? int(min((long long)s.nch, c.off + (c.end - c.pos))) : s.nch;
  s.pos = c.pos;
  c.pos += s.c1 - s.c0;
  if (s.c1 == s.nch) {
    next_tile<SA>(P, c);
  } else {
    c.done = true;  // the run ends inside this tile
  }
  return true;
}

// Warp 0: this block's run (collective over its lanes).
template <bool SA>
__device__ Start find_start(const Params& P) {
  const int lane = threadIdx.x & 31;
  long long total = 0, tiles = 0, first = 0;  // first: chunks of request `lane`
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    if (b0 + lane < P.B) {
      const Request r = load_request<SA>(P, b0 + lane, blockIdx.x == 0);
      if (r.n > 0) {
        const int nt = num_tiles(P, r);
        const long long x = P.Hkv * chunks_before<SA>(P, r, nt);
        if (b0 == 0) first = x;
        total += x;
        tiles += (long long)P.Hkv * nt;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  }
  Start s;
  const long long per = quotient(total + gridDim.x - 1, gridDim.x);
  s.cut = P.desc != nullptr && total >= tiles * kCutChunks;
  s.begin = per * blockIdx.x;
  s.end = min(total, s.begin + per);
  s.tile_off = 0;
  s.b = s.kvh = s.grp = 0;
  if (s.begin >= s.end) {
    s.begin = s.end = 0;
    return s;
  }
  long long before = 0;
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    long long x = b0 == 0 ? first : 0;
    if (b0 > 0 && b0 + lane < P.B) {
      const Request r = load_request<SA>(P, b0 + lane, false);
      if (r.n > 0) x = P.Hkv * chunks_before<SA>(P, r, num_tiles(P, r));
    }
    long long sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += a;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > s.begin);
    if (hit != 0u) {
      const int src = __ffs(hit) - 1;
      s.b = b0 + src;
      long long rel = s.begin - (before + __shfl_sync(0xffffffffu, sum - x, src));
      const Request r = load_request<SA>(P, s.b, false);
      const int nt = num_tiles(P, r);
      const long long per_head = chunks_before<SA>(P, r, nt);
      s.kvh = int(quotient(rel, per_head));
      rel -= s.kvh * per_head;
      // the last tile that starts at or before rel: 32 candidates at a time
      int lo = 0, hi = nt;  // lo starts at or before it, hi does not
      long long at = 0;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int k = min(lo + lane * step, hi);
        const long long v = k < hi ? chunks_before<SA>(P, r, k) : rel + 1;
        const unsigned low = __ballot_sync(0xffffffffu, v <= rel);
        const int last = 31 - __clz(int(low));  // (lane 0 is lo itself)
        at = __shfl_sync(0xffffffffu, v, last);
        hi = min(hi, lo + (last + 1) * step);
        lo = lo + last * step;
      }
      s.grp = lo;
      s.tile_off = rel - at;
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return s;
}

// ------------------------------------------------------------------ producer

// What a chunk's consumers need beside its rows (slot: chunk number mod 8).
// Its slot is written again for chunk n + 8, once the S MMAs of chunk n + 7 - NS
// are done, NS <= 4: they follow every reading of chunk n's.
constexpr int kKeySlots = 8;
struct Keys {
  uint32_t bad[4];  // bit j: key j of the chunk lies in a bad page
  int good;         // some key of the tile part, up to this chunk, does not
  int steps;        // 16-key steps that hold keys
  int pad[2];
};
struct SaKeys : Keys {
  uint32_t fresh[4];  // bit j: key j is one of the request's new tokens
  int toks[kKC];
};
template <bool SA>
struct KeysOf { using T = Keys; };
template <>
struct KeysOf<true> { using T = SaKeys; };

// Rows that load_run moves for a run of `len` rows, 1 <= len <= 128.
__device__ __forceinline__ int run_rows(int len) {
  const int step = 1 << min(kBoxes - 1, 31 - __clz(len));
  return len == step ? step : 2 * step;
}
// A run of `len` rows of a page from row `in` to rows r .. of a stage: a box of
// 2^i <= len rows from its start and one up to its end, which may overlap.
template <int D>
__device__ __forceinline__ void load_run(const CUtensorMap* maps, uint32_t dst, int r, int len, int in,
                                         int page, int kvh, uint32_t bar) {
  const int i = min(kBoxes - 1, 31 - __clz(len)), rest = len - (1 << i);
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb)
    tma_box4(dst + uint32_t(kb * (kKC * 128) + r * 128), maps + i, kb * 64, kvh, in, page, bar);
  if (rest > 0) {
#pragma unroll
    for (int kb = 0; kb < D / 64; ++kb)
      tma_box4(dst + uint32_t(kb * (kKC * 128) + (r + rest) * 128), maps + i, kb * 64, kvh, in + rest, page, bar);
  }
}

// Warp 0 brings Q, K and what the other roles need to know, warp 3 brings V.
template <int D, int NS>
__device__ void producer_role(const Params& P, const Start& start, const Cursor& first, const Seg& first_seg, bool have,
                              uint8_t* smem, uint32_t sbase, uint32_t bars, volatile int* abort_flag) {
  using BR = Bars<NS>;
  constexpr uint32_t kTile = kKC * D * 2;
  const int lane = threadIdx.x & 31;
  const bool is_v = threadIdx.x >= 32;
  const uint32_t full = is_v ? BR::kVfull : BR::kKfull, free = is_v ? BR::kVfree : BR::kKfree;
  const CUtensorMap* maps = is_v ? P.tv : P.tk;
  const uint32_t stages = sbase + (is_v ? P.off_v : P.off_k);
  auto wwait = [&](uint32_t bar, uint32_t parity) {
    const bool ok = bounded_wait(bars + 8 * bar, parity & 1u, P.timeout_cycles, P.err, abort_flag);
    return __all_sync(0xffffffffu, ok);
  };
  Cursor cur = first;
  Seg s = first_seg;
  int n = 0, x = 0;    // chunks and tiles so far
  int nq = 0, nk = 0;  // Q loads and loads of this warp's stages begun
  bool ok = true;
  for (; ok && have; ++x) {
    const bool more = more_segs(cur);
    const int lo = tile_lo<false>(P, s.r, s.grp), hi = tile_hi<false>(P, s.r, s.grp);
    const int i0 = s.grp * P.Bt;
    const int32_t* table = P.table + (long long)s.b * P.max_pages;
    // page of table column `col` (columns hi and on: not looked at)
    const int last_col = int(unsigned(hi - 1) / unsigned(P.page));
    auto page_at = [&](int col) { return col <= last_col ? table[col] : -1; };
    int page = page_at(int(unsigned(lo + s.c0 * kKC) / unsigned(P.page)) + lane);
    if (!is_v) {
      if (x > 3 && !(ok = wwait(BR::kSegFree + (x & 3), uint32_t((x >> 2) - 1)))) break;
      if (lane == 0) {
        Shared* sh = reinterpret_cast<Shared*>(smem + P.off_seg) + (x & 3);
        sh->t0 = s.r.q0 + i0;
        sh->nt = min(P.Bt, s.r.n - i0);
        sh->pos0 = s.r.len - s.r.n + i0;
        sh->lo = lo;
        sh->kvh = s.kvh;
        sh->c0 = s.c0;
        sh->c1 = s.c1;
        sh->nch = s.nch;
        sh->a[0] = sh->a[1] = sh->b[1] = s.c0;
        sh->b[0] = s.c1;
        if (min(P.Bt, s.r.n - i0) * P.g > kBM) sh->b[1] = s.c1;  // else half 1 has no rows
        sh->more = more;
        // a run that ends inside a tile is a full one
        sh->join = s.c1 < s.nch && s.c0 == 0 ? int((s.pos + s.nch - 1) / (start.end - start.begin)) : -1;
        mbar_arrive(bars + 8 * (BR::kSegFull + (x & 3)));
      }
      if (x > 0 && !(ok = wwait(BR::kQfree, uint32_t(x - 1)))) break;
      if (lane == 0) {
        // rows of other tokens behind the tile's are computed and not written
        mbar_arrive_expect_tx(bars + 8 * BR::kQfull, uint32_t(P.Bt * P.g) * D * 2);
        for (int kb = 0; kb < D / 64; ++kb)
          tma_box3(sbase + kb * (kRows * 128), &P.tq, kb * 64, s.kvh * P.g, s.r.q0 + i0, bars + 8 * BR::kQfull);
      }
      ++nq;
    }
    // a good key's place, which stands in for keys of bad pages (whose weight is 0)
    int gpage = 0, gin = 0;
    bool good = false;
    for (int c = s.c0; c < s.c1; ++c, ++n) {
      const int st = n % NS;
      const int j0 = lo + c * kKC, j1 = min(hi, j0 + kKC);
      const int col0 = int(unsigned(j0) / unsigned(P.page)), cols = int(unsigned(j1 - 1) / unsigned(P.page)) - col0 + 1;
      const int steps = (j1 - j0 + 15) / 16, fill = steps * 16 - (j1 - j0);
      // this lane's run of keys: those of table column col0 + i
      auto run = [&](int i, int& r, int& len, int& in) {
        const int a = max(j0, (col0 + i) * P.page);
        r = a - j0;
        len = min(j1 - a, P.page - (a - (col0 + i) * P.page));
        in = a - (col0 + i) * P.page;
      };
      // (pages of fewer than 5 tokens give some lanes more than one column)
      uint32_t bad[4] = {0, 0, 0, 0};
      bool any_bad = false;
      int last_good = -1;
      int rows = 0;  // that this lane's copies bring
      for (int i = lane; i < cols; i += 32) {
        const int pg = i < 32 ? page : table[col0 + i];
        int r, len, in;
        run(i, r, len, in);
        if (unsigned(pg) < unsigned(P.num_pages)) {
          last_good = i;
          rows += run_rows(len);
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) bad[w] |= band_bits(r, r + len - 1, w * 32);
          any_bad = true;
          rows += len;
        }
      }
      rows = __reduce_add_sync(0xffffffffu, rows);
      const unsigned fine = __ballot_sync(0xffffffffu, last_good >= 0);
      if (fine != 0u) {
        const int src = 31 - __clz(int(fine));
        const int i = __shfl_sync(0xffffffffu, last_good, src);
        int r, len;
        run(i, r, len, gin);
        gpage = i < 32 ? __shfl_sync(0xffffffffu, page, i) : table[col0 + i];
        good = true;
      }
      if (!is_v) {
        uint32_t words = 0;  // lanes 0-3: the chunk's bad keys
        if (__any_sync(0xffffffffu, any_bad)) {
          if (any_bad) atomicOr(P.err, SA_ERRBIT_RANGE);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t v = __reduce_or_sync(0xffffffffu, bad[w]);
            if (lane == w) words = v;
          }
        }
        Keys* keys = reinterpret_cast<Keys*>(smem + P.off_bad) + (n % kKeySlots);
        if (lane < 4) keys->bad[lane] = words;
        if (lane == 0) {
          keys->good = good;
          keys->steps = steps;
        }
      }
      if (n >= NS && !(ok = wwait(free + st, uint32_t(n / NS - 1)))) break;
      __syncwarp();
      // K rows past the last key keep what they held: their scores are masked.
      // The last step's V rows past it are copies of a real row, since weights of
      // 0 times what happens to be there need not be 0.
      const uint32_t bar = bars + 8 * (full + st), dst = stages + uint32_t(st) * kTile;
      if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(rows + (is_v ? fill : 0)) * D * 2);
      __syncwarp();
      for (int i = lane; i < cols; i += 32) {
        const int pg = i < 32 ? page : table[col0 + i];
        int r, len, in;
        run(i, r, len, in);
        if (unsigned(pg) < unsigned(P.num_pages)) {
          load_run<D>(maps, dst, r, len, in, pg, s.kvh, bar);
        } else {
          for (int e = 0; e < len; ++e) load_run<D>(maps, dst, r + e, 1, gin, gpage, s.kvh, bar);
        }
      }
      if (is_v && lane < fill) load_run<D>(maps, dst, j1 - j0 + lane, 1, gin, gpage, s.kvh, bar);
      ++nk;
      if (c + 1 < s.c1) page = page_at(int(unsigned(j0 + kKC) / unsigned(P.page)) + lane);
    }
    have = more && next_seg<false>(P, cur, s);
  }
  // A block must not exit with copies in flight (after a failed wait nobody
  // else may be left to wait for them): each barrier's last use, bounded.
  if (lane == 0) {
    auto drain = [&](uint32_t bar, int uses) {
      if (uses == 0) return;
      const long long t0 = clock64();
      while (!mbar_try_wait(bars + 8 * bar, uint32_t(uses - 1) & 1u) && clock64() - t0 < kDrainCycles) {
      }
    };
    drain(BR::kQfull, nq);
    for (int i = 0; i < NS; ++i) drain(full + i, nk > i ? (nk - i + NS - 1) / NS : 0);
  }
  __syncwarp();
}

// SA: rows from anywhere, so cp.async by four warps.  The list's entries of a
// chunk are read one chunk ahead, one key a thread.  (A warp issues one cp.async
// in 80 cycles here: two warps made 140 us of a gated call that takes 129 with
// four, and 131 with six.)
constexpr int kSaProducers = 128;
static_assert(kSaProducers == kKC, "a key a thread");

template <int D, int NS>
__device__ void sa_producer_role(const Params& P, const Start& start, const Cursor& first, const Seg& first_seg,
                                 bool have, uint8_t* smem, uint32_t sbase, uint32_t bars,
                                 volatile int* abort_flag, volatile int* vote) {
  using BR = Bars<NS>;
  constexpr uint32_t kTile = kKC * D * 2;
  constexpr int CPR = D / 8;               // 16-byte chunks per row
  constexpr int RPP = kSaProducers / CPR;  // rows per pass
  const int lane = threadIdx.x & 31;
  // warps 0, 3, 12 and 13
  const int tid = int(threadIdx.x) - (threadIdx.x < 32 ? 0 : threadIdx.x < 128 ? 64 : 320);
  const int cc = tid % CPR, r_first = tid / CPR;
  const uint32_t col = uint32_t(cc >> 3) * (kKC * 128), c8 = uint32_t(cc & 7);
  uint32_t* srow = reinterpret_cast<uint32_t*>(smem + P.off_seg + 4 * sizeof(Shared));  // [2][128]
  int* sq = reinterpret_cast<int*>(srow + 2 * kKC);  // [256] the tile's query rows
  int step = 0;
  // every producer learns whether thread 0's wait succeeded; also orders
  // their shared-memory writes before what follows
  auto agree = [&](uint32_t bar, uint32_t parity, bool need) {
    if (tid == 0)
      vote[step & 1] = !need || bounded_wait(bars + 8 * bar, parity & 1u, P.timeout_cycles, P.err, abort_flag) ? 1 : 0;
    asm volatile("bar.sync 1, %0;" ::"n"(kSaProducers) : "memory");
    const bool ok = vote[step & 1] != 0;
    ++step;
    return ok;
  };
  const char* kbase = reinterpret_cast<const char*>(P.k) + cc * 16;
  const char* vbase = reinterpret_cast<const char*>(P.v) + cc * 16;
  // row numbers of several keys first, then their copies (the copies' asm
  // would hold the shared-memory reads back)
  auto rows_in = [&](const char* base, uint32_t dst, const uint32_t* rows) {
    constexpr int kBatch = 8;
    for (int i0 = r_first; i0 < kKC; i0 += RPP * kBatch) {
      uint32_t r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) r[u] = i0 + u * RPP < kKC ? rows[i0 + u * RPP] : 0u;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * RPP;
        if (i < kKC) {
          const int bytes = r[u] != 0xffffffffu ? 16 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           dst + uint32_t(i) * 128 + ((c8 ^ uint32_t(i & 7)) << 4)),
                       "l"(base + uint64_t(bytes ? r[u] : 0u) * (D * 2)), "r"(bytes)
                       : "memory");
        }
      }
    }
  };
  Cursor cur = first;
  Seg s = first_seg;
  int n = 0, x = 0;
  bool ok = true;
  for (; ok && have; ++x) {
    const bool more = more_segs(cur);
    const int lo = tile_lo<true>(P, s.r, s.grp), hi = tile_hi<true>(P, s.r, s.grp);
    const int m0 = s.r.q0 + s.grp * P.Bt, nt = min(P.Bt, s.r.n - s.grp * P.Bt);
    const uint2* list = P.order.list + (long long)P.order.info[s.b].x * P.order.cap;
    const int first_new = s.r.len - (P.q_start[s.b + 1] - s.r.q0);
    auto entry = [&](int c, int at) {
      const int j = lo + c * kKC + at;
      return j < hi ? list[j] : make_uint2(0xffffffffu, 0x7fffffffu);
    };
    uint2 e = entry(s.c0, tid);
    const bool entry_used = x > 3;
    if (tid == 0) {
      // each half's chunks: from its first member's window to its last one's
      int a[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h] = b[h] = s.c0;
        const int rows = min(nt * P.g, (h + 1) * kBM) - h * kBM;
        if (rows > 0) {
          const int first = P.order.members[m0 + h * kBM / P.g].x;
          const int last = P.order.members[m0 + (h * kBM + rows - 1) / P.g].y;
          a[h] = max(s.c0, (first - lo) / kKC);
          b[h] = max(a[h], min(s.c1, (last - lo) / kKC + 1));
        }
      }
      if (!entry_used || bounded_wait(bars + 8 * (BR::kSegFree + (x & 3)), uint32_t((x >> 2) - 1) & 1u,
                                      P.timeout_cycles, P.err, abort_flag)) {
        Shared* sh = reinterpret_cast<Shared*>(smem + P.off_seg) + (x & 3);
        sh->t0 = m0;
        sh->nt = nt;
        sh->pos0 = 0;
        sh->lo = lo;
        sh->kvh = s.kvh;
        sh->c0 = s.c0;
        sh->c1 = s.c1;
        sh->nch = s.nch;
        for (int h = 0; h < 2; ++h) {
          sh->a[h] = a[h];
          sh->b[h] = b[h];
        }
        sh->more = more;
        sh->join = s.c1 < s.nch && s.c0 == 0 ? int((s.pos + s.nch - 1) / (start.end - start.begin)) : -1;
        mbar_arrive(bars + 8 * (BR::kSegFull + (x & 3)));
      }
    }
    for (int t = tid; t < nt; t += kSaProducers) sq[t] = P.order.members[m0 + t].z;
    if (!(ok = agree(BR::kQfree, uint32_t(x - 1), x > 0))) break;
    {
      constexpr int kBatch = 8;
      const int rows = nt * P.g;
      for (int i0 = r_first; i0 < rows; i0 += RPP * kBatch) {
        const __nv_bfloat16* src[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = min(i0 + u * RPP, rows - 1), t = r / P.g;
          src[u] = P.q + (long long)sq[t] * P.q_stride + (s.kvh * P.g + r - t * P.g) * D + cc * 8;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint32_t r = uint32_t(i0 + u * RPP);
          if (int(r) < rows)
            cp_async16(sbase + uint32_t(cc >> 3) * (kRows * 128) + r * 128 + ((c8 ^ (r & 7)) << 4), src[u]);
        }
      }
    }
    cp_async_arrive_noinc(bars + 8 * BR::kQfull);
    for (int c = s.c0; c < s.c1; ++c, ++n) {
      const int st = n % NS;
      SaKeys* keys = reinterpret_cast<SaKeys*>(smem + P.off_bad) + (n % kKeySlots);
      uint32_t* rows = srow + (n & 1) * kKC;
      {
        const int j = lo + c * kKC + tid;
        const uint32_t bad = __ballot_sync(0xffffffffu, j < hi && e.x == 0xffffffffu);
        const uint32_t fresh = __ballot_sync(0xffffffffu, j < hi && int(e.y) >= first_new);
        rows[tid] = e.x == 0xffffffffu ? e.x : e.x + uint32_t(s.kvh);
        keys->toks[tid] = int(e.y);
        if (lane == 0) {
          keys->bad[tid >> 5] = bad;
          keys->fresh[tid >> 5] = fresh;
        }
      }
      if (tid == 0) {
        keys->good = 1;  // rows that are not there are zeros
        keys->steps = kKC / 16;
      }
      if (c + 1 < s.c1) e = entry(c + 1, tid);
      if (!(ok = agree(BR::kKfree + st, uint32_t(n / NS - 1), n >= NS))) break;
      rows_in(kbase, sbase + P.off_k + uint32_t(st) * kTile + col, rows);
      cp_async_arrive_noinc(bars + 8 * (BR::kKfull + st));
      if (tid == 0) mbar_arrive(bars + 8 * (BR::kKfull + st));  // the key words
      if (!(ok = agree(BR::kVfree + st, uint32_t(n / NS - 1), n >= NS))) break;
      rows_in(vbase, sbase + P.off_v + uint32_t(st) * kTile + col, rows);
      cp_async_arrive_noinc(bars + 8 * (BR::kVfull + st));
    }
    have = more && next_seg<true>(P, cur, s);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // own copies land before exit
}

// ------------------------------------------------------------------ MMA issue
template <int D, int NS, bool SA>
__device__ void mma_role(const Params& P, int h, bool more, const Shared* seg, const typename KeysOf<SA>::T* keys,
                         uint32_t sbase, uint32_t tmem, uint32_t bars, volatile int* abort_flag) {
  using BR = Bars<NS>;
  constexpr uint32_t kTile = kKC * D * 2;
  constexpr uint32_t kIdescQk = idesc_bf16(kBM, kSub, 0), kIdescPv = idesc_bf16(kBM, D, 1);
  constexpr uint32_t kSubRows = kSub * 128 / 16;  // descriptor units between a chunk's parts
  // Q: column blocks of [256 rows x 128 B], half h from row 128 h
  const uint64_t qd = sdesc_sw128(sbase + uint32_t(h) * (kBM * 128), 16, 1024);
  const uint64_t kd = sdesc_sw128(sbase + P.off_k, 16, 1024);
  const uint64_t vd = sdesc_sw128(sbase + P.off_v, kKC * 128, 1024);
  const uint32_t ts = tmem + uint32_t(h * kKC), to = tmem + uint32_t(2 * kKC + h * D);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool ok = bounded_wait(bars + 8 * bar, parity & 1u, P.timeout_cycles, P.err, abort_flag);
    return __all_sync(0xffffffffu, ok);
  };
  int np[2] = {0, 0}, xh = 0;  // O MMAs of each part, tile parts so far
  // (P of a tile's first part says that the last tile's O has been read out, too;
  // without the wait for that the long prompt took 795 us instead of 775)
  auto pv_ready = [&](int u, bool first) {
    return wait(BR::kPfull + 2 * h + u, uint32_t(np[u]++)) &&
           !(first && xh > 0 && !wait(BR::kOfree + h, uint32_t(xh - 1)));
  };
  // O (+)= P V of part u of chunk number n, `steps` times 16 keys.  add: O holds
  // the sum of earlier parts (one of whose keys, at least, is real: the V rows
  // standing in for bad pages only may hold anything, and what they gave is
  // dropped).
  auto pv = [&](int n, int u, bool add, int steps) {
    if (SA) fence_proxy_async_smem();  // cp.async (generic proxy) data -> tensor core reads
    tc_fence_after();
    const uint64_t b = vd + uint64_t(n % NS) * (kTile / 16) + uint32_t(u) * kSubRows;
    const uint32_t p = ts + uint32_t(u * kSub);
    if (steps == kSub / 16) {
      mma_ts(to, p, b, kIdescPv, add ? 1u : 0u);
#pragma unroll
      for (int kk = 1; kk < kSub / 16; ++kk) mma_ts(to, p + 8 * kk, b + 128 * kk, kIdescPv, 1u);  // 16 keys of 128 B
    } else {
      for (int kk = 0; kk < steps; ++kk) mma_ts(to, p + 8 * kk, b + 128 * kk, kIdescPv, (add || kk > 0) ? 1u : 0u);
    }
    commit_elected(bars + 8 * (BR::kPVdone + 2 * h + u));
  };
  auto qk = [&](int n, int u) {
    if (SA) fence_proxy_async_smem();
    tc_fence_after();
    const uint64_t b = kd + uint64_t(n % NS) * (kTile / 16) + uint32_t(u) * kSubRows;
    const uint32_t d = ts + uint32_t(u * kSub);
    mma_ss<false>(d, qd, b, kIdescQk);
#pragma unroll
    for (int kk = 1; kk < D / 16; ++kk)
      mma_ss<true>(d, qd + uint64_t((kk >> 2) * (kRows * 128 / 16) + (kk & 3) * 2),
                   b + uint64_t((kk >> 2) * (kKC * 128 / 16) + (kk & 3) * 2), kIdescQk);
    commit_elected(bars + 8 * (BR::kSfull + 2 * h + u));
  };
  int n = 0;
  bool ok = true;
  for (int x = 0; ok && more; ++x) {
    if (!(ok = wait(BR::kSegFull + (x & 3), uint32_t(x >> 2)))) break;
    const Shared* sh = seg + (x & 3);
    const int c0 = sh->c0;
    const int chunks = __shfl_sync(0xffffffffu, sh->c1 - c0, 0);
    const int a = __shfl_sync(0xffffffffu, sh->a[h] - c0, 0), b = __shfl_sync(0xffffffffu, sh->b[h] - c0, 0);
    more = __shfl_sync(0xffffffffu, sh->more, 0) != 0;
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (BR::kSegFree + (x & 3)));
    if (!(ok = wait(BR::kQfull, uint32_t(x)))) break;
    bool good = false;  // some key up to the chunk before this one is real
    // (chunks the half has no part in are only waited for and given back)
    int parts = 2;      // of the current chunk
    for (int c = 0; ok && c < chunks; ++c, ++n) {
      const bool o = c > a && c <= b, sc = c >= a && c < b;  // O MMAs of chunk c - 1, S MMAs of chunk c
      bool good_last = true;
      if (c > 0) {
        ok = wait(BR::kVfull + (n - 1) % NS, uint32_t((n - 1) / NS));
        if (!SA && !good) good_last = __shfl_sync(0xffffffffu, keys[(n - 1) % kKeySlots].good, 0) != 0;
      }
      if (ok) ok = wait(BR::kKfull + n % NS, uint32_t(n / NS));
      if (!SA && c == chunks - 1) parts = (__shfl_sync(0xffffffffu, keys[n % kKeySlots].steps, 0) + 3) / 4;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (ok && o && (ok = pv_ready(u, u == 0 && c - 1 == a)))
          pv(n - 1, u, u == 0 ? c - 1 > a && good : good_last, kSub / 16);
        if (ok && sc && u < parts) qk(n, u);
      }
      if (ok) {
        if (c > 0) commit_elected(bars + 8 * (BR::kVfree + (n - 1) % NS));
        commit_elected(bars + 8 * (BR::kKfree + n % NS));
        if (c == chunks - 1) commit_elected(bars + 8 * BR::kQfree);
      }
      if (c > 0) good = good_last;
    }
    // the last O MMAs do not wait for the next tile's operands
    if (ok) ok = wait(BR::kVfull + (n - 1) % NS, uint32_t((n - 1) / NS));
    if (ok && b > a && b == chunks) {
      const bool good_last = SA || good || __shfl_sync(0xffffffffu, keys[(n - 1) % kKeySlots].good, 0) != 0;
      // (earlier chunks are full)
      const int steps = SA ? kKC / 16 : __shfl_sync(0xffffffffu, keys[(n - 1) % kKeySlots].steps, 0);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (ok && u < parts && (ok = pv_ready(u, u == 0 && chunks - 1 == a)))
          pv(n - 1, u, u == 0 ? chunks - 1 > a && good : good_last, min(kSub / 16, steps - u * (kSub / 16)));
    }
    if (b > a) ++xh;
    if (ok) commit_elected(bars + 8 * (BR::kVfree + (n - 1) % NS));
  }
  commit_elected(bars + 8 * (BR::kDrain + h));
  const long long t0 = clock64();
  while (!mbar_try_wait(bars + 8 * (BR::kDrain + h), 0) && clock64() - t0 < kDrainCycles) {
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
template <int D, int NS, bool SA>
__device__ void softmax_role(const Params& P, bool more, const Shared* seg, const typename KeysOf<SA>::T* keys,
                             uint32_t tmem, uint32_t bars, volatile int* abort_flag) {
  using BR = Bars<NS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (warp - kFirstSoftmaxWarp) >> 2, quad = warp & 3;
  const int row = h * kBM + quad * 32 + lane;
  const int t = row / P.g, j = row - t * P.g;
  const uint32_t lanes = uint32_t(quad * 32) << 16;
  const uint32_t sb = tmem + lanes + uint32_t(h * kKC);
  const uint32_t ob = tmem + lanes + uint32_t(2 * kKC + h * D);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool ok = bounded_wait(bars + 8 * bar, parity & 1u, P.timeout_cycles, P.err, abort_flag);
    return __all_sync(0xffffffffu, ok);
  };
  const uint64_t sl2 = f2_pack(P.scale_log2, P.scale_log2);
  int nbase = 0;         // chunks of earlier tile parts
  int k[2] = {0, 0};     // this half's S of each part so far
  for (int x = 0; more; ++x) {
    if (!wait(BR::kSegFull + (x & 3), uint32_t(x >> 2))) return;
    const Shared* sh = seg + (x & 3);
    more = sh->more != 0;
    const int c0 = sh->c0, c1 = sh->c1, a = sh->a[h], b = sh->b[h];
    const bool live = t < sh->nt;
    int4 mem = make_int4(0, -1, 0, 0);
    if (SA && live) mem = P.order.members[sh->t0 + t];
    const int pos = SA ? mem.w : sh->pos0 + t;
    // the row's keys as columns of chunk 0
    const int khi = live ? (SA ? mem.y : pos) - sh->lo : -1;
    const int klo = (SA ? mem.x : max(0, pos - P.w + 1)) - sh->lo;
    const bool whole = c0 == 0 && c1 == sh->nch;
    const int slot = int(blockIdx.x) * 2 + (c0 == 0 ? 1 : 0);
    const size_t orow = live ? size_t(SA ? mem.z : sh->t0 + t) * P.Hq + size_t(sh->kvh) * P.g + j : 0;
    if (sh->join >= 0 && warp == kFirstSoftmaxWarp && lane == 0) {
      Desc d;
      d.valid = 1;
      d.c1 = sh->join;
      d.t0 = sh->t0;
      d.rows = sh->nt * P.g;
      d.kvh = sh->kvh;
      d.pad = 0;
      P.desc[blockIdx.x] = d;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (BR::kSegFree + (x & 3)));
    float ref = -INFINITY, l = 0.f;
    int last_u = 0;
    for (int c = a; c < b; ++c) {
      const auto& key = keys[(nbase + c - c0) % kKeySlots];
      int parts = 2;
#pragma unroll 1  // (unrolled: slower by 8 %, see the top)
      for (int u = 0; u < 2; ++u) {
        if (u >= parts) break;
        if (!wait(BR::kSfull + 2 * h + u, uint32_t(k[u]))) return;
        tc_fence_after();
        if constexpr (SA) {  // the warp's rows have no keys here: most of its tile's parts
          const int at = c * kKC + u * kSub;
          if (__all_sync(0xffffffffu, khi < at || klo >= at + kSub)) {
            uint32_t zero[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) zero[e] = 0u;
            tmem_st16(sb + u * kSub, zero);
            tmem_st16(sb + u * kSub + 16, zero);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (BR::kPfull + 2 * h + u));
            ++k[u];
            last_u = u;
            continue;
          }
        }
        uint32_t v[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld32_async(sb + u * kSub + q * 32, v[q]);
        // (a chunk's words are there before its first S)
        if (!SA && u == 0 && c == c1 - 1) parts = (key.steps + 3) / 4;
        const uint2 bad = *reinterpret_cast<const uint2*>(&key.bad[2 * u]);
        const int lo = klo - c * kKC - u * kSub, hi = khi - c * kKC - u * kSub;
        bool clear = lo <= 0 && hi >= kSub - 1 && (bad.x | bad.y) == 0u;
        uint2 fresh = make_uint2(0u, 0u);
        if constexpr (SA) {
          fresh = *reinterpret_cast<const uint2*>(&key.fresh[2 * u]);
          clear = clear && (fresh.x | fresh.y) == 0u;
        }
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 2; ++q) reg_fence(v[q]);
        if (!__all_sync(0xffffffffu, clear)) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t keep = band_bits(lo, hi, q * 32) & ~(q == 0 ? bad.x : bad.y);
            if (!__all_sync(0xffffffffu, keep == 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((keep >> e) & 1u)) v[q][e] = __float_as_uint(-INFINITY);
            }
            if constexpr (SA) {  // of the new tokens, the later ones are left out (branches here cost more)
              const int4* tk = reinterpret_cast<const int4*>(key.toks + u * kSub + q * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int4 y = tk[e];
                if (y.x > pos) v[q][4 * e] = __float_as_uint(-INFINITY);
                if (y.y > pos) v[q][4 * e + 1] = __float_as_uint(-INFINITY);
                if (y.z > pos) v[q][4 * e + 2] = __float_as_uint(-INFINITY);
                if (y.w > pos) v[q][4 * e + 3] = __float_as_uint(-INFINITY);
              }
            }
          }
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t* y = &v[q >> 1][16 * (q & 1)];
          mx[q] = __uint_as_float(y[0]);
#pragma unroll
          for (int e = 1; e + 1 < 16; e += 2) mx[q] = fmax3(mx[q], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(y[15]));
        }
        const float msc = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * P.scale_log2;
        float alpha = 1.f;
        bool rescale = false;
        if (ref == -INFINITY) {
          ref = msc;  // nothing attended before: O and l are still 0 for this row
        } else if (msc > ref + kRescaleLog2) {
          alpha = fast_exp2(ref - msc);
          ref = msc;
          l *= alpha;
          rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // O must hold the O MMAs of every earlier part: they finish in order
          if (!wait(BR::kPVdone + 2 * h + (u ^ 1), uint32_t(u == 1 ? k[0] - 1 : k[1] - 1))) return;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
                "%13,%14,%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]),
                  "=r"(o[7]), "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]),
                  "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                : "r"(ob + q * 16)
                : "memory");
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(ob + q * 16, o);
          }
          tmem_wait_st();
        }
        const float nref = ref == -INFINITY ? 0.f : -ref;
        const uint64_t nms = f2_pack(nref, nref);
        uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = f2_unpack(f2_fma(
                f2_pack(__uint_as_float(v[q][2 * e]), __uint_as_float(v[q][2 * e + 1])), sl2, nms));
            const float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y);
            acc[e & 1] = f2_add(acc[e & 1], f2_pack(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st16(sb + u * kSub + q * 16, pk);
        }
        const float2 a0 = f2_unpack(acc[0]), a1 = f2_unpack(acc[1]);
        l += (a0.x + a0.y) + (a1.x + a1.y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (BR::kPfull + 2 * h + u));
        ++k[u];
        last_u = u;
      }
    }
    nbase += c1 - c0;
    // epilogue: the tile part is done when its last O MMA is
    if (b > a && !wait(BR::kPVdone + 2 * h + last_u, uint32_t(k[last_u] - 1))) return;
    tc_fence_after();
    float mul = l == 0.f ? 0.f : 1.f / l;
    if (P.gate != nullptr && live) mul *= 1.f / (1.f + expf(-P.gate[orow]));
    const uint64_t mul2 = f2_pack(mul, mul);
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
      uint32_t o[32];
      const int col = q * 32;
      tmem_ld32(ob + col, o);
      if (l == 0.f || b <= a) {  // a row without keys is 0, whatever bad pages left in O
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if (q == D / 32 - 1 && b > a) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (BR::kOfree + h));
      }
      if (!whole) {
        float4* dst = reinterpret_cast<float4*>(P.part) + (size_t(slot) * (D / 4) + col / 4) * kRows + row;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e * kRows] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
      } else if (live) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), mul2));
          o[2 * e] = __float_as_uint(y.x);
          o[2 * e + 1] = __float_as_uint(y.y);
        }
        if (SA && P.swa_part != nullptr) {
          const float4* add = reinterpret_cast<const float4*>(P.swa_part + orow * D + col);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 y = add[e];
            o[4 * e] = __float_as_uint(__uint_as_float(o[4 * e]) + y.x);
            o[4 * e + 1] = __float_as_uint(__uint_as_float(o[4 * e + 1]) + y.y);
            o[4 * e + 2] = __float_as_uint(__uint_as_float(o[4 * e + 2]) + y.z);
            o[4 * e + 3] = __float_as_uint(__uint_as_float(o[4 * e + 3]) + y.w);
          }
        }
        if (!SA && P.gate != nullptr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = o[8 * e + u];
            st_global_v8(P.part_out + orow * D + col + e * 8, w);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
              w[u] = pack_bf16x2(__uint_as_float(o[16 * e + 2 * u]), __uint_as_float(o[16 * e + 2 * u + 1]));
            st_global_2v4(P.out + orow * D + col + e * 16, w);
          }
        }
      }
    }
    if (!whole) {
      float2* ml = reinterpret_cast<float2*>(P.part + size_t(gridDim.x) * 2 * kRows * D) + size_t(slot) * kRows + row;
      *ml = make_float2(ref, l);
    }
  }
}

template <int D, int NS, bool SA>
__global__ void __launch_bounds__(SA ? kSaThreads : kThreads, 1) sa_paged_tiles_kernel(const __grid_constant__ Params P) {
  using BR = Bars<NS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Start s_start;
  __shared__ Cursor s_cursor;
  __shared__ Seg s_seg;
  __shared__ bool s_any;
  __shared__ int s_vote[2];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + P.off_bar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + P.off_bar + 8 * BR::kNum);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + P.off_bar + 8 * BR::kNum + 4);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 64) {
    mbar_init(bars + 8 * BR::kQfull, SA ? kSaProducers : 1);
    mbar_init(bars + 8 * BR::kQfree, 2);
    for (int i = 0; i < NS; ++i) {
      // SA: the producers' copies, and thread 0 for the key words
      mbar_init(bars + 8 * (BR::kKfull + i), SA ? kSaProducers + 1 : 1);
      mbar_init(bars + 8 * (BR::kKfree + i), 2);
      mbar_init(bars + 8 * (BR::kVfull + i), SA ? kSaProducers : 1);
      mbar_init(bars + 8 * (BR::kVfree + i), 2);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(bars + 8 * (BR::kOfree + h), 4);
      mbar_init(bars + 8 * (BR::kDrain + h), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bars + 8 * (BR::kSegFull + i), 1);
      mbar_init(bars + 8 * (BR::kSegFree + i), 8 + 2);
      mbar_init(bars + 8 * (BR::kSfull + i), 1);
      mbar_init(bars + 8 * (BR::kPfull + i), 4);
      mbar_init(bars + 8 * (BR::kPVdone + i), 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (!SA && warp == 3) {
    const int lane = threadIdx.x & 31, i = lane % kBoxes;  // (no boxes longer than a page)
    const CUtensorMap* m = lane == 2 * kBoxes ? &P.tq : lane < kBoxes ? &P.tk[i] : &P.tv[i];
    if (lane == 2 * kBoxes || (lane < 2 * kBoxes && 1 << i <= P.page))
      asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  } else if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  begin_after();  // (the order kernel, or the one for requests of few new tokens, may run beside the rest)
  if (threadIdx.x == 64 && P.desc != nullptr) P.desc[blockIdx.x].valid = 0;
  if (warp == 0) {
    const Start s = find_start<SA>(P);
    Cursor cur = make_cursor<SA>(P, s);
    Seg seg;
    const bool any = next_seg<SA>(P, cur, seg);
    if (threadIdx.x == 0) {
      s_start = s;
      s_cursor = cur;
      s_seg = seg;
      s_any = any;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool any = s_any;
  const Shared* seg = reinterpret_cast<const Shared*>(smem + P.off_seg);
  const auto* keys = reinterpret_cast<const typename KeysOf<SA>::T*>(smem + P.off_bad);

  if (warp >= kFirstSoftmaxWarp && warp < kFirstSoftmaxWarp + 8) {
    softmax_role<D, NS, SA>(P, any, seg, keys, tmem, bars, abort_flag);
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    mma_role<D, NS, SA>(P, warp - kMmaWarp, any, seg, keys, sbase, tmem, bars, abort_flag);
  } else if (SA) {
    sa_producer_role<D, NS>(P, s_start, s_cursor, s_seg, any, smem, sbase, bars, abort_flag, s_vote);
  } else {
    producer_role<D, NS>(P, s_start, s_cursor, s_seg, any, smem, sbase, bars, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

// Joins the parts of each tile that the runs cut, in block order.  Block
// (c, y) takes columns of the tile that starts in run c.
template <int D, bool SA>
__global__ void __launch_bounds__(kRows) sa_paged_tiles_join_kernel(const __grid_constant__ Params P) {
  begin_after();
  const int c0 = blockIdx.x;
  const Desc d = P.desc[c0];
  if (!d.valid) return;
  const int row = threadIdx.x, blocks = gridDim.x;
  if (row >= d.rows) return;
  const float2* ml = reinterpret_cast<const float2*>(P.part + size_t(blocks) * 2 * kRows * D);
  auto slot = [&](int c) { return size_t(c * 2 + (c == c0 ? 1 : 0)); };
  float m = -INFINITY;
  for (int c = c0; c <= d.c1; ++c) m = fmaxf(m, ml[slot(c) * kRows + row].x);
  float l = 0.f;
  float4 a[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= d.c1; ++c) {
    const float2 x = ml[slot(c) * kRows + row];
    const float f = x.x == -INFINITY ? 0.f : fast_exp2(x.x - m);
    l = fmaf(f, x.y, l);
    const float4* src = reinterpret_cast<const float4*>(P.part) + (slot(c) * (D / 4) + blockIdx.y * 4) * kRows + row;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 v = src[e * kRows];
      a[e].x = fmaf(f, v.x, a[e].x);
      a[e].y = fmaf(f, v.y, a[e].y);
      a[e].z = fmaf(f, v.z, a[e].z);
      a[e].w = fmaf(f, v.w, a[e].w);
    }
  }
  const int t = row / P.g, j = row - t * P.g;
  const int trow = SA ? P.order.members[d.t0 + t].z : d.t0 + t;
  const size_t orow = size_t(trow) * P.Hq + size_t(d.kvh) * P.g + j;
  float s = l == 0.f ? 0.f : 1.f / l;
  if (P.gate != nullptr) s *= 1.f / (1.f + expf(-P.gate[orow]));
  const int col = blockIdx.y * 16;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e].x *= s;
    a[e].y *= s;
    a[e].z *= s;
    a[e].w *= s;
    if (SA && P.swa_part != nullptr) {
      const float4 y = *reinterpret_cast<const float4*>(P.swa_part + orow * D + col + 4 * e);
      a[e].x += y.x;
      a[e].y += y.y;
      a[e].z += y.z;
      a[e].w += y.w;
    }
  }
  if (!SA && P.gate != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4*>(P.part_out + orow * D + col + 4 * e) =
          a[e];
  } else {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[2 * e] = pack_bf16x2(a[e].x, a[e].y);
      w[2 * e + 1] = pack_bf16x2(a[e].z, a[e].w);
    }
    st_global_2v4(P.out + orow * D + col, w);
  }
}

// ------------------------------------------------------------------ host

static bool may_cut(const PagedProblem& pb, bool sa) {
  const long long longest = (long long)pb.max_pages * pb.page;
  const long long keys = sa ? longest : min((long long)pb.window_swa + kRows, longest);
  return keys >= (long long)kCutChunks * kKC;
}

template <int D, int NS, bool SA>
static cudaError_t launch_one(Params& P, int sms, cudaStream_t stream) {
  using K = typename KeysOf<SA>::T;
  const uint32_t tile = kKC * D * 2;
  P.off_k = 2 * kBM * D * 2;
  P.off_v = P.off_k + NS * tile;
  P.off_bad = P.off_v + NS * tile;
  P.off_seg = P.off_bad + kKeySlots * uint32_t(sizeof(K));
  P.off_bar = P.off_seg + 4 * uint32_t(sizeof(Shared)) + (SA ? (2 * kKC + kRows) * 4 : 0);
  const uint32_t smem = P.off_bar + 8 * Bars<NS>::kNum + 16 + 1024;
  static_assert(2 * kBM * D * 2 + 2 * NS * kKC * D * 2 + kKeySlots * sizeof(K) + 4 * sizeof(Shared) + (2 * kKC + kRows) * 4 + 128 + 8 * Bars<NS>::kNum + 16 + 1024 + 64 <=
                    kMaxSmem, "shared memory");
  cudaError_t ce = allow_smem<sa_paged_tiles_kernel<D, NS, SA>>(smem);
  if (ce != cudaSuccess) return ce;
  // (a gated call's first kernel set up early made 123 us of 107: the order kernel
  // and the SA tiles behind it find their SMs in another order)
  ce = launch_kernel(sa_paged_tiles_kernel<D, NS, SA>, dim3(unsigned(sms)), SA ? kSaThreads : kThreads, smem, stream,
                     P, SA || P.gate == nullptr);
  if (ce != cudaSuccess || P.desc == nullptr) return ce;
  return launch_kernel(sa_paged_tiles_join_kernel<D, SA>, dim3(unsigned(sms), D / 16), kRows, 0, stream, P);
}

}  // namespace ptile

bool paged_tiles_supported(const PagedProblem& pb) {
  return pb.g <= ptile::kRows / 4;  // at least four tokens to a tile
}

size_t paged_tiles_workspace_bytes(const PagedProblem& pb, bool sa, int sms) {
  if (!ptile::may_cut(pb, sa)) return 0;
  const size_t part = size_t(sms) * 2 * ptile::kRows * (pb.d + 2) * 4;
  return (part + 255) / 256 * 256 + (size_t(sms) * sizeof(ptile::Desc) + 255) / 256 * 256;
}

namespace ptile {
static void common_params(Params* P, const PagedProblem& pb, bool sa, int row_limit, void* workspace, int sms) {
  std::memset(P, 0, sizeof(*P));
  P->table = pb.table;
  P->q_start = pb.q_start;
  P->seq_lens = pb.seq_lens;
  P->out = static_cast<__nv_bfloat16*>(pb.out);
  if (may_cut(pb, sa)) {
    const size_t part = size_t(sms) * 2 * kRows * (pb.d + 2) * 4;
    P->part = static_cast<float*>(workspace);
    P->desc = reinterpret_cast<Desc*>(static_cast<char*>(workspace) + (part + 255) / 256 * 256);
  }
  P->err = pb.err;
  P->B = pb.B;
  P->T = pb.T;
  P->max_new = pb.max_new;
  P->row_limit = row_limit;
  P->Hq = pb.Hq;
  P->Hkv = pb.Hkv;
  P->g = pb.g;
  P->Bt = paged_tile_tokens(pb);
  P->page = pb.page;
  P->num_pages = pb.num_pages;
  P->max_pages = pb.max_pages;
  P->w = pb.window_swa;
  P->scale_log2 = pb.scale * 1.4426950408889634f;
  P->timeout_cycles = wait_limit_cycles();
}
}  // namespace ptile

int paged_tile_tokens(const PagedProblem& pb) { return ptile::kRows / pb.g; }

sa_status_t launch_paged_tiles(const PagedProblem& pb, int row_limit, const float* gate,
                               float* part_out, void* workspace, int sms, cudaStream_t stream) {
  using namespace ptile;
  Params P;
  common_params(&P, pb, false, row_limit, workspace, sms);
  P.gate = gate;
  P.part_out = part_out;
  const uint64_t d2 = uint64_t(pb.d) * 2;
  const uint64_t qdims[3] = {uint64_t(pb.d), uint64_t(pb.Hq), uint64_t(pb.T)};
  const uint64_t qst[2] = {d2, uint64_t(pb.q_stride) * 2};
  const uint32_t qbox[3] = {64, uint32_t(pb.g), uint32_t(kRows / pb.g)};
  bool maps = encode_box_map(&P.tq, pb.q, 3, qdims, qst, qbox);
  const uint64_t dims[4] = {uint64_t(pb.d), uint64_t(pb.Hkv), uint64_t(pb.page), uint64_t(pb.num_pages)};
  const uint64_t st[3] = {d2, d2 * pb.Hkv, uint64_t(pb.page_stride) * 2};
  for (int i = 0; i < kBoxes && maps && 1 << i <= pb.page; ++i) {  // (no longer runs in a page)
    const uint32_t box[4] = {64, 1, 1u << i, 1};
    maps = encode_box_map(&P.tk[i], pb.k, 4, dims, st, box) && encode_box_map(&P.tv[i], pb.v, 4, dims, st, box);
  }
  if (!maps) return fail(SA_ERR_CUDA, "paged tile kernel: cannot encode the tensor maps");
  const cudaError_t ce =
      pb.d == 128 ? launch_one<128, 2, false>(P, sms, stream) : launch_one<64, 4, false>(P, sms, stream);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged tile kernel launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

sa_status_t launch_paged_sa_tiles(const PagedProblem& pb, const SaOrder& order, const float* gate,
                                  const float* swa_part, void* workspace, int sms, cudaStream_t stream) {
  using namespace ptile;
  Params P;
  common_params(&P, pb, true, 0, workspace, sms);
  P.gate = gate;
  P.swa_part = swa_part;
  P.q = static_cast<const __nv_bfloat16*>(pb.q);
  P.k = static_cast<const __nv_bfloat16*>(pb.k);
  P.v = static_cast<const __nv_bfloat16*>(pb.v);
  P.q_stride = pb.q_stride;
  P.order = order;
  const cudaError_t ce =
      pb.d == 128 ? launch_one<128, 2, true>(P, sms, stream) : launch_one<64, 4, true>(P, sms, stream);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged SA tile kernel launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
