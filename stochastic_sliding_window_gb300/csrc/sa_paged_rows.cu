// Row kernel of the paged-cache attention: SA, SWA or the gated pair for
// requests with few new tokens (decoding), any request when asked to.
//
// Mathematics.  A unit is up to 16 query rows that share a kv head: the g
// query heads of as many of a request's new tokens as fit (one token for SA,
// whose windows differ from token to token).  Its keys are cut into tiles of
// 16: positions max(0, pos - w + 1) .. for SWA, positions of sigma around
// p = sigma^{-1}(pos) for SA.  One pass over the tiles with a running maximum
// m and sum l per row:
//   S = Q K^T,  p = 2^(scale log2(e) S - m),  O <- 2^(m_old - m) O + p V.
// The weights p enter the second product as two bf16 terms, hi + lo, which
// keeps them to 2^-17: one bf16 would cost as much as the rounding of the
// result does, and the product is far from being what bounds the kernel.
//
// What bounds it: reading K and V once, 4 d bytes per key and kv head, for
// 4 g d multiply-adds.  So the split is by keys: every warp of the GPU (a
// "worker") takes an equal run of the tiles of all units laid end to end,
// found by a scan over the requests' lengths, so ragged batches balance
// whatever the lengths are and the host needs to know none.  A warp works
// alone -- its own ring of cp.async stages, no block barriers -- and its
// loads run ahead across the ends of units.  A unit cut by a run's end leaves
// fp32 partial (O, m, l) in the workspace; the second kernel joins them in
// worker order, so results do not depend on timing.  Where there are several
// units per worker the runs end at unit ends instead and one launch does all.
#include "sa_internal.h"
#include "sa_tc_common.cuh"

#include <cstring>

namespace sa {
namespace prow {

using namespace tcc;

constexpr int kKeys = 16;   // keys per tile
constexpr int kStages = 3;
constexpr uint32_t kMaxSmem = 232448;
constexpr int kMetaInts = 32;  // 16 key tokens, then the fields below
enum : int { kFlags = 16, kPos0, kRows, kTok0, kHr };
enum : int {
  kFirst = 1,     // first tile of a piece (a unit's run of one path): reset O, m, l
  kLast = 2,      // last tile of the piece: write it
  kNewQ = 4,      // first tile of the unit here: the stage holds its Q rows
  kIsSwa = 8,     // the piece is of the SWA path
  kWhole = 16,    // the whole unit is this worker's
  kTail = 32,     // the unit starts in this worker's run (partial slot 1, else 0)
  kAny = 64,      // some key of the tile is loaded
  kAddSwa = 128,  // gated: the SWA term comes from swa_part
  kNone = 256,    // no tile: the run is done
};

struct Desc {  // one per worker: the unit that starts in its run and ends beyond it
  int valid, c1, t0, hr, nrows, tsa, tsw, add_swa;
  long long u0, per;
};

struct Params {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_lens;
  const int32_t* perm;
  const int32_t* inv;
  const float* gate_sa;
  const float* gate_swa;
  const float* swa_part;  // [T, Hq, D] gated SWA terms of requests beyond row_limit
  __nv_bfloat16* out;
  int32_t* err;
  float* part;            // partial slots, then Desc[workers]; nullptr: never split
  Desc* desc;
  long long q_stride, page_stride, perm_stride;
  int B, T, max_new, row_limit, Hq, Hkv, g, page, num_pages, max_pages;
  int w, half, perm_len;
  int tb, rg, R;          // tokens and rows of a unit; row groups of a kv head (g > 16)
  int slot_floats;        // one partial: O [R, D], then (m, l) [R]; a multiple of 4
  int workers, min_tiles, snap;
  uint32_t stage_bytes, warp_bytes;
  float scale_log2;
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
               "{%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A request as the units see it; n = 0 where it has none here.
struct Request {
  int q0, n, len, tsa, tsw, groups;
};

template <int PATH>
__device__ __forceinline__ Request load_request(const Params& P, int b, bool report) {
  Request r;
  r.q0 = P.q_start[b];
  const int q1 = P.q_start[b + 1];
  r.len = P.seq_lens[b];
  r.n = q1 - r.q0;
  r.tsa = r.tsw = 0;
  const bool ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= P.T && r.n <= P.max_new && r.n <= r.len &&
                  (long long)r.len <= (long long)P.max_pages * P.page &&
                  (PATH == kPathSWA || r.len <= P.perm_len);
  if (!ok) {
    // (a request without new tokens is not looked at otherwise)
    if (report && q1 != r.q0) atomicOr(P.err, SA_ERRBIT_RANGE);
    r.n = 0;
  }
  const bool swa_here = r.n <= P.row_limit;
  if (PATH == kPathSWA && !swa_here) r.n = 0;
  if (PATH != kPathSWA) r.tsa = int((min(2LL * P.half + 1, (long long)P.perm_len) + kKeys - 1) / kKeys);
  if (PATH != kPathSA && swa_here)
    r.tsw = int((min((long long)r.len, (long long)P.w + P.tb - 1) + kKeys - 1) / kKeys);
  r.groups = ceil_div(r.n, P.tb);
  return r;
}

template <int D, int PATH>
__global__ void __launch_bounds__(D == 128 ? 256 : 512, 1) sa_paged_rows_kernel(const __grid_constant__ Params P) {
  constexpr int kPitch = D * 2 + 16;  // 16 bytes over: eight rows of a matrix hit all banks
  constexpr int kCpr = D / 8;         // 16-byte chunks per row
  constexpr uint32_t kOffV = kKeys * kPitch, kOffQ = 2 * kKeys * kPitch;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int worker = warp * int(gridDim.x) + int(blockIdx.x);
  if (worker >= P.workers) return;
  uint8_t* ring = smem_raw + size_t(warp) * P.warp_bytes;
  const uint32_t sring = smem_u32(ring);
  const uint32_t off_meta = kOffQ + uint32_t(P.R) * kPitch;
  const int HR = P.Hkv * P.rg;

  // ---- this worker's run of tiles: [begin, end) of all units' tiles
  long long total = 0, mine_sum = 0;
  {
    for (int b0 = 0; b0 < P.B; b0 += 32) {
      const int b = b0 + lane;
      if (b < P.B) {
        const Request r = load_request<PATH>(P, b, worker == 0);
        mine_sum += (long long)r.groups * HR * (r.tsa + r.tsw);
      }
    }
    total = mine_sum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  long long per = (total + P.workers - 1) / P.workers;
  if (per < P.min_tiles) per = P.min_tiles;
  const long long begin = per * worker;
  const long long end = min(total, begin + per);
  if (P.desc != nullptr && lane == 0) P.desc[worker].valid = 0;
  if (begin >= total) return;

  // ---- cursor: request, group, head and tile of the next tile to fetch
  int cb = 0;
  Request cr;
  long long cpos = begin;
  int cgrp = 0, chr_ = 0, ctile = 0;
  {
    long long before = 0;  // tiles of the requests before this chunk of 32
    for (int b0 = 0; b0 < P.B; b0 += 32) {
      const int b = b0 + lane;
      long long x = 0;
      if (b < P.B) {
        const Request r = load_request<PATH>(P, b, false);
        x = (long long)r.groups * HR * (r.tsa + r.tsw);
      }
      long long sum = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += a;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > begin);
      if (hit != 0u) {
        const int src = __ffs(hit) - 1;
        cb = b0 + src;
        const long long start = before + __shfl_sync(0xffffffffu, sum - x, src);
        cr = load_request<PATH>(P, cb, false);
        const int per_unit = cr.tsa + cr.tsw;
        const long long rel = begin - start;
        const long long uh = rel / per_unit;
        ctile = int(rel - uh * per_unit);
        cgrp = int(uh / HR);
        chr_ = int(uh - (long long)cgrp * HR);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  bool done = false;
  auto next_unit = [&]() {  // to the first tile of the next unit, if any
    ctile = 0;
    if (++chr_ < HR) return;
    chr_ = 0;
    if (++cgrp < cr.groups) return;
    cgrp = 0;
    do {
      if (++cb >= P.B) {
        done = true;
        return;
      }
      cr = load_request<PATH>(P, cb, false);
    } while (cr.groups == 0 || cr.tsa + cr.tsw == 0);
  };
  if (P.snap && ctile != 0) {  // the unit cut here is the previous worker's
    cpos += cr.tsa + cr.tsw - ctile;
    next_unit();
  }

  // ---- tiles on their way: A has its page ids, B its key tokens
  struct Tile {
    int flags, pos0, rows, t0, hr, b, tok;  // tok: this lane's key (lane & 15), -1: none
  };
  int upos0 = 0, urows = 0, ut0 = 0, slo = 0, shi = 0, wlo = 0, whi = 0;
  bool fresh = true;  // the cursor's unit has not been entered yet
  auto make = [&]() -> Tile {
    Tile t;
    t.tok = -1;
    t.flags = kNone;
    t.pos0 = t.rows = t.t0 = t.hr = t.b = 0;
    const int per_unit = cr.tsa + cr.tsw;
    if (done || (P.snap ? (ctile == 0 && cpos >= end) : cpos >= end)) return t;
    int flags = 0;
    if (fresh) {
      const int i0 = cgrp * P.tb, nt = min(P.tb, cr.n - i0);
      upos0 = cr.len - cr.n + i0;
      ut0 = cr.q0 + i0;
      urows = P.rg > 1 ? min(16, P.g - (chr_ % P.rg) * 16) : nt * P.g;
      if (PATH != kPathSA) {
        wlo = max(0, upos0 - P.w + 1);
        whi = upos0 + nt;
      }
      if (PATH != kPathSWA) {
        const int p = P.inv[(long long)cb * P.perm_stride + upos0];
        slo = shi = 0;
        if (unsigned(p) < unsigned(P.perm_len)) {
          slo = max(0, p - P.half);
          shi = int(min((long long)P.perm_len, (long long)p + P.half + 1));
        } else if (lane == 0) {
          atomicOr(P.err, SA_ERRBIT_RANGE);
        }
      }
      flags |= kNewQ;
    }
    const long long ustart = cpos - ctile;
    const bool whole = P.snap || (ustart >= begin && ustart + per_unit <= end);
    if (whole) flags |= kWhole;
    if (ustart >= begin) flags |= kTail;
    if (fresh && !whole && ustart >= begin && lane == 0) {
      Desc d;
      d.valid = 1;
      d.c1 = int((ustart + per_unit - 1) / per);
      d.t0 = ut0;
      d.hr = chr_;
      d.nrows = urows;
      d.tsa = cr.tsa;
      d.tsw = cr.tsw;
      d.add_swa = PATH == kPathGated && cr.tsw == 0;
      d.u0 = ustart;
      d.per = per;
      P.desc[worker] = d;
    }
    const bool is_swa = PATH == kPathSWA || (PATH == kPathGated && ctile >= cr.tsa);
    const int pt = is_swa ? ctile - cr.tsa : ctile;  // tile within the path
    if (pt == 0 || fresh) flags |= kFirst;
    if (is_swa) flags |= kIsSwa;
    if (PATH == kPathGated && cr.tsw == 0) flags |= kAddSwa;
    const bool path_end = ctile == (is_swa ? per_unit : cr.tsa) - 1;
    if (path_end || (!P.snap && cpos == end - 1)) flags |= kLast;
    // this lane's key
    const int key = pt * kKeys + (lane & 15);
    if (is_swa) {
      const int j = wlo + key;
      if (j < whi) t.tok = j;
    } else {
      const int j = slo + key;
      if (j < shi) {
        const int tok = P.perm[(long long)cb * P.perm_stride + j];
        if (unsigned(tok) >= unsigned(P.perm_len)) {
          atomicOr(P.err, SA_ERRBIT_RANGE);
        } else if (tok <= upos0) {
          t.tok = tok;
        }
      }
    }
    t.flags = flags;
    t.pos0 = upos0;
    t.rows = urows;
    t.t0 = ut0;
    t.hr = chr_;
    t.b = cb;
    fresh = false;
    ++cpos;
    if (++ctile == per_unit) {
      next_unit();
      fresh = true;
    }
    return t;
  };
  auto page_of = [&](const Tile& t) {  // -1: no key
    return t.tok >= 0 ? P.table[(long long)t.b * P.max_pages + int(unsigned(t.tok) / unsigned(P.page))] : -1;
  };
  auto issue = [&](const Tile& t, int page, int stage) {
    uint8_t* st = ring + uint32_t(stage) * P.stage_bytes;
    const uint32_t ss = sring + uint32_t(stage) * P.stage_bytes;
    int* meta = reinterpret_cast<int*>(st + off_meta);
    if (t.flags & kNone) {
      if (lane == 0) meta[kFlags] = kNone;
      return;
    }
    const int kvh = t.hr / P.rg;
    long long off = -1;
    if (t.tok >= 0) {
      if (unsigned(page) < unsigned(P.num_pages)) {
        const int in = int(unsigned(t.tok) % unsigned(P.page));
        off = (long long)page * P.page_stride + ((long long)in * P.Hkv + kvh) * D;
      } else {
        atomicOr(P.err, SA_ERRBIT_RANGE);
      }
    }
    const bool any = __any_sync(0xffffffffu, off >= 0);
    if (lane < kKeys) meta[lane] = off >= 0 ? t.tok : 0x7fffffff;
    if (lane == 0) {
      meta[kFlags] = t.flags | (any ? kAny : 0);
      meta[kPos0] = t.pos0;
      meta[kRows] = t.rows;
      meta[kTok0] = t.t0;
      meta[kHr] = t.hr;
    }
    if (any) {
      const int c = lane % kCpr;
#pragma unroll
      for (int i = 0; i < kKeys * kCpr / 32; ++i) {
        const int row = i * (32 / kCpr) + lane / kCpr;
        const long long o = __shfl_sync(0xffffffffu, off, row);
        const int bytes = o >= 0 ? 16 : 0;  // rows without a key are filled with zeros
        const long long at = (o >= 0 ? o : 0) + c * 8;
        cp_async16_zfill(ss + row * kPitch + c * 16, P.k + at, bytes);
        cp_async16_zfill(ss + kOffV + row * kPitch + c * 16, P.v + at, bytes);
      }
    }
    if (t.flags & kNewQ) {
      const int h0 = kvh * P.g + (P.rg > 1 ? (t.hr - kvh * P.rg) * 16 : 0);
      for (int i = lane; i < t.rows * kCpr; i += 32) {
        const int r = i / kCpr, c = i - r * kCpr;
        const int tk = P.rg > 1 ? 0 : r / P.g;
        cp_async16(ss + kOffQ + r * kPitch + c * 16,
                   P.q + (long long)(t.t0 + tk) * P.q_stride + (h0 + r - tk * P.g) * D + c * 8);
      }
    }
  };

  // ---- the pipeline
  Tile ta = make();
  int pa = page_of(ta);
  Tile tn = make();
  auto step = [&](int stage) {
    issue(ta, pa, stage);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ta = tn;
    pa = page_of(ta);
    tn = make();
  };
  step(0);
  step(1);

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float stash[PATH == kPathGated ? D / 8 : 1][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const int r0 = lane >> 2, r1 = r0 + 8;  // this lane's rows of the unit
  const int rt0 = P.rg > 1 ? 0 : r0 / P.g, rt1 = P.rg > 1 ? 0 : r1 / P.g;
  int stage = 0, fill = kStages - 1;
  while (true) {
    step(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    uint8_t* st = ring + uint32_t(stage) * P.stage_bytes;
    const uint32_t ss = sring + uint32_t(stage) * P.stage_bytes;
    const int* meta = reinterpret_cast<const int*>(st + off_meta);
    const int flags = meta[kFlags];
    if (flags & kNone) break;
    const int pos0 = meta[kPos0], rows = meta[kRows];
    if (flags & kFirst) {
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    if (flags & kNewQ) {
      // rows past the unit's last read its first: their weights are all masked
      int r = (lane & 7) + ((lane >> 3) & 1) * 8;
      if (r >= rows) r = 0;
      const uint32_t a = ss + kOffQ + r * kPitch + (lane >> 4) * 16;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) ldsm4(a + i * 32, qf[i]);
    }
    if (flags & kAny) {
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const uint32_t a = ss + ((lane & 7) + (lane >> 4) * 8) * kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t kf[4];
          ldsm4(a + i * 32, kf);
          mma16816(s[0], qf[i], kf[0], kf[1]);
          mma16816(s[1], qf[i], kf[2], kf[3]);
        }
      }
      const unsigned w = PATH == kPathSWA || (flags & kIsSwa) ? unsigned(P.w) : 0x7fffffffu;
      const int p0 = r0 < rows ? pos0 + rt0 : -1, p1 = r1 < rows ? pos0 + rt1 : -1;
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int2 tok = *reinterpret_cast<const int2*>(meta + t * 8 + (lane & 3) * 2);
        s[t][0] = unsigned(p0 - tok.x) < w ? s[t][0] * P.scale_log2 : -INFINITY;
        s[t][1] = unsigned(p0 - tok.y) < w ? s[t][1] * P.scale_log2 : -INFINITY;
        s[t][2] = unsigned(p1 - tok.x) < w ? s[t][2] * P.scale_log2 : -INFINITY;
        s[t][3] = unsigned(p1 - tok.y) < w ? s[t][3] * P.scale_log2 : -INFINITY;
        x0 = fmax3(x0, s[t][0], s[t][1]);
        x1 = fmax3(x1, s[t][2], s[t][3]);
      }
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
        const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float e0 = fast_exp2(s[t][0] - b0), e1 = fast_exp2(s[t][1] - b0);
        const float e2 = fast_exp2(s[t][2] - b1), e3 = fast_exp2(s[t][3] - b1);
        l0 += e0 + e1;
        l1 += e2 + e3;
        hi[2 * t] = pack_bf16x2(e0, e1);
        hi[2 * t + 1] = pack_bf16x2(e2, e3);
        lo[2 * t] = pack_bf16x2(e0 - __uint_as_float(hi[2 * t] << 16), e1 - __uint_as_float(hi[2 * t] & 0xffff0000u));
        lo[2 * t + 1] = pack_bf16x2(e2 - __uint_as_float(hi[2 * t + 1] << 16),
                                    e3 - __uint_as_float(hi[2 * t + 1] & 0xffff0000u));
      }
      const uint32_t a = ss + kOffV + ((lane & 7) + ((lane >> 3) & 1) * 8) * kPitch + (lane >> 4) * 16;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vf[4];
        ldsm4t(a + i * 32, vf);
        mma16816(o[2 * i], hi, vf[0], vf[1]);
        mma16816(o[2 * i + 1], hi, vf[2], vf[3]);
        mma16816(o[2 * i], lo, vf[0], vf[1]);
        mma16816(o[2 * i + 1], lo, vf[2], vf[3]);
      }
    }
    if (flags & kLast) {
      const int t0 = meta[kTok0], hr = meta[kHr];
      const int kvh = hr / P.rg;
      const int h0 = kvh * P.g + (P.rg > 1 ? (hr - kvh * P.rg) * 16 : 0);
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      if (!(flags & kWhole)) {
        const int slot = (worker * 2 + ((flags & kTail) ? 1 : 0)) * (PATH == kPathGated ? 2 : 1) +
                         (PATH == kPathGated && (flags & kIsSwa) ? 1 : 0);
        float* pw = P.part + size_t(slot) * P.slot_floats;
        if (r0 < rows) {
          if ((lane & 3) == 0) {
            pw[P.R * D + 2 * r0] = m0;
            pw[P.R * D + 2 * r0 + 1] = l0;
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(pw + r0 * D + i * 8 + (lane & 3) * 2) = make_float2(o[i][0], o[i][1]);
        }
        if (r1 < rows) {
          if ((lane & 3) == 0) {
            pw[P.R * D + 2 * r1] = m1;
            pw[P.R * D + 2 * r1 + 1] = l1;
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(pw + r1 * D + i * 8 + (lane & 3) * 2) = make_float2(o[i][2], o[i][3]);
        }
      } else {
        float f0 = l0 == 0.f ? 0.f : 1.f / l0, f1 = l1 == 0.f ? 0.f : 1.f / l1;
        const size_t row0 = size_t(t0 + rt0) * P.Hq + h0 + r0 - rt0 * P.g;
        const size_t row1 = size_t(t0 + rt1) * P.Hq + h0 + r1 - rt1 * P.g;
        bool write = true;
        if (PATH == kPathGated) {
          const float* gate = (flags & kIsSwa) ? P.gate_swa : P.gate_sa;
          if (r0 < rows) f0 *= 1.f / (1.f + expf(-gate[row0]));
          if (r1 < rows) f1 *= 1.f / (1.f + expf(-gate[row1]));
          write = (flags & (kIsSwa | kAddSwa)) != 0;
          if (flags & kIsSwa) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][0] = fmaf(o[i][0], f0, stash[i][0]);
              o[i][1] = fmaf(o[i][1], f0, stash[i][1]);
              o[i][2] = fmaf(o[i][2], f1, stash[i][2]);
              o[i][3] = fmaf(o[i][3], f1, stash[i][3]);
            }
            f0 = f1 = 1.f;
          } else if (!write) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              stash[i][0] = o[i][0] * f0;
              stash[i][1] = o[i][1] * f0;
              stash[i][2] = o[i][2] * f1;
              stash[i][3] = o[i][3] * f1;
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const int c = i * 8 + (lane & 3) * 2;
              const float2 z = make_float2(0.f, 0.f);
              const float2 a = r0 < rows ? *reinterpret_cast<const float2*>(P.swa_part + row0 * D + c) : z;
              const float2 b = r1 < rows ? *reinterpret_cast<const float2*>(P.swa_part + row1 * D + c) : z;
              o[i][0] = fmaf(o[i][0], f0, a.x);
              o[i][1] = fmaf(o[i][1], f0, a.y);
              o[i][2] = fmaf(o[i][2], f1, b.x);
              o[i][3] = fmaf(o[i][3], f1, b.y);
            }
            f0 = f1 = 1.f;
          }
        }
        if (write) {
          // through this stage's Q rows, whose fragments were taken, to whole 16-byte stores
          uint8_t* os = st + kOffQ;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const int c = (i * 8 + (lane & 3) * 2) * 2;
            if (r0 < rows) *reinterpret_cast<uint32_t*>(os + r0 * kPitch + c) = pack_bf16x2(o[i][0] * f0, o[i][1] * f0);
            if (r1 < rows) *reinterpret_cast<uint32_t*>(os + r1 * kPitch + c) = pack_bf16x2(o[i][2] * f1, o[i][3] * f1);
          }
          __syncwarp();
          for (int i = lane; i < rows * kCpr; i += 32) {
            const int r = i / kCpr, c = i - r * kCpr;
            const int tk = P.rg > 1 ? 0 : r / P.g;
            *reinterpret_cast<uint4*>(P.out + (size_t(t0 + tk) * P.Hq + h0 + r - tk * P.g) * D + c * 8) =
                *reinterpret_cast<const uint4*>(os + r * kPitch + c * 16);
          }
        }
      }
    }
    __syncwarp();  // the stage is read
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Joins the partials of each unit that the runs cut: block c takes the unit
// that starts in worker c's run.  Piece after piece in worker order.
template <int D, int PATH>
__global__ void __launch_bounds__(128) sa_paged_join_kernel(const __grid_constant__ Params P) {
  const Desc d = P.desc[blockIdx.x];
  if (!d.valid) return;
  const int c0 = blockIdx.x;
  const int kvh = d.hr / P.rg;
  const int h0 = kvh * P.g + (P.rg > 1 ? (d.hr - kvh * P.rg) * 16 : 0);
  constexpr int kPaths = PATH == kPathGated ? 2 : 1;
  for (int i = threadIdx.x; i < d.nrows * (D / 4); i += 128) {
    const int r = i / (D / 4), c4 = i - r * (D / 4);
    const int tk = P.rg > 1 ? 0 : r / P.g;
    const size_t row = size_t(d.t0 + tk) * P.Hq + h0 + r - tk * P.g;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int path = 0; path < kPaths; ++path) {
      const bool is_swa = PATH == kPathSWA || path == 1;
      const long long lo = d.u0 + (is_swa ? d.tsa : 0), hi = lo + (is_swa ? d.tsw : d.tsa);
      if (hi <= lo) continue;
      const int ca = int(lo / d.per), cz = int((hi - 1) / d.per);
      auto piece = [&](int c) {
        return P.part + (size_t(c * 2 + (c == c0 ? 1 : 0)) * kPaths + path) * P.slot_floats;
      };
      float m = -INFINITY;
      for (int c = ca; c <= cz; ++c) m = fmaxf(m, piece(c)[P.R * D + 2 * r]);
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = ca; c <= cz; ++c) {
        const float* pw = piece(c);
        const float pm = pw[P.R * D + 2 * r];
        const float f = pm == -INFINITY ? 0.f : fast_exp2(pm - m);
        l = fmaf(f, pw[P.R * D + 2 * r + 1], l);
        const float4 v = *reinterpret_cast<const float4*>(pw + r * D + c4 * 4);
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
    if (PATH == kPathGated && d.add_swa) {
      const float4 v = *reinterpret_cast<const float4*>(P.swa_part + row * D + c4 * 4);
      y.x += v.x;
      y.y += v.y;
      y.z += v.z;
      y.w += v.w;
    }
    *reinterpret_cast<uint2*>(P.out + row * D + c4 * 4) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  }
}

// ------------------------------------------------------------------ host

struct Config {
  int tb, rg, R, slot_floats, warps, workers, split, min_tiles;
  uint32_t stage_bytes, warp_bytes;
  size_t part_bytes, desc_bytes;
};

static Config make_config(const PagedProblem& pb, Path path, int row_limit, int sms) {
  Config c;
  c.rg = (pb.g + 15) / 16;
  // several tokens share a unit's 16 rows only where they share a window
  const int most_new = min(pb.max_new, row_limit);
  c.tb = path == kPathSWA && pb.g < 16 ? min(16 / pb.g, most_new) : 1;
  c.R = c.rg > 1 ? 16 : c.tb * pb.g;
  c.slot_floats = (c.R * (pb.d + 2) + 3) / 4 * 4;  // 16-byte aligned slots
  const uint32_t pitch = uint32_t(pb.d) * 2 + 16;
  c.stage_bytes = (2 * kKeys + uint32_t(c.R)) * pitch + kMetaInts * 4;
  c.warp_bytes = c.stage_bytes * kStages;
  c.warps = int(kMaxSmem / c.warp_bytes);
  const int most_warps = pb.d == 128 ? 8 : 16;
  if (c.warps > most_warps) c.warps = most_warps;
  c.workers = sms * c.warps;
  // Runs end at unit ends, without partials, where there are at least four
  // units per worker of at most 1024 keys each.
  const long long units = (pb.T + c.tb - 1) / c.tb * (long long)pb.Hkv * c.rg;
  const long long keys = path == kPathSA ? 2LL * pb.half + 1
                         : path == kPathSWA ? (long long)pb.window_swa
                                            : 2LL * pb.half + 1 + pb.window_swa;
  c.split = !(units >= 4LL * c.workers && keys <= 1024);
  c.min_tiles = 4;
  c.part_bytes = c.split ? (size_t(c.workers) * 2 * (path == kPathGated ? 2 : 1) * c.slot_floats * 4 + 255) / 256 * 256
                         : 0;
  c.desc_bytes = c.split ? size_t(c.workers) * sizeof(Desc) : 0;
  return c;
}

template <int D, int PATH>
static cudaError_t launch_one(const Params& P, const Config& c, int sms, cudaStream_t stream) {
  const uint32_t smem = c.warp_bytes * uint32_t(c.warps);
  cudaError_t ce = cudaFuncSetAttribute(sa_paged_rows_kernel<D, PATH>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
  if (ce != cudaSuccess) return ce;
  sa_paged_rows_kernel<D, PATH><<<sms, 32 * c.warps, smem, stream>>>(P);
  if ((ce = cudaGetLastError()) != cudaSuccess || !c.split) return ce;
  sa_paged_join_kernel<D, PATH><<<c.workers, 128, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace prow

size_t paged_rows_workspace_bytes(const PagedProblem& pb, Path path, int row_limit, int sms) {
  const prow::Config c = prow::make_config(pb, path, row_limit, sms);
  return c.part_bytes + c.desc_bytes;
}

sa_status_t launch_paged_rows(const PagedProblem& pb, Path path, int row_limit,
                              const float* swa_part, void* part, int sms, cudaStream_t stream) {
  using namespace prow;
  const Config c = make_config(pb, path, row_limit, sms);
  Params P;
  std::memset(&P, 0, sizeof(P));
  P.q = static_cast<const __nv_bfloat16*>(pb.q);
  P.k = static_cast<const __nv_bfloat16*>(pb.k);
  P.v = static_cast<const __nv_bfloat16*>(pb.v);
  P.table = pb.table;
  P.q_start = pb.q_start;
  P.seq_lens = pb.seq_lens;
  P.perm = pb.perm;
  P.inv = pb.inv;
  P.gate_sa = pb.gate_sa;
  P.gate_swa = pb.gate_swa;
  P.swa_part = swa_part;
  P.out = static_cast<__nv_bfloat16*>(pb.out);
  P.err = pb.err;
  if (c.split) {
    P.part = static_cast<float*>(part);
    P.desc = reinterpret_cast<Desc*>(static_cast<char*>(part) + c.part_bytes);
  }
  P.q_stride = pb.q_stride;
  P.page_stride = pb.page_stride;
  P.perm_stride = pb.perm_rows == 1 ? 0 : pb.perm_len;
  P.B = pb.B;
  P.T = pb.T;
  P.max_new = pb.max_new;
  P.row_limit = row_limit;
  P.Hq = pb.Hq;
  P.Hkv = pb.Hkv;
  P.g = pb.g;
  P.page = pb.page;
  P.num_pages = pb.num_pages;
  P.max_pages = pb.max_pages;
  P.w = pb.window_swa;
  P.half = pb.half;
  P.perm_len = pb.perm_len;
  P.tb = c.tb;
  P.rg = c.rg;
  P.R = c.R;
  P.slot_floats = c.slot_floats;
  P.workers = c.workers;
  P.min_tiles = c.min_tiles;
  P.snap = c.split ? 0 : 1;
  P.stage_bytes = c.stage_bytes;
  P.warp_bytes = c.warp_bytes;
  P.scale_log2 = pb.scale * 1.4426950408889634f;
  cudaError_t ce;
  if (pb.d == 128)
    ce = path == kPathSWA ? launch_one<128, kPathSWA>(P, c, sms, stream)
         : path == kPathSA ? launch_one<128, kPathSA>(P, c, sms, stream)
                           : launch_one<128, kPathGated>(P, c, sms, stream);
  else
    ce = path == kPathSWA ? launch_one<64, kPathSWA>(P, c, sms, stream)
         : path == kPathSA ? launch_one<64, kPathSA>(P, c, sms, stream)
                           : launch_one<64, kPathGated>(P, c, sms, stream);
  if (ce != cudaSuccess) return fail(SA_ERR_CUDA, "paged row kernel launch: %s", cudaGetErrorString(ce));
  return SA_OK;
}

}  // namespace sa
