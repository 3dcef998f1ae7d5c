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
// fp32 partials (O, m, l) in the workspace, which the second kernel joins in
// worker order, so results do not depend on timing.  Where there are several
// short units per worker the runs end at unit ends and there is nothing to
// join.  (Few short units: sa_paged_unit.cu.)  A token each of 48 requests of
// up to 32768 tokens, 32 q heads on 8 kv heads of 128, takes 604 us for 3.85 GB:
// 94 % of what a plain copy reaches.
#include "sa_paged_rows.cuh"

#include <cstring>

namespace sa {
namespace prow {

// Two stages a warp and eleven warps (d = 128) beat three and seven, or four
// and five: 621, 649 and 652 us for a decoding batch of 48 requests of up to
// 32768 tokens (3.85 GB; 32 / 8 heads).  A warp spends its time on its own
// instructions, not on waiting for its loads.
constexpr int kStages = 2;
// A stage: 16 K rows, 16 V rows, the unit's Q rows, 16 key tokens and a word of flags.
constexpr int kMetaInts = 32;
enum : int {
  kFirst = 1,    // first tile of a piece (a unit's run of one path): reset O, m, l
  kLast = 2,     // last tile of the piece: write it
  kNewQ = 4,     // first tile of the unit here: the stage holds its Q rows
  kAny = 8,      // some key of the tile is loaded
  kClear = 16,   // every row attends to all 16 keys
  kNone = 32,    // no tile: the run is done
  kRaw = 64,     // (one lane) the key is an entry of sigma not yet looked at
  kWithin = 128, // SWA: the keys lie in every row's window
  kPieceShift = 16,
};
// What the pieces under way have in common, eight at most from make() to the
// last tile's sums.
constexpr int kPieces = 8;
struct Piece {
  int flags, pos0, rows, t0, hr, pad[3];
};
enum : int {
  kIsSwa = 1,    // the piece is of the SWA path
  kWhole = 2,    // the whole unit is this worker's
  kTail = 4,     // the unit starts in this worker's run (partial slot 1, else 0)
  kAddSwa = 8,   // gated: the SWA term comes from swa_part
};

// Where a position of the laid-out tiles lies: request, its fields, and the
// position's offset in the request's tiles.  All lanes of a warp call it.
struct Place {
  int b;
  Request r;
  long long off;
};

// The lengths of up to 32 requests, one per lane, and the sum of their tiles.
struct Scan {
  Request r;
  long long x, sum;  // tiles of this lane's request; inclusive sum over the lanes
};
template <int PATH>
__device__ __forceinline__ Scan scan32(const Params& P, int b0, int HR, bool report) {
  const int lane = threadIdx.x & 31;
  Scan s;
  s.x = 0;
  s.r = Request{0, 0, 0, 0, 0, 0};
  if (b0 + lane < P.B) {
    s.r = load_request<PATH>(P, b0 + lane, report);
    s.x = (long long)s.r.groups * HR * (s.r.tsa + s.r.tsw);
  }
  s.sum = s.x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, s.sum, o);
    if (lane >= o) s.sum += a;
  }
  return s;
}

// pos is below the sum of all tiles; `head` is the scan of the first 32.
template <int PATH>
__device__ __forceinline__ Place locate(const Params& P, const Scan& head, int HR, long long pos) {
  Scan s = head;
  long long before = 0;
  Place p;
  for (int b0 = 0;; b0 += 32) {
    if (b0 > 0) s = scan32<PATH>(P, b0, HR, false);
    const unsigned hit = __ballot_sync(0xffffffffu, before + s.sum > pos);
    if (hit != 0u || b0 + 32 >= P.B) {
      const int src = hit != 0u ? __ffs(hit) - 1 : 0;
      p.b = b0 + src;
      p.off = pos - (before + __shfl_sync(0xffffffffu, s.sum - s.x, src));
      p.r.q0 = __shfl_sync(0xffffffffu, s.r.q0, src);
      p.r.n = __shfl_sync(0xffffffffu, s.r.n, src);
      p.r.len = __shfl_sync(0xffffffffu, s.r.len, src);
      p.r.tsa = __shfl_sync(0xffffffffu, s.r.tsa, src);
      p.r.tsw = __shfl_sync(0xffffffffu, s.r.tsw, src);
      p.r.groups = __shfl_sync(0xffffffffu, s.r.groups, src);
      return p;
    }
    before += __shfl_sync(0xffffffffu, s.sum, 31);
  }
}

// Warps of a block: as many as shared memory and registers hold.
__host__ __device__ constexpr int most_warps(int d, int nt) {
  return d == 128 ? (nt == 2 ? 8 : 12) : (nt == 2 ? 12 : 16);
}

template <int D, int PATH, int NT>
__device__ __forceinline__ void rows_role(const Params& P) {
  constexpr int kPitch = Pitch<D>;
  constexpr int kCpr = D / 8;  // 16-byte chunks per row
  constexpr uint32_t kOffQ = 2 * kKeys * kPitch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int worker = warp * int(gridDim.x) + int(blockIdx.x);
  uint8_t* ring = smem_raw + size_t(warp) * P.warp_bytes;
  const uint32_t sring = smem_u32(ring);
  const uint32_t off_meta = kOffQ + uint32_t(P.R) * kPitch;
  Piece* pieces = reinterpret_cast<Piece*>(ring + kStages * P.stage_bytes);
  const int HR = P.Hkv * P.rg;

  // ---- this worker's run [begin, end) of all units' tiles
  const Scan head = scan32<PATH>(P, 0, HR, worker == 0);
  long long total = __shfl_sync(0xffffffffu, head.sum, 31);
  if (P.B > 32) {
    long long more = 0;
    for (int b = 32 + lane; b < P.B; b += 32) {
      const Request r = load_request<PATH>(P, b, worker == 0);
      more += (long long)r.groups * HR * (r.tsa + r.tsw);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
    total += more;
  }
  const long long per = max((total + P.workers - 1) / P.workers, (long long)P.min_tiles);
  const long long begin = per * worker;
  const long long end = min(total, begin + per);
  const bool snap = P.snap != 0;
  if (P.desc != nullptr && lane == 0) P.desc[worker].valid = 0;
  if (begin >= total) return;

  // ---- cursor: request, group, head and tile of the next tile to fetch
  int cb, cgrp, chr_, ctile;
  Request cr;
  long long cpos = begin;
  {
    const Place p = locate<PATH>(P, head, HR, begin);
    cb = p.b;
    cr = p.r;
    const int per_unit = cr.tsa + cr.tsw;
    const long long uh = p.off / per_unit;
    ctile = int(p.off - uh * per_unit);
    cgrp = int(uh / HR);
    chr_ = int(uh - (long long)cgrp * HR);
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
  if (snap && ctile != 0) {  // the unit cut here is the previous worker's
    cpos += cr.tsa + cr.tsw - ctile;
    next_unit();
  }

  // ---- pieces: the cursor's unit, path by path
  int piece = -1, left = 0;          // tiles of the piece still to be made
  int kcur = 0, khi = 0;             // next key (a position, or one of sigma's), end
  int upos0 = 0, ulast = 0, urows = 0, ut0 = 0, slo = 0, shi = 0, wlo = 0, whi = 0;
  int ukvh = 0, have_b = -1, have_grp = -1, first_flags = 0;
  bool fresh = true, swa = PATH == kPathSWA;
  auto next_piece = [&]() {
    if (piece >= 0 && ctile == cr.tsa + cr.tsw) {
      next_unit();
      fresh = true;
    }
    if (done || (snap ? (ctile == 0 && cpos >= end) : cpos >= end)) return false;
    const int per_unit = cr.tsa + cr.tsw;
    if (fresh) {
      const int i0 = cgrp * P.tb, nt = min(P.tb, cr.n - i0);
      upos0 = cr.len - cr.n + i0;
      ulast = upos0 + nt - 1;
      ut0 = cr.q0 + i0;
      ukvh = chr_ / P.rg;
      urows = P.rg > 1 ? min(16, P.g - (chr_ - ukvh * P.rg) * 16) : nt * P.g;
      wlo = max(0, upos0 - P.w + 1);
      whi = ulast + 1;
      if (PATH != kPathSWA && (have_b != cb || have_grp != cgrp)) {  // one token's heads share it
        have_b = cb;
        have_grp = cgrp;
        const int p = P.inv[(long long)cb * P.perm_stride + upos0];
        slo = shi = 0;
        if (unsigned(p) < unsigned(P.perm_len)) {
          slo = max(0, p - P.half);
          shi = int(min((long long)P.perm_len, (long long)p + P.half + 1));
        } else if (lane == 0) {
          atomicOr(P.err, SA_ERRBIT_RANGE);
        }
      }
    }
    swa = PATH == kPathSWA || (PATH == kPathGated && ctile >= cr.tsa);
    const int path_end = swa ? per_unit : cr.tsa;
    const long long ustart = cpos - ctile;
    const bool whole = snap || (ustart >= begin && ustart + per_unit <= end);
    left = snap ? path_end - ctile : int(min((long long)(path_end - ctile), end - cpos));
    const int pt = swa ? ctile - cr.tsa : ctile;
    kcur = (swa ? wlo : slo) + pt * kKeys;
    khi = swa ? whi : shi;
    ++piece;
    if (lane == 0) {
      Piece pc;
      pc.flags = (swa ? kIsSwa : 0) | (whole ? kWhole : 0) | (ustart >= begin ? kTail : 0) |
                 (PATH == kPathGated && cr.tsw == 0 ? kAddSwa : 0);
      pc.pos0 = upos0;
      pc.rows = urows;
      pc.t0 = ut0;
      pc.hr = chr_;
      pc.pad[0] = pc.pad[1] = pc.pad[2] = 0;
      pieces[piece % kPieces] = pc;
      if (fresh && !whole && ustart >= begin) {
        Desc d;
        d.valid = 1;
        d.t0 = ut0;
        d.hr = chr_;
        d.nrows = urows;
        d.tsa = cr.tsa;
        d.tsw = cr.tsw;
        d.add_swa = PATH == kPathGated && cr.tsw == 0;
        d.pad = 0;
        d.u0 = ustart;
        d.per = per;
        P.desc[worker] = d;
      }
    }
    first_flags = kFirst | (fresh ? kNewQ : 0);
    fresh = false;
    cpos += left;
    ctile += left;
    return true;
  };

  // ---- tiles on their way: A has its page ids, B its key tokens
  struct Tile {
    int flags, tok, b, kvh, pos0;  // tok: this lane's key (lane & 15), -1: none
  };
  auto make = [&]() -> Tile {
    Tile t;
    t.tok = -1;
    t.flags = kNone;
    t.b = t.kvh = t.pos0 = 0;
    if (left == 0 && !next_piece()) return t;
    int flags = first_flags | (piece % kPieces) << kPieceShift;
    first_flags = 0;
    if (--left == 0) flags |= kLast;
    const int key = kcur + (lane & 15);
    if (swa) {
      if (kcur + kKeys - 1 <= upos0 && ulast - kcur < P.w) flags |= kWithin;
      if (key < khi) t.tok = key;
    } else if (key < khi) {
      t.tok = P.perm[(long long)cb * P.perm_stride + key];
      flags |= kRaw;
    }
    kcur += kKeys;
    t.flags = flags;
    t.b = cb;
    t.kvh = ukvh;
    t.pos0 = upos0;
    return t;
  };
  // sigma's entries are looked at a step after their loads began
  auto settle = [&](Tile& t) {
    if (PATH == kPathSWA || !(t.flags & kRaw)) return;
    t.flags = (t.flags & ~kRaw) | kWithin;
    if (unsigned(t.tok) >= unsigned(P.perm_len)) {
      atomicOr(P.err, SA_ERRBIT_RANGE);
      t.tok = -1;
    } else if (t.tok > t.pos0) {
      t.tok = -1;  // a later token
    }
  };
  auto page_of = [&](const Tile& t) {  // -1: no key
    return t.tok >= 0 ? P.table[(long long)t.b * P.max_pages + page_col(P, t.tok)] : -1;
  };
  auto issue = [&](const Tile& t, int page, int stage) {
    uint8_t* st = ring + uint32_t(stage) * P.stage_bytes;
    const uint32_t ss = sring + uint32_t(stage) * P.stage_bytes;
    int* meta = reinterpret_cast<int*>(st + off_meta);
    if (t.flags & kNone) {
      if (lane == 0) meta[kKeys] = kNone;
      return;
    }
    uint32_t row = 0xffffffffu;
    if (t.tok >= 0) {
      if (unsigned(page) < unsigned(P.num_pages))
        row = uint32_t(page) * uint32_t(P.page_rows) + uint32_t(page_in(P, t.tok)) * uint32_t(P.Hkv) + uint32_t(t.kvh);
      else
        atomicOr(P.err, SA_ERRBIT_RANGE);
    }
    const unsigned have = __ballot_sync(0xffffffffu, row != 0xffffffffu);
    const bool clear = __all_sync(0xffffffffu, row != 0xffffffffu && (t.flags & kWithin));
    if (lane < kKeys) meta[lane] = row != 0xffffffffu ? t.tok : 0x7fffffff;
    if (lane == 0) meta[kKeys] = (t.flags & ~kRaw) | (have != 0u ? kAny : 0) | (clear ? kClear : 0);
    if (have != 0u) load_tile<D>(P.k, P.v, ss, row);
    if (t.flags & kNewQ) {
      __syncwarp();
      const Piece* pc = pieces + ((t.flags >> kPieceShift) & (kPieces - 1));
      const int rows = pc->rows, t0 = pc->t0;
      const int h0 = t.kvh * P.g + (P.rg > 1 ? (pc->hr - t.kvh * P.rg) * 16 : 0);
      for (int i = lane; i < rows * kCpr; i += 32) {
        const int r = i / kCpr, c = i - r * kCpr;
        const int tk = P.rg > 1 ? 0 : r / P.g;
        cp_async16(ss + kOffQ + r * kPitch + c * 16,
                   P.q + (long long)(t0 + tk) * P.q_stride + (h0 + r - tk * P.g) * D + c * 8);
      }
    }
  };

  // ---- the pipeline
  Tile ta = make();
  settle(ta);
  int pa = page_of(ta);
  Tile tn = make();
  auto step = [&](int stage) {
    issue(ta, pa, stage);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ta = tn;
    settle(ta);
    pa = page_of(ta);
    tn = make();
  };
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) step(i);

  Acc<D, NT> acc;
  float stash[PATH == kPathGated ? D / 16 : 1][NT][4];
  acc.reset();
  int stage = 0, fill = kStages - 1;
  int pflags = 0, rows = 0, t0 = 0, h0 = 0;
  unsigned w = 0;
  while (true) {
    step(fill);
    fill = fill + 1 == kStages ? 0 : fill + 1;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    uint8_t* st = ring + uint32_t(stage) * P.stage_bytes;
    const uint32_t ss = sring + uint32_t(stage) * P.stage_bytes;
    const int* meta = reinterpret_cast<const int*>(st + off_meta);
    const int flags = meta[kKeys];
    if (flags & kNone) break;
    if (flags & kFirst) {
      const Piece* pc = pieces + ((flags >> kPieceShift) & (kPieces - 1));
      pflags = pc->flags;
      rows = pc->rows;
      t0 = pc->t0;
      const int hr = pc->hr, kvh = hr / P.rg;
      h0 = kvh * P.g + (P.rg > 1 ? (hr - kvh * P.rg) * 16 : 0);
      w = pflags & kIsSwa ? unsigned(P.w) : 0x7fffffffu;
      acc.reset();
      if (flags & kNewQ) acc.rows_of(ss + kOffQ, rows, pc->pos0, P.g, P.rg > 1);
    }
    if (flags & kAny) acc.tile(ss, meta, w, (flags & kClear) != 0, P.scale_log2);
    if (flags & kLast) {
      acc.sum_rows();
      if (!(pflags & kWhole)) {
        const int slot = (worker * 2 + ((pflags & kTail) ? 1 : 0)) * (PATH == kPathGated ? 2 : 1) +
                         (PATH == kPathGated && (pflags & kIsSwa) ? 1 : 0);
        acc.write(P.part + size_t(slot) * P.slot_floats, P.R, rows);
      } else {
        const bool write = PATH != kPathGated || (pflags & (kIsSwa | kAddSwa)) != 0;
        uint8_t* os = st + kOffQ;  // this stage's Q rows, whose fragments were taken
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = t * 8 + 2 * (lane & 3) + e;
            const int tk = P.rg > 1 ? 0 : r / P.g;
            const size_t orow = size_t(t0 + tk) * P.Hq + h0 + r - tk * P.g;
            float f = acc.l[t][e] == 0.f ? 0.f : 1.f / acc.l[t][e];
            if (PATH == kPathGated && r < rows)
              f *= 1.f / (1.f + expf(-((pflags & kIsSwa) ? P.gate_swa : P.gate_sa)[orow]));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float y = acc.o[i][t][2 * h + e] * f;
                const int col = i * 16 + (lane >> 2) + 8 * h;
                if (PATH == kPathGated) {
                  if (pflags & kIsSwa)
                    y += stash[i][t][2 * h + e];
                  else if (!write)
                    stash[i][t][2 * h + e] = y;
                  else if (r < rows)
                    y += P.swa_part[orow * D + col];
                }
                if (write && r < rows)
                  *reinterpret_cast<__nv_bfloat16*>(os + r * kPitch + col * 2) = __float2bfloat16_rn(y);
              }
            }
          }
        }
        if (write) {
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

template <int D, int PATH, int NT>
__global__ void __launch_bounds__(32 * most_warps(D, NT), 1)
    sa_paged_rows_kernel(const __grid_constant__ Params P) {
  if (P.beside) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else {
    begin_after();
  }
  rows_role<D, PATH, NT>(P);
  end_beside();
}

// Joins the parts of each unit that the runs cut, piece after piece in worker
// order: block c takes the unit that starts in worker c's run.
template <int D, int PATH>
__global__ void __launch_bounds__(128) sa_paged_join_kernel(const __grid_constant__ Params P) {
  begin_after();
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
#pragma unroll 4
      for (int c = ca; c <= cz; ++c) m = fmaxf(m, piece(c)[P.R * D + 2 * r]);
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
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
  int tb, rg, R, slot_floats, warps, workers, snap;
  uint32_t stage_bytes, warp_bytes;
  size_t part_bytes, desc_bytes;
};

static Config make_config(const PagedProblem& pb, Path path, int row_limit, int sms) {
  Config c;
  paged_unit_shape(pb, path, row_limit, &c.tb, &c.rg, &c.R);
  c.slot_floats = (c.R * (pb.d + 2) + 3) / 4 * 4;  // 16-byte aligned slots
  const uint32_t pitch = uint32_t(pb.d) * 2 + 16;
  c.stage_bytes = (2 * kKeys + uint32_t(c.R)) * pitch + kMetaInts * 4;
  c.warp_bytes = c.stage_bytes * kStages + kPieces * uint32_t(sizeof(Piece));
  c.warps = int(kMaxSmem / c.warp_bytes);
  c.warps = min(c.warps, most_warps(pb.d, c.R > 8 ? 2 : 1));
  c.workers = sms * c.warps;
  // Short units are left whole where there are at least four for each worker.
  const long long units = (pb.T + c.tb - 1) / c.tb * (long long)pb.Hkv * c.rg;
  c.snap = units >= 4LL * c.workers && paged_unit_keys(pb, path, c.tb) <= 1280;
  c.part_bytes =
      c.snap ? 0 : (size_t(c.workers) * 2 * (path == kPathGated ? 2 : 1) * c.slot_floats * 4 + 255) / 256 * 256;
  c.desc_bytes = c.snap ? 0 : size_t(c.workers) * sizeof(Desc);
  return c;
}

template <int D, int PATH, int NT>
static cudaError_t launch_rows(const Params& P, const Config& c, int sms, cudaStream_t stream) {
  const uint32_t smem = c.warp_bytes * uint32_t(c.warps);
  const cudaError_t ce = allow_smem<sa_paged_rows_kernel<D, PATH, NT>>(kMaxSmem);
  if (ce != cudaSuccess) return ce;
  return launch_kernel(sa_paged_rows_kernel<D, PATH, NT>, dim3(unsigned(sms)), unsigned(32 * c.warps), smem, stream,
                       P);
}

template <int D, int PATH>
static cudaError_t launch_one(const Params& P, const Config& c, int sms, cudaStream_t stream) {
  const cudaError_t ce = c.R <= 8 ? launch_rows<D, PATH, 1>(P, c, sms, stream) : launch_rows<D, PATH, 2>(P, c, sms, stream);
  if (ce != cudaSuccess || c.snap) return ce;
  // its blocks may be set up while the row kernel's last ones finish
  return launch_kernel(sa_paged_join_kernel<D, PATH>, dim3(unsigned(c.workers)), 128, 0, stream, P);
}

void fill_params(Params* out, const PagedProblem& pb, Path path, int row_limit, const float* swa_part) {
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
  P.q_stride = pb.q_stride;
  P.page_rows = int(pb.page_stride / pb.d);
  P.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (pb.page == 1 << i) P.page_shift = i;
  P.perm_stride = pb.perm_rows == 1 ? 0 : pb.perm_len;
  P.B = pb.B;
  P.T = pb.T;
  P.max_new = pb.max_new;
  P.row_limit = row_limit;
  P.sa_limit = pb.sa_limit;
  P.beside = pb.beside;
  P.Hq = pb.Hq;
  P.Hkv = pb.Hkv;
  P.g = pb.g;
  P.page = pb.page;
  P.num_pages = pb.num_pages;
  P.max_pages = pb.max_pages;
  P.w = pb.window_swa;
  P.half = pb.half;
  P.perm_len = pb.perm_len;
  paged_unit_shape(pb, path, row_limit, &P.tb, &P.rg, &P.R);
  P.scale_log2 = pb.scale * 1.4426950408889634f;
  *out = P;
}

}  // namespace prow

// Units: several tokens share the 16 rows only where they share a window.
void paged_unit_shape(const PagedProblem& pb, Path path, int row_limit, int* tb, int* rg, int* rows) {
  *rg = (pb.g + 15) / 16;
  *tb = path == kPathSWA && pb.g < 16 ? min(16 / pb.g, min(pb.max_new, row_limit)) : 1;
  *rows = *rg > 1 ? 16 : *tb * pb.g;
}

// The most keys that a unit attends to.
long long paged_unit_keys(const PagedProblem& pb, Path path, int tb) {
  const long long swa = min((long long)pb.window_swa + tb - 1, (long long)pb.max_pages * pb.page);
  const long long near = min(2LL * pb.half + 1, (long long)pb.perm_len);
  return path == kPathSWA ? swa : path == kPathSA ? near : swa + near;
}

size_t paged_rows_workspace_bytes(const PagedProblem& pb, Path path, int row_limit, int sms) {
  const prow::Config c = prow::make_config(pb, path, row_limit, sms);
  return c.part_bytes + c.desc_bytes;
}

sa_status_t launch_paged_rows(const PagedProblem& pb, Path path, int row_limit,
                              const float* swa_part, void* part, int sms, cudaStream_t stream) {
  using namespace prow;
  const Config c = make_config(pb, path, row_limit, sms);
  Params P;
  fill_params(&P, pb, path, row_limit, swa_part);
  if (!c.snap) {
    P.part = static_cast<float*>(part);
    P.desc = reinterpret_cast<Desc*>(static_cast<char*>(part) + c.part_bytes);
  }
  P.slot_floats = c.slot_floats;
  P.workers = c.workers;
  P.min_tiles = 4;
  P.snap = c.snap;
  P.stage_bytes = c.stage_bytes;
  P.warp_bytes = c.warp_bytes;
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
