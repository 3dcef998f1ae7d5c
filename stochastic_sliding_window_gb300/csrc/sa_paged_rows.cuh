// Device pieces shared by the kernels on the warp-level matrix instructions
// (sa_paged_rows.cu, sa_paged_unit.cu, sa_paged_members.cu): the request's fields, the warp-level
// matrix instructions, and one 16-key tile of the online softmax of a unit of
// up to 16 query rows.
#pragma once

#include "sa_internal.h"
#include "sa_tc_common.cuh"

namespace sa {
namespace prow {

using namespace tcc;

constexpr int kKeys = 16;   // keys per tile
constexpr uint32_t kMaxSmem = 232448;

struct Desc {  // one per worker: the unit that starts in its run and ends beyond it
  int valid, t0, hr, nrows, tsa, tsw, add_swa, pad;
  long long u0, per;  // its first tile; tiles per run
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
  long long q_stride, perm_stride;
  int B, T, max_new, row_limit, sa_limit, Hq, Hkv, g, page, page_shift, num_pages, max_pages;
  int page_rows;          // rows of D elements between pages
  int w, half, perm_len;
  int tb, rg, R;          // tokens and rows of a unit; row groups of a kv head (g > 16)
  int slot_floats;        // one partial: O [R, D], then (m, l) [R]; a multiple of 4
  int workers, min_tiles, snap;  // snap: runs end at unit ends
  uint32_t stage_bytes, warp_bytes;
  int beside;             // launched beside the tile kernel
  int gmax, list_keys, stages;    // unit kernel: groups per request, key list, stages per warp
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
  if (PATH != kPathSWA && paged_sa_tiled(r.n, r.len, P.half, P.sa_limit)) r.n = 0;
  const bool swa_here = r.n <= P.row_limit;
  if (PATH == kPathSWA && !swa_here) r.n = 0;
  if (PATH != kPathSWA) r.tsa = int((min(2LL * P.half + 1, (long long)P.perm_len) + kKeys - 1) / kKeys);
  if (PATH != kPathSA && swa_here)
    r.tsw = int((min((long long)r.len, (long long)P.w + P.tb - 1) + kKeys - 1) / kKeys);
  r.groups = ceil_div(r.n, P.tb);
  return r;
}

// Bytes between rows of a tile in shared memory: 16 over, so that the eight
// rows of a matrix load hit all banks.
template <int D>
constexpr int Pitch = D * 2 + 16;

// Page and row of a position (page_shift: log2 of a page size that is a power
// of two, else -1).
__device__ __forceinline__ int page_col(const Params& P, int tok) {
  return P.page_shift >= 0 ? tok >> P.page_shift : int(unsigned(tok) / unsigned(P.page));
}
__device__ __forceinline__ int page_in(const Params& P, int tok) {
  return P.page_shift >= 0 ? tok & (P.page - 1) : int(unsigned(tok) % unsigned(P.page));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Loads 16 keys' rows of K and V (row numbers of D elements in lanes 0-15,
// 0xffffffff: none, filled with zeros) into a stage.
template <int D>
__device__ __forceinline__ void load_tile(const __nv_bfloat16* k, const __nv_bfloat16* v, uint32_t stage,
                                          uint32_t row) {
  constexpr int kCpr = D / 8;
  const int lane = threadIdx.x & 31, c = lane % kCpr;
  const uint32_t dst = stage + (lane / kCpr) * Pitch<D> + c * 16;
  const char* kc = reinterpret_cast<const char*>(k + c * 8);
  const char* vc = reinterpret_cast<const char*>(v + c * 8);
  if (__all_sync(0xffffffffu, row != 0xffffffffu)) {
#pragma unroll
    for (int i = 0; i < kKeys * kCpr / 32; ++i) {
      const uint32_t r = __shfl_sync(0xffffffffu, row, i * (32 / kCpr) + lane / kCpr);
      const uint64_t at = uint64_t(r) * uint32_t(D * 2);
      cp_async16(dst + i * (32 / kCpr) * Pitch<D>, kc + at);
      cp_async16(dst + (kKeys + i * (32 / kCpr)) * Pitch<D>, vc + at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kKeys * kCpr / 32; ++i) {
      const uint32_t r = __shfl_sync(0xffffffffu, row, i * (32 / kCpr) + lane / kCpr);
      const int bytes = r != 0xffffffffu ? 16 : 0;
      const uint64_t at = uint64_t(r != 0xffffffffu ? r : 0u) * uint32_t(D * 2);
      cp_async16_zfill(dst + i * (32 / kCpr) * Pitch<D>, kc + at, bytes);
      cp_async16_zfill(dst + (kKeys + i * (32 / kCpr)) * Pitch<D>, vc + at, bytes);
    }
  }
}

// A warp's running softmax of 8 NT query rows.  Both products are taken
// transposed, so that the 16 of the matrix instruction's M are keys, then
// columns of O, and its 8 of N are query rows -- a unit of up to 8 rows (any
// decoding with up to 8 query heads per kv head) wastes nothing:
//   S^T [16 keys, 8 rows] = K Q^T,   O^T [D, 8 rows] += V^T P^T.
// This lane's rows are 8 nt + 2 (lane % 4) + {0, 1}; its keys lane / 4 and
// lane / 4 + 8; its columns of O 16 i + lane / 4 and 8 more.  P turns from the
// first product's result layout to the second's operand layout by a transpose
// of 8 x 8 blocks in registers.
template <int D, int NT>
struct Acc {
  uint32_t qf[D / 16][NT][2];  // Q^T fragments
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];    // maxima in log2 units; sums: this lane's share
  int pos[NT][2];              // the rows' positions (-1: no row)

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
#pragma unroll
      for (int t = 0; t < NT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
    }
  }

  // The unit's rows: Q at sq; row r is of the token r / g (of the one token
  // where a unit holds one) from position pos0 on.  Rows past the last read
  // the first: all their weights are masked.
  __device__ __forceinline__ void rows_of(uint32_t sq, int rows, int pos0, int g, bool one) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int r = t * 8 + (lane & 7);
      if (r >= rows) r = 0;
      const uint32_t a = sq + r * Pitch<D> + (lane >> 3) * 16;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t f[4];
        ldsm4(a + i * 64, f);
        qf[2 * i][t][0] = f[0];
        qf[2 * i][t][1] = f[1];
        qf[2 * i + 1][t][0] = f[2];
        qf[2 * i + 1][t][1] = f[3];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = t * 8 + 2 * (lane & 3) + e;
        pos[t][e] = row < rows ? pos0 + (one ? 0 : row / g) : -1;
      }
    }
  }

  // Scores, in log2 units, of 16 keys whose K rows are at sk.
  __device__ __forceinline__ void scores(uint32_t sk, float scale_log2, float (&s)[NT][4]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    {
      const uint32_t a = sk + ((lane & 7) + ((lane >> 3) & 1) * 8) * Pitch<D> + (lane >> 4) * 16;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t kf[4];
        ldsm4(a + i * 32, kf);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(s[t], kf, qf[i][t][0], qf[i][t][1]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] *= scale_log2;
    }
  }

  // 16 keys: K rows at sk, V rows behind them, their tokens in toks
  // (0x7fffffff: no key); a row attends to tokens p - w + 1 .. p of its
  // position p.  clear: every real row attends to all of them.
  __device__ __forceinline__ void tile(uint32_t sk, const int* toks, unsigned w, bool clear, float scale_log2) {
    const int lane = threadIdx.x & 31;
    float s[NT][4];
    scores(sk, scale_log2, s);
    if (!clear) {
      const int ta = toks[lane >> 2], tb = toks[(lane >> 2) + 8];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (unsigned(pos[t][0] - ta) >= w) s[t][0] = -INFINITY;
        if (unsigned(pos[t][1] - ta) >= w) s[t][1] = -INFINITY;
        if (unsigned(pos[t][0] - tb) >= w) s[t][2] = -INFINITY;
        if (unsigned(pos[t][1] - tb) >= w) s[t][3] = -INFINITY;
      }
    }
    absorb<true>(sk, s);
  }

  // Takes 16 masked scores per row, and the V rows behind the K rows at sk, into
  // the running softmax.  kLow: P's rounding to bf16 is made up for by a second
  // product with what it left out.
  template <bool kLow>
  __device__ __forceinline__ void absorb(uint32_t sk, float (&s)[NT][4]) {
    const int lane = threadIdx.x & 31;
    float x[NT][2];
    bool up = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      x[t][0] = fmaxf(s[t][0], s[t][2]);
      x[t][1] = fmaxf(s[t][1], s[t][3]);
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        x[t][0] = fmaxf(x[t][0], __shfl_xor_sync(0xffffffffu, x[t][0], d));
        x[t][1] = fmaxf(x[t][1], __shfl_xor_sync(0xffffffffu, x[t][1], d));
      }
      up = up || x[t][0] > m[t][0] || x[t][1] > m[t][1];
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float n = fmaxf(m[t][e], x[t][e]);
          f[e] = m[t][e] == -INFINITY ? 0.f : fast_exp2(m[t][e] - n);
          m[t][e] = n;
          l[t][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][t][0] *= f[0];
          o[i][t][1] *= f[1];
          o[i][t][2] *= f[0];
          o[i][t][3] *= f[1];
        }
      }
    }
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float b0 = m[t][0] == -INFINITY ? 0.f : m[t][0], b1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = fast_exp2(s[t][2 * h] - b0), p1 = fast_exp2(s[t][2 * h + 1] - b1);
        l[t][0] += p0;
        l[t][1] += p1;
        const uint32_t a = pack_bf16x2(p0, p1);
        hi[t][h] = transpose8(a);
        if (kLow) lo[t][h] = transpose8(pack_bf16x2(p0 - __uint_as_float(a << 16), p1 - __uint_as_float(a & 0xffff0000u)));
      }
    }
    const uint32_t a = sk + (kKeys + (lane & 7) + (lane >> 4) * 8) * Pitch<D> + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t vf[4];
      ldsm4t(a + i * 32, vf);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16816(o[i][t], vf, hi[t][0], hi[t][1]);
        if (kLow) mma16816(o[i][t], vf, lo[t][0], lo[t][1]);
      }
    }
  }

  // The lanes' shares of the rows' sums to every lane of the row.
  __device__ __forceinline__ void sum_rows() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        l[t][0] += __shfl_xor_sync(0xffffffffu, l[t][0], d);
        l[t][1] += __shfl_xor_sync(0xffffffffu, l[t][1], d);
      }
    }
  }

  // O [R, D], then (m, l) [R], of the first `rows` rows.
  __device__ __forceinline__ void write(float* pw, int R, int rows) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = t * 8 + 2 * (lane & 3) + e;
        if (r >= rows) continue;
        if (lane < 4) {
          pw[R * D + 2 * r] = m[t][e];
          pw[R * D + 2 * r + 1] = l[t][e];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          pw[r * D + i * 16 + (lane >> 2)] = o[i][t][e];
          pw[r * D + i * 16 + (lane >> 2) + 8] = o[i][t][2 + e];
        }
      }
    }
  }
};

void fill_params(Params* out, const PagedProblem& pb, Path path, int row_limit, const float* swa_part);

}  // namespace prow
}  // namespace sa
