// Device pieces shared by the two kernels for requests with few new tokens
// (sa_paged_rows.cu, sa_paged_unit.cu): the request's fields, the warp-level
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
  long long q_stride, page_stride, perm_stride;
  int B, T, max_new, row_limit, Hq, Hkv, g, page, num_pages, max_pages;
  int w, half, perm_len;
  int tb, rg, R;          // tokens and rows of a unit; row groups of a kv head (g > 16)
  int slot_floats;        // one partial: O [R, D], then (m, l) [R]; a multiple of 4
  int workers, min_tiles, snap;  // snap: runs end at unit ends
  uint32_t stage_bytes, warp_bytes;
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

// A fragments of a unit's query rows.  Rows past the last read the first:
// their weights are all masked.
template <int D>
__device__ __forceinline__ void load_q(uint32_t sq, int rows, uint32_t (&qf)[D / 16][4]) {
  const int lane = threadIdx.x & 31;
  int r = (lane & 7) + ((lane >> 3) & 1) * 8;
  if (r >= rows) r = 0;
  const uint32_t a = sq + r * Pitch<D> + (lane >> 4) * 16;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) ldsm4(a + i * 32, qf[i]);
}

// A warp's running softmax of 16 rows: this lane's rows are lane / 4 and
// lane / 4 + 8, its columns 8 i + 2 (lane % 4) and the next.
template <int D>
struct Acc {
  float o[D / 8][4];
  float m0, m1, l0, l1;  // maxima in log2 units; the sums are this lane's share

  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // 16 keys: K rows at sk, V rows at sv, their tokens in tok (0x7fffffff: no
  // key).  p0, p1: the positions of this lane's rows (-1: no row); a row
  // attends to tokens p - w + 1 .. p.
  __device__ __forceinline__ void tile(uint32_t sk, uint32_t sv, const int* toks,
                                       const uint32_t (&qf)[D / 16][4], int p0, int p1, unsigned w,
                                       float scale_log2) {
    constexpr int kPitch = Pitch<D>;
    const int lane = threadIdx.x & 31;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const uint32_t a = sk + ((lane & 7) + (lane >> 4) * 8) * kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t kf[4];
        ldsm4(a + i * 32, kf);
        mma16816(s[0], qf[i], kf[0], kf[1]);
        mma16816(s[1], qf[i], kf[2], kf[3]);
      }
    }
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int2 tok = *reinterpret_cast<const int2*>(toks + t * 8 + (lane & 3) * 2);
      s[t][0] = unsigned(p0 - tok.x) < w ? s[t][0] * scale_log2 : -INFINITY;
      s[t][1] = unsigned(p0 - tok.y) < w ? s[t][1] * scale_log2 : -INFINITY;
      s[t][2] = unsigned(p1 - tok.x) < w ? s[t][2] * scale_log2 : -INFINITY;
      s[t][3] = unsigned(p1 - tok.y) < w ? s[t][3] * scale_log2 : -INFINITY;
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
    const uint32_t a = sv + ((lane & 7) + ((lane >> 3) & 1) * 8) * kPitch + (lane >> 4) * 16;
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

  // The lanes' shares of the rows' sums to every lane of the row.
  __device__ __forceinline__ void sum_rows() {
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
  }

  // O [R, D], then (m, l) [R], of the first `rows` rows.
  __device__ __forceinline__ void write(float* pw, int R, int rows) const {
    const int lane = threadIdx.x & 31;
    const int r0 = lane >> 2, r1 = r0 + 8;
    if (r0 < rows) {
      if ((lane & 3) == 0) {
        pw[R * D + 2 * r0] = m0;
        pw[R * D + 2 * r0 + 1] = l0;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(pw + r0 * D + i * 8 + (lane & 3) * 2) = make_float2(o[i][0], o[i][1]);
    }
    if (r1 < rows) {
      if ((lane & 3) == 0) {
        pw[R * D + 2 * r1] = m1;
        pw[R * D + 2 * r1 + 1] = l1;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(pw + r1 * D + i * 8 + (lane & 3) * 2) = make_float2(o[i][2], o[i][3]);
    }
  }
};

void fill_params(Params* out, const PagedProblem& pb, Path path, int row_limit, const float* swa_part);

}  // namespace prow
}  // namespace sa
