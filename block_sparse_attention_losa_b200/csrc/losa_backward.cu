// losa_backward.cu - the gradient of block-sparse attention over a frozen
// pattern (losa_sparse_attn_bwd), probabilities recomputed.
//
// Mathematics, per head, over the kept (query, key) pairs:
//   P_ij = exp(scale q_i.k_j - lse_i)         the forward pass's weights
//   D_i  = dO_i . O_i                         = sum_j P_ij dP_ij
//   dV_j = sum_i P_ij dO_i
//   dS_ij = P_ij (dO_i.v_j - D_i)
//   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i.
// dK and dV sum over queries and dQ over keys, so two kernels run, each
// owning its output rows: no atomics, the same bits every time, and no fp32
// gradient buffer that has to be cleared and converted. The price is that
// scores and dP are computed twice (seven products instead of five).
#include <algorithm>

#include "losa_device.cuh"
#include "losa_internal.h"

namespace losa {
namespace {

// ------------------------------------------------------------------ D

// D_i = dO_i . O_i, one warp per row; rows of the padding get 0. The sum is
// held in fp32. With `rounded`, dO (fp32) is first rounded to bf16, the form
// in which the products of the bf16 path read it, and that copy is written:
// D then cancels against the same dO that dP is made of.
template <int D>
__device__ __forceinline__ void load_row(const void* base, bool bf16, size_t row, int lane,
                                         float (&v)[D / 32]) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p + e));
      v[e] = __uint_as_float(u << 16);
      v[e + 1] = __uint_as_float(u & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(base) + row * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      const float2 u = __ldg(reinterpret_cast<const float2*>(p + e));
      v[e] = u.x;
      v[e + 1] = u.y;
    }
  }
}

// Three bf16 terms whose sum is x to 24 bits, as the first columns of a
// 16-column operand row (the other columns 0).
__device__ __forceinline__ uint4 split3(float x) {
  const uint32_t h = pack_bf16x2(x, 0.f) & 0xffffu;
  const float r1 = x - __uint_as_float(h << 16);
  const uint32_t m = pack_bf16x2(r1, 0.f) & 0xffffu;
  const float r2 = r1 - __uint_as_float(m << 16);
  const uint32_t l = pack_bf16x2(r2, 0.f) & 0xffffu;
  return make_uint4(h | (m << 16), l, 0u, 0u);
}

// The bf16 path's further operand rows, which carry -lse / scale and -D into
// its products: 8-row groups of two 8 x 16-byte core matrices each.
struct AugRows {
  uint4 *q, *d_o;  // null on the fp32 path
  const float* lse;
  float inv_scale;
};

template <int D>
__global__ void __launch_bounds__(256)
    delta_kernel(const void* o, bool o_bf16, const void* d_o, bool do_bf16, int64_t rows,
                 int L, int L_pad, float* delta, uint16_t* rounded, const AugRows aug) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  float sum = 0.f;
  if (row % L_pad < L) {
    float a[D / 32], b[D / 32];
    load_row<D>(o, o_bf16, row, lane, a);
    load_row<D>(d_o, do_bf16, row, lane, b);
    if (rounded) {
      uint32_t* w = reinterpret_cast<uint32_t*>(rounded + row * D + lane * (D / 32));
#pragma unroll
      for (int e = 0; e < D / 32; e += 2) {
        w[e / 2] = pack_bf16x2(b[e], b[e + 1]);
        b[e] = __uint_as_float(w[e / 2] << 16);
        b[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) sum = fmaf(a[e], b[e], sum);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) delta[row] = sum;
  if (aug.q && lane < 4) {
    // Lanes 0, 1: the row's two halves of q's columns; 2, 3: of dO's. Padded
    // rows get a score far below any other, so their weight is 0; values are
    // kept inside bf16's range.
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) {
      const float a = row % L_pad < L ? -aug.lse[row] * aug.inv_scale : -3e38f;
      x = split3(fminf(fmaxf(a, -3e38f), 3e38f));
    } else if (lane == 2) {
      x = split3(fminf(fmaxf(-sum, -3e38f), 3e38f));
    }
    (lane < 2 ? aug.q : aug.d_o)[(row >> 3) * 16 + (lane & 1) * 8 + (row & 7)] = x;
  }
}

// ------------------------------------------------------------------ fp32

struct SimtParams {
  const float *q, *k, *v;
  const void* d_o;
  bool do_bf16, out_bf16;
  const float *lse, *delta;
  int L, L_pad, n_qt, block;
  float scale;
  const int *ptr, *entry, *order;
  void *dq, *dk, *dv;
};

__device__ __forceinline__ float load_value(const void* p, bool bf16, size_t i) {
  return bf16 ? __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + i)) << 16)
              : __ldg(static_cast<const float*>(p) + i);
}

__device__ __forceinline__ void store4(void* p, bool bf16, size_t i, float4 x) {
  if (bf16) {
    uint2 w;
    w.x = pack_bf16x2(x.x, x.y);
    w.y = pack_bf16x2(x.z, x.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = x;
  }
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 64;  // rows a CTA owns, and rows per step

template <int D> struct SimtSmem {
  float x[kSimtRows][D + 4], x2[kSimtRows][D + 4];  // own rows: K, V or Q, dO
  float y[kSimtRows][D + 4], y2[kSimtRows][D + 4];  // a step's rows: Q, dO or K, V
  float p[kSimtRows][kSimtRows + 4], ds[kSimtRows][kSimtRows + 4];  // [step row][own row]
};

// One CTA owns half of a 128-row tile: 64 key rows (kKeys: dK and dV) or 64
// query rows (dQ), and walks the tile's list 64 rows of the other side at a
// time: two segments of 32 rows, the unit in which a block of any size (32,
// 64, 128) starts and ends. Every product is fp32 FMA: 256 threads hold a
// 64 x 64 score tile (4 x 4 each) and a 64 x D gradient tile (4 x D / 16
// each).
template <int D, bool kKeys>
__global__ void __launch_bounds__(kSimtThreads)
    bwd_simt_kernel(const SimtParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem_raw);
  constexpr int NC = D / 64;  // float4 groups of a gradient row per thread
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int tile = p.order[blockIdx.x >> 1], half = blockIdx.x & 1;
  const int bh = tile / p.n_qt;
  const int own0 = (tile - bh * p.n_qt) * 128 + half * 64;
  if (own0 >= p.L_pad) return;
  const size_t base = size_t(bh) * p.L_pad;
  const int e1 = p.ptr[tile + 1];
  const int per_entry = p.block / 32;

  auto fill = [&](float (&dst)[kSimtRows][D + 4], const void* src, bool bf16, int r0, int first,
                  int rows) {
    for (int i = tid; i < rows * D; i += kSimtThreads) {
      const int r = i / D, c = i - r * D;
      dst[first + r][c] =
          (r0 >= 0 && r0 + r < p.L) ? load_value(src, bf16, (base + r0 + r) * D + c) : 0.f;
    }
  };
  fill(sm.x, kKeys ? p.k : p.q, false, own0, 0, kSimtRows);
  fill(sm.x2, kKeys ? p.v : p.d_o, kKeys ? false : p.do_bf16, own0, 0, kSimtRows);

  float acc[4][NC * 4] = {}, acc2[kKeys ? 4 : 1][NC * 4] = {};
  float own_lse[4], own_delta[4];
  if (!kKeys) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = own0 + ty * 4 + a;
      own_lse[a] = r < p.L ? p.lse[base + r] : 0.f;
      own_delta[a] = r < p.L ? p.delta[base + r] : 0.f;
    }
  }

  // The list's segments that touch this half, two at a time.
  int e = p.ptr[tile], part = 0;
  while (true) {
    int row0[2] = {-1, -1};
    bool keep[2][2] = {};  // [segment][32-row group of the own rows]
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      while (e < e1 && row0[s] < 0) {
        const int ent = p.entry[e];
        const unsigned m = unsigned(ent) >> 16;
        const bool k0 = (m >> ((half * 2) * 32 / p.block)) & 1;
        const bool k1 = (m >> ((half * 2 + 1) * 32 / p.block)) & 1;
        if (k0 || k1) {
          row0[s] = (ent & 0xFFFF) * p.block + part * 32;
          keep[s][0] = k0;
          keep[s][1] = k1;
          if (++part == per_entry) part = 0, ++e;
        } else {
          ++e;
        }
      }
    }
    if (row0[0] < 0) break;
    __syncthreads();  // the step before has read y, y2, p and ds
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fill(sm.y, kKeys ? p.q : p.k, false, row0[s], 32 * s, 32);
      fill(sm.y2, kKeys ? p.d_o : p.v, kKeys ? p.do_bf16 : false, row0[s], 32 * s, 32);
    }
    __syncthreads();
    // Scores and dP: own rows 4 ty + a, step rows tx + 16 c.
    float s_[4][4] = {}, dp[4][4] = {};
    for (int c = 0; c < D; c += 4) {
      float4 xv[4], yv[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) xv[a] = *reinterpret_cast<const float4*>(&sm.x[ty * 4 + a][c]);
#pragma unroll
      for (int a = 0; a < 4; ++a) yv[a] = *reinterpret_cast<const float4*>(&sm.y[tx + 16 * a][c]);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s_[a][i] = dot4(xv[a], yv[i], s_[a][i]);
#pragma unroll
      for (int a = 0; a < 4; ++a) xv[a] = *reinterpret_cast<const float4*>(&sm.x2[ty * 4 + a][c]);
#pragma unroll
      for (int a = 0; a < 4; ++a) yv[a] = *reinterpret_cast<const float4*>(&sm.y2[tx + 16 * a][c]);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dp[a][i] = dot4(xv[a], yv[i], dp[a][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tx + 16 * i, s = r >> 5;
      const int row = row0[s] + (r & 31);
      const bool in = row0[s] >= 0 && row < p.L;
      const float lse_i = kKeys && in ? p.lse[base + row] : 0.f;
      const float delta_i = kKeys && in ? p.delta[base + row] : 0.f;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int own = ty * 4 + a;
        const bool on = in && keep[s][own >> 5] && own0 + own < p.L;
        // expf, not ex2.approx of a product: dQ is a sum in which the keys'
        // mean cancels, which magnifies a rounding of the exponent.
        const float x = fmaf(s_[a][i], p.scale, -(kKeys ? lse_i : own_lse[a]));
        const float w = on ? expf(x) : 0.f;
        sm.p[r][own] = w;
        sm.ds[r][own] = on ? w * (dp[a][i] - (kKeys ? delta_i : own_delta[a])) : 0.f;
      }
    }
    __syncthreads();
    // acc += dS^T y (dK or dQ), acc2 += P^T y2 (dV): own rows 4 ty + a,
    // features 4 tx + 64 c.
    for (int r = 0; r < kSimtRows; ++r) {
      const float4 ds4 = *reinterpret_cast<const float4*>(&sm.ds[r][ty * 4]);
      const float dsa[4] = {ds4.x, ds4.y, ds4.z, ds4.w};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 yv = *reinterpret_cast<const float4*>(&sm.y[r][tx * 4 + 64 * c]);
        const float ya[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[a][c * 4 + i] = fmaf(dsa[a], ya[i], acc[a][c * 4 + i]);
      }
      if constexpr (kKeys) {
        const float4 p4 = *reinterpret_cast<const float4*>(&sm.p[r][ty * 4]);
        const float pa[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 yv = *reinterpret_cast<const float4*>(&sm.y2[r][tx * 4 + 64 * c]);
          const float ya[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc2[a][c * 4 + i] = fmaf(pa[a], ya[i], acc2[a][c * 4 + i]);
        }
      }
    }
  }

#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int row = own0 + ty * 4 + a;
    if (row >= p.L_pad) continue;
    const float f = row < p.L ? p.scale : 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const size_t at = (base + row) * D + tx * 4 + 64 * c;
      store4(kKeys ? p.dk : p.dq, p.out_bf16, at,
             make_float4(acc[a][c * 4] * f, acc[a][c * 4 + 1] * f, acc[a][c * 4 + 2] * f,
                         acc[a][c * 4 + 3] * f));
      if constexpr (kKeys)
        store4(p.dv, p.out_bf16, at, make_float4(acc2[a][c * 4], acc2[a][c * 4 + 1],
                                                 acc2[a][c * 4 + 2], acc2[a][c * 4 + 3]));
    }
  }
}

template <int D, bool kKeys>
cudaError_t run_simt(const SimtParams& p, int64_t tiles, cudaStream_t stream) {
  auto kern = bwd_simt_kernel<D, kKeys>;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(sizeof(SimtSmem<D>)));
  if (err != cudaSuccess) return err;
  kern<<<unsigned(2 * tiles), kSimtThreads, sizeof(SimtSmem<D>), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace {
// Offsets of a call's workspace: D, the bf16 path's further operand rows and
// its bf16 copy of a fp32 dO. Rows come in multiples of 32, so each part is
// aligned to 128 bytes.
struct Workspace {
  size_t q_aug, do_aug, rounded, bytes;
  Workspace(const losa_pattern* p, int d, bool in_bf16, bool do_bf16) {
    const size_t rows = size_t(p->B) * p->H * p->n_blocks * p->block;
    q_aug = rows * 4;
    do_aug = q_aug + (in_bf16 ? rows * 32 : 0);
    rounded = do_aug + (in_bf16 ? rows * 32 : 0);
    bytes = rounded + (in_bf16 && !do_bf16 ? rows * d * 2 : 0);
  }
};
}  // namespace

size_t backward_workspace(const losa_pattern* p, int d, bool in_bf16, bool do_bf16) {
  return Workspace(p, d, in_bf16, do_bf16).bytes;
}

cudaError_t launch_backward(const BackwardCall& c, cudaStream_t stream) {
  const losa_pattern* pat = c.p;
  const int L_pad = pat->n_blocks * pat->block;
  const int64_t rows = int64_t(pat->B) * pat->H * L_pad;
  const Workspace at(pat, c.d, c.in_bf16, c.do_bf16);
  char* ws = static_cast<char*>(c.workspace);
  float* delta = reinterpret_cast<float*>(ws);
  uint16_t* rounded =
      c.in_bf16 && !c.do_bf16 ? reinterpret_cast<uint16_t*>(ws + at.rounded) : nullptr;
  AugRows aug{};
  if (c.in_bf16)
    aug = {reinterpret_cast<uint4*>(ws + at.q_aug), reinterpret_cast<uint4*>(ws + at.do_aug), c.lse,
           1.f / c.scale};
  const unsigned grid = unsigned((rows + 7) / 8);
  (c.d == 64 ? delta_kernel<64> : delta_kernel<128>)<<<grid, 256, 0, stream>>>(
      c.o, c.o_bf16, c.d_o, c.do_bf16, rows, c.L, L_pad, delta, rounded, aug);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  if (c.in_bf16)
    return launch_backward_mma(c, {rounded ? rounded : c.d_o, delta,
                                   reinterpret_cast<const uint16_t*>(ws + at.q_aug),
                                   reinterpret_cast<const uint16_t*>(ws + at.do_aug)},
                               stream);
  SimtParams p{};
  p.q = static_cast<const float*>(c.q);
  p.k = static_cast<const float*>(c.k);
  p.v = static_cast<const float*>(c.v);
  p.d_o = c.d_o;
  p.do_bf16 = c.do_bf16;
  p.out_bf16 = c.out_bf16;
  p.lse = c.lse;
  p.delta = delta;
  p.L = c.L;
  p.L_pad = L_pad;
  p.n_qt = pat->n_qt;
  p.block = pat->block;
  p.scale = c.scale;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.ptr = pat->key_ptr;
  p.entry = pat->key_entry;
  p.order = pat->key_order;
  err = c.d == 64 ? run_simt<64, true>(p, pat->n_tiles, stream)
                  : run_simt<128, true>(p, pat->n_tiles, stream);
  if (err != cudaSuccess) return err;
  p.ptr = pat->tile_ptr;
  p.entry = pat->tile_entry;
  p.order = pat->tile_order;
  return c.d == 64 ? run_simt<64, false>(p, pat->n_tiles, stream)
                   : run_simt<128, false>(p, pat->n_tiles, stream);
}

}  // namespace losa
