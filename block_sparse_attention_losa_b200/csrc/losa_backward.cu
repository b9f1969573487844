// losa_backward.cu - the gradient of block-sparse attention over a frozen
// pattern (losa_sparse_attn_bwd), probabilities recomputed.
//
// Mathematics, per head, over the kept (query, key) pairs:
//   P_ij = exp(scale q_i.k_j - lse_i)         the forward pass's weights
//   D_i  = dO_i . O_i                         = sum_j P_ij dP_ij
//   dV_j = sum_i P_ij dO_i
//   dS_ij = P_ij (dO_i.v_j - D_i)
//   dQ_i = scale sum_j dS_ij k_j,  dK_j = scale sum_i dS_ij q_i.
// dK and dV sum over queries and dQ over keys, so key tiles and query tiles
// run side by side, each owning its output rows: no atomics, the same bits
// every time, and no fp32 gradient buffer that has to be cleared and
// converted. The price is that scores and dP are computed twice (seven
// products instead of five). It buys speed too on the tensor cores: per 128 x
// 128 scores at d = 128 the seven products take 3,584 cycles of the tensor
// core, while a single pass with five (2,560) would have to write dS and read
// it back as an operand and to move fp32 dQ tiles through shared memory,
// about 3,840 cycles of its 128 bytes each.
//
// This file holds the prepass (D, and what the tensor-core path reads beside
// it) and the fp32 path; losa_backward_mma.cu the bf16 path.
//
// fp32 calls without o and lse form lse_i and D_i themselves, from the scores
// that P is made of. The forward call's own come from tf32 products: with them
// a row of P does not sum to 1 and sum_j dS_ij is not 0, so what a head's keys
// have in common stands in dQ, magnified by its size over the keys' spread.
#include <algorithm>

#include "losa_device.cuh"
#include "losa_internal.h"

namespace losa {
namespace {

// ------------------------------------------------------------------ D

// Eight features of a row, as loaded and in fp32.
struct Eight {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* base, bool bf16, size_t at) {
    if (bf16) {
      a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      a = __ldg(p);
      b = __ldg(p + 1);
    }
  }
  __device__ __forceinline__ void get(bool bf16, float (&v)[8]) const {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = !bf16 ? __uint_as_float(u[e])
                   : __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
  }
};

// Three bf16 terms whose sum is x to 24 bits, as the first columns of a
// 16-column operand row (the other columns 0). Finite values are kept inside
// bf16's range; an infinity or NaN is the first term.
__device__ __forceinline__ uint4 split3(float x) {
  if (!isfinite(x)) return make_uint4(pack_bf16x2(x, 0.f) & 0xffffu, 0u, 0u, 0u);
  x = fminf(fmaxf(x, -3e38f), 3e38f);
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
  uint4 *q, *d_o;
  const float* lse;
  float inv_scale;
};

// D_i = dO_i . O_i for all rows (0 in the padding), the sum in fp32. Where
// dO's type is not that of q, k and v, `copy` receives it in theirs: a fp32 dO
// is rounded to bf16, as the tensor cores read it, before D is formed, so that
// D cancels against the same dO that dP is made of; a bf16 one is widened.
// Without o (fp32 path, D formed later) dO is converted only.
// Bound: HBM. D / 8 lanes share a row, and a warp has four sets of rows in
// flight (one row per warp at a time took 20 us at 75,776 rows of 64), three CTAs
// to an SM (two, with 86 registers a thread, cost a fifth more).
constexpr int kDeltaSets = 4;
// kAug: the bf16 path.
template <int D, bool kAug>
__global__ void __launch_bounds__(256, 3)
    delta_kernel(const void* o, bool o_bf16, const void* d_o, bool do_bf16, int64_t rows,
                 int L, int L_pad, float* delta, void* copy, const AugRows aug) {
  constexpr int LANES = D / 8, SET = 32 / LANES;  // lanes of a row, rows of a set
  const int lane = threadIdx.x & 31, part = lane % LANES;
  const int64_t row0 =
      (int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (kDeltaSets * SET) + lane / LANES;
  Eight a[kDeltaSets], b[kDeltaSets];
  bool valid[kDeltaSets];
  float lse[kDeltaSets];
#pragma unroll
  for (int s = 0; s < kDeltaSets; ++s) {
    const int64_t row = row0 + s * SET;
    valid[s] = row < rows && row % L_pad < L;
    lse[s] = kAug && valid[s] ? __ldg(aug.lse + row) : 0.f;
    if (valid[s]) {
      if (o) a[s].load(o, o_bf16, size_t(row) * D + part * 8);
      b[s].load(d_o, do_bf16, size_t(row) * D + part * 8);
    }
  }
#pragma unroll
  for (int s = 0; s < kDeltaSets; ++s) {
    const int64_t row = row0 + s * SET;
    float sum = 0.f;
    if (valid[s]) {
      float x[8] = {}, y[8];
      if (o) a[s].get(o_bf16, x);
      b[s].get(do_bf16, y);
      if (copy) {
        const size_t at = size_t(row) * D + part * 8;
        if (do_bf16) {
          float4* w = reinterpret_cast<float4*>(static_cast<float*>(copy) + at);
          w[0] = make_float4(y[0], y[1], y[2], y[3]);
          w[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
          Eight r;
          r.a = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                           pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(copy) + at) = r.a;
          r.get(true, y);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (row >= rows) continue;
    if (kAug && isnan(lse[s])) sum = NAN;  // into dQ, whichever its columns
    if (part == 0) delta[row] = sum;
    if (kAug && part < 4) {
      // Parts 0, 1: the row's two halves of q's columns; 2, 3: of dO's. Padded
      // rows get a score far below any other, so their weight is 0. A lse that
      // is NaN becomes an infinite score: its exponential is inf or NaN in
      // every column, that of a NaN is not (exp2_fma2's clamp drops it).
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (part == 0) {
        const float t = valid[s] ? -lse[s] * aug.inv_scale : -3e38f;
        w = split3(isnan(t) ? INFINITY : t);
      } else if (part == 2) {
        w = split3(-sum);
      }
      (part < 2 ? aug.q : aug.d_o)[(row >> 3) * 16 + (part & 1) * 8 + (row & 7)] = w;
    }
  }
}

// ------------------------------------------------------------------ fp32

struct FmaParams {
  const float *q, *k, *v, *d_o, *lse, *delta;
  float *lse_out, *delta_out;  // row_stats_kernel's results
  int L, L_pad, n_qt, n_tiles, block;
  float scale;
  const int *key_ptr, *key_entry, *key_order;        // by key tile
  const int *tile_ptr, *tile_entry, *tile_order;     // by query tile
  void *dq, *dk, *dv;
  bool out_bf16;
};

__device__ __forceinline__ void store4(void* p, bool bf16, size_t i, const float* x, float f) {
  if (bf16) {
    uint2 w;
    w.x = pack_bf16x2(x[0] * f, x[1] * f);
    w.y = pack_bf16x2(x[2] * f, x[3] * f);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) =
        make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
  }
}

// 16 bytes from global to shared memory, asynchronously; zeros if !valid.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

constexpr int kOwn = 32;   // rows a CTA owns
constexpr int kStep = 64;  // rows of the other side per step

// Own rows are padded by one 16-byte chunk, and the others hold their chunks
// permuted (chunk c of row r at place c ^ (r & 7)), so that eight rows' equal
// chunks lie in different banks. 113 KB at D = 128: just two CTAs per SM.
template <int D> struct FmaSmem {
  float x[kOwn][D + 4], x2[kOwn][D + 4];  // own rows: K, V or Q, dO
  float y[kStep][D], y2[kStep][D];  // a step's rows: Q, dO or K, V
  float p[kStep][kOwn], ds[kStep][kOwn];
};
// acc += a . b of four features as two pairs of partial sums.
__device__ __forceinline__ void dot4(const float4& a, const float4& b, f32x2& acc) {
  acc = f2_fma(f2_make(a.x, a.y), f2_make(b.x, b.y), acc);
  acc = f2_fma(f2_make(a.z, a.w), f2_make(b.z, b.w), acc);
}

// Running maximum m of a row's scores, and of exp(s - m) the sum l and the sum
// t of its products with dP. lse = m + log l, D = t / l.
struct RowStats {
  float m, l, t;
};
// exp(from - to), 0 for a sum that is still empty.
__device__ __forceinline__ float raised(float from, float to) {
  return from == to ? 1.f : from == -INFINITY ? 0.f : expf(from - to);
}
__device__ __forceinline__ RowStats join(const RowStats& a, const RowStats& b) {
  const float m = fmaxf(a.m, b.m), fa = raised(a.m, m), fb = raised(b.m, m);
  return {m, a.l * fa + b.l * fb, a.t * fa + b.t * fb};
}

// What fma_tile forms: dK and dV of key rows, dQ of query rows, or their lse
// and D.
enum class Fma { kKeys, kQueries, kStats };

// One CTA owns 32 rows (a quarter of a 128-row tile, always inside one block)
// of keys (kKeys: dK and dV) or of queries (dQ) and walks those list entries
// whose blocks meet, 64 rows of the other side at a time: two segments of 32
// rows, the unit in which blocks of 32, 64 and 128 rows start and end.
// Every product is fp32 FMA, bound by the FMA units and the reads of its
// operands from shared memory. A 16-byte read of a warp takes two cycles of
// shared memory where each lane wants what lane ^ 1 or each what lane ^ 2
// wants, else four (measured, whatever the number of distinct addresses), so
// bit 0 of a lane picks among own rows alone and bit 1 among the other
// operand's alone (before: 3.0 a read, and 2.43 ms for the case below); and
// few threads hold large tiles. With T = 128:
//   scores: a warp has 16 x 32 of the 32 x 64, a thread 4 x 4 of it;
//   gradients: a thread has 8 own rows x 8 features; the threads hold both
//   products (keys) and, with what is left, parts of the step's rows, summed
//   at the end.
// 5,000 tokens, 8 heads, d 64, half the blocks kept: 2.38 ms, 27 TFLOP/s of
// the five products that the gradient needs, 38 of the seven that run.
template <int D, int T, Fma kWhat>
__device__ __forceinline__ void fma_tile(const FmaParams& p, FmaSmem<D>& sm, int tile,
                                         int quarter) {
  constexpr bool kKeys = kWhat == Fma::kKeys, kStats = kWhat == Fma::kStats;
  constexpr int CH = D / 4;                           // chunks of a row
  constexpr int PER = CH / 2 * (kOwn / 8);            // threads that hold a gradient
  constexpr int GROUPS = T / PER;
  constexpr int PARTS = kKeys ? GROUPS / 2 : GROUPS;  // of a step's rows
  constexpr int WARP_ROWS = kStep / (T / 64);         // step rows of a warp's scores
  constexpr int NI = WARP_ROWS / 8;                   // of a thread's
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = tile / p.n_qt;
  const int own0 = (tile - bh * p.n_qt) * 128 + quarter * kOwn;
  if (own0 >= p.L_pad) return;
  const size_t base = size_t(bh) * p.L_pad;
  const int* ptr = kKeys ? p.key_ptr : p.tile_ptr;
  const int* entry = kKeys ? p.key_entry : p.tile_entry;
  const unsigned bit = 1u << (16 + quarter * kOwn / p.block);
  const int per_entry = p.block / 32;
  int e = ptr[tile];
  const int e1 = own0 < p.L ? ptr[tile + 1] : e;  // padding alone: nothing to sum

  // The list's entries, 32 at a time in the lanes of each warp (one by one,
  // each would cost a load's latency), and the next 32.
  auto entries = [&](int at) { return at + lane < e1 ? __ldg(entry + at + lane) : 0; };
  int word = 0, ahead = entries(e), ent = 0, part = 0;
  unsigned meets = 0;  // lanes of `word` whose block meets the own rows
  // First row of the list's next segment of 32 rows, -1 at its end.
  auto next_segment = [&]() -> int {
    while (true) {
      if (part == 0) {
        while (meets == 0) {
          if (e >= e1) return -1;
          word = ahead;
          meets = __ballot_sync(0xffffffffu, (unsigned(word) & bit) != 0);
          e += 32;
          ahead = entries(e);
        }
        ent = __shfl_sync(0xffffffffu, word, __ffs(meets) - 1);
        meets &= meets - 1;
      }
      const int row = (ent & 0xFFFF) * p.block + part * 32;
      if (++part == per_entry) part = 0;
      if (row < p.L) return row;
    }
  };
  // 32 rows from r0 on (none if r0 < 0), rows of the padding as zeros.
  auto fill = [&](float* dst, const float* src, int r0, bool padded) {
#pragma unroll
    for (int n = 0; n < 32 * CH / T; ++n) {
      const int r = (tid + n * T) / CH, c = tid % CH;
      const bool in = r0 >= 0 && r0 + r < p.L;
      copy16(dst + (padded ? r * (D + 4) + c * 4 : r * D + (c ^ (r & 7)) * 4),
             src + (base + (in ? r0 + r : 0)) * D + c * 4, in);
    }
  };
  fill(&sm.x[0][0], kKeys ? p.k : p.q, own0, true);
  fill(&sm.x2[0][0], kKeys ? p.v : p.d_o, own0, true);

  // Scores: the warp's 16 own rows and WARP_ROWS step rows, the thread's rows
  // so + 4 a and si + 8 i, four own rows by bits 0 and 2 of the lane, eight
  // step rows by the others.
  const int so = 16 * (warp / (T / 64)) + (lane & 1) + 2 * (lane >> 2 & 1);
  const int si = WARP_ROWS * (warp % (T / 64)) + (lane >> 1 & 1) + 2 * (lane >> 3);
  // Gradients: own rows go.. and chunks gc and gc + CH / 2, for the group's
  // product and part.
  const int group = tid / PER, within = tid % PER;
  const int go = 8 * ((within & 1) + 2 * (within / CH)), gc = (within >> 1) % (CH / 2);
  const bool use_p = kKeys && (group & 1);
  const int gpart = kKeys ? group >> 1 : group;
  f32x2 acc[4][8] = {};  // pairs of own rows x features
  RowStats stats[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) stats[a] = {-INFINITY, 0.f, 0.f};
  float own_lse[4], own_delta[4];
  if (kWhat == Fma::kQueries) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = own0 + so + 4 * a;
      own_lse[a] = r < p.L ? p.lse[base + r] : 0.f;
      own_delta[a] = r < p.L ? p.delta[base + r] : 0.f;
    }
  }

  int seg[2] = {next_segment(), next_segment()};
  while (seg[0] >= 0) {
    const int row0[2] = {seg[0], seg[1]};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fill(&sm.y[32 * s][0], kKeys ? p.q : p.k, row0[s], false);
      fill(&sm.y2[32 * s][0], kKeys ? p.d_o : p.v, row0[s], false);
    }
    // A warp's step rows lie in one segment.
    float step_lse[NI], step_delta[NI];
    bool on[NI];
    const int seg0 = si >= 32 ? row0[1] : row0[0];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = seg0 + (si & 31) + 8 * i;
      on[i] = seg0 >= 0 && row < p.L;
      step_lse[i] = kKeys && on[i] ? __ldg(p.lse + base + row) : 0.f;
      step_delta[i] = kKeys && on[i] ? __ldg(p.delta + base + row) : 0.f;
    }
    seg[0] = next_segment();
    seg[1] = next_segment();
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    f32x2 s2[4][NI] = {}, d2[4][NI] = {};
#pragma unroll 4
    for (int c = 0; c < CH; ++c) {
      const int yc = (c ^ (si & 7)) * 4;
      float4 xv[4], yv[NI];
#pragma unroll
      for (int a = 0; a < 4; ++a) xv[a] = *reinterpret_cast<const float4*>(&sm.x[so + 4 * a][4 * c]);
#pragma unroll
      for (int i = 0; i < NI; ++i) yv[i] = *reinterpret_cast<const float4*>(&sm.y[si + 8 * i][yc]);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < NI; ++i) dot4(xv[a], yv[i], s2[a][i]);
#pragma unroll
      for (int a = 0; a < 4; ++a) xv[a] = *reinterpret_cast<const float4*>(&sm.x2[so + 4 * a][4 * c]);
#pragma unroll
      for (int i = 0; i < NI; ++i) yv[i] = *reinterpret_cast<const float4*>(&sm.y2[si + 8 * i][yc]);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < NI; ++i) dot4(xv[a], yv[i], d2[a][i]);
    }
    if constexpr (kStats) {
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        RowStats& z = stats[a];
        float m = z.m;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (on[i]) m = fmaxf(m, f2_sum(s2[a][i]) * p.scale);
        const float f = raised(z.m, m);
        z = {m, z.l * f, z.t * f};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (!on[i]) continue;
          const float w = expf(fmaf(f2_sum(s2[a][i]), p.scale, -m));
          z.l += w;
          z.t = fmaf(w, f2_sum(d2[a][i]), z.t);
        }
      }
      __syncthreads();  // before the next step's rows arrive
      continue;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = si + 8 * i;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int o = so + 4 * a;
        // expf, not ex2.approx of a product: dQ is a sum in which the keys'
        // mean cancels, which magnifies a rounding of the exponent.
        const float x = fmaf(f2_sum(s2[a][i]), p.scale, -(kKeys ? step_lse[i] : own_lse[a]));
        const float w = on[i] && own0 + o < p.L ? expf(x) : 0.f;
        const float g = f2_sum(d2[a][i]) - (kKeys ? step_delta[i] : own_delta[a]);
        const int at = o ^ (4 * (r & 7));
        if (kKeys) sm.p[r][at] = w;
        sm.ds[r][at] = w != 0.f ? w * g : 0.f;
      }
    }
    __syncthreads();
    const float* wts = use_p ? &sm.p[0][0] : &sm.ds[0][0];
    const float* rows = use_p ? &sm.y2[0][0] : &sm.y[0][0];
#pragma unroll 4
    for (int r = gpart * (kStep / PARTS); r < (gpart + 1) * (kStep / PARTS); ++r) {
      const int k = r & 7;
      const float4 a0 = *reinterpret_cast<const float4*>(wts + r * kOwn + (go ^ (4 * k)));
      const float4 a1 = *reinterpret_cast<const float4*>(wts + r * kOwn + ((go + 4) ^ (4 * k)));
      const f32x2 av[4] = {f2_make(a0.x, a0.y), f2_make(a0.z, a0.w), f2_make(a1.x, a1.y),
                           f2_make(a1.z, a1.w)};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float4 yv =
            *reinterpret_cast<const float4*>(rows + r * D + ((gc ^ k) + n * (CH / 2)) * 4);
        const f32x2 yy[4] = {f2_make(yv.x, yv.x), f2_make(yv.y, yv.y), f2_make(yv.z, yv.z),
                             f2_make(yv.w, yv.w)};
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[a][4 * n + i] = f2_fma(av[a], yy[i], acc[a][4 * n + i]);
      }
    }
    __syncthreads();  // before the next step's rows arrive
  }

  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if constexpr (kStats) {
    // A row's sums lie in eight lanes of the T / 64 warps that share it.
    constexpr int SHARES = T / 64;
    static_assert(SHARES * kOwn * sizeof(RowStats) <= sizeof(sm.p), "room for the rows' sums");
    RowStats* sums = reinterpret_cast<RowStats*>(&sm.p[0][0]);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
      for (int bit : {2, 8, 16}) {
        const RowStats& z = stats[a];
        stats[a] = join(z, {__shfl_xor_sync(0xffffffffu, z.m, bit),
                            __shfl_xor_sync(0xffffffffu, z.l, bit),
                            __shfl_xor_sync(0xffffffffu, z.t, bit)});
      }
      if ((lane & ~5) == 0) sums[(warp % SHARES) * kOwn + so + 4 * a] = stats[a];
    }
    __syncthreads();
    if (tid < kOwn && own0 + tid < p.L) {
      RowStats z = sums[tid];
#pragma unroll
      for (int s = 1; s < SHARES; ++s) z = join(z, sums[s * kOwn + tid]);
      p.lse_out[base + own0 + tid] = z.m + logf(z.l);
      p.delta_out[base + own0 + tid] = z.t / z.l;
    }
    return;
  }

  // Parts of a gradient meet in shared memory; the first one writes the rows.
  float out[8][8];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 8; ++i) f2_split(acc[a][i], out[2 * a][i], out[2 * a + 1][i]);
  if constexpr (PARTS > 1) {
    constexpr int N = PER * (kKeys ? 2 : 1);  // threads of a part
    const int mine = within + (use_p ? PER : 0);
    float4* buf = reinterpret_cast<float4*>(&sm.y[0][0]);
    static_assert(16 * N * sizeof(float4) <= sizeof(sm.y), "room for a part's sums");
#pragma unroll
    for (int s = 1; s < PARTS; ++s) {
      if (gpart == s) {
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            buf[(2 * a + n) * N + mine] =
                make_float4(out[a][4 * n], out[a][4 * n + 1], out[a][4 * n + 2], out[a][4 * n + 3]);
      }
      __syncthreads();
      if (gpart == 0) {
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float4 z = buf[(2 * a + n) * N + mine];
            out[a][4 * n] += z.x, out[a][4 * n + 1] += z.y;
            out[a][4 * n + 2] += z.z, out[a][4 * n + 3] += z.w;
          }
      }
      __syncthreads();
    }
  }
  if (gpart == 0) {
    void* dst = kKeys ? (use_p ? p.dv : p.dk) : p.dq;
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      const int row = own0 + go + a;
      if (row >= p.L_pad) continue;
      const float f = use_p ? 1.f : p.scale;
      if (row >= p.L) {  // 0 whatever the sums hold: 0 times NaN is not
#pragma unroll
        for (int i = 0; i < 8; ++i) out[a][i] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
        store4(dst, p.out_bf16, (base + row) * D + (gc + n * (CH / 2)) * 4, &out[a][4 * n], f);
    }
  }
}

// The key quarters of all tiles, longest lists first within a head, then the
// query quarters.
template <int D, int T>
__global__ void __launch_bounds__(T, T == 128 ? 2 : 1) bwd_fma_kernel(const FmaParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FmaSmem<D>& sm = *reinterpret_cast<FmaSmem<D>*>(smem_raw);
  const int i = blockIdx.x >> 2, quarter = blockIdx.x & 3;
  if (i < p.n_tiles)
    fma_tile<D, T, Fma::kKeys>(p, sm, p.key_order[i], quarter);
  else
    fma_tile<D, T, Fma::kQueries>(p, sm, p.tile_order[i - p.n_tiles], quarter);
}

// lse and D of the query quarters, in a launch of its own since the key tiles
// need every row's: two products more for the gradient's seven (2,200 tokens, 4
// heads, d 128, half the blocks kept: 531 -> 729 us).
template <int D, int T>
__global__ void __launch_bounds__(T, T == 128 ? 2 : 1) row_stats_kernel(const FmaParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  fma_tile<D, T, Fma::kStats>(p, *reinterpret_cast<FmaSmem<D>*>(smem_raw),
                              p.tile_order[blockIdx.x >> 2], blockIdx.x & 3);
}

template <int D, int T> cudaError_t run_fma(const FmaParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0}, stats_allowed{0};
  cudaError_t err;
  if (p.lse_out) {
    err = allow_smem(reinterpret_cast<const void*>(row_stats_kernel<D, T>),
                     int(sizeof(FmaSmem<D>)), stats_allowed);
    if (err != cudaSuccess) return err;
    row_stats_kernel<D, T><<<4u * unsigned(p.n_tiles), T, sizeof(FmaSmem<D>), stream>>>(p);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  err = allow_smem(reinterpret_cast<const void*>(bwd_fma_kernel<D, T>),
                                     int(sizeof(FmaSmem<D>)), allowed);
  if (err != cudaSuccess) return err;
  bwd_fma_kernel<D, T><<<8u * unsigned(p.n_tiles), T, sizeof(FmaSmem<D>), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

namespace {
// Offsets of a call's workspace: D, the bf16 path's further operand rows, and
// dO in the type of q, k and v where it has the other one, and the fp32 path's
// own lse. Rows come in multiples of 32, so each part is aligned to 128 bytes.
struct Workspace {
  size_t q_aug, do_aug, copy, lse, bytes;
  Workspace(const losa_pattern* p, int d, bool in_bf16, bool do_bf16) {
    const size_t rows = size_t(p->B) * p->H * p->n_blocks * p->block;
    q_aug = rows * 4;
    do_aug = q_aug + (in_bf16 ? rows * 32 : 0);
    copy = do_aug + (in_bf16 ? rows * 32 : 0);
    lse = copy + (in_bf16 != do_bf16 ? rows * d * (in_bf16 ? 2 : 4) : 0);
    bytes = lse + (in_bf16 ? 0 : rows * 4);
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
  void* copy = c.in_bf16 != c.do_bf16 ? ws + at.copy : nullptr;
  const void* d_o = copy ? copy : c.d_o;
  AugRows aug{};
  if (c.in_bf16)
    aug = {reinterpret_cast<uint4*>(ws + at.q_aug), reinterpret_cast<uint4*>(ws + at.do_aug), c.lse,
           1.f / c.scale};
  const int64_t per_cta = 8 * kDeltaSets * (256 / c.d);
  const unsigned grid = unsigned((rows + per_cta - 1) / per_cta);
  if (c.o || copy) {
    auto kernel = c.d == 64 ? (c.in_bf16 ? delta_kernel<64, true> : delta_kernel<64, false>)
                            : (c.in_bf16 ? delta_kernel<128, true> : delta_kernel<128, false>);
    kernel<<<grid, 256, 0, stream>>>(c.o, c.o_bf16, c.d_o, c.do_bf16, rows, c.L, L_pad, delta, copy,
                                     aug);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (c.in_bf16)
    return launch_backward_mma(c, {d_o, delta,
                                   reinterpret_cast<const uint16_t*>(ws + at.q_aug),
                                   reinterpret_cast<const uint16_t*>(ws + at.do_aug)},
                               stream);
  FmaParams p{};
  p.q = static_cast<const float*>(c.q);
  p.k = static_cast<const float*>(c.k);
  p.v = static_cast<const float*>(c.v);
  p.d_o = static_cast<const float*>(d_o);
  p.lse_out = c.o ? nullptr : reinterpret_cast<float*>(ws + at.lse);
  p.delta_out = delta;
  p.lse = c.o ? c.lse : p.lse_out;
  p.delta = delta;
  p.L = c.L;
  p.L_pad = L_pad;
  p.n_qt = pat->n_qt;
  p.n_tiles = int(pat->n_tiles);
  p.block = pat->block;
  p.scale = c.scale;
  p.key_ptr = pat->key_ptr;
  p.key_entry = pat->key_entry;
  p.key_order = pat->key_order;
  p.tile_ptr = pat->tile_ptr;
  p.tile_entry = pat->tile_entry;
  p.tile_order = pat->tile_order;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.out_bf16 = c.out_bf16;
  // At most one CTA per SM or a few more: a CTA's own speed counts, and 256
  // threads hide more latency (600 tokens, 4 heads, d 128, 160 CTAs: 76 us
  // against 103 with 128). More: two CTAs of 128 threads share an SM, and their
  // larger tiles read less shared memory (3,048 tokens, one head, d 64, 192
  // CTAs: 343 us against 404).
  if (8 * pat->n_tiles <= kSms + kSms / 8)
    return c.d == 64 ? run_fma<64, 256>(p, stream) : run_fma<128, 256>(p, stream);
  return c.d == 64 ? run_fma<64, 128>(p, stream) : run_fma<128, 128>(p, stream);
}

}  // namespace losa
