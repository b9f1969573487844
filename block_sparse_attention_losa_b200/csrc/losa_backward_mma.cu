// losa_backward_mma.cu - the tensor-core kernel of losa_sparse_attn_bwd
// (bf16 operands, fp32 accumulation in tensor memory): a CTA owns 128 key
// rows, for dK and dV, and walks the query blocks that keep them, or 128 query
// rows, for dQ, and walks the key blocks they keep.
#include <algorithm>

#include "losa_device.cuh"
#include "losa_internal.h"

namespace losa {
namespace {

constexpr int kBwdThreads = 384;
// Launched with 168 registers a thread (checked at build time); the control
// warpgroup gives some back to the two that hold scores.
constexpr int kBwdLaunchRegs = 168, kScoreRegs = 216, kControlRegs = 72;
static_assert(2 * 128 * kScoreRegs + 128 * kControlRegs == kBwdThreads * kBwdLaunchRegs,
              "register split must use exactly the launch allocation");
constexpr int kTile = 128;  // rows a CTA owns, and rows of a step
constexpr int kAugBytes = kTile * 32;

// A pattern's lists by key tile or by query tile.
struct BwdLists {
  const int *ptr, *entry, *order;
};

struct BwdParams {
  int L, L_pad, n_qt, n_tiles;
  float scale, scale_log2;
  BwdLists keys, queries;
  const float *lse, *delta;
  const uint16_t *q_aug, *do_aug;
  const void *q, *d_o;  // dQ kernel: its own rows
  void *dq, *dk, *dv;
  int* status;
  long long wait_limit;
};

// cp.async.bulk of `bytes` (a multiple of 16, both sides 16-byte aligned).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// Shared-memory matrix descriptors in two halves. The low one is the start
// address and the stride LBO, both in units of 16 bytes; a shared-memory
// address needs 14 bits in those units, so a step along an operand is an
// addition to it. The high half is a constant per layout: SBO, the
// descriptor's version (bit 46) and the swizzle (bits 61 to 63).
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return (saddr >> 4) | ((lbo_bytes >> 4) << 16);
}
// Rows of 128 bytes, 128-byte swizzle, 8-row groups 1 KB apart (K-major with
// any LBO, MN-major with LBO the distance of 64-column slabs).
constexpr uint32_t kDescSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major operand of 16 bf16 columns without swizzle: 8-row groups of 256
// bytes (SBO), each two 8 x 16-byte core matrices 128 bytes apart (LBO).
constexpr uint32_t kDescAug = (256u >> 4) | (1u << 14);

template <uint32_t kHiA, uint32_t kHiB>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kHiA), "n"(kHiB)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescSw128)
      : "memory");
}

__device__ __forceinline__ void zero32(float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = 0.f;
}
__device__ __forceinline__ void mul32(float (&x)[32], const float (&w)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    f2_split(f2_mul(f2_make(x[i], x[i + 1]), f2_make(w[i], w[i + 1])), x[i], x[i + 1]);
}
// x = (x + c) * w
__device__ __forceinline__ void add_mul32(float (&x)[32], float c, const float (&w)[32]) {
  const f32x2 c2 = f2_make(c, c);
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    f2_split(f2_mul(f2_add(f2_make(x[i], x[i + 1]), c2), f2_make(w[i], w[i + 1])), x[i], x[i + 1]);
}

// One arrival per warp: every lane's tensor-memory accesses are complete
// (tcgen05.wait) and ordered before it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A wait of a whole warp, with one answer for all its lanes, so that none
// goes on alone into the warp-wide tensor-memory accesses after a wait that
// others gave up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// Of every 16 column pairs, how many take exp2 on the FMA pipe.
constexpr int kPolyPairs = 4;

// e = 2^(x * c) of 32 values.
__device__ __forceinline__ void exp2_scaled(float (&x)[32], float c) {
  const f32x2 c2 = f2_make(c, c);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a, b;
    f2_split(f2_mul(f2_make(x[i], x[i + 1]), c2), a, b);
    if ((i >> 1) < kPolyPairs) {
      exp2_fma2(a, b, x[i], x[i + 1]);
    } else {
      x[i] = ex2_approx(a);
      x[i + 1] = ex2_approx(b);
    }
  }
}
// e = 2^(x * c + o) of 32 values.
__device__ __forceinline__ void exp2_shifted(float (&x)[32], float c, float o) {
  const f32x2 c2 = f2_make(c, c), o2 = f2_make(o, o);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float a, b;
    f2_split(f2_fma(f2_make(x[i], x[i + 1]), c2, o2), a, b);
    if ((i >> 1) < kPolyPairs) {
      exp2_fma2(a, b, x[i], x[i + 1]);
    } else {
      x[i] = ex2_approx(a);
      x[i + 1] = ex2_approx(b);
    }
  }
}

// Stores 32 values as bf16 pairs over 16 columns.
__device__ __forceinline__ void tmem_st_bf16(uint32_t taddr, const float (&x)[32]) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  tmem_st16(taddr, pk);
}

// What that rounding leaves, rounded likewise: with it the pairs hold 16 bits
// of each value.
__device__ __forceinline__ void tmem_st_bf16_rest(uint32_t taddr, const float (&x)[32]) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t h = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    pk[i] = pack_bf16x2(x[2 * i] - __uint_as_float(h << 16),
                        x[2 * i + 1] - __uint_as_float(h & 0xffff0000u));
  }
  tmem_st16(taddr, pk);
}

// Writes one row's 32 accumulator columns, times f, to the result.
template <bool kOutBf16>
__device__ __forceinline__ void store_row32(void* out, size_t at, const float (&x)[32], float f) {
  if constexpr (kOutBf16) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      uint4 w;
      w.x = pack_bf16x2(x[e] * f, x[e + 1] * f);
      w.y = pack_bf16x2(x[e + 2] * f, x[e + 3] * f);
      w.z = pack_bf16x2(x[e + 4] * f, x[e + 5] * f);
      w.w = pack_bf16x2(x[e + 6] * f, x[e + 7] * f);
      dst[e / 8] = w;
    }
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      dst[e / 4] = make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f);
  }
}
template <bool kOutBf16>
__device__ __forceinline__ void store_zero32(void* out, size_t at) {
  const float zero[32] = {};
  store_row32<kOutBf16>(out, at, zero, 0.f);
}

// ------------------------------------------------------------------ dK, dV

// Shared memory of the dK/dV kernel: its K and V tiles, the constant operand
// that adds lse and D, and a ring of steps (Q and dO tiles with their rows of
// lse and D).
template <int D> struct KeyLayout {
  static constexpr int NS = D == 128 ? 2 : 4;  // stages
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + TILE_BYTES;
  static constexpr int OFF_Q = OFF_V + TILE_BYTES;
  static constexpr int OFF_DO = OFF_Q + NS * TILE_BYTES;
  static constexpr int OFF_QA = OFF_DO + NS * TILE_BYTES;
  static constexpr int OFF_DA = OFF_QA + NS * kAugBytes;
  static constexpr int OFF_ONE = OFF_DA + NS * kAugBytes;
  static constexpr int OFF_BAR = OFF_ONE + kAugBytes;
  static constexpr int N_BARS = 4 * NS + 12;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  // 1 KB of slack for alignment; above 116 KB, so that one CTA runs per SM
  // (each allocates all 512 TMEM columns).
  static constexpr int SMEM_ALLOC = BYTES + 1024;
  static_assert(SMEM_ALLOC > 116 * 1024 && SMEM_ALLOC <= 227 * 1024, "shared memory");
};

// Scores are formed transposed (rows are keys), so that P^T and dS^T lie in
// tensor memory as the A operands of dV and dK. The row constants lse_i and
// D_i then run along the columns, where a thread would have to load one per
// score; instead they enter the products: Q and dO get 16 further columns
// that hold -lse_i / scale and -D_i as three bf16 terms each (24 bits), and
// K and V matching columns of ones, so S^T arrives as q.k - lse / scale and
// dP^T as dO.v - D for 1/8 of a product's time each.
//
// Per step j the MMA warp issues dV(j), S(j+1), dK(j), dP(j+1): the softmax's
// first half (P from S) runs under dK(j-1) and dP(j), its second (dS from P
// and dP) under dV(j) and S(j+1), with one buffer of each in the 512 columns
// of tensor memory: S/P, dP/dS, dV, dK. At D = 64 there is room for a second
// S/P, and S(j+1) comes first.
//
// Warps 0-7 hold the scores, thread t of a warp one key row and half the
// query columns; warp 8 loads, warp 9 issues the MMAs.
template <int D, int BLK, bool kOutBf16>
__device__ __forceinline__ void key_tile(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         const CUtensorMap& tm_q, const CUtensorMap& tm_do,
                                         const BwdParams& p, const BwdLists& list, int tile) {
  using Lay = KeyLayout<D>;
  constexpr int NS = Lay::NS;
  constexpr int EPI = kTile / BLK;  // list entries per step
  constexpr int SLABS = D / 64;
  constexpr uint32_t C_DP = 128, C_DV = 256, C_DK = 256 + D;
  // S and P of step j: at D = 64 two buffers fit, and S(j+1) is formed while
  // step j's are in use.
  constexpr bool kTwoS = D == 64;
  auto buffer = [](int j) -> int { return kTwoS ? j & 1 : 0; };
  auto c_s = [&](int j) -> uint32_t { return 384u * buffer(j); };
  // Parity of step j's use of its buffer's barriers.
  auto use = [](int j) -> uint32_t { return (kTwoS ? j >> 1 : j) & 1; };
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kTile, kTile, false, false);
  constexpr uint32_t IDESC_G = idesc_bf16_f32(kTile, D, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* q_full = bars;             // [NS]
  uint64_t* q_empty = q_full + NS;     // [NS]
  uint64_t* do_full = q_empty + NS;    // [NS]
  uint64_t* do_empty = do_full + NS;   // [NS]
  uint64_t* k_full = do_empty + NS;
  uint64_t* v_full = k_full + 1;
  // Scores and weights, one set per buffer of S: with two, S(j+1) may be
  // complete before a slow warp has seen S(j), and a fast warp may deliver
  // P(j+1) before a slow one P(j). A buffer's next use comes after all warps'
  // last one, whose P the MMA warp has waited for.
  uint64_t* s_full = v_full + 1;   // [2]
  uint64_t* p_full = s_full + 2;   // [2][2] first, second 32 columns of each half
  uint64_t* dp_full = p_full + 4;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* drain_bar = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bh = tile / p.n_qt;
  const int kt = tile - bh * p.n_qt;
  const int e0 = list.ptr[tile];
  const int n_ent = list.ptr[tile + 1] - e0;
  const int n_it = (n_ent + EPI - 1) / EPI;

  // Step j's rows: slots past the end of the list repeat its last entry; the
  // softmax masks their columns.
  auto load_step = [&](const CUtensorMap* map, const uint16_t* aug, uint64_t* full, int off,
                       int off_aug, int st, const int (&row)[EPI]) {
    mbar_arrive_expect_tx(full, Lay::TILE_BYTES + kAugBytes);
#pragma unroll
    for (int e = 0; e < EPI; ++e) {
#pragma unroll
      for (int s = 0; s < SLABS; ++s)
        tma_load_3d(smem + off + st * Lay::TILE_BYTES + s * (kTile * 128) + e * (BLK * 128), map,
                    full, s * 64, row[e], bh);
      bulk_load(smem + off_aug + st * kAugBytes + e * (BLK * 32),
                aug + (size_t(bh) * p.L_pad + row[e]) * 16, BLK * 32, full);
    }
  };
  auto step_rows = [&](int j, int (&row)[EPI]) {
#pragma unroll
    for (int e = 0; e < EPI; ++e)
      row[e] = (list.entry[e0 + min(j * EPI + e, n_ent - 1)] & 0xFFFF) * BLK;
  };
  auto load_own = [&](const CUtensorMap* map, uint64_t* full, int off) {
    mbar_arrive_expect_tx(full, Lay::TILE_BYTES);
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
      tma_load_3d(smem + off + s * (kTile * 128), map, full, s * 64, kt * kTile, bh);
  };

  // The loading thread sets the barriers up and sends off what the first step
  // needs before the CTA meets, so that the copies run under the rest of the
  // set-up.
  if (warp == 8 && lane == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    mbar_init(k_full, 1);
    mbar_init(v_full, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 8);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(acc_full, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    if (n_it > 0) {
      int row[EPI];
      load_own(&tm_k, k_full, Lay::OFF_K);
      step_rows(0, row);
      load_step(&tm_q, p.q_aug, &q_full[0], Lay::OFF_Q, Lay::OFF_QA, 0, row);
      load_own(&tm_v, v_full, Lay::OFF_V);
      load_step(&tm_do, p.do_aug, &do_full[0], Lay::OFF_DO, Lay::OFF_DA, 0, row);
    }
  }
  // The ones: columns 0 to 2 of every row.
  for (int i = threadIdx.x; i < kAugBytes / 16; i += kBwdThreads) {
    const bool first = (i & 15) < 8;  // the row group's first core matrix
    reinterpret_cast<uint4*>(smem + Lay::OFF_ONE)[i] =
        first ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.wait_limit};

  if (warp >= 8) {
  reg_dealloc<kControlRegs>();
  if (warp == 8) {
    // ================================================================ producer
    if (lane == 0 && n_it > 0) {
      bool ok = true;
      int loaded_q = 1, loaded_do = 1;
      for (int j = 1; ok && j < n_it; ++j) {
        const int st = j % NS;
        const uint32_t parity = ((j / NS) & 1) ^ 1;
        int row[EPI];
        step_rows(j, row);
        if (!(ok = mbar_wait(&q_empty[st], parity, wc))) break;
        load_step(&tm_q, p.q_aug, &q_full[st], Lay::OFF_Q, Lay::OFF_QA, st, row);
        ++loaded_q;
        if (!(ok = mbar_wait(&do_empty[st], parity, wc))) break;
        load_step(&tm_do, p.do_aug, &do_full[st], Lay::OFF_DO, Lay::OFF_DA, st, row);
        ++loaded_do;
      }
      // The last copies land before the CTA ends, also when another warp gave
      // up a wait after all of them had been sent.
      mbar_wait_drain(k_full, 0);
      mbar_wait_drain(v_full, 0);
      for (int i = max(loaded_q - NS, 0); i < loaded_q; ++i)
        mbar_wait_drain(&q_full[i % NS], (i / NS) & 1);
      for (int i = max(loaded_do - NS, 0); i < loaded_do; ++i)
        mbar_wait_drain(&do_full[i % NS], (i / NS) & 1);
    }
  } else if (warp == 9) {
    // ================================================================ MMA issuer
    // The whole warp walks the loop and one elected lane issues, so that the
    // descriptors are warp-uniform values (issued from a branch of one lane,
    // an MMA instruction took about 100 cycles instead of its 64).
    if (n_it > 0) {
      const uint32_t base = smem_addr(smem);
      const uint32_t one_lo = sdesc_lo(base + Lay::OFF_ONE, 128);
      // D[col] = own (A) * step's rows (B)^T + ones * aug^T
      auto issue_scores = [&](uint32_t col, int own, int off, int off_aug, int st,
                              uint64_t* done) {
        const uint32_t a = sdesc_lo(base + own, 16);
        const uint32_t b = sdesc_lo(base + off + st * Lay::TILE_BYTES, 16);
        const uint32_t g = sdesc_lo(base + off_aug + st * kAugBytes, 128);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
            mma_ss<kDescSw128, kDescSw128>(tmem + col, a + o, b + o, IDESC_S, kk > 0 ? 1u : 0u);
          }
          mma_ss<kDescAug, kDescAug>(tmem + col, one_lo, g, IDESC_S, 1u);
          umma_commit(done);
        }
        __syncwarp();
      };
      // D[col] += P^T or dS^T (A, tensor memory: 32 columns of each half of
      // the queries) * step's rows (B), over the first (part 0) or second 32
      // query rows of each half.
      auto issue_grad = [&](uint32_t col, uint32_t a, int off, int st, int part, bool first,
                            uint64_t* done) {
        const uint32_t b = sdesc_lo(base + off + st * Lay::TILE_BYTES + part * (32 * 128),
                                    kTile * 128);
        const uint32_t at = tmem + a + part * 16;
        const uint32_t acc = first ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ts(tmem + col, at + (i >> 1) * 64 + (i & 1) * 8,
                   b + (((i >> 1) * 64 + (i & 1) * 16) * 128 >> 4), IDESC_G, i > 0 ? 1u : acc);
          if (done) umma_commit(done);
        }
        __syncwarp();
      };
      bool ok = warp_wait(k_full, 0, wc) && warp_wait(&q_full[0], 0, wc);
      if (ok) {
        tc_fence_after();
        issue_scores(c_s(0), Lay::OFF_K, Lay::OFF_Q, Lay::OFF_QA, 0, &s_full[0]);
        ok = warp_wait(v_full, 0, wc) && warp_wait(&do_full[0], 0, wc);
      }
      if (ok) {
        tc_fence_after();
        issue_scores(C_DP, Lay::OFF_V, Lay::OFF_DO, Lay::OFF_DA, 0, dp_full);
      }
      for (int j = 0; ok && j < n_it; ++j) {
        const int st = j % NS, nx = (j + 1) % NS;
        const uint32_t nx_parity = ((j + 1) / NS) & 1;
        auto next_scores = [&]() -> bool {
          if (!warp_wait(&q_full[nx], nx_parity, wc)) return false;
          tc_fence_after();
          issue_scores(c_s(j + 1), Lay::OFF_K, Lay::OFF_Q, Lay::OFF_QA, nx,
                       &s_full[buffer(j + 1)]);
          return true;
        };
        if (kTwoS && j + 1 < n_it && !(ok = next_scores())) break;
        if (!(ok = warp_wait(&p_full[2 * buffer(j)], use(j), wc))) break;
        tc_fence_after();
        issue_grad(C_DV, c_s(j), Lay::OFF_DO, st, 0, j == 0, nullptr);
        if (!(ok = warp_wait(&p_full[2 * buffer(j) + 1], use(j), wc))) break;
        tc_fence_after();
        issue_grad(C_DV, c_s(j), Lay::OFF_DO, st, 1, false, &do_empty[st]);
        if (!kTwoS && j + 1 < n_it && !(ok = next_scores())) break;
        if (!(ok = warp_wait(ds_full, j & 1, wc))) break;
        tc_fence_after();
        issue_grad(C_DK, C_DP, Lay::OFF_Q, st, 0, j == 0, nullptr);
        issue_grad(C_DK, C_DP, Lay::OFF_Q, st, 1, false, &q_empty[st]);
        if (j + 1 < n_it) {
          if (!(ok = warp_wait(&do_full[nx], nx_parity, wc))) break;
          tc_fence_after();
          issue_scores(C_DP, Lay::OFF_V, Lay::OFF_DO, Lay::OFF_DA, nx, dp_full);
        }
      }
      // The end of the MMAs: for the results, and before TMEM is freed, also
      // when the warps that want the results gave up waiting for them.
      uint64_t* end = ok ? acc_full : drain_bar;
      if (elect_one()) umma_commit(end);
      mbar_wait_drain(end, 0);
    }
  }
  } else {
    reg_alloc<kScoreRegs>();
    // ================================================================ scores
    const int wl = warp & 3, half = warp >> 2;
    const int r = wl * 32 + lane;        // key row within the tile, TMEM lane
    const uint32_t at = tmem + (uint32_t(wl * 32) << 16);
    const uint32_t dp_col = at + C_DP + 64 * half;
    const int kb = (wl * 32) / BLK;      // key block within the tile (warp-uniform)
    bool ok = true;
    // The two 32-column groups' entries of step j + 1 are fetched in step j.
    const int slot[2] = {(64 * half) / BLK, (64 * half + 32) / BLK};
    int ent[2], next[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) next[g] = slot[g] < n_ent ? __ldg(list.entry + e0 + slot[g]) : 0;
    for (int j = 0; j < n_it; ++j) {
      bool on[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        ent[g] = next[g];
        const int idx = (j + 1) * EPI + slot[g];
        next[g] = idx < n_ent ? __ldg(list.entry + e0 + idx) : 0;
        on[g] = ((ent[g] >> 16) >> kb) & 1;
      }
      const uint32_t s_col = at + c_s(j) + 64 * half;
      if (!(ok = warp_wait(&s_full[buffer(j)], use(j), wc))) break;
      tc_fence_after();
      // Two groups of 32 columns, the second loaded and the first stored
      // under the other's arithmetic; the first can feed dV at once. A group
      // whose query block does not keep this key block has weight 0.
      float w[64];
      float (&w0)[32] = *reinterpret_cast<float(*)[32]>(&w[0]);
      float (&w1)[32] = *reinterpret_cast<float(*)[32]>(&w[32]);
      tmem_ld32(s_col, w0);
      tmem_ld_wait();
      tmem_ld32(s_col + 32, w1);
      if (on[0])
        exp2_scaled(w0, p.scale_log2);
      else
        zero32(w0);
      tmem_st_bf16(s_col, w0);
      tmem_ld_wait();
      tmem_st_wait();
      warp_arrive(&p_full[2 * buffer(j)], lane);
      if (on[1])
        exp2_scaled(w1, p.scale_log2);
      else
        zero32(w1);
      tmem_st_bf16(s_col + 16, w1);
      tmem_st_wait();
      warp_arrive(&p_full[2 * buffer(j) + 1], lane);
      if (!(ok = warp_wait(dp_full, j & 1, wc))) break;
      tc_fence_after();
      float y0[32], y1[32];
      tmem_ld32(dp_col, y0);
      tmem_ld_wait();
      tmem_ld32(dp_col + 32, y1);
      if (on[0])
        mul32(y0, w0);
      else
        zero32(y0);
      tmem_st_bf16(dp_col, y0);
      tmem_ld_wait();
      if (on[1])
        mul32(y1, w1);
      else
        zero32(y1);
      tmem_st_bf16(dp_col + 16, y1);
      tmem_st_wait();
      warp_arrive(ds_full, lane);
    }
    // ---- results: warps 0-3 dV, warps 4-7 dK; rows of the padding are 0
    const int row = kt * kTile + r;
    const size_t out_at = (size_t(bh) * p.L_pad + row) * D;
    void* out = half ? p.dk : p.dv;
    if (n_it > 0 && ok && (ok = warp_wait(acc_full, 0, wc))) {
      tc_fence_after();
      const float f = half ? p.scale : 1.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float x[32];
        tmem_ld32(at + (half ? C_DK : C_DV) + 32 * c, x);
        tmem_ld_wait();
        if (row < p.L)
          store_row32<kOutBf16>(out, out_at + 32 * c, x, f);
        else if (row < p.L_pad)
          store_zero32<kOutBf16>(out, out_at + 32 * c);
      }
    } else if (n_it == 0 && row < p.L_pad) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) store_zero32<kOutBf16>(out, out_at + 32 * c);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dQ

template <int D> struct QueryLayout {
  static constexpr int NS = D == 128 ? 3 : 4;  // stages of K and of V
  static constexpr int TILE_BYTES = kTile * D * 2;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + NS * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + NS * TILE_BYTES;
  static constexpr int N_BARS = 4 * NS + 8;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM_ALLOC = BYTES + 1024;  // one CTA per SM, as above
  static_assert(SMEM_ALLOC > 116 * 1024 && SMEM_ALLOC <= 227 * 1024, "shared memory");
};

// The CTA's own Q and dO rows are the A operands of every S and dP: they stay
// in tensor memory (64 columns each at D = 128), which halves what those
// products read from shared memory. Per step j the MMA thread issues S(j+1)
// as soon as the softmax has S(j) in registers, then dQ(j) and dP(j+1); dS
// takes dP's place as the A operand of dQ += dS K.
// kRest: dS is followed by what its rounding to bf16 left, and dQ is the sum
// of both products (see launch_backward_mma).
template <int D, int BLK, bool kOutBf16, bool kRest>
__device__ __forceinline__ void query_tile(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                           const BwdParams& p, const BwdLists& list, int tile) {
  using Lay = QueryLayout<D>;
  constexpr int NS = Lay::NS;
  constexpr int EPI = kTile / BLK;
  constexpr int SLABS = D / 64;
  constexpr uint32_t C_S = 0, C_DP = 128, C_DQ = 256, C_Q = 256 + D, C_DO = C_Q + D / 2;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(kTile, kTile, false, false);
  constexpr uint32_t IDESC_G = idesc_bf16_f32(kTile, D, false, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::OFF_BAR);
  uint64_t* k_full = bars;            // [NS]
  uint64_t* k_empty = k_full + NS;    // [NS]
  uint64_t* v_full = k_empty + NS;    // [NS]
  uint64_t* v_empty = v_full + NS;    // [NS]
  uint64_t* own_full = v_empty + NS;  // Q and dO in tensor memory
  uint64_t* s_full = own_full + 1;
  uint64_t* s_free = s_full + 1;
  uint64_t* dp_full = s_free + 1;
  uint64_t* ds_full = dp_full + 1;  // [2] first, second 32 columns of each half
  uint64_t* acc_full = ds_full + 2;
  uint64_t* drain_bar = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bh = tile / p.n_qt;
  const int qt = tile - bh * p.n_qt;
  const int e0 = list.ptr[tile];
  const int n_ent = list.ptr[tile + 1] - e0;  // at least 1: every query block keeps one
  const int n_it = (n_ent + EPI - 1) / EPI;

  auto load_step = [&](const CUtensorMap* map, uint64_t* full, int off, int st,
                       const int (&row)[EPI]) {
    mbar_arrive_expect_tx(full, Lay::TILE_BYTES);
#pragma unroll
    for (int e = 0; e < EPI; ++e)
#pragma unroll
      for (int s = 0; s < SLABS; ++s)
        tma_load_3d(smem + off + st * Lay::TILE_BYTES + s * (kTile * 128) + e * (BLK * 128), map,
                    full, s * 64, row[e], bh);
  };
  auto step_rows = [&](int j, int (&row)[EPI]) {
#pragma unroll
    for (int e = 0; e < EPI; ++e)
      row[e] = (list.entry[e0 + min(j * EPI + e, n_ent - 1)] & 0xFFFF) * BLK;
  };

  // First copies before the CTA meets, as in key_tile.
  if (warp == 8 && lane == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(own_full, 8);
    mbar_init(s_full, 1);
    mbar_init(s_free, 8);
    mbar_init(dp_full, 1);
    mbar_init(&ds_full[0], 8);
    mbar_init(&ds_full[1], 8);
    mbar_init(acc_full, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    int row[EPI];
    step_rows(0, row);
    load_step(&tm_k, &k_full[0], Lay::OFF_K, 0, row);
    load_step(&tm_v, &v_full[0], Lay::OFF_V, 0, row);
  }
  // The score warps' own rows, on their way to tensor memory: warps 0-3 Q,
  // warps 4-7 dO; zero past L.
  uint4 own[D / 8];
  if (warp < 8) {
    const int row = qt * kTile + (warp & 3) * 32 + lane;
    const uint16_t* src =
        static_cast<const uint16_t*>(warp >> 2 ? p.d_o : p.q) + (size_t(bh) * p.L_pad + row) * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      own[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row < p.L) own[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
    }
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.wait_limit};

  if (warp >= 8) {
  reg_dealloc<kControlRegs>();
  if (warp == 8) {
    // ================================================================ producer
    if (lane == 0) {
      bool ok = true;
      int loaded_k = 1, loaded_v = 1;
      for (int j = 1; ok && j < n_it; ++j) {
        const int st = j % NS;
        const uint32_t parity = ((j / NS) & 1) ^ 1;
        int row[EPI];
        step_rows(j, row);
        if (!(ok = mbar_wait(&k_empty[st], parity, wc))) break;
        load_step(&tm_k, &k_full[st], Lay::OFF_K, st, row);
        ++loaded_k;
        if (!(ok = mbar_wait(&v_empty[st], parity, wc))) break;
        load_step(&tm_v, &v_full[st], Lay::OFF_V, st, row);
        ++loaded_v;
      }
      // The last copies land before the CTA ends, as in key_tile.
      for (int i = max(loaded_k - NS, 0); i < loaded_k; ++i)
        mbar_wait_drain(&k_full[i % NS], (i / NS) & 1);
      for (int i = max(loaded_v - NS, 0); i < loaded_v; ++i)
        mbar_wait_drain(&v_full[i % NS], (i / NS) & 1);
    }
  } else if (warp == 9) {
    // ================================================================ MMA issuer
    const uint32_t base = smem_addr(smem);
    auto issue_scores = [&](uint32_t col, uint32_t own, int off, int st, uint64_t* done,
                            uint64_t* free) {
      const uint32_t b = sdesc_lo(base + off + st * Lay::TILE_BYTES, 16);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ts(tmem + col, tmem + own + kk * 8,
                 b + (((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4), IDESC_S,
                 kk > 0 ? 1u : 0u);
        umma_commit(done);
        if (free) umma_commit(free);
      }
      __syncwarp();
    };
    // dQ += dS (A, tensor memory) * K_j (B), over the first (part 0) or second
    // 32 keys of each half.
    auto issue_grad = [&](int st, int part, bool first, uint64_t* done) {
      const uint32_t b = sdesc_lo(base + Lay::OFF_K + st * Lay::TILE_BYTES + part * (32 * 128),
                                  kTile * 128);
      const uint32_t at = tmem + C_DP + part * 16;
      const uint32_t acc = first ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma_ts(tmem + C_DQ, at + (i >> 1) * 64 + (i & 1) * 8,
                 b + (((i >> 1) * 64 + (i & 1) * 16) * 128 >> 4), IDESC_G, i > 0 ? 1u : acc);
        if constexpr (kRest) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ts(tmem + C_DQ, at + 32 + (i >> 1) * 64 + (i & 1) * 8,
                   b + (((i >> 1) * 64 + (i & 1) * 16) * 128 >> 4), IDESC_G, 1u);
        }
        if (done) umma_commit(done);
      }
      __syncwarp();
    };
    bool ok = warp_wait(own_full, 0, wc) && warp_wait(&k_full[0], 0, wc);
    if (ok) {
      tc_fence_after();
      issue_scores(C_S, C_Q, Lay::OFF_K, 0, s_full, nullptr);
      ok = warp_wait(&v_full[0], 0, wc);
    }
    if (ok) {
      tc_fence_after();
      issue_scores(C_DP, C_DO, Lay::OFF_V, 0, dp_full, &v_empty[0]);
    }
    for (int j = 0; ok && j < n_it; ++j) {
      const int st = j % NS, nx = (j + 1) % NS;
      const uint32_t nx_parity = ((j + 1) / NS) & 1;
      if (j + 1 < n_it) {
        if (!(ok = warp_wait(&k_full[nx], nx_parity, wc) && warp_wait(s_free, j & 1, wc))) break;
        tc_fence_after();
        issue_scores(C_S, C_Q, Lay::OFF_K, nx, s_full, nullptr);
      }
      if (!(ok = warp_wait(&ds_full[0], j & 1, wc))) break;
      tc_fence_after();
      issue_grad(st, 0, j == 0, nullptr);
      if (!(ok = warp_wait(&ds_full[1], j & 1, wc))) break;
      tc_fence_after();
      issue_grad(st, 1, false, &k_empty[st]);
      if (j + 1 < n_it) {
        if (!(ok = warp_wait(&v_full[nx], nx_parity, wc))) break;
        tc_fence_after();
        issue_scores(C_DP, C_DO, Lay::OFF_V, nx, dp_full, &v_empty[nx]);
      }
    }
    uint64_t* end = ok ? acc_full : drain_bar;
    if (elect_one()) umma_commit(end);
    mbar_wait_drain(end, 0);
  }
  } else {
    reg_alloc<kScoreRegs>();
    // ================================================================ scores
    const int wl = warp & 3, half = warp >> 2;
    const int r = wl * 32 + lane;
    const int row = qt * kTile + r;
    const bool valid = row < p.L;
    const size_t flat = size_t(bh) * p.L_pad + row;
    const uint32_t at = tmem + (uint32_t(wl * 32) << 16);
    const uint32_t s_col = at + C_S + 64 * half, dp_col = at + C_DP + 64 * half;
    const int qb = (wl * 32) / BLK;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t u[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = own[4 * c + i];
        u[4 * i] = x.x, u[4 * i + 1] = x.y, u[4 * i + 2] = x.z, u[4 * i + 3] = x.w;
      }
      tmem_st16(at + (half ? C_DO : C_Q) + 16 * c, u);
    }
    tmem_st_wait();
    warp_arrive(own_full, lane);
    const float NEG_INF = -__int_as_float(0x7f800000);
    const float shift = valid ? -p.lse[flat] * 1.4426950408889634f : NEG_INF;
    const float delta = valid ? p.delta[flat] : 0.f;
    bool ok = true;
    const int slot[2] = {(64 * half) / BLK, (64 * half + 32) / BLK};
    int next[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) next[g] = slot[g] < n_ent ? __ldg(list.entry + e0 + slot[g]) : 0;
    // Valid columns of step j's two 32-column groups (0: not kept), from the
    // entries fetched a step before.
    auto columns = [&](int j, int (&lim)[2]) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int ent = next[g];
        const int idx = (j + 1) * EPI + slot[g];
        next[g] = idx < n_ent ? __ldg(list.entry + e0 + idx) : 0;
        const int left = p.L - (ent & 0xFFFF) * BLK - (64 * half + 32 * g) % BLK;
        lim[g] = ((ent >> 16) >> qb) & 1 ? max(left, 0) : 0;
      }
    };
    // Weights of step j into w, in two groups, the second loaded under the
    // first one's arithmetic.
    float w0[32], w1[32];
    int lim[2];
    auto weights = [&](int j) -> bool {
      columns(j, lim);
      if (!warp_wait(s_full, j & 1, wc)) return false;
      tc_fence_after();
      tmem_ld32(s_col, w0);
      tmem_ld_wait();
      tmem_ld32(s_col + 32, w1);
      if (lim[0] > 0) exp2_shifted(w0, p.scale_log2, shift);
      tmem_ld_wait();
      warp_arrive(s_free, lane);
      if (lim[1] > 0) exp2_shifted(w1, p.scale_log2, shift);
      return true;
    };
    // dS of one group: y = w (dP - D); keys of the padding score 0, whose
    // weight can overflow.
    auto gradient = [&](float (&y)[32], const float (&w)[32], int left) {
      if (left > 0) {
        add_mul32(y, -delta, w);
        if (left < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i >= left) y[i] = 0.f;
        }
      } else {
        zero32(y);
      }
    };
    ok = weights(0);
    for (int j = 0; ok && j < n_it; ++j) {
      if (!(ok = warp_wait(dp_full, j & 1, wc))) break;
      tc_fence_after();
      float y0[32], y1[32];
      tmem_ld32(dp_col, y0);
      tmem_ld_wait();
      tmem_ld32(dp_col + 32, y1);
      gradient(y0, w0, lim[0]);
      tmem_st_bf16(dp_col, y0);
      tmem_ld_wait();
      if constexpr (kRest) tmem_st_bf16_rest(dp_col + 32, y0);  // where y1 was
      tmem_st_wait();
      warp_arrive(&ds_full[0], lane);
      gradient(y1, w1, lim[1]);
      tmem_st_bf16(dp_col + 16, y1);
      if constexpr (kRest) tmem_st_bf16_rest(dp_col + 48, y1);
      tmem_st_wait();
      warp_arrive(&ds_full[1], lane);
      if (j + 1 < n_it) ok = weights(j + 1);
    }
    if (ok && (ok = warp_wait(acc_full, 0, wc))) {
      tc_fence_after();
      // The two halves of the columns; rows of the padding are 0.
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float x[32];
        const int col = half * (D / 2) + 32 * c;
        tmem_ld32(at + C_DQ + col, x);
        tmem_ld_wait();
        if (valid)
          store_row32<kOutBf16>(p.dq, flat * D + col, x, p.scale);
        else if (row < p.L_pad)
          store_zero32<kOutBf16>(p.dq, flat * D + col);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Both halves of the gradient in one launch: the key tiles first, whose steps
// have four products, then the query tiles, whose steps have three. The
// query tiles fill the SMs that the last key tiles leave idle, and a small
// call's two halves run side by side.
template <int D, int BLK, bool kOutBf16, bool kRest>
__global__ void __launch_bounds__(kBwdThreads, 1)
    bwd_tiles_kernel(const __grid_constant__ CUtensorMap own_k,
                     const __grid_constant__ CUtensorMap own_v,
                     const __grid_constant__ CUtensorMap step_q,
                     const __grid_constant__ CUtensorMap step_do,
                     const __grid_constant__ CUtensorMap step_k,
                     const __grid_constant__ CUtensorMap step_v, const BwdParams p) {
  const int i = blockIdx.x;
  if (i < p.n_tiles)
    key_tile<D, BLK, kOutBf16>(own_k, own_v, step_q, step_do, p, p.keys, p.keys.order[i]);
  else
    query_tile<D, BLK, kOutBf16, kRest>(step_k, step_v, p, p.queries, p.queries.order[i - p.n_tiles]);
}

template <int D, int BLK, bool kOutBf16, bool kRest>
cudaError_t run_mma(const BackwardCall& c, const BackwardOperands& w, const BwdParams& p,
                    cudaStream_t stream) {
  const int BH = c.p->B * c.p->H;
  CUtensorMap own_k, own_v, step_q, step_do, step_k, step_v;
  // Rows past L read as zero, whatever they hold.
  if (!make_slab_map(&own_k, c.k, BH, c.L, p.L_pad, D, kTile, 2, false) ||
      !make_slab_map(&own_v, c.v, BH, c.L, p.L_pad, D, kTile, 2, false) ||
      !make_slab_map(&step_q, c.q, BH, c.L, p.L_pad, D, BLK, 2, false) ||
      !make_slab_map(&step_do, w.d_o, BH, c.L, p.L_pad, D, BLK, 2, false) ||
      !make_slab_map(&step_k, c.k, BH, c.L, p.L_pad, D, BLK, 2, false) ||
      !make_slab_map(&step_v, c.v, BH, c.L, p.L_pad, D, BLK, 2, false))
    return cudaErrorInvalidValue;
  auto kern = bwd_tiles_kernel<D, BLK, kOutBf16, kRest>;
  constexpr int smem = std::max(KeyLayout<D>::SMEM_ALLOC, QueryLayout<D>::SMEM_ALLOC);
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed);
  if (err != cudaSuccess) return err;
  kern<<<2u * unsigned(p.n_tiles), kBwdThreads, smem, stream>>>(own_k, own_v, step_q, step_do,
                                                               step_k, step_v, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_backward_mma(const BackwardCall& c, const BackwardOperands& w,
                                cudaStream_t stream) {
  const losa_pattern* pat = c.p;
  BwdParams p{};
  p.L = c.L;
  p.L_pad = pat->n_blocks * pat->block;
  p.n_qt = pat->n_qt;
  p.n_tiles = int(pat->n_tiles);
  p.scale = c.scale;
  p.scale_log2 = c.scale * 1.4426950408889634f;
  p.lse = c.lse;
  p.delta = w.delta;
  p.q_aug = w.q_aug;
  p.do_aug = w.do_aug;
  p.q = c.q;
  p.d_o = w.d_o;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.keys = {pat->key_ptr, pat->key_entry, pat->key_order};
  p.queries = {pat->tile_ptr, pat->tile_entry, pat->tile_order};
  p.status = device_status_word();
  if (!p.status) return cudaErrorInvalidDevice;
  p.wait_limit = wait_limit();
  // dQ is a sum that cancels (each row of dS sums to 0), and dS's rounding to
  // bf16 shows in it: a head's dQ is off by 0.35 % of its norm, and where few
  // rows carry that norm by up to 1.3 % (modelled on random heads of 64
  // tokens, 0.6 % at 1,024, 0.45 % at 4,096). So in heads of up to 32 tiles of
  // 128 rows the query tiles, which have one product less than the key tiles
  // beside them, take dS's remainder as well: 0.17 to 0.19 %, the result's own
  // rounding. The rule looks at the head alone, whose dQ has the same bits
  // beside any others. It costs 3 to 5 % of the time in a call of one such head
  // (2,000 tokens, half the blocks kept: d 128 26.8 -> 28.1 us, d 64 24.1 ->
  // 24.9) and 9 to 17 % in one of 24 (d 128, 60 % of blocks of 64 kept: 1,000
  // tokens 52.5 -> 61.4 us, 4,000 493 -> 559); in longer heads, whose error is
  // the smaller one, it would cost 11 to 14 %.
  const bool rest = p.n_qt <= 32;
#define LOSA_BWD_CASE(D_, BLK_)                                                    \
  if (c.d == D_ && pat->block == BLK_) {                                           \
    auto run = c.out_bf16                                                          \
                   ? (rest ? run_mma<D_, BLK_, true, true> : run_mma<D_, BLK_, true, false>)    \
                   : (rest ? run_mma<D_, BLK_, false, true> : run_mma<D_, BLK_, false, false>); \
    return run(c, w, p, stream);                                                   \
  }
  LOSA_BWD_CASE(128, 128)
  LOSA_BWD_CASE(128, 64)
  LOSA_BWD_CASE(128, 32)
  LOSA_BWD_CASE(64, 128)
  LOSA_BWD_CASE(64, 64)
  LOSA_BWD_CASE(64, 32)
#undef LOSA_BWD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace losa
