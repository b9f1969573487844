// losa_rope.cu - rotary positions with several axes, between the token-major
// tensors of a model's projections and the head-major padded layout of the
// attention calls (losa_rope_pack), and the way back (losa_rope_unpack).
//
// Mathematics: pair i of axis a, at position p_a of the token, turns by
// p_a * scale_a * theta^(-2 i / dim_a): (x, y) -> (x cos - y sin, x sin + y
// cos). The way back, which is also the gradient (a rotation's transpose is
// its inverse), turns by the negative angle.
//
// Bound: HBM. Each value is read once and written once. A thread owns eight
// adjacent features (16 bytes of bf16) of one token, a row's threads side by
// side, and walks the heads of Q, K and V in batches of four loads, the first
// issued before the angles are computed: these are computed once per token
// and pair and stay in registers for every head of both tensors. Pairs by
// halves meet in different threads of a warp: they exchange through shared
// memory.
// Measured on a B200 with cold caches, bf16, launch included: 102 us at the
// Wan2.1-1.3B shape (12 heads, 32,760 tokens, d 128: 5.9 TB/s), 686 us at
// the HunyuanVideo one (24 heads, 118,800 tokens: 6.4 TB/s, 0.99 of the
// measured copy rate); by halves 110 us at the first. Tried and slower: 16
// features a thread in two groups of 128 contiguous bytes a row (862 us at
// the second; the rows' halves then move apart), two features a thread (250
// us by halves at the first), and one loop over all tensors' heads with its
// addresses formed per row (950 us at the second).
// Angles are reduced in 64 bits (the position times the frequency in turns,
// less the nearest integer), since a far position times a frequency of 1
// loses in 32 bits what the sine needs; what is left, at most half a turn,
// goes through sincospif in 32 bits.
#include <cuda_bf16.h>

#include <cmath>

#include <algorithm>

#include "losa_device.cuh"
#include "losa_internal.h"

namespace losa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 16;  // CTAs per SM over which a call's work is spread

struct RopeParams {
  int n_tensors;      // given ones, the first in the arrays below
  bool turns[3];      // Q and K
  const void* in[3];
  void* out[3];
  // Element strides (batch, token, head) of the token-major side; the packed
  // side is [B, H, L_pad, d].
  long long sb[3], sl[3], sh[3];
  const int* positions;   // [B, L, n_axes] or null (grid)
  int n_axes;
  int H, L, L_pad, d;
  int n_text;
  int head_step;          // heads per CTA
  int grid_h, grid_w;     // extents of the inner axes (absent axes: 1)
  int start[3];
  double freq[64];        // turns per position of each pair, in feature order
  unsigned char axis[64]; // its axis
  short half[3];          // features of an axis / 2
  short base[3];          // first feature of an axis
  int n_rot;              // features that turn (the rest pass through)
};

// The token of a thread, or the padding after the last one.
struct Place {
  long long pos[3];
  bool text;
};
__device__ __forceinline__ Place place_of(const RopeParams& p, int b, int l) {
  Place x{{0, 0, 0}, l < p.n_text};
  if (p.positions) {
    const int* q = p.positions + (size_t(b) * p.L + l) * p.n_axes;
    x.pos[0] = q[0];
    if (p.n_axes > 1) x.pos[1] = q[1];
    if (p.n_axes > 2) x.pos[2] = q[2];
  } else {
    const int i = l - p.n_text;
    x.pos[0] = (long long)(i / (p.grid_h * p.grid_w)) + p.start[0];
    x.pos[1] = (long long)(i / p.grid_w % p.grid_h) + p.start[1];
    x.pos[2] = (long long)(i % p.grid_w) + p.start[2];
  }
  return x;
}
// cos and sin of pair `pair`.
__device__ __forceinline__ void turn_of(const RopeParams& p, const Place& x, int pair, float& c,
                                        float& s) {
  const int axis = p.axis[pair];
  const long long pos = axis == 0 ? x.pos[0] : axis == 1 ? x.pos[1] : x.pos[2];
  const double turn = double(pos) * p.freq[pair];
  sincospif(2.f * float(turn - rint(turn)), &s, &c);
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 w;
  w.x = pack_bf16x2(v[0], v[1]);
  w.y = pack_bf16x2(v[2], v[3]);
  w.z = pack_bf16x2(v[4], v[5]);
  w.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = w;
}

// Element offsets of row (b, l) of head h: of tensor t in token order, and of
// the packed layout.
__device__ __forceinline__ size_t flat_at(const RopeParams& p, int t, int b, int l, int h) {
  return size_t(b) * p.sb[t] + size_t(l) * p.sl[t] + size_t(h) * p.sh[t];
}
__device__ __forceinline__ size_t packed_at(const RopeParams& p, int b, int l, int h) {
  return ((size_t(b) * p.H + h) * p.L_pad + l) * p.d;
}

template <typename T> struct Raw;  // eight features as loaded
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_any(const float* p) {
    a = make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
    b = make_float4(__ldg(p + 4), __ldg(p + 5), __ldg(p + 6), __ldg(p + 7));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_any(const __nv_bfloat16* p) {
    const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
    a = make_uint4(__ldg(u) | uint32_t(__ldg(u + 1)) << 16, __ldg(u + 2) | uint32_t(__ldg(u + 3)) << 16,
                   __ldg(u + 4) | uint32_t(__ldg(u + 5)) << 16,
                   __ldg(u + 6) | uint32_t(__ldg(u + 7)) << 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store_any(float* p, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = v[e];
}
__device__ __forceinline__ void store_any(__nv_bfloat16* p, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = __float2bfloat16_rn(v[e]);
}

// kUnpack: packed -> token-major by the negative angle. kHalves: pair i of an
// axis is its features (i, i + dim/2) instead of (2i, 2i + 1). kVec: every
// group of eight features is 16-byte aligned on both sides.
// kFew: the CTA has at most two heads, and the loads of all three tensors go
// out together (with one head after another's three round trips to memory, a
// single head of 118,800 tokens took 85 us, now 71, most of it angles).
template <typename TI, typename TO, bool kUnpack, bool kHalves, bool kVec, bool kFew>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int BATCH = kFew ? 2 : 4;
  const int groups = p.d / 8;
  const int f0 = 8 * (threadIdx.x % groups);
  const int lane = threadIdx.x & 31;
  const int l = blockIdx.x * (kRopeThreads / groups) + threadIdx.x / groups;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * p.head_step;
  const int h1 = min(h0 + p.head_step, p.H);
  const bool valid = l < p.L;

  if (!kUnpack && !valid && l < p.L_pad) {  // padding rows are zero
    const float zero[8] = {};
    for (int t = 0; t < p.n_tensors; ++t)
      for (int h = h0; h < h1; ++h) {
        TO* out = static_cast<TO*>(p.out[t]) + packed_at(p, b, l, h) + f0;
        if constexpr (kVec)
          store8(out, zero);
        else
          store_any(out, zero);
      }
  }
  if constexpr (!kHalves) {
    if (!valid) return;
  }  // by halves a warp's threads stay together for the exchange

  // Heads first .. first + BATCH - 1 of tensor t.
  Raw<TI> raws[kFew ? 3 : 1][BATCH];
  auto load = [&](int t, int first, Raw<TI> (&raw)[BATCH]) {
    const TI* in = static_cast<const TI*>(p.in[t]) + f0 +
                   (kUnpack ? packed_at(p, b, l, first) : flat_at(p, t, b, l, first));
    const size_t step = kUnpack ? size_t(p.L_pad) * p.d : size_t(p.sh[t]);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (valid && first + i < h1) {
        if constexpr (kVec)
          raw[i].load(in + i * step);
        else
          raw[i].load_any(in + i * step);
      }
    }
  };
  load(0, h0, raws[0]);
  if constexpr (kFew) {
    if (p.n_tensors > 1) load(1, h0, raws[1]);
    if (p.n_tensors > 2) load(2, h0, raws[2]);
  }

  // The thread's four pairs in feature order. Adjacent: cs[e], sn[e] of the
  // pair (2e, 2e + 1). By halves, per feature: y[e] = x[e] cs[e] + partner
  // sn[e], the partner at word from[e] of the exchange (feature 8 g + e of the
  // row at word 32 e + g); the pairs' values come from the threads of the row
  // that computed them.
  constexpr int NA = kHalves ? 8 : 4;
  float cs[NA], sn[NA];
  int from[kHalves ? 8 : 1];
  __shared__ float2 turned[kHalves ? kRopeThreads * 4 : 1];
  int n_turn = 0;  // features of this thread that turn
  if (valid) {
    const Place x = place_of(p, b, l);
    if (!x.text) n_turn = min(max(p.n_rot - f0, 0), 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float c = 1.f, s = 0.f;
      if (2 * e < n_turn) turn_of(p, x, f0 / 2 + e, c, s);
      if (kUnpack) s = -s;
      if constexpr (kHalves) {
        turned[threadIdx.x * 4 + e] = make_float2(c, s);
      } else {
        cs[e] = c;
        sn[e] = s;
      }
    }
  }
  if constexpr (kHalves) {
    __syncwarp();
    const float2* row = turned + (threadIdx.x - threadIdx.x % groups) * 4;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
      from[e] = 32 * e + lane;
      const int f = f0 + e;
      if (e >= n_turn) continue;
      const int axis = (p.n_axes > 2 && f >= p.base[2]) ? 2 : (p.n_axes > 1 && f >= p.base[1]);
      const int half = p.half[axis], i = f - p.base[axis];
      const bool second = i >= half;
      const float2 t = row[p.base[axis] / 2 + (second ? i - half : i)];
      cs[e] = t.x;
      sn[e] = second ? t.y : -t.y;  // minus sin of the first feature
      const int other = second ? f - half : f + half;
      from[e] = 32 * (other & 7) + (lane & ~(groups - 1)) + (other >> 3);
    }
  }

  __shared__ float exchange[kHalves ? kRopeThreads / 32 : 1][4][kHalves ? 8 * 32 : 1];
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    if (t >= p.n_tensors) break;
    const size_t step = kUnpack ? size_t(p.sh[t]) : size_t(p.L_pad) * p.d;
    for (int first = h0; first < h1; first += BATCH) {
      Raw<TI>(&raw)[BATCH] = raws[kFew ? t : 0];
      if (!kFew && (t > 0 || first > h0)) load(t, first, raw);
      TO* out = static_cast<TO*>(p.out[t]) + f0 +
                (kUnpack ? flat_at(p, t, b, l, first) : packed_at(p, b, l, first));
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (first + i >= h1) break;
        float x[8];
        raw[i].get(x);
        if (p.turns[t]) {
          if constexpr (kHalves) {
            float* buf = exchange[warp][kFew ? 2 * (t & 1) + i : i];
#pragma unroll
            for (int e = 0; e < 8; ++e) buf[32 * e + lane] = x[e];
            __syncwarp();
            if (valid) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (e < n_turn) x[e] = fmaf(x[e], cs[e], buf[from[e]] * sn[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (2 * e < n_turn) {
                const float u = x[2 * e], v = x[2 * e + 1];
                x[2 * e] = fmaf(u, cs[e], -v * sn[e]);
                x[2 * e + 1] = fmaf(u, sn[e], v * cs[e]);
              }
            }
          }
        }
        if (valid) {
          if constexpr (kVec)
            store8(out + i * step, x);
          else
            store_any(out + i * step, x);
        }
      }
      // The next batch's exchange writes where this one's is read.
      if constexpr (kHalves) __syncwarp();
    }
  }
}

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename TI, typename TO>
cudaError_t launch(const RopeParams& p, bool unpack, bool halves, bool vec, dim3 grid,
                   cudaStream_t stream) {
#define LOSA_ROPE(U_, H_, V_)                                                   \
  if (unpack == U_ && halves == H_ && vec == V_) {                              \
    (p.head_step <= 2 ? rope_kernel<TI, TO, U_, H_, V_, true>                   \
                      : rope_kernel<TI, TO, U_, H_, V_, false>)                 \
        <<<grid, kRopeThreads, 0, stream>>>(p);                                 \
    return cudaGetLastError();                                                  \
  }
  LOSA_ROPE(false, false, true)
  LOSA_ROPE(false, false, false)
  LOSA_ROPE(false, true, true)
  LOSA_ROPE(false, true, false)
  LOSA_ROPE(true, false, true)
  LOSA_ROPE(true, false, false)
  LOSA_ROPE(true, true, true)
  LOSA_ROPE(true, true, false)
#undef LOSA_ROPE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, cudaStream_t stream) {
  RopeParams p{};
  const losa_rope_spec& s = *c.spec;
  const int in_size = c.in_bf16 ? 2 : 4, out_size = c.out_bf16 ? 2 : 4;
  const int flat_size = c.unpack ? out_size : in_size;
  bool vec = true;
  for (int i = 0; i < 3; ++i) {
    if (!c.in[i]) continue;
    const int t = p.n_tensors++;
    p.turns[t] = i < 2;
    p.in[t] = c.in[i];
    p.out[t] = c.out[i];
    p.sb[t] = c.strides[3 * i];
    p.sl[t] = c.strides[3 * i + 1];
    p.sh[t] = c.strides[3 * i + 2];
    vec = vec && multiple16(c.in[i]) && multiple16(c.out[i]) &&
          (c.B == 1 || p.sb[t] * flat_size % 16 == 0) &&
          (c.L == 1 || p.sl[t] * flat_size % 16 == 0) &&
          (c.H == 1 || p.sh[t] * flat_size % 16 == 0);
  }
  p.positions = c.positions;
  p.n_axes = s.n_axes;
  p.H = c.H;
  p.L = c.L;
  p.L_pad = c.L_pad;
  p.d = c.d;
  p.n_text = s.n_text;
  // The grid's axes, outermost first. Absent ones, at the end, have extent 1:
  // place_of divides by it, and no pair refers to them.
  int ext[3] = {1, 1, 1};
  for (int a = 0; a < s.n_axes; ++a) {
    ext[a] = std::max(1, s.grid[a]);  // 0: text alone, or positions listed
    p.start[a] = s.start[a];
  }
  p.grid_h = ext[1];
  p.grid_w = ext[2];
  int f = 0;
  for (int a = 0; a < s.n_axes; ++a) {
    p.base[a] = short(f);
    p.half[a] = short(s.dim[a] / 2);
    const double step = -2.0 * std::log(s.theta) / s.dim[a];
    for (int i = 0; i < s.dim[a] / 2; ++i) {
      p.axis[f / 2 + i] = (unsigned char)a;
      p.freq[f / 2 + i] = s.scale[a] * std::exp(step * i) / (2.0 * M_PI);
    }
    f += s.dim[a];
  }
  p.n_rot = f;
  const bool halves = s.pairing == LOSA_ROPE_HALVES;
  const int tokens = kRopeThreads / (c.d / 8);
  const int nx = ((c.unpack ? c.L : c.L_pad) + tokens - 1) / tokens;
  // All heads of a token in one CTA share its angles; they are split over
  // CTAs where that leaves too few of them to even out over the SMs, down to
  // four heads each (CogVideoX shape, 48 heads: 118 us unsplit, 112 split),
  // and further where not even every SM would have one.
  const int64_t per_split = int64_t(nx) * c.B;
  int64_t split = std::max<int64_t>(1, std::min<int64_t>((kSms * kRopeCtas + per_split - 1) / per_split,
                                                         c.H / 4));
  if (split * per_split < kSms) split = std::min<int64_t>(c.H, (kSms + per_split - 1) / per_split);
  p.head_step = int((c.H + split - 1) / split);
  split = (c.H + p.head_step - 1) / p.head_step;
  const dim3 grid(nx, unsigned(split), c.B);
  if (c.in_bf16)
    return c.out_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, c.unpack, halves, vec, grid, stream)
                      : launch<__nv_bfloat16, float>(p, c.unpack, halves, vec, grid, stream);
  return c.out_bf16 ? launch<float, __nv_bfloat16>(p, c.unpack, halves, vec, grid, stream)
                    : launch<float, float>(p, c.unpack, halves, vec, grid, stream);
}

}  // namespace losa
