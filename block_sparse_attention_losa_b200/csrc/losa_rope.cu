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
// adjacent features (16 bytes of bf16) of one token and walks the heads of
// Q, K and V, so an angle is computed once per token and pair, stays in
// registers, and serves every head of both tensors. Angles are reduced in
// 64 bits (the position times the frequency in turns, less the nearest
// integer), since a far position times a frequency of 1 loses in 32 bits
// what the sine needs; what is left, at most half a turn, goes through
// sincospif in 32 bits.
#include <cuda_bf16.h>

#include <cmath>

#include <algorithm>

#include "losa_device.cuh"
#include "losa_internal.h"

namespace losa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kFeat = 8;  // features of a thread

struct RopeParams {
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

template <typename T> struct Chunk;
template <> struct Chunk<float> {
  float v[kFeat];
  template <bool kVec> __device__ __forceinline__ void load(const float* p) {
    if constexpr (kVec) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < kFeat; ++e) v[e] = __ldg(p + e);
    }
  }
};
template <> struct Chunk<__nv_bfloat16> {
  float v[kFeat];
  template <bool kVec> __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (kVec) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(u[e] << 16);
        v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kFeat; ++e) v[e] = __bfloat162float(p[e]);
    }
  }
};

template <bool kVec> __device__ __forceinline__ void store_chunk(float* p, const float (&v)[kFeat]) {
  if constexpr (kVec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int e = 0; e < kFeat; ++e) p[e] = v[e];
  }
}
template <bool kVec>
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&v)[kFeat]) {
  if constexpr (kVec) {
    uint4 w;
    w.x = pack_bf16x2(v[0], v[1]);
    w.y = pack_bf16x2(v[2], v[3]);
    w.z = pack_bf16x2(v[4], v[5]);
    w.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
#pragma unroll
    for (int e = 0; e < kFeat; ++e) p[e] = __float2bfloat16_rn(v[e]);
  }
}

// kUnpack: packed -> token-major by the negative angle. kHalves: pair i of an
// axis is its features (i, i + dim/2) instead of (2i, 2i + 1). kVec: every
// 8-feature group is 16-byte aligned on both sides.
template <typename TI, typename TO, bool kUnpack, bool kHalves, bool kVec>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  const int groups = p.d / kFeat;
  const int g = threadIdx.x % groups;
  const int f0 = g * kFeat;
  const int l = blockIdx.x * (kRopeThreads / groups) + threadIdx.x / groups;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * p.head_step;
  const int h1 = min(h0 + p.head_step, p.H);
  if (l >= (kUnpack ? p.L : p.L_pad)) return;

  if (!kUnpack && l >= p.L) {  // padding rows are zero
    const float zero[kFeat] = {};
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      if (!p.out[t]) continue;
      TO* out = static_cast<TO*>(p.out[t]) + (size_t(b) * p.H * p.L_pad + l) * p.d + f0;
      for (int h = h0; h < h1; ++h) store_chunk<kVec>(out + size_t(h) * p.L_pad * p.d, zero);
    }
    return;
  }

  // Interleaved: cs[e / 2], sn[e / 2] of the pair (e, e + 1). Halves: per
  // feature, with its partner's place.
  constexpr int NA = kHalves ? kFeat : kFeat / 2;
  float cs[NA], sn[NA];
  int partner[kHalves ? kFeat : 1];
  bool turns[NA];
  bool any = false;
  bool whole = true;  // halves: the partners are one aligned group of 8
  {
    const bool text = l < p.n_text;
    long long pos[3] = {0, 0, 0};
    if (p.positions) {
      const int* q = p.positions + (size_t(b) * p.L + l) * p.n_axes;
      for (int a = 0; a < p.n_axes; ++a) pos[a] = q[a];
    } else {
      const int i = l - p.n_text;
      pos[0] = (long long)(i / (p.grid_h * p.grid_w)) + p.start[0];
      pos[1] = (long long)(i / p.grid_w % p.grid_h) + p.start[1];
      pos[2] = (long long)(i % p.grid_w) + p.start[2];
    }
#pragma unroll
    for (int e = 0; e < NA; ++e) {
      const int f = kHalves ? f0 + e : f0 + 2 * e;
      turns[e] = !text && f < p.n_rot;
      any |= turns[e];
      cs[e] = 1.f;
      sn[e] = 0.f;
      if constexpr (kHalves) partner[e] = f;
      if (!turns[e]) {
        if (f >= p.n_rot) whole = false;
        continue;
      }
      int pair, axis;
      bool second = false;
      if constexpr (kHalves) {
        axis = (p.n_axes > 2 && f >= p.base[2]) ? 2 : (p.n_axes > 1 && f >= p.base[1]) ? 1 : 0;
        int i = f - p.base[axis];
        second = i >= p.half[axis];
        partner[e] = second ? f - p.half[axis] : f + p.half[axis];
        if (second) i -= p.half[axis];
        pair = p.base[axis] / 2 + i;
        if (partner[e] != partner[0] + e || (partner[0] & (kFeat - 1))) whole = false;
      } else {
        pair = f / 2;
        axis = p.axis[pair];
      }
      const double turn = double(axis == 0 ? pos[0] : axis == 1 ? pos[1] : pos[2]) * p.freq[pair];
      float s, c;
      sincospif(2.f * float(turn - rint(turn)), &s, &c);
      cs[e] = c;
      sn[e] = (kUnpack != second) ? -s : s;  // of the first feature: minus sin
    }
  }

#pragma unroll
  for (int t = 0; t < 3; ++t) {
    if (!p.in[t]) continue;
    const size_t packed = (size_t(b) * p.H * p.L_pad + l) * p.d;
    const size_t flat = size_t(b) * p.sb[t] + size_t(l) * p.sl[t];
    const size_t packed_step = size_t(p.L_pad) * p.d, flat_step = p.sh[t];
    const TI* in = static_cast<const TI*>(p.in[t]) + (kUnpack ? packed : flat);
    TO* out = static_cast<TO*>(p.out[t]) + (kUnpack ? flat : packed) + f0;
    const size_t in_step = kUnpack ? packed_step : flat_step;
    const size_t out_step = kUnpack ? flat_step : packed_step;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      Chunk<TI> x;
      x.template load<kVec>(in + h * in_step + f0);
      float y[kFeat];
#pragma unroll
      for (int e = 0; e < kFeat; ++e) y[e] = x.v[e];
      if (t < 2 && any) {
        if constexpr (kHalves) {
          Chunk<TI> z;
          if (kVec && whole) {
            z.template load<kVec>(in + h * in_step + partner[0]);
          } else {
#pragma unroll
            for (int e = 0; e < kFeat; ++e) z.v[e] = float(in[h * in_step + partner[e]]);
          }
#pragma unroll
          for (int e = 0; e < kFeat; ++e)
            if (turns[e]) y[e] = fmaf(x.v[e], cs[e], -z.v[e] * sn[e]);
        } else {
#pragma unroll
          for (int e = 0; e < kFeat; e += 2) {
            if (turns[e / 2]) {
              y[e] = fmaf(x.v[e], cs[e / 2], -x.v[e + 1] * sn[e / 2]);
              y[e + 1] = fmaf(x.v[e], sn[e / 2], x.v[e + 1] * cs[e / 2]);
            }
          }
        }
      }
      store_chunk<kVec>(out + h * out_step, y);
    }
  }
}

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename TI, typename TO>
cudaError_t launch(const RopeParams& p, bool unpack, bool halves, bool vec, dim3 grid,
                   cudaStream_t stream) {
#define LOSA_ROPE(U_, H_, V_)                                          \
  if (unpack == U_ && halves == H_ && vec == V_) {                     \
    rope_kernel<TI, TO, U_, H_, V_><<<grid, kRopeThreads, 0, stream>>>(p); \
    return cudaGetLastError();                                         \
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
  for (int t = 0; t < 3; ++t) {
    p.in[t] = c.in[t];
    p.out[t] = c.out[t];
    if (!c.in[t]) continue;
    p.sb[t] = c.strides[3 * t];
    p.sl[t] = c.strides[3 * t + 1];
    p.sh[t] = c.strides[3 * t + 2];
    vec = vec && multiple16(c.in[t]) && multiple16(c.out[t]) &&
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
  // The grid's axes, outermost first, right-aligned to (t, h, w) so that an
  // absent axis has extent 1 and its position is never used.
  int ext[3] = {1, 1, 1};
  for (int a = 0; a < s.n_axes; ++a) {
    ext[a] = s.grid[a];
    p.start[a] = s.start[a];
  }
  p.grid_h = ext[1];
  p.grid_w = ext[2];
  int f = 0;
  for (int a = 0; a < s.n_axes; ++a) {
    p.base[a] = short(f);
    p.half[a] = short(s.dim[a] / 2);
    for (int i = 0; i < s.dim[a] / 2; ++i) {
      p.axis[f / 2 + i] = (unsigned char)a;
      p.freq[f / 2 + i] = s.scale[a] * std::pow(s.theta, -2.0 * i / s.dim[a]) / (2.0 * M_PI);
    }
    f += s.dim[a];
  }
  p.n_rot = f;
  const int tokens = kRopeThreads / (c.d / kFeat);
  const int nx = ((c.unpack ? c.L : c.L_pad) + tokens - 1) / tokens;
  // All heads of a token in one CTA share its angles; with too few tokens to
  // give every SM several CTAs the heads are split.
  const int64_t want = 148 * 4;
  int split = int(std::min<int64_t>(c.H, std::max<int64_t>(1, want / (int64_t(nx) * c.B))));
  p.head_step = (c.H + split - 1) / split;
  split = (c.H + p.head_step - 1) / p.head_step;
  const dim3 grid(nx, split, c.B);
  const bool halves = s.pairing == LOSA_ROPE_HALVES;
  if (c.in_bf16)
    return c.out_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, c.unpack, halves, vec, grid, stream)
                      : launch<__nv_bfloat16, float>(p, c.unpack, halves, vec, grid, stream);
  return c.out_bf16 ? launch<float, __nv_bfloat16>(p, c.unpack, halves, vec, grid, stream)
                    : launch<float, float>(p, c.unpack, halves, vec, grid, stream);
}

}  // namespace losa
