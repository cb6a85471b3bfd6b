// pa_rope_write.cu -- norms of queries and keys for each head, position rotation and paged write in
// one pass: the step between the q/k/v projection and the attention.
//
// Mathematics, per head row x of D values at position p (fp32): y = x / sqrt(mean(x^2) + eps) * w;
// pairs (u, v) of the first rot values become (u cos - v sin, v cos + u sin) by the angles of row p
// of a table; one rounding to the output's type at the end.  Values of v are stored as they are.
//
// A pass over the data, bound by HBM: each value is read once and written once.  D / 8 lanes hold a head
// row, 8 values each, so the sum of squares is a few shuffles.  Where a pair lies rot / 2 apart, a lane's
// values are two pieces of 4 that far apart (and from rot on 8 in a row): both values of a pair are in one
// lane, at the price of 8-byte accesses.  A warp takes a segment of a token's heads, 256 / D head rows at a
// time (a group): the token's position, slot and angles are loaded once for the segment, and the next three
// groups' loads are in flight while three are worked on (two, or four, with as many blocks on an SM as the
// registers allow: 5 to 11% slower).  The warps of one wave stride over the (token,
// segment) pairs.  8192 tokens of 64 + 8 + 8 heads of 128 into FP8: 67 us, 4.8 TB/s of reads and writes mixed, at
// 65% of the issue slots; 61 tokens of 32 + 8 + 8: 2.4 us in a graph, a launch.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_launch.h"
#include "pa_quant.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
enum RopeFmt { ROPE_BF16 = 0, ROPE_FP8 = 1, ROPE_NVFP4 = 2 };

struct RopeArgs {
  const uint16_t *q, *k, *v;    // token strides below; heads dense
  const uint16_t *q_weight, *k_weight;  // [D] bf16 or null
  const float *cos_sin;         // [max_position, rot]
  const int32_t *positions;
  const int64_t *slots;
  uint16_t *q_out;
  uint8_t *k_pool, *v_pool;
  uint32_t *status;             // or null
  long long q_stride, k_stride, v_stride, n_slots;
  int tokens, Hq, Hkv, rot, max_position;
  int v0;                     // the values' first row of a token, behind the queries' and keys'
  int groups, segs, per_seg;  // groups of head rows per token, segments of them, groups per segment
  float eps;
  Fp8Scale v_scale;
  float2 k_inv;  // 1 / the keys' scale, and what its rounding left out
};

__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ void unpack8(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// f / s, correctly rounded; the way of dividing (see Fp8Scale) is the same for the whole launch.
__device__ __forceinline__ void quot8(const float (&f)[8], Fp8Scale s, float (&q)[8]) {
  if (s.rcp != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = f[i] * s.rcp;
  } else if (s.rcpn != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = markstein_quot(f[i], s.sc, s.rcpn);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(f[i], s.sc);
  }
}

// E4M3 codes of quotients, nearest with ties to even, saturated.
__device__ __forceinline__ uint2 fp8_codes8(const float (&q)[8]) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2((c[0] & 0xffffu) | (c[1] << 16), (c[2] & 0xffffu) | (c[3] << 16));
}

// NVFP4: this lane's 8 quotients f / s, whose block of 16 it shares with the lane beside it (all lanes of the
// warp): the scale code of amax / 6, then each value's code of its quotient over E4M3(scale code), every
// step correctly rounded; a NaN in the block gives the NaN scale code and zero codes.
__device__ __forceinline__ uint32_t nvfp4_codes8(const float (&q)[8], uint32_t *scale_code) {
  float amax = 0.f;  // of the quotients: the division is monotone, so it is the quotient of the largest
  int nan = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(q[i]));
    nan |= q[i] != q[i];
  }
  // every lane takes part in both exchanges
  amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
  nan |= __shfl_xor_sync(FULL, nan, 1);
  *scale_code = 0x7Fu;
  if (nan) return 0u;
  *scale_code = (uint32_t)__nv_cvt_float_to_fp8(markstein_quot(amax, 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
  const float ds = e4m3_value(*scale_code);
  if (ds == 0.f) return 0u;
  const float r = __frcp_rn(ds);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= e2m1_pair(markstein_quot(q[2 * i], ds, r), markstein_quot(q[2 * i + 1], ds, r)) << (8 * i);
  return c;
}

template <int D, int FMT, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 3) qk_norm_rope_write_kernel(const RopeArgs a) {
  constexpr int LPH = D / 8;     // lanes per head row
  constexpr int HPG = 32 / LPH;  // head rows per group
  constexpr int AHEAD = 3;       // groups loaded together
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPH, g = lane / LPH;
  const int v0 = a.v0, HK = a.Hq + a.Hkv, H = v0 + a.Hkv, half = a.rot >> 1;
  constexpr bool PIECES = !IL;
  const bool turned = l * 8 < a.rot;
  // where this lane's two pieces of 4 values start (8 in a row where pairs are adjacent, and from rot on)
  const int at0 = PIECES && turned ? l * 4 : l * 8, at1 = PIECES && turned ? half + l * 4 : l * 8 + 4;
  const int e0 = turned ? l * 4 : 0;  // the first angle of this lane's 4 pairs
  // 16 bytes of bf16 values of a row: one access, or one of each piece
  auto load8 = [&](const uint16_t *row) {
    if constexpr (!PIECES) return *reinterpret_cast<const uint4 *>(row + at0);
    const uint2 lo = *reinterpret_cast<const uint2 *>(row + at0), hi = *reinterpret_cast<const uint2 *>(row + at1);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  };
  auto store8 = [&](uint16_t *row, uint4 v) {
    if constexpr (!PIECES) {
      *reinterpret_cast<uint4 *>(row + at0) = v;
    } else {
      *reinterpret_cast<uint2 *>(row + at0) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2 *>(row + at1) = make_uint2(v.z, v.w);
    }
  };
  const bool norm_q = a.q_weight != nullptr, norm_k = a.k_weight != nullptr;
  const uint4 wq = norm_q ? load8(a.q_weight) : make_uint4(0, 0, 0, 0), wk = norm_k ? load8(a.k_weight) : make_uint4(0, 0, 0, 0);
  const int items = a.tokens * a.segs, stride = (int)gridDim.x * (kRopeThreads / 32);
  int item = (int)blockIdx.x * (kRopeThreads / 32) + (int)(threadIdx.x >> 5);
  long long next_slot = item < items ? a.slots[item / a.segs] : 0;
  int next_pos = item < items ? a.positions[item / a.segs] : 0;
  for (; item < items; item += stride) {
    const int t = item / a.segs, g0 = (item - t * a.segs) * a.per_seg, g1 = min(g0 + a.per_seg, a.groups);
    const long long slot = next_slot;
    const int pos = next_pos;
    auto fetch = [&](int grp) {  // this lane's values of a group's rows
      const int h = grp * HPG + g;
      const uint16_t *row = h < a.Hq ? a.q + t * a.q_stride + h * D
                            : h < v0 ? a.k + t * a.k_stride + (h - a.Hq) * D
                                     : a.v + t * a.v_stride + (h - v0) * D;
      const bool there = grp < g1 && h < H && (FMT == ROPE_BF16 || h < HK || h >= v0);
      if (FMT == ROPE_NVFP4 && PIECES && h >= v0)  // (see the keys' exchange below)
        return there ? *reinterpret_cast<const uint4 *>(row + l * 8) : make_uint4(0, 0, 0, 0);
      return there ? load8(row) : make_uint4(0, 0, 0, 0);
    };
    uint4 raw[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) raw[i] = fetch(g0 + i);
    if (item + stride < items) {
      next_slot = a.slots[(item + stride) / a.segs];
      next_pos = a.positions[(item + stride) / a.segs];
    }
    if (slot < 0) continue;  // padding
    if (slot >= a.n_slots || pos < 0 || pos >= a.max_position) {
      if (a.status && lane == 0) atomicOr(a.status, slot >= a.n_slots ? PA_DEV_BAD_SLOT : PA_DEV_BAD_POS);
      continue;
    }
    float co[4], si[4];
    {
      const float *cs = a.cos_sin + (size_t)pos * a.rot + e0;
      const float4 c = *reinterpret_cast<const float4 *>(cs), s = *reinterpret_cast<const float4 *>(cs + half);
      co[0] = c.x, co[1] = c.y, co[2] = c.z, co[3] = c.w;
      si[0] = s.x, si[1] = s.y, si[2] = s.z, si[3] = s.w;
    }
    // norm and rotation of one lane's values of a row (all lanes of the warp; sums: some row has a norm;
    // norm, on: this row has one, is turned)
    auto turn = [&](float (&x)[8], bool sums, uint4 weight, bool norm, bool on) {
      if (sums) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) s2 = pair_fma(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
        if (norm) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          float w[8];
          unpack8(weight, w);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 y = pair_mul(pair_mul(make_float2(x[e], x[e + 1]), make_float2(r, r)), make_float2(w[e], w[e + 1]));
            x[e] = y.x, x[e + 1] = y.y;
          }
        }
      }
      if (on && turned) {
        if constexpr (IL) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * co[e] - v * si[e];
            x[2 * e + 1] = v * co[e] + u * si[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 u = make_float2(x[e], x[e + 1]), v = make_float2(x[4 + e], x[5 + e]), c = make_float2(co[e], co[e + 1]),
                         s = make_float2(si[e], si[e + 1]);
            const float2 p = pair_fma(make_float2(-v.x, -v.y), s, pair_mul(u, c)), q = pair_fma(u, s, pair_mul(v, c));
            x[e] = p.x, x[e + 1] = p.y, x[4 + e] = q.x, x[5 + e] = q.y;
          }
        }
      }
    };
    // A key as the quotient by its pool's scale, (x w cos - x' w' sin) (1 / (rms scale)): a step of a code is a sixteenth of
    // the value, so a key beside the middle of two codes goes by its last bits, and fewer roundings put fewer of them on
    // the wrong side: x w is exact, the factor is a pair of floats, a product's rounding is made good.  (Of 50 million keys 21
    // codes are not those of 64 bits, 94 with norm, rotation and division one after the other; that cost 63 -> 68 us.)
    auto turn_quot = [&](float (&x)[8], bool norm) {
      const float2 inv = a.k_inv;
      float2 f = inv;
      if (norm_q || norm_k) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) s2 = pair_fma(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
        if (norm) {
          // one step of Newton's method on 1 / sqrt(m), its change kept apart
          const float m = ss * (1.f / D) + a.eps, r = rsqrtf(m), r2 = r * r;
          const float left = fmaf(-m, fmaf(r, r, -r2), fmaf(-m, r2, 1.f)), rl = fabsf(left) < 1.f ? 0.5f * r * left : 0.f;
          f.x = r * inv.x;
          f.y = fmaf(rl, inv.x, fmaf(r, inv.y, fmaf(r, inv.x, -f.x)));
          float w[8];
          unpack8(wk, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= w[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = IL ? 2 * e : e, j = IL ? 2 * e + 1 : 4 + e;
        float u = x[i], v = x[j], ul = 0.f, vl = 0.f;
        if (turned) {
          const float uc = u * co[e], vc = v * co[e];
          ul = fmaf(u, co[e], -uc);
          vl = fmaf(v, co[e], -vc);
          const float us = fmaf(u, si[e], vc);
          u = fmaf(-v, si[e], uc);
          v = us;
        }
        const float rest_u = fmaf(ul, f.x, u * f.y), rest_v = fmaf(vl, f.x, v * f.y);
        x[i] = fmaf(u, f.x, fabsf(rest_u) < INFINITY ? rest_u : 0.f);
        x[j] = fmaf(v, f.x, fabsf(rest_v) < INFINITY ? rest_v : 0.f);
      }
    };
    for (int grp = g0; grp < g1; grp += AHEAD) {
      uint4 cur[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        cur[i] = raw[i];
        raw[i] = fetch(grp + AHEAD + i);
      }
      if ((grp + AHEAD) * HPG <= a.Hq) {  // queries only
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (grp + i >= g1) break;
          float x[8];
          unpack8(cur[i], x);
          turn(x, norm_q, wq, norm_q, true);
          store8(a.q_out + ((size_t)t * a.Hq + (grp + i) * HPG + g) * D, pack8(x));
        }
        continue;
      }
#pragma unroll 1
      for (int i = 0; i < AHEAD && grp + i < g1; ++i) {
        const int h = (grp + i) * HPG + g, hw = h - g;  // hw: the warp's first row
        const bool is_v = (FMT == ROPE_BF16 ? h : hw) >= v0, is_q = h < a.Hq;
        float x[8];
        unpack8(cur[0], x);
#pragma unroll
        for (int e = 0; e + 1 < AHEAD; ++e) cur[e] = cur[e + 1];
        if (hw < (FMT != ROPE_BF16 ? a.Hq : v0)) {  // some row is a query's (or a key's that stays bf16)
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e];
          const bool still = FMT == ROPE_BF16 && is_v;  // (a value beside a key)
          turn(y, norm_q || norm_k, is_q ? wq : wk, is_q ? norm_q : norm_k && !still, !still);
          if (FMT == ROPE_BF16 || is_q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[e];
          }
        }
        if (is_q) store8(a.q_out + ((size_t)t * a.Hq + h) * D, pack8(x));
        if (hw + HPG <= a.Hq) continue;
        // some row of the warp goes into a pool
        const bool store = !is_q && h < H && (FMT == ROPE_BF16 || h < HK || is_v);
        uint8_t *pool = is_v ? a.v_pool : a.k_pool;
        const size_t row = (size_t)slot * a.Hkv + (is_v ? h - v0 : h - a.Hq);
        if constexpr (FMT == ROPE_BF16) {
          if (store) store8(reinterpret_cast<uint16_t *>(pool) + row * D, pack8(x));
        } else {
          float q[8];
          if (!is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = x[e];
            turn_quot(q, norm_k && !is_q);
          } else {
            quot8(x, a.v_scale, q);
          }
          if constexpr (FMT == ROPE_NVFP4 && PIECES) {
            // keys: from two pieces to 8 values in a row, so that a block is two lanes' (values were read so)
            const bool first = l * 8 < half;
            float y[8];
            const int src = lane - l + (turned ? 2 * (first ? l : l - half / 8) : l);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = q[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int nb = turned ? src + 1 : lane;
              const float a0 = __shfl_sync(FULL, y[e], src), a1 = __shfl_sync(FULL, y[e], nb),
                          b0 = __shfl_sync(FULL, y[4 + e], src), b1 = __shfl_sync(FULL, y[4 + e], nb);
              if (turned && !is_v) {
                q[e] = first ? a0 : b0;
                q[4 + e] = first ? a1 : b1;
              }
            }
          }
          if constexpr (FMT == ROPE_FP8) {
            const uint2 c = fp8_codes8(q);
            if (store) {
              uint8_t *p = pool + row * D;
              if constexpr (PIECES) {
                *reinterpret_cast<uint32_t *>(p + at0) = c.x;
                *reinterpret_cast<uint32_t *>(p + at1) = c.y;
              } else {
                *reinterpret_cast<uint2 *>(p + at0) = c;
              }
            }
          } else {
            constexpr int CODES = D / 2, SCALES = D / 16, ROW = (CODES + SCALES + 15) / 16 * 16;
            uint8_t *p = pool + row * ROW;
            uint32_t sb;
            const uint32_t codes = nvfp4_codes8(q, &sb);
            // four blocks' scales to the first of their eight lanes
            const uint32_t s1 = __shfl_down_sync(FULL, sb, 2), s2 = __shfl_down_sync(FULL, sb, 4),
                           s3 = __shfl_down_sync(FULL, sb, 6);
            if (store) {
              *reinterpret_cast<uint32_t *>(p + l * 4) = codes;
              if (l % 8 == 0) *reinterpret_cast<uint32_t *>(p + CODES + l / 2) = sb | (s1 << 8) | (s2 << 16) | (s3 << 24);
              if (l > 0 && l <= (ROW - CODES - SCALES) / 4)
                *reinterpret_cast<uint32_t *>(p + CODES + SCALES + (l - 1) * 4) = 0u;
            }
          }
        }
      }
    }
  }
}

// Blocks of one wave: the device's SMs times the kernel's resident blocks (asked once per device).
template <auto kernel>
int wave_blocks() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  if (const int n = known[dev].load(std::memory_order_relaxed)) return n;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kRopeThreads, 0) != cudaSuccess)
    return -1;
  known[dev].store(sms * per_sm, std::memory_order_relaxed);
  return sms * per_sm;
}

template <int D, int FMT, bool IL>
cudaError_t launch_rope(RopeArgs &a, cudaStream_t stream) {
  constexpr int HPG = 256 / D, WARPS = kRopeThreads / 32;
  constexpr auto kernel = qk_norm_rope_write_kernel<D, FMT, IL>;
  const int wave = wave_blocks<kernel>();
  if (wave <= 0) return cudaErrorUnknown;
  // Into codes a group's rows are all values or none is: the values' quotients are formed as the plain write's.
  a.v0 = FMT == ROPE_BF16 ? a.Hq + a.Hkv : (a.Hq + a.Hkv + HPG - 1) / HPG * HPG;
  a.groups = (a.v0 + a.Hkv + HPG - 1) / HPG;
  // Segments per token, by the time of the longest warp: rounds of (token, segment) pairs, each the segment's
  // groups and a start (position, slot, angles and first rows from memory) worth about four of them.  (One
  // group a segment everywhere takes 117 us where this takes 65, 8192 tokens of 64 + 8 + 8 heads of 128.)
  const long long warps = (long long)wave * WARPS;
  long long best = LLONG_MAX;
  for (int per = a.groups; per >= 1; per = per > 1 ? per * 3 / 4 : 0) {
    const int segs = (a.groups + per - 1) / per;
    const long long cost = ((long long)a.tokens * segs + warps - 1) / warps * (per + 4);
    if (cost < best) best = cost, a.per_seg = per, a.segs = segs;
  }
  const long long items = (long long)a.tokens * a.segs, blocks = (items + WARPS - 1) / WARPS;
  if (items > INT_MAX - wave * WARPS) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < wave ? blocks : wave));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int FMT>
cudaError_t launch_rope_any(RopeArgs &a, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch_rope<D, FMT, true>(a, stream) : launch_rope<D, FMT, false>(a, stream);
}

template <int FMT>
cudaError_t launch_rope_dim(int D, RopeArgs &a, bool interleaved, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_rope_any<64, FMT>(a, interleaved, stream);
    case 128: return launch_rope_any<128, FMT>(a, interleaved, stream);
    default: return launch_rope_any<256, FMT>(a, interleaved, stream);
  }
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool overlap(const void *p, size_t np, const void *q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

int rope_call(const void *q, const void *k, const void *v, const void *q_weight, const void *k_weight,
              const float *cos_sin, const int32_t *positions, const int64_t *slot_mapping, void *q_out, void *k_pool,
              void *v_pool, int T, int Hq, int Hkv, int D, long long q_stride, long long k_stride, long long v_stride,
              int rot, int interleaved, int max_position, float eps, int fmt, float k_scale, float v_scale,
              int page_size, int num_pages, uint32_t *status, cudaStream_t stream) {
  note_launches(0);
  if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || max_position <= 0 || rot <= 0 ||
      !std::isfinite(eps) || eps < 0.f)
    return PA_ERR_INVALID_ARGUMENT;
  if (fmt != ROPE_BF16 && !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return PA_ERR_INVALID_ARGUMENT;
  if (D != 64 && D != 128 && D != 256) return PA_ERR_UNSUPPORTED;
  if (rot > D) return PA_ERR_INVALID_ARGUMENT;
  if (rot % 16 != 0 || Hq > 65536 || Hkv > 65536) return PA_ERR_UNSUPPORTED;
  // (so that 1 / (rms scale) is no infinity, which would make NaN of a key's zeros)
  if (fmt != ROPE_BF16 && !(k_scale >= 0x1p-50f && k_scale <= 0x1p50f && v_scale >= 0x1p-50f && v_scale <= 0x1p50f))
    return PA_ERR_UNSUPPORTED;
  if (T == 0) return PA_OK;
  if (!q || !k || !v || !cos_sin || !positions || !slot_mapping || !q_out || !k_pool || !v_pool)
    return PA_ERR_INVALID_ARGUMENT;
  const long long nq = (long long)Hq * D, nk = (long long)Hkv * D;
  if (q_stride < nq || k_stride < nk || v_stride < nk) return PA_ERR_INVALID_ARGUMENT;
  if (q_stride % 8 || k_stride % 8 || v_stride % 8) return PA_ERR_MISALIGNED;
  const void *vecs[] = {q, k, v, q_weight, k_weight, cos_sin, q_out, k_pool, v_pool};
  for (const void *p : vecs)
    if (!aligned_to(p, 16)) return PA_ERR_MISALIGNED;
  if (!aligned_to(positions, 4) || !aligned_to(slot_mapping, 8) || !aligned_to(status, 4)) return PA_ERR_MISALIGNED;
  // nothing that is written may be something else that is read or written, but q_out may be q
  const size_t row = fmt == ROPE_BF16 ? 2 * (size_t)D : fmt == ROPE_FP8 ? (size_t)D : (size_t)(D / 2 + D / 16 + 15) / 16 * 16;
  const size_t pool = (size_t)num_pages * page_size * Hkv * row, out = (size_t)T * nq * 2;
  const size_t sq = ((size_t)(T - 1) * q_stride + nq) * 2, sk = ((size_t)(T - 1) * k_stride + nk) * 2,
               sv = ((size_t)(T - 1) * v_stride + nk) * 2;
  const bool in_place = q_out == q && (q_stride == nq || T == 1);
  if (!in_place && overlap(q_out, out, q, sq)) return PA_ERR_INVALID_ARGUMENT;
  if (overlap(q_out, out, k, sk) || overlap(q_out, out, v, sv) || overlap(k_pool, pool, v_pool, pool))
    return PA_ERR_INVALID_ARGUMENT;
  const void *pools[] = {k_pool, v_pool};
  for (const void *p : pools)
    if (overlap(p, pool, q, sq) || overlap(p, pool, k, sk) || overlap(p, pool, v, sv) || overlap(p, pool, q_out, out))
      return PA_ERR_INVALID_ARGUMENT;
  const struct {
    const void *p;
    size_t n;
  } more[] = {{cos_sin, (size_t)max_position * rot * 4}, {positions, (size_t)T * 4}, {slot_mapping, (size_t)T * 8},
              {q_weight, q_weight ? (size_t)D * 2 : 0}, {k_weight, k_weight ? (size_t)D * 2 : 0}, {status, status ? 4u : 0u}};
  for (const auto &m : more)
    if (overlap(q_out, out, m.p, m.n) || overlap(k_pool, pool, m.p, m.n) || overlap(v_pool, pool, m.p, m.n))
      return PA_ERR_INVALID_ARGUMENT;
  RopeArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.q_weight = static_cast<const uint16_t *>(q_weight);
  a.k_weight = static_cast<const uint16_t *>(k_weight);
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.slots = slot_mapping;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.k_pool = static_cast<uint8_t *>(k_pool);
  a.v_pool = static_cast<uint8_t *>(v_pool);
  a.status = status;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_slots = (long long)num_pages * page_size;
  a.tokens = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.rot = rot;
  a.max_position = max_position;
  a.v0 = a.groups = a.segs = a.per_seg = 0;
  a.eps = eps;
  a.k_inv.x = 1.f / k_scale;
  a.k_inv.y = std::fma(-k_scale, a.k_inv.x, 1.f) * a.k_inv.x;
  a.v_scale = fp8_scale(v_scale);
  const cudaError_t e = fmt == ROPE_BF16  ? launch_rope_dim<ROPE_BF16>(D, a, interleaved != 0, stream)
                        : fmt == ROPE_FP8 ? launch_rope_dim<ROPE_FP8>(D, a, interleaved != 0, stream)
                                          : launch_rope_dim<ROPE_NVFP4>(D, a, interleaved != 0, stream);
  if (e == cudaErrorInvalidConfiguration) return PA_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return cuda_fail(e);
  note_launches(1);
  return PA_OK;
}

}  // namespace

}  // namespace pa

extern "C" int pa_qk_norm_rope_write(const void *q, const void *k, const void *v, const void *q_weight,
                                     const void *k_weight, const float *cos_sin, const int32_t *positions,
                                     const int64_t *slot_mapping, void *q_out, void *k_pool, void *v_pool,
                                     int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                     long long q_stride, long long k_stride, long long v_stride, int rot_dim,
                                     int interleaved, int max_position, float eps, int page_size, int num_pages,
                                     uint32_t *status, cudaStream_t stream) {
  return pa::rope_call(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, num_tokens,
                       num_q_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride, rot_dim, interleaved,
                       max_position, eps, pa::ROPE_BF16, 1.f, 1.f, page_size, num_pages, status, stream);
}

extern "C" int pa_qk_norm_rope_write_fp8(const void *q, const void *k, const void *v, const void *q_weight,
                                         const void *k_weight, const float *cos_sin, const int32_t *positions,
                                         const int64_t *slot_mapping, void *q_out, void *k_pool, void *v_pool,
                                         int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                         long long q_stride, long long k_stride, long long v_stride, int rot_dim,
                                         int interleaved, int max_position, float eps, float k_scale, float v_scale,
                                         int page_size, int num_pages, uint32_t *status, cudaStream_t stream) {
  return pa::rope_call(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, num_tokens,
                       num_q_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride, rot_dim, interleaved,
                       max_position, eps, pa::ROPE_FP8, k_scale, v_scale, page_size, num_pages, status, stream);
}

extern "C" int pa_qk_norm_rope_write_nvfp4(const void *q, const void *k, const void *v, const void *q_weight,
                                           const void *k_weight, const float *cos_sin, const int32_t *positions,
                                           const int64_t *slot_mapping, void *q_out, void *k_pool, void *v_pool,
                                           int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                           long long q_stride, long long k_stride, long long v_stride, int rot_dim,
                                           int interleaved, int max_position, float eps, float k_scale, float v_scale,
                                           int page_size, int num_pages, uint32_t *status, cudaStream_t stream) {
  return pa::rope_call(q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping, q_out, k_pool, v_pool, num_tokens,
                       num_q_heads, num_kv_heads, head_dim, q_stride, k_stride, v_stride, rot_dim, interleaved,
                       max_position, eps, pa::ROPE_NVFP4, k_scale, v_scale, page_size, num_pages, status, stream);
}
