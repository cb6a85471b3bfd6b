// pa_rope_write.cu -- norms of queries and keys for each head, position rotation and paged write in
// one pass: the step between the q/k/v projection and the attention.
//
// Mathematics, per head row x of D values at position p (fp32): y = x / sqrt(mean(x^2) + eps) * w;
// pairs (u, v) of the first rot values become (u cos - v sin, v cos + u sin) by the angles of row p
// of a table; one rounding to the output's type at the end.  Values of v are stored as they are.
//
// A pass over the data, bound by HBM: each value is read once and written once.  A lane holds 8
// consecutive values (one 16-byte load), D / 8 lanes a head row, so the sum of squares is a few
// shuffles, an adjacent pair lies in one lane, and a pair rot / 2 apart is one shuffle away (rot is a
// multiple of 16, so whole lanes face each other).  A warp takes one token and IT x (256 / D) of its
// heads: the token's position, slot and angles are loaded once for all of them, and the IT rows'
// loads are in flight together.
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
  const uint4 *q_weight, *k_weight;  // [D] bf16 or null
  const float *cos_sin;         // [max_position, rot]
  const int32_t *positions;
  const int64_t *slots;
  uint16_t *q_out;
  uint8_t *k_pool, *v_pool;
  uint32_t *status;             // or null
  long long q_stride, k_stride, v_stride, n_slots;
  int tokens, Hq, Hkv, rot, max_position, chunks;  // chunks: warps per token
  float eps;
  Fp8Scale k_scale, v_scale;
};

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

// E4M3 codes of f / s, nearest with ties to even, saturated.
__device__ __forceinline__ uint2 fp8_codes8(const float (&f)[8], Fp8Scale s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(quot(f[2 * i], s), quot(f[2 * i + 1], s)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2((c[0] & 0xffffu) | (c[1] << 16), (c[2] & 0xffffu) | (c[3] << 16));
}

// NVFP4 codes of this lane's 8 values and the scale code of its block of 16, which it shares with the
// lane beside it (all lanes of the warp): the scale code of (amax / s) / 6, then each value's code of
// (f / s) / E4M3(scale code), every step correctly rounded; a NaN in the block gives the NaN scale
// code and zero codes.
__device__ __forceinline__ uint32_t nvfp4_codes8(const float (&f)[8], Fp8Scale s, uint32_t *scale_code) {
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(f[i]));
    nan = nan || f[i] != f[i];
  }
  // every lane takes part in both exchanges
  const float both = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
  const int other_nan = __shfl_xor_sync(FULL, (int)nan, 1);
  const bool any_nan = nan || other_nan != 0;
  *scale_code = 0x7Fu;
  if (any_nan) return 0u;
  *scale_code = (uint32_t)__nv_cvt_float_to_fp8(markstein_quot(quot(both, s), 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
  const float ds = e4m3_value(*scale_code);
  if (ds == 0.f) return 0u;
  const float r = __frcp_rn(ds);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c |= e2m1_pair(markstein_quot(quot(f[2 * i], s), ds, r), markstein_quot(quot(f[2 * i + 1], s), ds, r)) << (8 * i);
  return c;
}

template <int D, int FMT, bool IL, int IT>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_write_kernel(const RopeArgs a) {
  constexpr int LPH = D / 8;     // lanes per head row
  constexpr int HPI = 32 / LPH;  // head rows per warp and iteration
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPH, g = lane / LPH;
  const int item = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int t = item / a.chunks, h0 = (item - t * a.chunks) * (HPI * IT);
  if (t >= a.tokens) return;
  const long long slot = a.slots[t];
  const int pos = a.positions[t];
  const int H = a.Hq + 2 * a.Hkv;
  uint4 raw[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int h = h0 + i * HPI + g;
    const uint16_t *row = h < a.Hq          ? a.q + t * a.q_stride + h * D
                          : h < a.Hq + a.Hkv ? a.k + t * a.k_stride + (h - a.Hq) * D
                                             : a.v + t * a.v_stride + (h - a.Hq - a.Hkv) * D;
    raw[i] = h < H ? *reinterpret_cast<const uint4 *>(row + l * 8) : make_uint4(0, 0, 0, 0);
  }
  if (slot < 0) return;  // padding
  if (slot >= a.n_slots || pos < 0 || pos >= a.max_position) {
    if (a.status && lane == 0) atomicOr(a.status, slot >= a.n_slots ? PA_DEV_BAD_SLOT : PA_DEV_BAD_POS);
    return;
  }
  // this lane's angles: those of its 8 values (or 4 adjacent pairs)
  const int half = a.rot >> 1;
  const bool turned = l * 8 < a.rot;
  float co[IL ? 4 : 8], si[IL ? 4 : 8];
  {
    const int e0 = IL ? l * 4 : (l * 8 < half ? l * 8 : l * 8 - half);
    const float *cs = a.cos_sin + (size_t)pos * a.rot + (turned ? e0 : 0);
#pragma unroll
    for (int i = 0; i < (IL ? 4 : 8); i += 4) {
      const float4 c = *reinterpret_cast<const float4 *>(cs + i);
      const float4 s = *reinterpret_cast<const float4 *>(cs + half + i);
      co[i] = c.x, co[i + 1] = c.y, co[i + 2] = c.z, co[i + 3] = c.w;
      si[i] = s.x, si[i + 1] = s.y, si[i + 2] = s.z, si[i + 3] = s.w;
    }
  }
  // pairs half a turn apart: this lane's partner, and the sign of the sine for its side
  const int partner = !turned ? lane : l * 8 < half ? lane + half / 8 : lane - half / 8;
  const float side = l * 8 < half ? -1.f : 1.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int hw = h0 + i * HPI;  // the warp's first row of this iteration
    if (hw >= H) break;
    const int h = hw + g;
    const bool is_v = h >= a.Hq + a.Hkv;
    float x[8];
    unpack8(raw[i], x);
    if (hw < a.Hq + a.Hkv) {  // some row of the warp is a query's or a key's
      const uint4 *weight = h < a.Hq ? a.q_weight : a.k_weight;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
      if (!is_v && weight) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float w[8];
        unpack8(weight[l], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
      }
      if constexpr (IL) {
        if (!is_v && turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = x[2 * e], v = x[2 * e + 1];
            x[2 * e] = u * co[e] - v * si[e];
            x[2 * e + 1] = v * co[e] + u * si[e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_sync(FULL, x[e], partner);
          if (!is_v && turned) x[e] = x[e] * co[e] + side * y * si[e];
        }
      }
    }
    if (h < a.Hq) *reinterpret_cast<uint4 *>(a.q_out + ((size_t)t * a.Hq + h) * D + l * 8) = pack8(x);
    if (hw + HPI > a.Hq) {  // some row of the warp goes into a pool
      const bool store = h >= a.Hq && h < H;
      uint8_t *pool = is_v ? a.v_pool : a.k_pool;
      const Fp8Scale sc = is_v ? a.v_scale : a.k_scale;
      const size_t row = (size_t)slot * a.Hkv + (is_v ? h - a.Hq - a.Hkv : h - a.Hq);
      if constexpr (FMT == ROPE_BF16) {
        if (store) *reinterpret_cast<uint4 *>(pool + row * (2 * D) + l * 16) = pack8(x);
      } else if constexpr (FMT == ROPE_FP8) {
        if (store) *reinterpret_cast<uint2 *>(pool + row * D + l * 8) = fp8_codes8(x, sc);
      } else {
        constexpr int CODES = D / 2, SCALES = D / 16, ROW = (CODES + SCALES + 15) / 16 * 16;
        uint32_t sb;
        const uint32_t codes = nvfp4_codes8(x, sc, &sb);
        // four blocks' scales to the first of their eight lanes
        const uint32_t s1 = __shfl_down_sync(FULL, sb, 2), s2 = __shfl_down_sync(FULL, sb, 4),
                       s3 = __shfl_down_sync(FULL, sb, 6);
        if (store) {
          uint8_t *p = pool + row * ROW;
          *reinterpret_cast<uint32_t *>(p + l * 4) = codes;
          if (l % 8 == 0) *reinterpret_cast<uint32_t *>(p + CODES + l / 2) = sb | (s1 << 8) | (s2 << 16) | (s3 << 24);
          if (l > 0 && l <= (ROW - CODES - SCALES) / 4)
            *reinterpret_cast<uint32_t *>(p + CODES + SCALES + (l - 1) * 4) = 0u;
        }
      }
    }
  }
}

template <int D, int FMT, bool IL, int IT>
cudaError_t launch_rope(RopeArgs &a, cudaStream_t stream) {
  constexpr int ROWS = 256 / D * IT;
  const int H = a.Hq + 2 * a.Hkv;
  a.chunks = (H + ROWS - 1) / ROWS;
  const long long items = (long long)a.tokens * a.chunks;
  const long long grid = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > INT_MAX / (kRopeThreads / 32)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_write_kernel<D, FMT, IL, IT>, a);
}

template <int D, int FMT>
cudaError_t launch_rope_any(RopeArgs &a, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch_rope<D, FMT, true, 1>(a, stream) : launch_rope<D, FMT, false, 1>(a, stream);
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
  RopeArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.q_weight = static_cast<const uint4 *>(q_weight);
  a.k_weight = static_cast<const uint4 *>(k_weight);
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
  a.chunks = 0;
  a.eps = eps;
  a.k_scale = fp8_scale(k_scale);
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
