// New rows into the paged cache (mla_kv_append): per token, RMS norm of the
// 512 latent values, RoPE, conversion to the cache's format, and the scatter to
// the token's slot, the key's counterpart of mla_q_norm_rope.
//
//   y    = latent * (1 / sqrt(mean(latent^2) + eps)) * gamma      (norm)
//   bf16 = RNE(y), the rotated pairs RNE(x0 c - x1 s), RNE(x0 s + x1 c)
//   FP8  per 128 values: scale = amax * (1 / 448) (1 if amax = 0), code = RNE(x / scale)
//   FP4  per 16 values:  scale = e4m3(amax * (1 / 6)),             code = RNE(x / scale)
// 1 / 448 and 1 / 6 are rounded to fp32. For E2M1 the product decides like the
// quotient; an FP8 scale may differ from amax / 448 in its last bit (55 % of bf16
// mantissas), and is the same as torch's amax / 448 on the GPU, which multiplies
// by the reciprocal of a scalar: programs that fill a cache with torch get these bytes.
//
// A row map, for 4-bit records 1152 bytes in and 416 out per token. One warp per
// token: lane l holds latent values 8l..8l+7 and 256+8l.. (an FP4 block is two
// lanes, an FP8 tile sixteen) and RoPE pair l, so every access of the warp is
// contiguous. 32768 rows, without / with the stored values written too: 20 / 23 us
// into 4-bit records, 21 / 23 FP8, 16 / 21 BF16 (floors at the measured copy rate
// 9 / 15, 10 / 16, 13 / 19). Quantised rows are bound by instruction issue (4 bits:
// 557 warp instructions a row, 3.1 a clock of 4; DRAM 26 %); the norm's 64-bit sum
// is 1 us of it.
// The codes are functions of the inputs alone, whatever the order of the sum:
// the sum of squares is taken in 64 bits (squares of bf16 values; its rounding
// reaches the fp32 factor about once in 2^29 rows), every fp32 operation after
// it is rounded once, uncontracted.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "mla_kernels.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 128;  // four tokens per block (eight: 256 rows 2.5 us instead of 2.3)
constexpr int kRope = 64;

struct AppendParams {
  const __nv_bfloat16* kv;
  const float *gamma, *cos_t, *sin_t;
  const int32_t* slots;
  uint8_t *cache, *cache_scale;
  __nv_bfloat16* values;
  uint32_t* status;
  long long stride;
  int tokens, num_slots;
  float eps;
};

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  a = x;
}

// x / s rounded as the E2M1 conversion needs it. x has 8 significant bits, s 4,
// and a midpoint m of the code's grid 3: x / s is m itself or at least 2^-8 of
// it away. The product with 1 / s is off by 2^-23 at most, and rounding it to
// 12 bits (Veltkamp's split) gives m exactly in the first case and keeps its
// side in the second, so RNE decides as for the exact quotient.
__device__ __forceinline__ float quotient(float x, float inv) {
  const float q = fminf(fmaxf(__fmul_rn(x, inv), -8.f), 8.f);
  const float c = __fmul_rn(q, 4097.f);
  return __fsub_rn(c, __fsub_rn(c, q));
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  constexpr bool kFull = FMT != MLA_KV_NVFP4;  // 576-value rows; else 512 with RoPE on the last 64
  constexpr int kD = kFull ? kDqk : kNvfp4D;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int tok = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.tokens) return;
  const int slot = p.slots[tok];
  const __nv_bfloat16* src = p.kv + (size_t)tok * p.stride;
  const uint4 a = reinterpret_cast<const uint4*>(src)[lane], b = reinterpret_cast<const uint4*>(src)[32 + lane];
  uint32_t rope = 0;
  float c = 1.f, s = 0.f;
  if (kFull) {
    rope = reinterpret_cast<const uint32_t*>(src + kDv)[lane];
    if (p.cos_t) c = p.cos_t[(size_t)tok * (kRope / 2) + lane], s = p.sin_t[(size_t)tok * (kRope / 2) + lane];
  }
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1 && lane == 0 && p.status) atomicOr(p.status, (uint32_t)MLA_DEVICE_STATUS_BOUNDS);
    return;
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack(w[i]);
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
  if (p.gamma) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fma((double)y[i], (double)y[i], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = (float)(1.0 / sqrt(ss / (double)kDv + (double)p.eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 g = reinterpret_cast<const float4*>(p.gamma)[(i >> 1) * 64 + 2 * lane + (i & 1)];
      y[4 * i] = __fmul_rn(__fmul_rn(y[4 * i], r), g.x);
      y[4 * i + 1] = __fmul_rn(__fmul_rn(y[4 * i + 1], r), g.y);
      y[4 * i + 2] = __fmul_rn(__fmul_rn(y[4 * i + 2], r), g.z);
      y[4 * i + 3] = __fmul_rn(__fmul_rn(y[4 * i + 3], r), g.w);
    }
  }
  if (!kFull && p.cos_t && lane >= 24) {  // dims 448..511
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = (size_t)tok * (kRope / 2) + 4 * (lane - 24) + i;
      rotate(y[8 + 2 * i], y[9 + 2 * i], p.cos_t[at], p.sin_t[at]);
    }
  }
  // rows are rounded to bf16 before anything else is made of them
  uint32_t v[8];
  float amax[2] = {0.f, 0.f};  // of each half row's values
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    const float2 f = unpack(v[i]);
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
    amax[i >> 2] = fmaxf(amax[i >> 2], fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  if (kFull && p.cos_t) {
    float2 f = unpack(rope);
    rotate(f.x, f.y, c, s);
    rope = pack_bf16x2(f.x, f.y);
  }
  if (FMT == MLA_KV_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(p.cache + (size_t)slot * (kDqk * 2)) + lane;
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[32] = make_uint4(v[4], v[5], v[6], v[7]);
    reinterpret_cast<uint32_t*>(p.cache + (size_t)slot * (kDqk * 2) + kDv * 2)[lane] = rope;
  } else if (FMT == MLA_KV_FP8_E4M3) {
    uint8_t* rec = p.cache + (size_t)slot * kFp8RecordBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax[h] = fmaxf(amax[h], __shfl_xor_sync(0xffffffffu, amax[h], o));
      const float scale = amax[h] > 0.f ? __fmul_rn(amax[h], 1.f / 448.f) : 1.f;
      uint32_t pk[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t q = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(y[8 * h + 2 * i], scale), __fdiv_rn(y[8 * h + 2 * i + 1], scale)), __NV_SATFINITE,
            __NV_E4M3);
        pk[i >> 1] |= (uint32_t)q << (16 * (i & 1));
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(q, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        v[4 * h + i] = pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
      }
      reinterpret_cast<uint2*>(rec)[32 * h + lane] = make_uint2(pk[0], pk[1]);
      if ((lane & 15) == 0) reinterpret_cast<float*>(rec + kDv)[2 * h + (lane >> 4)] = scale;
    }
    reinterpret_cast<uint32_t*>(rec + kDv + 16)[lane] = rope;
  } else {
    uint8_t* codes = p.cache + (size_t)slot * (kFull ? kFp4RecordBytes : kNvfp4RowBytes);
    uint8_t* scales = kFull ? codes + kFp4ScaleOff : p.cache_scale + (size_t)slot * kNvfp4ScaleBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      amax[h] = fmaxf(amax[h], __shfl_xor_sync(0xffffffffu, amax[h], 1));
      const __nv_fp8_storage_t sc = __nv_cvt_float_to_fp8(__fmul_rn(amax[h], 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
      const __half_raw sr = __nv_cvt_fp8_to_halfraw(sc, __NV_E4M3);
      const float sf = __half2float(*reinterpret_cast<const __half*>(&sr));
      const float inv = sf > 0.f ? __fdiv_rn(1.f, sf) : 0.f;
      uint32_t pk = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_fp4x2_storage_t q = 0;  // a block whose scale rounds to 0 has codes 0
        if (sf > 0.f)
          q = __nv_cvt_float2_to_fp4x2(make_float2(quotient(y[8 * h + 2 * i], inv), quotient(y[8 * h + 2 * i + 1], inv)),
                                       __NV_E2M1, cudaRoundNearest);
        pk |= (uint32_t)q << (8 * i);
        const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2(q, __NV_E2M1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        v[4 * h + i] = pack_bf16x2(f.x * sf, f.y * sf);  // exact
      }
      reinterpret_cast<uint32_t*>(codes)[32 * h + lane] = pk;
      if ((lane & 1) == 0) scales[16 * h + (lane >> 1)] = sc;
    }
    if (kFull) reinterpret_cast<uint32_t*>(codes + kFp4RopeOff)[lane] = rope;
  }
  if (p.values) {
    uint4* dst = reinterpret_cast<uint4*>(p.values + (size_t)tok * kD) + lane;
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[32] = make_uint4(v[4], v[5], v[6], v[7]);
    if (kFull) reinterpret_cast<uint32_t*>(p.values + (size_t)tok * kD + kDv)[lane] = rope;
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_kv_append(const void* kv, long long kv_stride, int tokens, int d_qk, const float* gamma,
                                      float eps, const float* rope_cos, const float* rope_sin, const int32_t* slots,
                                      void* kcache, void* kv_scale, int kv_format, int num_pages, void* kv_out,
                                      uint32_t* status, mla_stream_t stream) {
  if (!kv || !slots || !kcache || tokens <= 0 || num_pages <= 0) return MLA_ERR_INVALID_ARG;
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_E4M3 && kv_format != MLA_KV_NVFP4 &&
      kv_format != MLA_KV_FP4_E2M1)
    return MLA_ERR_INVALID_ARG;
  const bool nvfp4 = kv_format == MLA_KV_NVFP4;
  if (d_qk != (nvfp4 ? kNvfp4D : kDqk) || kv_stride < d_qk || kv_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (!al16(kv) || !al16(kcache) || !al16(kv_out) || !al16(gamma) || !al4(slots) || !al4(status) || !al4(rope_cos) ||
      !al4(rope_sin))
    return MLA_ERR_INVALID_ARG;
  if ((rope_cos == nullptr) != (rope_sin == nullptr)) return MLA_ERR_INVALID_ARG;
  if (gamma && !(eps >= 0.f)) return MLA_ERR_INVALID_ARG;
  if (nvfp4 && (!kv_scale || !al16(kv_scale))) return MLA_ERR_INVALID_ARG;
  if ((long long)num_pages * kPage > 0x7fffffffLL || tokens > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  const size_t T = (size_t)tokens, rows = (size_t)num_pages * kPage;
  const size_t row_bytes = kv_format == MLA_KV_BF16       ? kDqk * 2
                           : kv_format == MLA_KV_FP8_E4M3 ? kFp8RecordBytes
                           : nvfp4                        ? kNvfp4RowBytes
                                                          : kFp4RecordBytes;
  const size_t angles = rope_cos ? T * (kRope / 2) * 4 : 0;
  const struct { const void* p; size_t n; } in[] = {{kv, ((T - 1) * (size_t)kv_stride + d_qk) * 2}, {gamma, gamma ? kDv * 4 : 0},
                                                    {rope_cos, angles}, {rope_sin, angles}, {slots, T * 4}};
  const struct { const void* p; size_t n; } out[] = {{kcache, rows * row_bytes}, {kv_scale, nvfp4 ? rows * kNvfp4ScaleBytes : 0},
                                                     {kv_out, kv_out ? T * d_qk * 2 : 0}, {status, status ? sizeof(*status) : 0}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j)
      // rows are read whole before they are written: kv_out may be kv itself
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n) && !(i == 2 && j == 0 && kv_out == kv && kv_stride == d_qk))
        return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MLA_ERR_INVALID_ARG;
  }
  const AppendParams p{static_cast<const __nv_bfloat16*>(kv), gamma, rope_cos, rope_sin, slots,
                       static_cast<uint8_t*>(kcache), static_cast<uint8_t*>(kv_scale),
                       static_cast<__nv_bfloat16*>(kv_out), status, kv_stride, tokens, num_pages * kPage, eps};
  const dim3 grid((tokens - 1) / (kThreads / 32) + 1);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      kv_format == MLA_KV_BF16        ? launch_pdl(kv_append_kernel<MLA_KV_BF16>, grid, dim3(kThreads), 0, st, p)
      : kv_format == MLA_KV_FP8_E4M3  ? launch_pdl(kv_append_kernel<MLA_KV_FP8_E4M3>, grid, dim3(kThreads), 0, st, p)
      : kv_format == MLA_KV_NVFP4     ? launch_pdl(kv_append_kernel<MLA_KV_NVFP4>, grid, dim3(kThreads), 0, st, p)
                                      : launch_pdl(kv_append_kernel<MLA_KV_FP4_E2M1>, grid, dim3(kThreads), 0, st, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
